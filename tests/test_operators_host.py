"""Refusals of the decode-step operators, which all happen on the host before a
GPU is touched, and the 64-bit reference forms against hand-worked values."""

import math

import numpy as np
import pytest

import group_quantized_mat_gb300 as g
import operators_reference as ref

FAKE = 1 << 20  # an aligned address that validation must reject before any use


@pytest.fixture(scope="module")
def lib():
    from group_quantized_mat_gb300 import build
    build.build()
    return g.load()


def call(lib, name, pointers, scalars, kw):
    vals = {**{p: FAKE for p in pointers}, **scalars, "workspace": None, "workspace_bytes": 0, "flags": 0, "stream": None}
    assert set(kw) <= set(vals), kw
    vals.update(kw)
    return getattr(lib, name)(*vals.values())


LORA = (["w_q", "scales", "biases", "x", "a", "b", "adapter", "c", "y"],
        dict(M=2, N=64, K=1024, bits=4, gs=64, L=3, R=8))


@pytest.mark.parametrize("kw,code", [
    *[({p: None}, 1) for p in LORA[0]],
    (dict(bits=3), 2), (dict(gs=32), 3), (dict(K=1000), 4), (dict(N=0), 4), (dict(K=0), 4), (dict(M=0), 5), (dict(M=257), 5),
    (dict(L=0), 11), (dict(L=65537), 11), (dict(R=0), 11), (dict(R=257), 11), (dict(flags=2), 10), (dict(flags=0x10), 10),
    *[({p: FAKE + 8}, 6) for p in ("w_q", "scales", "biases", "x", "a", "b", "workspace")],
    (dict(adapter=FAKE + 2), 6), (dict(c=FAKE + 1), 6), (dict(y=FAKE + 1), 6), (dict(y=FAKE + 2, flags=1), 6),
])
def test_lora_refusals(lib, kw, code):
    assert call(lib, "qmv_lora_run", *LORA, kw) == code


MOE = (["x", "router", "gu_w", "gu_s", "gu_b", "dn_w", "dn_s", "dn_b", "y", "ids", "weights"],
       dict(M=2, K=512, inter=256, E=8, k=2, bits=4, gs=64))


@pytest.mark.parametrize("kw,code", [
    *[({p: None}, 1) for p in MOE[0][:9]],
    (dict(bits=8), 2), (dict(gs=96), 3), (dict(K=100), 4), (dict(inter=100), 4), (dict(inter=0), 4), (dict(K=0), 4),
    (dict(inter=192, gs=128), 4), (dict(M=0), 5), (dict(M=257), 5), (dict(E=0), 11), (dict(E=1025), 11), (dict(k=0), 11),
    (dict(k=9), 11), (dict(E=64, k=33), 11), (dict(M=256, E=64, k=17), 11), (dict(K=1 << 20, inter=1 << 20), 4), (dict(flags=2), 10), (dict(flags=0x40), 10),
    *[({p: FAKE + 8}, 6) for p in MOE[0][:8] + ["workspace"]],
    (dict(y=FAKE + 1), 6), (dict(y=FAKE + 2, flags=1), 6), (dict(ids=FAKE + 2), 6), (dict(weights=FAKE + 2), 6),
])
def test_moe_refusals(lib, kw, code):
    assert call(lib, "qmv_moe_run", *MOE, kw) == code


VERIFY = (["target", "draft", "draft_tokens", "draft_len", "temperature", "uniform", "noise", "tokens", "accepted", "logprob"],
          dict(B=2, S=3, V=1000, ld_target=1000, ld_draft=1000, ld_noise=1000))


@pytest.mark.parametrize("kw,code", [
    *[({p: None}, 1) for p in ("target", "draft_tokens", "uniform", "noise", "tokens", "accepted")],
    (dict(B=0), 11), (dict(B=65536), 11), (dict(S=-1), 11), (dict(S=64), 11), (dict(V=0), 4), (dict(V=(1 << 24) + 1), 4),
    (dict(ld_target=999), 4), (dict(ld_draft=999), 4), (dict(ld_noise=-1), 4), (dict(ld_noise=1 << 41), 4),
    (dict(flags=1), 10), (dict(target=FAKE + 1), 6), (dict(target=FAKE + 2, flags=0x40), 6), (dict(draft=FAKE + 1), 6),
    (dict(workspace=FAKE + 8), 6), *[({p: FAKE + 2}, 6) for p in VERIFY[0][2:]],
])
def test_verify_refusals(lib, kw, code):
    assert call(lib, "qmv_verify_run", *VERIFY, kw) == code


def test_workspace_sizes(lib):
    assert g.qmv_lora_workspace_size(1, 64, 1024, 4, 64, 8) > 0 and g.qmv_lora_workspace_size(0, 64, 1024, 4, 64, 8) == 0
    assert g.qmv_lora_workspace_size(1, 64, 1024, 4, 64, 0) == 0 and g.qmv_lora_workspace_size(1, 64, 1000, 4, 64, 8) == 0
    assert g.qmv_moe_workspace_size(1, 512, 256, 8, 2, 4, 64) > 0 and g.qmv_moe_workspace_size(1, 512, 256, 8, 9, 4, 64) == 0
    assert g.qmv_verify_workspace_size(1, 0, 10) > 0 and g.qmv_verify_workspace_size(0, 0, 10) == 0
    sizes = [g.qmv_verify_workspace_size(B, 4, 50000) for B in (1, 2, 64, 1000)]
    assert sizes == sorted(sizes)


def test_errors_carry_their_names(lib):
    with pytest.raises(g.QmvError) as e:
        g.qmv_verify_run(FAKE, None, None, None, None, None, FAKE, FAKE, FAKE, None, 0, 0, 10, stream=0)
    assert e.value.code == 11 and "QMV_ERR_COUNT" in str(e.value)


# ------------------------------------------------------ the reference forms --
def test_reference_routing():
    ids, w = ref.route(np.array([1.0, 3.0, 3.0, math.nan]), 2, False)
    assert ids == [1, 2] and np.allclose(w, 0.5)
    _, w = ref.route(np.array([0.0, math.log(3.0)]), 1, True)
    assert np.allclose(w, 0.75)


def test_reference_verify():
    ln = math.log
    t = np.array([[[ln(0.5), ln(0.5), -math.inf], [ln(0.1), ln(0.2), ln(0.7)]]])
    d = np.array([[[ln(0.8), ln(0.2), -math.inf]]])
    args = dict(lens=[1], temp=np.array([1.0]), big=3e38)
    # accepted at u 0.8 < 0.5, refused above; what is left after a refusal is token 1 alone
    tok, n, lp, _ = ref.verify(t, d, np.array([[0]]), uniform=np.array([[0.6]]), noise=np.array([[1.0, 1.0, 1.0]]), **args)
    assert tok.tolist() == [[0, 2]] and n[0] == 1 and np.allclose(lp, [[ln(0.5), ln(0.7)]])
    tok, n, _, _ = ref.verify(t, d, np.array([[0]]), uniform=np.array([[0.7]]), noise=np.array([[1e-9, 1.0, 1.0]]), **args)
    assert tok.tolist() == [[1, -1]] and n[0] == 0
