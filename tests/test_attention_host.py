"""Refusals of an attention layer's operators, which all happen on the host before a
GPU is touched, and the 64-bit reference forms against hand-worked values."""

import math

import numpy as np
import pytest
import torch

import attention_reference as ref
import group_quantized_mat_gb300 as g
from test_operators_host import FAKE, call, lib  # noqa: F401

ROPE = (["qkv", "q_norm", "k_norm", "positions", "inv_freq", "axis", "slots", "q", "k_cache", "v_cache"],
        dict(T=3, heads=8, kv_heads=2, head_dim=128, rope_dim=128, page_size=16, pages=4, axes=2, eps=1e-6, ld_qkv=12 * 128,
             page_stride=16 * 256, token_stride=256, head_stride=128))


def rope(lib, kw):  # noqa: F811
    vals = {**{p: FAKE for p in ROPE[0]}, **ROPE[1], "flags": 0, "stream": None}
    assert set(kw) <= set(vals), kw
    vals.update(kw)
    return lib.qmv_rope_run(*vals.values())


@pytest.mark.parametrize("kw,code", [
    *[({p: None}, 1) for p in ("qkv", "positions", "inv_freq", "q", "k_cache", "v_cache")],
    (dict(T=0), 11), (dict(T=(1 << 22) + 1), 11), (dict(heads=0), 11), (dict(heads=9), 11), (dict(kv_heads=0), 11), (dict(kv_heads=257, heads=257), 11),
    (dict(heads=130, kv_heads=2), 11), (dict(T=1 << 22, heads=512, kv_heads=256), 11), (dict(axes=0), 11), (dict(axes=5), 11),
    (dict(head_dim=96), 4), (dict(head_dim=0), 4), (dict(rope_dim=-16), 4), (dict(rope_dim=144), 4), (dict(rope_dim=24), 4),
    (dict(eps=-1.0), 4), (dict(eps=math.nan), 4), (dict(eps=math.inf), 4), (dict(ld_qkv=12 * 128 - 8), 4), (dict(ld_qkv=12 * 128 + 4), 4),
    (dict(page_size=0), 4), (dict(page_size=4), 4), (dict(page_size=12), 4), (dict(page_size=65544), 4), (dict(pages=0), 4),
    (dict(token_stride=64), 4), (dict(token_stride=260), 4), (dict(head_stride=0), 4), (dict(head_stride=-128), 4), (dict(page_stride=16 * 256 - 8), 4),
    (dict(token_stride=1 << 39), 4), (dict(page_stride=1 << 47), 4), (dict(token_stride=128), 4),
    (dict(flags=1), 10), (dict(flags=0x400), 10),
    *[({p: FAKE + 8}, 6) for p in ("qkv", "q_norm", "k_norm", "q", "k_cache", "v_cache")],
    (dict(positions=FAKE + 2), 6), (dict(inv_freq=FAKE + 2), 6), (dict(slots=FAKE + 4), 6),
])
def test_rope_refusals(lib, kw, code):  # noqa: F811
    assert rope(lib, kw) == code


ATTEND = (["q", "k_cache", "v_cache", "page_table", "q_start", "kv_len", "out", "lse"],
          dict(B=2, T=6, max_new=3, heads=8, kv_heads=2, head_dim=128, page_size=16, pages=4, max_pages=2, scale=0.1, window=0, sinks=0,
               ld_q=1024, ld_out=1024, page_stride=16 * 256, token_stride=256, head_stride=128))


@pytest.mark.parametrize("kw,code", [
    *[({p: None}, 1) for p in ATTEND[0][:4] + ATTEND[0][5:7]],
    (dict(B=0), 11), (dict(B=1025), 11), (dict(T=0), 11), (dict(max_new=0), 11), (dict(max_new=7), 11), (dict(heads=7), 11), (dict(kv_heads=0), 11),
    (dict(heads=260, ld_q=1 << 20), 11), (dict(q_start=None, T=5), 11),
    (dict(head_dim=32), 4), (dict(page_size=20), 4), (dict(page_size=7), 4), (dict(pages=0), 4), (dict(max_pages=0), 4), (dict(max_pages=(1 << 22) + 1), 4),
    (dict(scale=math.nan), 4), (dict(scale=math.inf), 4), (dict(window=-1), 4), (dict(sinks=-1), 4), (dict(window=(1 << 30) + 1), 4),
    (dict(ld_q=1023), 4), (dict(ld_q=1028), 4), (dict(ld_out=1016), 4), (dict(page_stride=128), 4), (dict(head_stride=132), 4),
    (dict(flags=1), 10), *[({p: FAKE + 8}, 6) for p in ("q", "k_cache", "v_cache", "out", "workspace")],
    *[({p: FAKE + 2}, 6) for p in ("page_table", "q_start", "kv_len", "lse")],
])
def test_attend_refusals(lib, kw, code):  # noqa: F811
    assert call(lib, "qmv_attend_run", *ATTEND, kw) == code


def test_attend_workspace_size(lib):  # noqa: F811
    size = g.qmv_attend_workspace_size
    assert size(1, 1, 1, 8, 2, 128, 16, 4) > 0
    assert size(0, 1, 1, 8, 2, 128, 16, 4) == 0 and size(1, 1, 2, 8, 2, 128, 16, 4) == 0 and size(1, 1, 1, 8, 3, 128, 16, 4) == 0
    sizes = [size(B, 4 * B, 4, 8, 2, 128, 16, 500) for B in (1, 2, 64, 1000)]
    assert sizes == sorted(sizes)
    assert size(4, 16, 4, 8, 2, 128, 64, 2000, 1024, 4) <= size(4, 16, 4, 8, 2, 128, 64, 2000)


# ------------------------------------------------------ the reference forms --
def test_reference_rope():
    x = np.zeros((1, 3, 4))
    x[0, 0] = [3.0, 0.0, 4.0, 0.0]
    x[0, 1] = [0.0, 2.0, 0.0, 0.0]
    x[0, 2] = [1.0, 2.0, 3.0, 4.0]
    pos, freq = np.array([[1], [2]]), np.array([math.pi / 2, math.pi / 4])
    (q, k, v), _ = ref.rope(x, None, np.ones(4), pos, freq, None, 1, 1, 0.0, 0.0, False)
    assert np.allclose(q, [[[-4.0, 0.0, 3.0, 0.0]]]) and np.allclose(k, [[[0.0, math.sqrt(2), 0.0, math.sqrt(2)]]]) and (v == x[:, 2:]).all()
    (q, _, _), _ = ref.rope(x, None, None, pos, freq, np.array([1, 1]), 1, 1, 0.0, 0.0, True)
    assert np.allclose(q, [[[-3.0, 0.0, 0.0, 4.0]]])


def test_reference_attend():
    k = torch.zeros(3, 8, 1, 2, dtype=torch.float64)
    v = torch.arange(24, dtype=torch.float64).view(3, 8, 1, 1).expand(3, 8, 1, 2).clone()
    k[2, 0] = math.log(3.0)  # key 8 of the sequence, whose pages are 0 and 2
    q = torch.tensor([[[1.0, 0.0]]] * 2, dtype=torch.float64)
    args = (q, k, v, [[0, 2]], [0, 2], [9], 1, 1.0)
    out, lse, _, _ = ref.attend(*args)
    assert torch.allclose(out[:, 0, 0], torch.tensor([3.5, (28 + 3 * 16) / 11], dtype=torch.float64))
    assert torch.allclose(lse[:, 0], torch.tensor([math.log(8), math.log(11)], dtype=torch.float64))
    out, _, _, _ = ref.attend(*args, window=2, sinks=1)
    assert torch.allclose(out[:, 0, 0], torch.tensor([(0 + 6 + 7) / 3, (0 + 7 + 3 * 16) / 5], dtype=torch.float64))
    out, lse, _, _ = ref.attend(q, k, v, [[0, 2]], [0, 2], [1], 1, 1.0)
    assert out[0, 0, 0] == 0 and lse[0, 0] == -math.inf and lse[1, 0] == 0
