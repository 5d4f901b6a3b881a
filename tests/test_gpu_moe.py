"""qmv_moe_run on the GPU: a whole mixture-of-experts layer over group-quantized
experts, against the 64-bit formula, with bounds carried through both products."""

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g
import operators_reference as ref
from gpu_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    g.load()


class Layer:
    def __init__(self, M, K, I, E, k, bits, gs, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.shape = (M, K, I, E, k, bits, gs)
        self.gu = [ref.Matrix(2 * I, K, bits, gs, seed * 1000 + 2 * e) for e in range(E)]
        self.dn = [ref.Matrix(K, I, bits, gs, seed * 1000 + 2 * e + 1) for e in range(E)]
        self.x = ref.to_bf16(rng.standard_normal((M, K)) * spread)
        self.router = ref.to_bf16(rng.standard_normal((E, K)) * 1.5 / np.sqrt(K))
        self.w = [dev(a) for ms in (self.gu, self.dn)
                  for a in (np.stack([g.qmv_pack(m.q, bits) for m in ms]), np.stack([m.scales for m in ms]),
                            np.stack([m.biases for m in ms]))]

    def run(self, rows=None, flags=0, x=None, router=None, routing=True, **kw):
        M, K, I, E, k, bits, gs = self.shape
        x = self.x if x is None else x
        rows = list(range(M)) if rows is None else rows
        n = len(rows)
        y = torch.full((n + 1, K), 7, dtype=torch.float32 if flags & g.F32_OUT else torch.bfloat16, device="cuda")
        ids = torch.full((n, k), -5, dtype=torch.int32, device="cuda")
        w = torch.full((n, k), -5, dtype=torch.float32, device="cuda")
        g.qmv_moe_run(dev(x[rows]), dev(self.router if router is None else router), *self.w, y, ids if routing else None,
                      w if routing else None, n, K, I, E, k, bits, gs, flags=flags, **kw)
        torch.cuda.synchronize()
        assert (y[-1] == 7).all(), "wrote past the last token"
        return y[:-1].float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy()

    def check(self, flags=0):
        M, K, I, E, k, bits, gs = self.shape
        y, err, ids, w, margin = ref.moe(ref.bf(self.x), ref.bf(self.router), self.gu, self.dn, I, k,
                                         bool(flags & g.MOE_GELU), bool(flags & g.MOE_SOFTMAX_ALL))
        # sqrt(K) roundings of the largest magnitude sum is more than K roundings of either sign add up to
        assert margin > 1, "the inputs leave the routing undecided"
        got, gi, gw = self.run(flags=flags | g.F32_OUT)
        assert np.array_equal(gi, ids)
        assert np.allclose(gw, w, rtol=2e-5, atol=1e-9)
        assert np.all(np.abs(got - y) <= err), float(np.max(np.abs(got - y) / err))
        # the bound is not slack beyond use: as a whole the result is much closer
        assert np.linalg.norm(got - y) <= 1e-4 * np.linalg.norm(y)
        got16, _, _ = self.run(flags=flags)
        assert np.all(np.abs(got16 - y) <= err + 2.0 ** -8 * np.abs(y))


# one expert, all experts, one group each way, odd group counts, more tokens
# than one tile for an expert, every weight form
SHAPES = [
    (1, 64, 64, 1, 1, 4, 64), (1, 128, 128, 4, 2, 2, 128), (2, 320, 192, 5, 5, 4, 64), (5, 640, 384, 8, 2, 2, 64),
    (8, 512, 256, 3, 2, 4, 128), (16, 1024, 448, 16, 4, 4, 64), (17, 384, 128, 2, 1, 2, 128), (33, 256, 320, 4, 3, 4, 64),
    (70, 192, 64, 3, 2, 4, 64), (3, 2048, 768, 12, 8, 4, 64), (1, 3840, 1920, 4, 2, 2, 128), (256, 128, 128, 7, 2, 2, 64),
    (4, 256, 128, 40, 32, 4, 64), (2, 1088, 1344, 4, 2, 2, 64),
]


@pytest.mark.parametrize("M,K,I,E,k,bits,gs", SHAPES)
def test_moe_matches_the_formula(M, K, I, E, k, bits, gs):
    Layer(M, K, I, E, k, bits, gs, seed=M + K + E).check()


@pytest.mark.parametrize("flags", [g.MOE_GELU, g.MOE_SOFTMAX_ALL, g.MOE_GELU | g.MOE_SOFTMAX_ALL])
def test_activation_and_weights(flags):
    Layer(6, 512, 320, 10, 3, 4, 64, seed=21).check(flags)


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_small_and_large_activations(spread):
    """Large ones saturate the activation and spread h over many orders of magnitude."""
    Layer(5, 512, 256, 6, 2, 4, 64, seed=22, spread=spread).check()


def test_equal_logits_take_the_lowest_expert():
    lay = Layer(3, 256, 64, 9, 4, 4, 64, seed=23)
    r = lay.router.copy()
    r[5] = r[2]
    r[8] = r[2]
    r[7] = r[0]
    _, ids, w = lay.run(router=r)
    l = ref.bf(lay.x) @ ref.bf(r).T
    for m in range(3):
        assert list(ids[m]) == sorted(range(9), key=lambda e: (-l[m, e], e))[:4]
    _, ids, w = lay.run(router=np.zeros_like(r))
    assert (ids == np.arange(4)).all() and np.allclose(w, 0.25)


def test_nan_logits_are_never_chosen_before_numbers():
    lay = Layer(2, 256, 64, 6, 3, 4, 64, seed=24)
    r = lay.router.copy()
    r[1] = 0x7fc0
    r[4] = 0x7fc0
    y, ids, w = lay.run(router=r)
    assert not np.isin(ids, (1, 4)).any() and np.isfinite(w).all() and np.isfinite(y).all()


def test_one_expert_for_all_tokens():
    """All tokens on one expert: more tokens than a tile, every other expert empty."""
    lay = Layer(40, 256, 128, 6, 1, 4, 64, seed=25)
    x = np.abs(ref.bf(lay.x))
    lay.x = ref.to_bf16(x)
    r = np.zeros((6, 256))
    r[3] = 1.0 / 16
    lay.router = ref.to_bf16(r)
    lay.check()


@pytest.mark.parametrize("bits,gs", [(4, 64), (2, 128)])
def test_a_token_does_not_depend_on_its_batch(bits, gs):
    lay = Layer(21, 640, 256, 6, 2, bits, gs, seed=26)
    full, ids, w = lay.run(flags=g.F32_OUT)
    for rows in ([0], [20], [3, 2], list(range(4, 13)), list(range(20, 2, -1))):
        y, i, ww = lay.run(rows, flags=g.F32_OUT)
        assert np.array_equal(y, full[rows]) and np.array_equal(i, ids[rows]) and np.array_equal(ww, w[rows])


def test_routing_outputs_are_optional_and_runs_repeat():
    lay = Layer(7, 512, 192, 8, 3, 4, 64, seed=27)
    want, _, _ = lay.run(flags=g.F32_OUT)
    M, K, I, E, k, bits, gs = lay.shape
    need = g.qmv_moe_workspace_size(M, K, I, E, k, bits, gs)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(4):
            y, _, _ = lay.run(flags=g.F32_OUT, routing=False, workspace=ws, workspace_bytes=need, stream=st)
            assert np.array_equal(y, want)
    assert torch.isnan(ws[need // 4:]).all(), "wrote past the workspace"
    with pytest.raises(g.QmvError) as e:
        lay.run(workspace=ws, workspace_bytes=need - 1)
    assert e.value.code == 8
    assert g.qmv_device_error() == 0


def test_capture_in_a_graph():
    lay = Layer(3, 512, 256, 8, 2, 4, 64, seed=28)
    M, K, I, E, k, bits, gs = lay.shape
    want, _, _ = lay.run()
    x, r = dev(lay.x), dev(lay.router)
    y = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    need = g.qmv_moe_workspace_size(M, K, I, E, k, bits, gs)
    ws = torch.empty(need // 4 + 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.qmv_moe_run(x, r, *lay.w, y, None, None, M, K, I, E, k, bits, gs, workspace=ws, workspace_bytes=need)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(want, y.float().cpu().numpy())


@pytest.mark.parametrize("M,E,k,bits", [(256, 1024, 16, 4), (256, 3, 1, 2), (128, 1024, 32, 4)])
def test_the_most_choices(M, E, k, bits):
    """As many choices as a call takes, over few and over the most experts: the lists
    fill shared memory. Tokens alone and in a small batch give the same rows."""
    lay = Layer(M, 64, 64, E, k, bits, 64, seed=29)
    full, ids, _ = lay.run(flags=g.F32_OUT)
    assert np.isfinite(full).all()
    for rows in ([0], [M - 1], [M // 2, 1, 7, 64]):
        got, got_ids, _ = lay.run(rows, flags=g.F32_OUT)
        assert np.array_equal(got, full[rows]) and np.array_equal(got_ids, ids[rows])
