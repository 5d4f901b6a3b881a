"""qmv_lora_run on the GPU: a shared projection with each vector's own low-rank
adapter, against the 64-bit formula, with bounds from the fp32 arithmetic."""

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


class Problem:
    def __init__(self, M, N, K, bits, gs, L, R, ids=None, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.shape = (M, N, K, bits, gs, L, R)
        self.m = ref.Matrix(N, K, bits, gs, seed)
        self.x = ref.to_bf16(rng.standard_normal((M, K)) * spread ** rng.uniform(-1, 1, (M, 1)))
        self.a = ref.to_bf16(rng.standard_normal((L, R, K)) / np.sqrt(K))
        self.b = ref.to_bf16(rng.standard_normal((L, N, R)) * 0.5)
        self.ids = np.asarray(rng.integers(-1, L, M) if ids is None else ids, dtype=np.int32)
        self.c = rng.uniform(0.5, 2.0, L).astype(np.float32)
        self.dev = [dev(g.qmv_pack(self.m.q, bits)), dev(self.m.scales), dev(self.m.biases)]
        self.dev2 = [dev(self.a), dev(self.b)]
        self.dc = torch.from_numpy(self.c).cuda()

    def run(self, rows=None, flags=0, **kw):
        M, N, K, bits, gs, L, R = self.shape
        rows = list(range(M)) if rows is None else rows
        x, ids = dev(self.x[rows]), torch.from_numpy(self.ids[rows]).cuda()
        f32 = bool(flags & g.F32_OUT)
        y = torch.full((len(rows) + 1, N), 7, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        g.qmv_lora_run(*self.dev, x, *self.dev2, ids, self.dc, y, len(rows), N, K, bits, gs, L, R, flags=flags, **kw)
        torch.cuda.synchronize()
        assert (y[-1] == 7).all(), "wrote past the last vector"
        return y[:-1].float().cpu().numpy()

    def expect(self):
        return ref.lora(self.m, ref.bf(self.x), ref.bf(self.a), ref.bf(self.b), self.ids, self.c.astype(np.float64))

    def check(self):
        y, err = self.expect()
        got32, got16 = self.run(flags=g.F32_OUT), self.run()
        assert np.all(np.abs(got32 - y) <= err), float(np.max(np.abs(got32 - y) / err))
        assert np.all(np.abs(got16 - y) <= err + 2.0 ** -8 * np.abs(y))
        return got32


# one group of K; one row; rows that end inside a tile; every weight form; odd
# ranks; more vectors than one tile of them; long K
SHAPES = [
    (1, 1, 64, 4, 64, 1, 1), (1, 17, 128, 2, 128, 2, 3), (2, 16, 192, 4, 64, 2, 16), (3, 250, 1088, 4, 64, 3, 8),
    (8, 33, 2048, 2, 64, 4, 27), (9, 100, 3840, 4, 128, 4, 64), (16, 257, 1024, 2, 128, 5, 16),
    (17, 40, 5120, 4, 64, 16, 32), (33, 130, 960, 2, 64, 3, 5), (65, 48, 640, 4, 64, 7, 12), (13, 64, 15360, 4, 64, 4, 16),
    (5, 31, 17408, 2, 128, 2, 256), (256, 20, 256, 4, 128, 9, 7), (1, 15360, 3840, 4, 64, 8, 16),
]


@pytest.mark.parametrize("M,N,K,bits,gs,L,R", SHAPES)
def test_lora_matches_the_formula(M, N, K, bits, gs, L, R):
    Problem(M, N, K, bits, gs, L, R, seed=M + N + K).check()


@pytest.mark.parametrize("M,bits,gs", [(1, 4, 64), (7, 2, 64), (16, 4, 128), (40, 4, 64)])
def test_no_adapter_is_the_projection_alone(M, bits, gs):
    """Ids below 0 and from the adapter count on mean none, whatever the adapters hold."""
    pr = Problem(M, 70, 1280, bits, gs, 3, 16, ids=[(-1, 3, -2 ** 31, 2 ** 31 - 1)[i % 4] for i in range(M)], seed=5)
    y, err = pr.m.product(ref.bf(pr.x))
    assert np.all(np.abs(pr.run(flags=g.F32_OUT) - y) <= err)
    clean = pr.run(flags=g.F32_OUT)
    for t in pr.dev2:
        t.fill_(0x7fc0)  # NaN
    assert np.array_equal(clean, pr.run(flags=g.F32_OUT))


def test_adapters_of_other_vectors_do_not_leak():
    """A NaN adapter touches only its own vectors."""
    pr = Problem(12, 64, 640, 4, 64, 3, 8, ids=[0, 1, 2, -1] * 3, seed=6)
    clean = pr.run(flags=g.F32_OUT)
    pr.dev2[0][1].fill_(0x7fc0)
    got = pr.run(flags=g.F32_OUT)
    keep = pr.ids != 1
    assert np.array_equal(clean[keep], got[keep]) and np.isnan(got[~keep]).all()


@pytest.mark.parametrize("bits,gs", [(4, 64), (4, 128), (2, 64), (2, 128)])
def test_a_vector_does_not_depend_on_its_batch(bits, gs):
    """Every row of a batch equals the call on that row alone, and on other subsets, bit for bit."""
    pr = Problem(37, 96, 3840, bits, gs, 5, 24, seed=7)
    full = pr.run(flags=g.F32_OUT)
    for rows in ([0], [36], [8, 1], [5, 3, 4, 2], list(range(20, 29)), list(range(16, 0, -1))):
        assert np.array_equal(pr.run(rows, flags=g.F32_OUT), full[rows]), rows


@pytest.mark.parametrize("bits", [4, 2])
def test_wide_ranges_of_x(bits):
    """Vectors of very different size, elements of very different size in one group, zeros, a zero vector."""
    pr = Problem(10, 48, 1280, bits, 64, 2, 8, seed=8, spread=1e9)
    x = ref.bf(pr.x)
    x[1] = 0.0
    x[2, ::3] *= 2.0 ** -60
    x[3, :64] = 0.0
    x[4, 5] = 2.0 ** 100
    x[6] *= 2.0 ** -80
    pr.x = ref.to_bf16(x)
    got = pr.check()
    assert np.all(got[1] == 0)


def test_inputs_on_another_stream_and_own_workspace():
    pr = Problem(6, 200, 3840, 4, 64, 4, 16, seed=9)
    want = pr.run(flags=g.F32_OUT)
    M, N, K, bits, gs, L, R = pr.shape
    need = g.qmv_lora_workspace_size(M, N, K, bits, gs, R)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            assert np.array_equal(want, pr.run(flags=g.F32_OUT, workspace=ws, workspace_bytes=need, stream=st))
    assert torch.isnan(ws[need // 4:]).all(), "wrote past the workspace"
    with pytest.raises(g.QmvError) as e:
        pr.run(workspace=ws, workspace_bytes=need - 1)
    assert e.value.code == 8


def test_capture_in_a_graph():
    pr = Problem(4, 512, 2048, 4, 64, 4, 16, seed=10)
    want = pr.run()
    M, N, K, bits, gs, L, R = pr.shape
    x, ids = dev(pr.x), torch.from_numpy(pr.ids).cuda()
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    need = g.qmv_lora_workspace_size(M, N, K, bits, gs, R)
    ws = torch.empty(need // 4 + 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.qmv_lora_run(*pr.dev, x, *pr.dev2, ids, pr.dc, y, M, N, K, bits, gs, L, R, workspace=ws, workspace_bytes=need)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(want, y.float().cpu().numpy())
    assert g.qmv_device_error() == 0


def test_few_ring_slots():
    """The widest range of K with 16 vectors and the highest rank leaves room for
    two slots of weights: a single vector's call, which has more, gives the same rows."""
    pr = Problem(16, 17408, 4096, 4, 64, 2, 256, ids=[0, -1, 1, 1] * 4, seed=11)
    full = pr.run(flags=g.F32_OUT)
    assert np.isfinite(full).all()
    for row in (0, 5, 15):
        assert np.array_equal(pr.run([row], flags=g.F32_OUT)[0], full[row])


@pytest.mark.parametrize("N,R", [(19, 3), (23, 1), (130, 27), (77, 254), (1201, 13), (8, 255)])
def test_adapters_whose_rows_start_anywhere(N, R):
    """Odd ranks and row counts: pieces of an adapter off 16-byte boundaries, and the array's last bytes."""
    Problem(6, N, 320, 4, 64, 3, R, ids=[2, 0, 1, 2, -1, 0], seed=N + R).check()


@pytest.mark.parametrize("M,N,K,bits,gs,R", [(40, 20008, 4224, 4, 64, 27), (200, 19992, 1344, 2, 64, 64), (33, 20000, 5120, 2, 128, 200)])
def test_passes_over_several_tiles(M, N, K, bits, gs, R):
    """More vectors than a pass and more rows than a round of tiles, over one range of
    K and several: the same rows as single vectors, and on another run."""
    pr = Problem(M, N, K, bits, gs, 7, R, seed=12)
    full = pr.run(flags=g.F32_OUT)
    assert np.isfinite(full).all()
    for row in (0, 16, M - 1):
        assert np.array_equal(pr.run([row], flags=g.F32_OUT)[0], full[row])
    assert np.array_equal(pr.run(flags=g.F32_OUT), full)
