"""qmv_lora_run over projections of full width: more vectors than a pass serves, so that
a CTA goes through several, and rings of three slots. Against the 64-bit formula, with
the bounds of operators_reference, formed on the GPU."""

import functools

import pytest
import torch

import group_quantized_mat_gb300 as g
from lora_shapes import FEW_SLOTS, PASSES, THREE_SLOTS
from operators_reference import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    g.load()


@functools.lru_cache(maxsize=1)
def weights(N, K, bits, gs):
    """Packed words, scales, biases; the matrix and the sum of its terms' magnitudes in 64 bits."""
    gen = torch.Generator("cuda").manual_seed(N + K + bits + gs)
    w = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=gen, device="cuda", dtype=torch.int64).int()
    s = (torch.rand((N, K // gs), generator=gen, device="cuda") * 0.02 + 0.001).bfloat16()
    b = (-(2 ** (bits - 1) - 0.5) * s.float() + 1e-3 * torch.randn(s.shape, generator=gen, device="cuda")).bfloat16()
    shifts = torch.arange(0, 32, bits, device="cuda", dtype=torch.int32)
    q = ((w.unsqueeze(-1) >> shifts) & (2 ** bits - 1)).reshape(N, K // gs, gs).double()
    sq, bb = s.double().unsqueeze(-1) * q, b.double().unsqueeze(-1)
    return w, s, b, (sq + bb).view(N, K), (sq.abs() + bb.abs()).view(N, K)


def problem(M, N, K, bits, gs, R, adapters=6):
    gen = torch.Generator("cuda").manual_seed(M + R)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    x, a, b = randn(M, K).bfloat16(), (randn(adapters, R, K) / K ** 0.5).bfloat16(), (randn(adapters, N, R) * 0.5).bfloat16()
    ids = torch.randint(-1, adapters, (M,), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.rand((adapters,), generator=gen, device="cuda") * 1.5 + 0.5
    return x, a, b, ids, c


def run(wsb, x, a, b, ids, c, shape):
    M, N, K, bits, gs, R = shape
    y = torch.full((M + 1, N), 7.0, device="cuda")
    g.qmv_lora_run(*wsb, x, a, b, ids, c, y, M, N, K, bits, gs, len(c), R, flags=g.F32_OUT)
    torch.cuda.synchronize()
    assert g.qmv_device_error() == 0
    assert (y[-1] == 7).all(), "wrote past the last vector"
    return y[:-1]


def expect(shape, wide, mag, x, a, b, ids, c):
    M, N, K, bits, gs, R = shape
    x = x.double()
    y, err = x @ wide.T, (20 + 2 * (K // gs) + 32) * U * (x.abs() @ mag.T)
    for m, ad in enumerate(ids.tolist()):
        if ad >= 0:
            aa, bb, cc = a[ad].double(), b[ad].double(), float(c[ad])
            v = aa @ x[m]
            verr = (K + 2) * U * (aa.abs() @ x[m].abs())
            y[m] += cc * (bb @ v)
            err[m] += cc * (bb.abs() @ (verr + (R + 4) * U * v.abs())) + 4 * U * y[m].abs()
    return y, err


@pytest.mark.parametrize("shape", sorted(PASSES, key=lambda s: s[1:]) + THREE_SLOTS + FEW_SLOTS, ids=lambda s: "x".join(map(str, s)))
def test_passes_match_the_formula(shape):
    M, N, K, bits, gs, R = shape
    w, s, b, wide, mag = weights(N, K, bits, gs)
    p = problem(M, N, K, bits, gs, R)
    got = run((w, s, b), *p, shape)
    y, err = expect(shape, wide, mag, *p)
    assert bool((((got - y).abs() <= err).all())), float(((got - y).abs() / err).max())
    # the bound allows every rounding the worst sign: as a whole the result is much closer
    assert float((got - y).norm()) <= 3e-6 * float(y.norm())
    # a vector's result is that of a call with it alone, whichever pass it is in
    for m in {0, M // 2, M - 1}:
        x, a, bb, ids, c = p
        assert torch.equal(run((w, s, b), x[m:m + 1].contiguous(), a, bb, ids[m:m + 1].contiguous(), c, (1, *shape[1:]))[0], got[m]), m


@pytest.mark.parametrize("R", [16, 24, 72, 128, 200])
def test_rows_do_not_depend_on_the_tiles_they_are_in(R):
    """The first rows of a larger matrix, whose tiles are higher, give the same bits."""
    M, N, K, more = 5, 1000, 1024, 5000
    w, s, b, _, _ = weights(more, K, 4, 64)
    x, a, bb, ids, c = problem(M, more, K, 4, 64, R)
    ids.copy_(torch.arange(M) % 3)
    large = run((w, s, b), x, a, bb, ids, c, (M, more, K, 4, 64, R))
    small = run((w[:N].contiguous(), s[:N].contiguous(), b[:N].contiguous()), x, a, bb[:, :N].contiguous(), ids, c, (M, N, K, 4, 64, R))
    assert torch.equal(large[:, :N], small)
