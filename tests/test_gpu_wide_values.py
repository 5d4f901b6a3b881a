"""The operators over packed weights at the ends of the number range: vectors, and the
experts' inner values, up to bf16's and fp32's largest and down to subnormal numbers.
Bounds are operators_reference's, relative to the sums of magnitudes."""

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g
import operators_reference as ref
from gpu_helpers import dev
from test_gpu_lora import Problem
from test_gpu_moe import Layer

pytestmark = pytest.mark.gpu

MAX = ref.bf(np.array([0x7f7f], dtype=np.uint16))[0]  # bf16's largest


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    g.load()


def rescale(m, factor):
    """The matrix times a power of two."""
    m.scales, m.biases = ref.to_bf16(ref.bf(m.scales) * factor), ref.to_bf16(ref.bf(m.biases) * factor)
    m.w, m.mag = m.w * factor, m.mag * factor


def lora_problem(x, bits, gs, factor):
    M, K = x.shape
    pr = Problem(M, 70, K, bits, gs, 2, 8, ids=[-1] * M, seed=bits + gs)
    rescale(pr.m, factor)
    pr.x = ref.to_bf16(x)
    pr.dev = [pr.dev[0], dev(pr.m.scales), dev(pr.m.biases)]
    return pr


@pytest.mark.parametrize("bits,gs", [(4, 64), (4, 128), (2, 64), (2, 128)])
def test_vectors_up_to_the_largest_number(bits, gs):
    """Weights of about 2^-35: no result overflows, though sums of q x and of x do."""
    K = 640
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, K))
    x[0, 5] = 1.5 * 2.0 ** 126
    x[1, 70] = -1.75 * 2.0 ** 127
    x[2] = MAX
    x[3] = MAX * rng.choice([-1, 1], K)
    x[4, 64:128] = -MAX
    x[5] *= 2.0 ** 125
    x[6, ::2] *= 2.0 ** 124
    pr = lora_problem(x, bits, gs, 2.0 ** -30)
    y, err = pr.m.product(ref.bf(pr.x))
    assert np.abs(y).max() < 2.0 ** 120
    got = pr.run(flags=g.F32_OUT)
    assert np.all(np.abs(got - y) <= err), float(np.max(np.abs(got - y) / err))


@pytest.mark.parametrize("bits,gs", [(4, 64), (2, 128)])
def test_vectors_down_to_the_smallest_number(bits, gs):
    K = 640
    rng = np.random.default_rng(2)
    tiny = 2.0 ** -133  # bf16's smallest
    x = rng.integers(-200, 201, (4, K)) * tiny
    x[1] = 0.0
    x[1, 9] = tiny
    x[2] = rng.standard_normal(K) * 2.0 ** -120
    x[3, 64:128] = rng.standard_normal(64)
    pr = lora_problem(x, bits, gs, 2.0 ** 40)
    y, err = pr.m.product(ref.bf(pr.x))
    got = pr.run(flags=g.F32_OUT)
    assert np.all(np.abs(got - y) <= err + 2.0 ** -130), float(np.max(np.abs(got - y) / (err + 2.0 ** -130)))
    assert np.abs(got[1]).max() > 0


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_vector_that_is_no_number_gives_nan_and_leaves_the_others(bad):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 512))
    pr = lora_problem(x, 4, 64, 1.0)
    clean = pr.run(flags=g.F32_OUT)
    x[2, 100] = bad
    pr.x = ref.to_bf16(x)
    got = pr.run(flags=g.F32_OUT)
    keep = [0, 1, 3, 4]
    assert np.array_equal(got[keep], clean[keep]) and np.isnan(got[2]).all()


@pytest.mark.parametrize("bits,gs", [(4, 64), (2, 128)])
@pytest.mark.parametrize("gelu", [False, True])
def test_inner_values_up_to_the_largest_number(bits, gs, gelu):
    """h = act(gate x) (up x) whose largest is in fp32's highest binades."""
    lay = Layer(3, 256, 256, 2, 2, bits, gs, seed=31)
    h = 0.0
    for m in lay.gu:
        r = ref.bf(lay.x) @ m.w.T
        h = max(h, float((np.maximum(r[:, :256], 0) * np.abs(r[:, 256:])).max()))
    top = 2 * int(np.floor((127.9 - np.log2(h)) / 2))  # twice a whole power for gate and up
    for m in lay.gu:
        rescale(m, 2.0 ** (top // 2))
    for m in lay.dn:
        rescale(m, 2.0 ** -40)
    assert 2.0 ** 125.9 <= h * 2.0 ** top < 2.0 ** 128
    for i, ms in ((0, lay.gu), (3, lay.dn)):
        lay.w[i + 1], lay.w[i + 2] = dev(np.stack([m.scales for m in ms])), dev(np.stack([m.biases for m in ms]))
    with np.errstate(over="ignore"):
        y, err, _, _, _ = ref.moe(ref.bf(lay.x), ref.bf(lay.router), lay.gu, lay.dn, 256, 2, gelu, False)
    got, _, _ = lay.run(flags=g.F32_OUT | (g.MOE_GELU if gelu else 0))
    assert np.all(np.abs(got - y) <= err), float(np.max(np.abs(got - y) / err))
    assert np.linalg.norm(got - y) <= 1e-4 * np.linalg.norm(y)


def test_tokens_up_to_the_largest_number():
    """x of bf16's largest through all three products (equal logits: no router weight)."""
    lay = Layer(4, 320, 128, 3, 2, 4, 64, seed=32)
    x = ref.bf(lay.x)
    x[0, 3] = MAX
    x[1] = MAX * np.sign(x[1] + 1e-9)
    x[2] *= 2.0 ** 124
    lay.x, lay.router = ref.to_bf16(x), np.zeros_like(lay.router)
    for m in lay.gu:
        rescale(m, 2.0 ** -100)
    lay.w[1], lay.w[2] = dev(np.stack([m.scales for m in lay.gu])), dev(np.stack([m.biases for m in lay.gu]))
    with np.errstate(over="ignore"):
        y, err, ids, _, _ = ref.moe(ref.bf(lay.x), ref.bf(lay.router), lay.gu, lay.dn, 128, 2, False, False)
    got, gi, _ = lay.run(flags=g.F32_OUT)
    assert np.array_equal(gi, ids)
    # (of the last token, whose x is small, h falls below the least number)
    assert np.all(np.abs(got - y) <= err + 2.0 ** -130), float(np.max(np.abs(got - y) / (err + 2.0 ** -130)))


@pytest.mark.parametrize("bits,gs", [(4, 64), (4, 128), (2, 64), (2, 128)])
@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_sums_of_exact_products_are_exact(M, bits, gs):
    """Scales 1, biases 0, whole numbers: every sum is a whole number below 2^24, though a
    group's terms lie up to 2^21 apart, so any bit that an accumulator dropped would show."""
    K = 256
    pr = Problem(M, 150, K, bits, gs, 1, 8, ids=[-1] * M, seed=M)
    rng = np.random.default_rng(M + bits)
    x = rng.integers(-255, 256, (M, K)).astype(np.float64)
    for m in range(M):
        for sub in range(0, K, 64):
            x[m, sub + 2 * rng.integers(32)] = rng.choice([-1, 1]) * 2.0 ** 17
    pr.x = ref.to_bf16(x)
    pr.m.scales, pr.m.biases = np.full_like(pr.m.scales, 0x3f80), np.zeros_like(pr.m.biases)
    pr.dev = [pr.dev[0], dev(pr.m.scales), dev(pr.m.biases)]
    want = x @ pr.m.q.astype(np.float64).T
    assert np.abs(x).max() == 2.0 ** 17 and np.abs(want).max() < 2 ** 24
    assert np.array_equal(pr.run(flags=g.F32_OUT), want)


@pytest.mark.parametrize("M,K,I,E,k,bits,gs,gelu", [(3, 1024, 14336, 2, 1, 4, 64, False), (9, 4096, 2048, 3, 2, 4, 128, True),
                                                    (2, 65536, 64, 2, 1, 2, 64, False), (2, 64, 65536, 2, 2, 2, 64, True),
                                                    (40, 128, 14336, 2, 1, 2, 128, False)])
def test_experts_wider_than_any_other_test(M, K, I, E, k, bits, gs, gelu):
    Layer(M, K, I, E, k, bits, gs, seed=M + E).check(g.MOE_GELU if gelu else 0)
