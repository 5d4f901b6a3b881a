"""More of qmv_verify_run on the GPU against the 64-bit rule: what test_gpu_verify leaves out."""

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g
from test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    g.load()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("draft", [True, False])
def test_the_smallest_temperatures(dtype, draft):
    """Above 0 every temperature samples, in the limit the argmax."""
    b = Batch(8, 3, 900, dtype, draft=draft, seed=31, lens=[3] * 8)
    b.temp[:] = np.array([1e-30, 1e-37, 1e-38, 4.2e-39, 2.9e-39, 1e-40, 1e-42, 1e-45], dtype=np.float32)
    assert (b.temp > 0).all()
    best = np.argmax(b.target, -1)
    b.tokens[:, 0] = best[:, 0]
    if draft:
        b.draft[:, 0] = b.target[:, 0]
    out, acc, lp = b.check()
    assert (acc >= 1).all() and (out[:, 0] == best[:, 0]).all() and (lp[:, 0] == 0).all()


def part(b, rows):
    """The sequences `rows` of a batch alone."""
    c = object.__new__(Batch)
    c.__dict__.update(b.__dict__)
    c.B = len(rows)
    for name in ("target", "draft", "tokens", "lens", "temp", "uniform", "noise"):
        v = getattr(b, name)
        setattr(c, name, None if v is None else v[rows].copy())
    return c


@pytest.mark.parametrize("B,S,V,dtype,draft,pad", [(37, 4, 5003, "bf16", True, 0), (24, 3, 4099, "f32", True, 5),
                                                   (600, 2, 2111, "bf16", True, 1), (19, 5, 40001, "bf16", False, 3)])
def test_a_sequence_does_not_depend_on_its_batch(B, S, V, dtype, draft, pad):
    """Bit for bit, log-probabilities too, however the batch splits a sequence's race over
    blocks and wherever its rows lie."""
    b = Batch(B, S, V, dtype, pad=pad, draft=draft, greedy=0.3, seed=B + V)
    full = b.run()
    for rows in ([0], [B - 1], [B // 2, 1], list(range(min(B, 9)))[::-1]):
        for got, want in zip(part(b, rows).run(), full):
            assert np.array_equal(got, want[rows]), rows


@pytest.mark.parametrize("B,S,V,dtype,draft", [(2, 3, 262144, "bf16", True), (3, 1, 262147, "f32", True), (1, 2, 1 << 20, "bf16", False)])
def test_vocabularies_above_any_tested(B, S, V, dtype, draft):
    Batch(B, S, V, dtype, draft=draft, seed=V % 97).check()


def test_the_largest_vocabulary():
    """2^24 tokens, fp32, two certain ones: the last of the row, and after it the first."""
    V = 1 << 24
    target = torch.zeros((1, 2, V), device="cuda")
    target[0, 0, V - 1] = 200.0
    target[0, 1, 0] = 200.0
    out = torch.full((1, 2), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((1, 2), 7.0, device="cuda")
    drafted = torch.tensor([[V - 1]], dtype=torch.int32, device="cuda")
    g.qmv_verify_run(target, None, drafted, None, None, torch.full((1, 1), 0.5, device="cuda"), torch.ones((1, V), device="cuda"),
                     out, acc, lp, 1, 1, V, flags=g.VERIFY_F32_LOGITS)
    torch.cuda.synchronize()
    assert out.tolist() == [[V - 1, 0]] and acc.tolist() == [1] and lp.tolist() == [[0.0, 0.0]]
