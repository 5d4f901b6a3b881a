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
