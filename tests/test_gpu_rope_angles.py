"""Angles of qmv_rope_run at frequencies of any size and sign, against turns in 60 decimal digits."""

import decimal
import math

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g
from test_gpu_rope import lib  # noqa: F401

pytestmark = pytest.mark.gpu

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def angles(positions, freq):
    """positions * freq modulo a turn, in radians: the product is exact, as is its remainder to some 40 digits."""
    with decimal.localcontext() as c:
        c.prec = 70
        turns = [[decimal.Decimal(p) * decimal.Decimal(f) / (2 * PI) for f in freq] for p in positions]
        return np.array([[float((t - t.to_integral_value(decimal.ROUND_FLOOR)) * 2 * PI) for t in row] for row in turns])


@pytest.mark.parametrize("far", [10, 100000, (1 << 31) - 1])
@pytest.mark.parametrize("least,most", [(1e-6, 1.0), (1.0, 100.0), (1e3, 1e6), (1e-38, 1e-10)])
def test_frequencies_of_any_size(far, least, most):
    """|error| <= |position| max(1, |inv_freq|) 2^-50 + 2 pi 2^-24 radians, and 4 roundings of the products and the sum."""
    gen = torch.Generator().manual_seed(61)
    T, D = 24, 128
    positions = torch.randint(-far, far, (T,), generator=gen, dtype=torch.int32)
    positions[0], positions[1] = far, -far
    freq = torch.tensor(least).double().mul((most / least) ** torch.rand(D // 2, generator=gen).double()).float()
    freq[::3] *= -1
    freq[0], freq[1] = most, -most
    x = torch.randn(T, 3, D, generator=gen)
    q = torch.empty(T, 1, D, dtype=torch.bfloat16, device="cuda")
    g.qmv_rope_run(x.cuda(), None, None, positions.cuda(), freq.cuda(), None, None, q, None, None, T, 1, 1, D, D, 8, 1, flags=g.ROPE_F32_IN)
    a, b = x[:, 0, :D // 2].double().numpy(), x[:, 0, D // 2:].double().numpy()
    angle = angles(positions.tolist(), freq.tolist())
    want = np.concatenate([a * np.cos(angle) - b * np.sin(angle), a * np.sin(angle) + b * np.cos(angle)], -1)
    off = np.abs(positions.double().numpy())[:, None] * np.maximum(1.0, np.abs(freq.double().numpy())) * 2.0 ** -50 + (2 * math.pi + 4) * 2.0 ** -24
    bound = (1 + 2.0 ** -8) * np.tile(off * (np.abs(a) + np.abs(b)), 2) + 2.0 ** -8 * np.abs(want)  # (and the result is rounded)
    assert (np.abs(q[:, 0].double().cpu().numpy() - want) <= bound).all()
    assert g.qmv_device_error() == 0
