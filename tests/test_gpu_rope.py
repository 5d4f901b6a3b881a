"""qmv_rope_run against its formula in 64 bits, and what it leaves alone."""

import math

import numpy as np
import pytest
import torch

import attention_reference as ref
import group_quantized_mat_gb300 as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    return g.load()


def make(T, heads, kv, D, rot, axes, f32, norms, page, seed, far=100000, pad=0, order="tokens", scale=1.0):
    """A problem on the GPU, with a cache in the given order of its dimensions."""
    gen = torch.Generator().manual_seed(seed)
    width = (heads + 2 * kv) * D
    x = torch.randn(T, width + pad, generator=gen) * scale
    x = x if f32 else x.bfloat16()
    pages = -(-T // page) + 2
    shape = (pages, page, kv, D) if order == "tokens" else (pages, kv, page, D)
    cache = torch.randn(2, *shape, generator=gen).bfloat16()
    half = rot // 2
    p = dict(T=T, heads=heads, kv=kv, D=D, rot=rot, axes=axes, f32=f32, page=page, pages=pages, order=order, ld=width + pad,
             x=x, q_norm=(torch.rand(D, generator=gen) + 0.5).bfloat16() if norms & 1 else None,
             k_norm=(torch.rand(D, generator=gen) + 0.5).bfloat16() if norms & 2 else None,
             positions=torch.randint(0, far, (axes, T), generator=gen, dtype=torch.int32),
             inv_freq=(10000.0 ** (-torch.arange(half) / max(half, 1))).float(),
             axis=torch.randint(0, axes + 1, (half,), generator=gen).to(torch.uint8) if axes > 1 else None,
             slots=torch.randperm(pages * page, generator=gen)[:T], cache=cache)
    p["slots"][T // 2::5] = -1 if T > 2 else p["slots"][T // 2::5]
    return p


def strides(p):
    if p["order"] == "tokens":
        return dict(page_stride=p["page"] * p["kv"] * p["D"], token_stride=p["kv"] * p["D"], head_stride=p["D"])
    return dict(page_stride=p["page"] * p["kv"] * p["D"], token_stride=p["D"], head_stride=p["page"] * p["D"])


def run(p, flags=0, eps=1e-6, rows=slice(None), stream=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    T = len(range(p["T"])[rows])
    q = torch.full((T, p["heads"], p["D"]), math.nan, dtype=torch.bfloat16, device="cuda")
    cache = dev(p["cache"]).clone()
    args = [dev(p["x"][rows].contiguous()), dev(p["q_norm"]), dev(p["k_norm"]), dev(p["positions"][:, rows].contiguous()), dev(p["inv_freq"]), dev(p["axis"]),
            dev(p["slots"][rows].contiguous())]
    g.qmv_rope_run(*args, q, cache[0], cache[1], T, p["heads"], p["kv"], p["D"], p["rot"], p["page"], p["pages"], p["axes"], eps, p["ld"],
                   flags=flags | (g.ROPE_F32_IN if p["f32"] else 0), stream=stream, **strides(p))
    torch.cuda.synchronize()
    return q.cpu(), cache.cpu()


def by_place(p, cache):
    """[pages * page_size, kv, D]"""
    c = cache if p["order"] == "tokens" else cache.transpose(-2, -3)
    return c.reshape(p["pages"] * p["page"], p["kv"], p["D"])


def check(p, q, cache, eps=1e-6, one=0.0, neighbours=False):
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    x = f64(p["x"])[:, :(p["heads"] + 2 * p["kv"]) * p["D"]].reshape(p["T"], -1, p["D"])
    out, err = ref.rope(x, f64(p["q_norm"]), f64(p["k_norm"]), p["positions"].numpy(), f64(p["inv_freq"]),
                        None if p["axis"] is None else p["axis"].numpy().astype(int), p["heads"], p["kv"], eps, one, neighbours)
    # |position| 2^-50 radians more for the positions
    more = float(p["positions"].abs().max()) * 2.0 ** -50
    assert (np.abs(q.double().numpy() - out[0]) <= err[0] + more * np.abs(out[0]).max() + 1e-38).all()
    for c, before, want, bound in ((cache[0], p["cache"][0], out[1], err[1]), (cache[1], p["cache"][1], out[2], err[2])):
        got, old = by_place(p, c), by_place(p, before).clone()
        at = p["slots"] >= 0
        assert (np.abs(got[p["slots"][at]].double().numpy() - want[at.numpy()]) <= bound[at.numpy()] + more * np.abs(want).max() + 1e-38).all()
        got[p["slots"][at]] = old[p["slots"][at]]
        assert torch.equal(got.view(torch.int16), old.view(torch.int16)), "places that no token has are left alone"


@pytest.mark.parametrize("T,heads,kv,D,rot,axes,f32,norms,page,pad,order", [
    (1, 40, 8, 128, 128, 1, False, 3, 16, 0, "tokens"),
    (1, 1, 1, 64, 64, 1, True, 3, 8, 0, "heads"),
    (2, 3, 1, 64, 16, 2, False, 1, 24, 8, "heads"),
    (13, 16, 8, 256, 64, 1, True, 3, 32, 24, "tokens"),
    (5, 64, 1, 256, 256, 4, False, 2, 16, 0, "tokens"),
    (7, 12, 4, 128, 96, 3, False, 3, 8, 0, "heads"),
    (300, 6, 2, 64, 48, 1, False, 0, 64, 0, "tokens"),
    (1155, 32, 4, 128, 128, 3, False, 3, 64, 0, "tokens"),
    (700, 5, 5, 128, 112, 2, True, 3, 40, 8, "heads"),
    (65, 2, 2, 256, 0, 1, False, 3, 16, 0, "tokens"),
    (3, 1, 1, 256, 208, 1, False, 3, 128, 0, "tokens"),
])
@pytest.mark.parametrize("neighbours,plus_one", [(False, False), (True, True)])
def test_against_the_formula(T, heads, kv, D, rot, axes, f32, norms, page, pad, order, neighbours, plus_one):
    p = make(T, heads, kv, D, rot, axes, f32, norms, page, seed=T + D + rot, pad=pad, order=order)
    flags = (g.ROPE_NEIGHBOURS if neighbours else 0) | (g.ROPE_NORM_PLUS_ONE if plus_one else 0)
    q, cache = run(p, flags)
    check(p, q, cache, one=float(plus_one), neighbours=neighbours)


@pytest.mark.parametrize("far", [1 << 20, 1 << 30, (1 << 31) - 1])
def test_far_and_negative_positions(far):
    p = make(40, 4, 2, 128, 128, 1, True, 0, 16, seed=3, far=far)
    p["positions"][0, ::3] *= -1
    q, cache = run(p)
    check(p, q, cache)


def test_wide_values():
    """Values whose squares neither overflow nor vanish in 32 bits; a row of zeros stays zero."""
    for scale in (1e-15, 1e15):
        p = make(9, 4, 2, 128, 128, 1, True, 3, 16, seed=4, scale=scale)
        p["x"][3] = 0.0
        q, cache = run(p, eps=0.0 if scale > 1 else 1e-36)
        if scale > 1:
            q, p["x"] = q.clone(), p["x"].clone()
            assert torch.isnan(q[3]).all()  # 0 / 0 without an eps
            keep = [i for i in range(9) if i != 3]
            sub = {**p, "T": 8, "x": p["x"][keep], "positions": p["positions"][:, keep], "slots": p["slots"][keep]}
            f64 = lambda t: t.double().numpy()  # noqa: E731
            out, err = ref.rope(f64(sub["x"]).reshape(8, -1, 128), f64(p["q_norm"]), f64(p["k_norm"]), sub["positions"].numpy(), f64(p["inv_freq"]), None, 4, 2, 0.0, 0.0, False)
            assert (np.abs(f64(q[keep]) - out[0]) <= err[0] + 1e-38).all()
        else:
            check(p, q, cache, eps=1e-36)
            assert (q[3] == 0).all()


def test_a_token_does_not_depend_on_the_others():
    p = make(500, 10, 2, 128, 128, 3, False, 3, 16, seed=5)
    q, cache = run(p)
    for t in (0, 1, 250, 499):
        q1, c1 = run(p, rows=slice(t, t + 1))
        assert torch.equal(q1[0].view(torch.int16), q[t].view(torch.int16))
        s = int(p["slots"][t])
        if s >= 0:
            for i in range(2):
                assert torch.equal(by_place(p, c1[i])[s].view(torch.int16), by_place(p, cache[i])[s].view(torch.int16))


def test_places_outside_the_cache_and_no_cache():
    p = make(6, 4, 2, 64, 64, 1, False, 3, 8, seed=6)
    places = p["pages"] * p["page"]
    p["slots"] = torch.tensor([places, -7, 0, places - 1, 1 << 40, -(1 << 40)])
    q, cache = run(p)
    q2, _ = run({**p, "slots": torch.tensor([-1] * 6)})
    assert torch.equal(q.view(torch.int16), q2.view(torch.int16))
    p["slots"] = torch.where((p["slots"] >= 0) & (p["slots"] < places), p["slots"], -1)
    check(p, q, cache)
    q3 = torch.empty_like(q, device="cuda")
    g.qmv_rope_run(p["x"].cuda(), p["q_norm"].cuda(), p["k_norm"].cuda(), p["positions"].cuda(), p["inv_freq"].cuda(), None, None, q3, None, None,
                   6, 4, 2, 64, 64, 8, 1)
    assert torch.equal(q3.cpu().view(torch.int16), q.view(torch.int16))


def test_streams_and_graphs():
    p = make(33, 8, 2, 128, 128, 1, False, 3, 16, seed=7)
    want, wc = run(p)
    s = torch.cuda.Stream()
    got, gc = run(p, stream=s)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(gc.view(torch.int16), wc.view(torch.int16))
    x, q, cache = p["x"].cuda(), torch.zeros(33, 8, 128, dtype=torch.bfloat16, device="cuda"), p["cache"].cuda()
    args = [x, p["q_norm"].cuda(), p["k_norm"].cuda(), p["positions"].cuda(), p["inv_freq"].cuda(), None, p["slots"].cuda(), q, cache[0], cache[1],
            33, 8, 2, 128, 128, 16, p["pages"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.qmv_rope_run(*args)
    for _ in range(2):
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.cpu().view(torch.int16), want.view(torch.int16))
    x.mul_(2)  # new data, same graph
    graph.replay()
    torch.cuda.synchronize()
    check({**p, "x": p["x"] * 2}, q.cpu(), cache.cpu())
