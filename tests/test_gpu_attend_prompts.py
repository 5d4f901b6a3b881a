"""qmv_attend_run on batches of prompts whose work items differ: short last items, empty parts, rows that are not computed."""

import math

import pytest
import torch

from test_gpu_attend import Problem, lib, same  # noqa: F401

pytestmark = pytest.mark.gpu


def check_rows(p, got, b, first, n, **kw):
    """Rows first .. first + n - 1 (more than 16) of sequence b against the formula."""
    keys, at = p.keys[b] - p.new[b] + first + n, p.start[b] + first
    one = Problem([n], [keys], p.heads, p.kv, p.D, page=p.page, seed=0)
    one.k, one.v, one.pages, one.most = p.k, p.v, p.pages, p.most
    one.table, one.q = p.table[b:b + 1], p.q[at:at + n]
    one.check([x[at:at + n] for x in got], **kw)


@pytest.mark.parametrize("heads,kv,D,lengths", [(8, 4, 128, (100, 40, 130, 64, 65)), (16, 8, 64, (20, 129, 17, 90)), (10, 2, 128, (60, 20, 51, 26)), (4, 4, 256, (130, 17, 40))])
def test_second_tiles_that_come_and_go(heads, kv, D, lengths):
    """Blocks take items with one tile of rows behind items with two: totals of the one are not those of the other."""
    B = 480
    new = [lengths[(b * 7 + b // 11) % len(lengths)] for b in range(B)]
    keys = [n + (b % 4) * 37 for b, n in enumerate(new)]
    p = Problem(new, keys, heads, kv, D, page=16, seed=41)
    d = p.device()
    got = p.run(d)
    for b in list(range(0, B, 53)) + [B - 1]:
        check_rows(p, got, b, 0, new[b])
    for _ in range(10):
        assert same(p.run(d), got)


@pytest.mark.parametrize("heads,kv,D", [(16, 8, 64), (16, 8, 128), (8, 4, 256)])
def test_parts_without_keys(heads, kv, D):
    """A prompt in three parts of its last rows' keys: of its first rows' one tile two parts are empty."""
    p = Problem([3000, 17], [3000, 2900], heads, kv, D, page=64, seed=42)
    d = p.device()
    got = p.run(d)
    for first in (0, 100, 1480, 2960):
        check_rows(p, got, 0, first, 40)
    check_rows(p, got, 1, 0, 17)
    for _ in range(10):
        assert same(p.run(d), got)


@pytest.mark.parametrize("heads,kv,D", [(4, 2, 128), (4, 1, 64), (2, 2, 256)])
@pytest.mark.parametrize("new,keys,most", [([5, 2], [100, 50], 3), ([40, 2], [100, 50], 20), ([300, 31], [900, 400], 150)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_keys_of_rows_that_are_not_computed(heads, kv, D, new, keys, most, window, sinks):
    """Of a sequence with more rows than max_new the last rows' own keys are seen by no query: whatever they hold, it has no
    influence."""
    a, b = (Problem(new, keys, heads, kv, D, page=48, seed=43) for _ in range(2))
    for s, n in enumerate(new):
        for j in range(keys[s] - n + min(n, most), keys[s]):
            for c in (a.k, a.v):
                c[a.table[s, j // 48], j % 48] = math.nan if j % 2 else -math.inf
    got = a.run(max_new=most, window=window, sinks=sinks)
    assert same(got, b.run(max_new=most, window=window, sinks=sinks))
    b.check(got, max_new=most, window=window, sinks=sinks)


@pytest.mark.parametrize("heads,kv,D", [(4, 2, 128), (4, 1, 64), (2, 2, 256)])
@pytest.mark.parametrize("new,keys", [([5], [700]), ([40], [700]), ([300, 20], [300, 2100])])
@pytest.mark.parametrize("size,scale", [(2.0 ** 13, None), (2.0 ** 15, 1.0), (2.0 ** 17, 1.0), (2.0 ** 17, -1.0), (2.0 ** 30, 0.5)])
def test_scores_of_any_size(heads, kv, D, new, keys, size, scale):
    """Queries of which some are so large that the softmax is a choice of the largest score: that key's value, whatever the size; the
    others as ever."""
    p = Problem(new, keys, heads, kv, D, seed=44)
    p.k = torch.where(torch.isnan(p.k), p.k, (p.k.float() * size).bfloat16())
    p.q[::2] = (p.q[::2].float() * size).bfloat16()
    p.q[1::2] = (p.q[1::2].float() / size).bfloat16()
    d = p.device()
    out, lse = p.run(d, scale=scale)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    s = scale if scale is not None else D ** -0.5
    chosen = 0
    for b, n in enumerate(new):
        for i in range(n):
            t, L = p.start[b] + i, keys[b] - n + i + 1
            j = torch.arange(L)
            at = p.table[b].long()[j // p.page], j % p.page
            k, v = (c[at].double().repeat_interleave(heads // kv, 1) for c in (p.k, p.v))
            q = p.q[t].double()
            z, S = torch.einsum("hd,lhd->lh", q, k) * s, (torch.einsum("hd,lhd->lh", q.abs(), k.abs()) * abs(s)).amax(0)
            top, where = z.sort(0, descending=True)
            for h in range(heads):
                # a score is within (D + 16) steps of an accumulator of S; weights below 2^-200 are none
                if t % 2 == 0 and L > 1 and float(top[0, h] - top[1, h]) > 2 * (D + 16) * 2.0 ** -23 * float(S[h]) + 200:
                    chosen += 1
                    # (one weight, rounded to bf16 in prompts while the total is not, then the result: (1 + 2^-8)^2)
                    assert ((out[t, h].double() - v[where[0, h], h]).abs() <= (2.0 ** -7 + 2.0 ** -15) * v[where[0, h], h].abs()).all()
                    assert abs(float(lse[t, h]) - float(top[0, h])) <= 2 * (D + 16) * 2.0 ** -23 * float(S[h])
    assert chosen > 0.5 * heads * sum(n // 2 for n in new) or size < 2.0 ** 14
    # the ordinary rows, by the formula
    if size <= 2.0 ** 17:
        y, z, oe, le = p.want(scale=scale)
        rows = torch.arange(p.T) % 2 == 1
        assert ((out.double() - y).abs()[rows] <= oe[rows] + 1e-30).all() and ((lse.double() - z).abs()[rows] <= le[rows]).all()


@pytest.mark.parametrize("heads,kv,D", [(4, 2, 128), (4, 1, 64), (2, 2, 256)])
@pytest.mark.parametrize("new,keys", [([100], [128]), ([17, 128, 40], [17, 128, 120])])
@pytest.mark.parametrize("sharp", [0.5, 3.0, 10.0])
def test_the_largest_weight_has_no_rounding(heads, kv, D, new, keys, sharp):
    """Rows whose keys lie in one tile: what the weights' rounding (2^-8 of each) may change is what the other keys than the
    largest give; of a row with one key it is nothing."""
    p = Problem(new, keys, heads, kv, D, seed=45, sharp=sharp)
    out, lse = p.run()
    p.check((out, lse))
    for b, n in enumerate(new):
        for i in range(n):
            t, L = p.start[b] + i, keys[b] - n + i + 1
            j = torch.arange(L)
            at = p.table[b].long()[j // p.page], j % p.page
            k, v = (c[at].double().repeat_interleave(heads // kv, 1) for c in (p.k, p.v))
            q = p.q[t].double()
            z, S = torch.einsum("hd,lhd->lh", q, k) * D ** -0.5, (torch.einsum("hd,lhd->lh", q.abs(), k.abs()) * D ** -0.5).amax(0)
            w = torch.softmax(z, 0)
            y, A = torch.einsum("lh,lhd->hd", w, v), torch.einsum("lh,lhd->hd", w, v.abs())
            e = (D + 16) * 2.0 ** -23 * S + 16 * 2.0 ** -24
            # (where two scores are so close that either may be the largest in 32 bits, no weight counts as it)
            top = z.topk(min(L, 2), 0).values
            clear = top[0] - top[-1] > 2 * e if L > 1 else torch.ones(heads, dtype=torch.bool)
            least = w.masked_fill(clear & (torch.arange(L)[:, None] == w.argmax(0)), 0.0)
            rest = torch.einsum("lh,lhd->hd", least, v.abs())
            bound = 2.0 ** -8 * y.abs() + 2.0 ** -8 * rest + ((2 * e + (L + 64) * 2.0 ** -23)[:, None] * A) * (1 + 2.0 ** -7)
            assert ((out[t].double() - y).abs() <= (1 + 2.0 ** -8) * bound + 1e-30).all()
            if L == 1:
                assert torch.equal(out[t].double(), v[0])
