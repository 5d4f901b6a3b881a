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
