"""Calls that hold sequences of a few new tokens and prompts together: what workspace they need, and that a decoded
token has the bits that it has alone."""

import pytest
import torch

import group_quantized_mat_gb300 as g
from test_operators_host import lib  # noqa: F401

SIZE = 16  # of a page


def size(B, T, max_new, heads, kv, D, room, window=0, sinks=0):
    return g.qmv_attend_workspace_size(B, T, max_new, heads, kv, D, SIZE, -(-room // SIZE), window, sinks)


@pytest.mark.parametrize("heads,kv,D", [(40, 8, 128), (8, 1, 64), (16, 8, 256), (64, 1, 128)])
@pytest.mark.parametrize("singles,chunk", [(64, 512), (255, 512), (1023, 512), (7, 17), (1, 100000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4)])
def test_the_workspace_follows_the_rows(lib, heads, kv, D, singles, chunk, window, sinks):  # noqa: F811
    """Sums of single tokens and a prompt: no more than as many single tokens as the call has rows need, or than the
    prompt's parts (of 128 rows, two tiles of them at head_dim 64 and 128; fewer than 1216 parts)."""
    B, T = singles + 1, singles + chunk
    apart = size(min(T, 1024), min(T, 1024), 1, heads, kv, D, 131072, window, sinks) * -(-T // 1024)
    parts = 1216 * 256 * (4 * D + 8) + 8192
    got = size(B, T, chunk, heads, kv, D, 131072, window, sinks)
    assert got <= max(2 * apart if window else apart, parts)  # (a window's units: one more for a sequence of 16 tokens)
    # and never more than 16 rows for each sequence
    assert got <= max(size(B, 16 * B, 16, heads, kv, D, 131072, window, sinks), parts)


def test_the_workspace_of_few_tokens(lib):  # noqa: F811
    """Sums of head_dim floats, a maximum and a total for each row, head and unit (1024 keys here)."""
    units = 131072 // 1024
    for B, n in ((1, 1), (64, 1), (4, 5), (3, 16)):
        assert size(B, B * n, n, 40, 8, 128, 131072) <= B * n * 40 * units * (128 * 4 + 8) + 512
    assert size(256, 767, 512, 40, 8, 128, 131072) <= 2.05e9


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv,D", [(10, 2, 128), (16, 8, 256), (8, 1, 64), (64, 1, 128)])
@pytest.mark.parametrize("chunk", [17, 60, 300])  # (17: sums by the rows of q, else by sequences)
def test_a_decoded_token_in_a_call_with_a_prompt(heads, kv, D, chunk):
    from test_gpu_attend import Problem, same

    def one(p, b, i):
        q = Problem([1], [p.keys[b] - p.new[b] + i + 1], heads, kv, D, seed=0)
        q.k, q.v, q.pages, q.most, q.table = p.k, p.v, p.pages, p.most, p.table[b:b + 1]
        q.q = p.q[p.start[b] + i:p.start[b] + i + 1]
        return q

    p = Problem([1, 3, chunk, 1, 16], [1500, 700, 900, 2049, 40], heads, kv, D, seed=51)
    d = p.device()
    for window, sinks in ((0, 0), (300, 5)):
        bytes_ = g.qmv_attend_workspace_size(5, p.T, chunk, heads, kv, D, p.page, p.most, window, sinks)
        ws = torch.full((bytes_ + 4096,), 0xff, dtype=torch.uint8, device="cuda")
        got = p.run(d, window=window, sinks=sinks, workspace=ws, workspace_bytes=bytes_)
        assert (ws[bytes_:] == 0xff).all(), "what lies behind the workspace is left alone"
        p.check(got, window=window, sinks=sinks)
        for b in (0, 1, 3, 4):
            for i in range(p.new[b]):
                t = p.start[b] + i
                assert same(one(p, b, i).run(window=window, sinks=sinks), [x[t:t + 1] for x in got]), (b, i)
