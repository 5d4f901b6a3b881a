"""qmv_attend_run at the ends of its ranges: many sequences, wide groups, wide values, lists that make no sense, and a
whole attention layer."""

import math

import pytest
import torch

import group_quantized_mat_gb300 as g
from test_gpu_attend import Problem, bits, lib, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,D,new,window", [(40, 8, 128, 1, 0), (4, 4, 64, 2, 100), (10, 2, 256, 3, 0), (64, 1, 256, 1, 0), (8, 1, 128, 16, 50)])
def test_as_many_sequences_as_there_may_be(heads, kv, D, new, window):
    B = 1024
    keys = [new + (37 * b) % 300 for b in range(B)]
    p = Problem([new] * B, keys, heads, kv, D, page=16, seed=21)
    got = p.run(window=window, sinks=3)
    # (the formula for a few of them)
    for b in (0, 1, 500, 1023):
        one = Problem([new], [keys[b]], heads, kv, D, page=16, seed=0)
        one.k, one.v, one.pages, one.most = p.k, p.v, p.pages, p.most
        one.table, one.q = p.table[b:b + 1], p.q[b * new:(b + 1) * new]
        one.check((got[0][b * new:(b + 1) * new], got[1][b * new:(b + 1) * new]), window=window, sinks=3)


def test_many_prompts():
    B = 1024
    p = Problem([17 + b % 5 for b in range(B)], [20 + b % 7 + b % 5 for b in range(B)], 2, 1, 64, page=8, seed=22)
    got = p.run()
    for b in (0, 511, 1023):
        n, at = p.new[b], p.start[b]
        one = Problem([n], [p.keys[b]], 2, 1, 64, page=8, seed=0)
        one.k, one.v, one.pages, one.most = p.k, p.v, p.pages, p.most
        one.table, one.q = p.table[b:b + 1], p.q[at:at + n]
        one.check((got[0][at:at + n], got[1][at:at + n]))


@pytest.mark.parametrize("heads,kv,D", [(64, 1, 64), (64, 1, 256), (33, 1, 128), (17, 1, 256), (7, 1, 64)])
@pytest.mark.parametrize("new", [1, 3, 16, 50])
def test_wide_groups(heads, kv, D, new):
    p = Problem([new, 2], [600 + new, 40], heads, kv, D, page=40, seed=23)
    p.check(p.run())


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("value", [3.0e38, 1e-30])
def test_wide_values(new, value):
    """Values near the ends of the type: their mean is one of them, not an infinity."""
    p = Problem([new], [1000], 4, 2, 128, seed=24)
    p.v = torch.where(torch.isnan(p.v), p.v, (p.v.float().sign() * 0 + value).bfloat16())
    out, _ = p.run()
    assert torch.isfinite(out).all()
    assert ((out.double() - p.v[p.table[0, 0], 0, 0, 0].double()).abs() <= 2.0 ** -7 * value).all()


@pytest.mark.parametrize("new", [1, 5, 40, 300])
@pytest.mark.parametrize("window,sinks", [(100, 0), (100, 5), (37, 130), (1, 1)])
def test_unseen_keys_of_pages_that_are_seen(new, window, sinks):
    """Of a page that is seen in part, the keys before every window and behind the first tokens may be anything."""
    def problem():
        return Problem([new], [900], 4, 2, 128, page=48, seed=25)
    a, b = problem(), problem()
    low = 900 - new - window + 1
    for j in range(sinks, low):
        page, place = int(a.table[0, j // 48]), j % 48
        for c in (a.k, a.v):
            c[page, place] = math.nan if j % 2 else math.inf
    assert same(a.run(window=window, sinks=sinks), b.run(window=window, sinks=sinks))
    b.check(b.run(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("drafts", [1, 5])
def test_drafts_that_begin_a_part_of_their_own(drafts):
    """A token whose keys are one part of the work by themselves, and two with the drafts behind it: the same bits, also
    where a result is close to the middle of two bf16 (2 million of them: a last bit of fp32 shows in some)."""
    B, heads = 512, 32
    p = Problem([1 + drafts] * B, [256 + drafts] * B, heads, 1, 128, page=16, seed=28)
    out, lse = p.run()
    one = Problem([1] * B, [256] * B, heads, 1, 128, page=16, seed=0)
    one.k, one.v, one.pages, one.most, one.table = p.k, p.v, p.pages, p.most, p.table
    one.q = p.q[::1 + drafts].contiguous()
    assert same((out[::1 + drafts], lse[::1 + drafts]), one.run())


@pytest.mark.parametrize("heads,kv,D", [(8, 2, 128), (4, 4, 64), (10, 2, 256)])
@pytest.mark.parametrize("new,keys", [([1, 3], [5, 700]), ([2, 16], [2, 6000]), ([40, 300], [700, 300]), ([33], [9000])])
def test_queries_that_are_not_numbers(heads, kv, D, new, keys):
    """A query with a NaN has NaN as its result, and leaves the others' as they are."""
    a, b = (Problem(new, keys, heads, kv, D, seed=27) for _ in range(2))
    bad = torch.zeros(a.T, heads, dtype=torch.bool)
    bad[::3, 1] = bad[1::4, heads - 1] = True
    a.q[bad] = math.nan
    got, want = a.run(), b.run()
    assert all(torch.isnan(x[bad]).all() for x in got)
    assert same([x[~bad] for x in got], [x[~bad] for x in want])


def test_lists_that_make_no_sense():
    """Rows, lengths and pages out of range or of several sequences: what comes out means nothing, but nothing else is touched."""
    gen = torch.Generator().manual_seed(26)
    p = Problem([5, 40, 16, 3], [300, 900, 1000, 64], 8, 2, 128, seed=26)
    d = p.device()
    for trial in range(12):
        big = 1 << 31
        d["start"] = torch.randint(-big, big, (5,), generator=gen).int().cuda() if trial % 3 == 0 else torch.randint(-5, p.T + 5, (5,), generator=gen).int().cuda()
        if trial % 3 == 2:
            d["start"] = torch.tensor([0, p.T, 0, p.T, 0], dtype=torch.int32).cuda()
        d["keys"] = torch.randint(-big, big, (4,), generator=gen).int().cuda() if trial % 2 else torch.tensor([1, 10 ** 6, -3, 0], dtype=torch.int32).cuda()
        d["table"] = torch.randint(-3, p.pages + 3, p.table.shape, generator=gen).int().cuda()
        guard = torch.full((64 << 20,), 0x5a, dtype=torch.uint8, device="cuda")
        size = g.qmv_attend_workspace_size(4, p.T, 40, 8, 2, 128, p.page, p.most)
        assert size + 4096 < guard.numel()
        ws = guard[:size]
        p.run(d, window=(0, 70)[trial & 1], sinks=4, max_new=40, workspace=ws, workspace_bytes=size)
        assert (guard[size:] == 0x5a).all()


def test_strides_of_queries_and_results_of_their_own():
    p = Problem([3, 30], [200, 500], 4, 2, 128, seed=27)
    want = p.run()
    d = p.device()
    q = torch.zeros(p.T, 1024, dtype=torch.bfloat16, device="cuda")
    q[:, :512] = d["q"][:, :512]
    out, lse = torch.zeros(p.T, 640, dtype=torch.bfloat16, device="cuda"), torch.zeros(p.T, 4, device="cuda")
    g.qmv_attend_run(q, d["k"], d["v"], d["table"], d["start"], d["keys"], out, lse, 2, p.T, 30, 4, 2, 128, 16, p.pages, p.most, ld_q=1024, ld_out=640)
    assert same((out[:, :512].reshape(p.T, 4, 128).cpu(), lse.cpu()), want) and (out[:, 512:] == 0).all()
    out2 = torch.zeros(p.T, 512, dtype=torch.bfloat16, device="cuda")
    g.qmv_attend_run(q, d["k"], d["v"], d["table"], d["start"], d["keys"], out2, None, 2, p.T, 30, 4, 2, 128, 16, p.pages, p.most, ld_q=1024)
    assert torch.equal(out2, out[:, :512].contiguous())


def test_keys_shared_by_sequences():
    """A page in several sequences' tables, and twice in one's."""
    p = Problem([2, 2], [128, 128], 4, 2, 128, seed=28)
    p.table[1] = p.table[0]
    p.table[0, 5] = p.table[0, 2]
    p.check(p.run())


# ------------------------------------------------------------------ a layer --
class Layer:
    """Quantized projections around the two operators, on the GPU, and the same in 64 bits on what they were given."""

    def __init__(self, width, heads, kv, D, page, pages, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.width, self.heads, self.kv, self.D, self.page, self.pages = width, heads, kv, D, page, pages
        self.qkv, self.wqkv = self.matrix((heads + 2 * kv) * D, width, gen)
        self.o, self.wo = self.matrix(width, heads * D, gen)
        self.q_norm, self.k_norm = ((torch.rand(D, device="cuda", generator=gen) + 0.5).bfloat16() for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))).float()
        self.k, self.v = (torch.full((pages, page, kv, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    @staticmethod
    def matrix(N, K, gen):
        w = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=gen, device="cuda", dtype=torch.int64).int()
        s = ((torch.rand((N, K // 64), generator=gen, device="cuda") + 0.5) * 0.2 / K ** 0.5).bfloat16()
        b = (-7.5 * s.float()).bfloat16()
        q = ((w.unsqueeze(-1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).reshape(N, K // 64, 64)
        return (w, s, b), (q * s.double().unsqueeze(-1) + b.double().unsqueeze(-1)).flatten(-2)

    def __call__(self, x, table, start, kv_len, positions, max_new):
        T, B = len(x), len(kv_len)
        h, kv, D, n = self.heads, self.kv, self.D, (self.heads + 2 * self.kv) * self.D
        both = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
        q, a = (torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        y = torch.empty(T, self.width, dtype=torch.bfloat16, device="cuda")
        slots = table.long().gather(1, (positions // self.page).long().view(B, -1)).flatten() * self.page + positions.flatten() % self.page
        g.qmv_run(*self.qkv, x, both, T, n, self.width, 4, 64)
        g.qmv_rope_run(both, self.q_norm, self.k_norm, positions, self.inv_freq, None, slots, q, self.k, self.v, T, h, kv, D, D, self.page, self.pages)
        g.qmv_attend_run(q, self.k, self.v, table, start, kv_len, a, None, B, T, max_new, h, kv, D, self.page, self.pages, table.shape[1])
        g.qmv_run(*self.o, a, y, T, self.width, h * D, 4, 64)
        return y

    def want(self, x):
        """One sequence from its first token on, all in 64 bits (without the roundings between the operators)."""
        L, h, kv, D = len(x), self.heads, self.kv, self.D
        both = (x.double() @ self.wqkv.T).view(L, -1, D)
        angle = torch.arange(L, device="cuda").double()[:, None] * self.inv_freq.double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]

        def turned(v, w):
            v = v / (v.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            a, b = v[..., :D // 2], v[..., D // 2:]
            return torch.cat([a * c - b * s, a * s + b * c], -1)
        q, k = turned(both[:, :h], self.q_norm), turned(both[:, h:h + kv], self.k_norm).repeat_interleave(h // kv, 1)
        v = both[:, h + kv:].repeat_interleave(h // kv, 1)
        z = torch.einsum("thd,jhd->htj", q, k) / D ** 0.5
        z = z.masked_fill(torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        return torch.einsum("htj,jhd->thd", torch.softmax(z, -1), v).reshape(L, -1) @ self.wo.T


@pytest.mark.parametrize("heads,kv,D", [(8, 2, 128), (4, 4, 64), (4, 2, 256)])
def test_a_layer(heads, kv, D):
    """Prompts in chunks, then drafts, over one cache: near the formula; drafted tokens bit for bit as one at a time."""
    width, page, B, L = 512, 16, 2, 150
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(B, L, width, generator=gen, device="cuda").bfloat16()

    def fill(steps):
        layer = Layer(width, heads, kv, D, page, 24)
        table = torch.randperm(24, generator=torch.Generator().manual_seed(4))[:20].int().view(2, 10).cuda()
        out, at = [], 0
        for n in steps:
            start = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
            positions = torch.arange(at, at + n, dtype=torch.int32, device="cuda").repeat(B).view(1, -1)
            out.append(layer(x[:, at:at + n].reshape(B * n, width).contiguous(), table, start, torch.full((B,), at + n, dtype=torch.int32, device="cuda"),
                             positions, n).view(B, n, width))
            at += n
        assert at == L and g.qmv_device_error() == 0
        return layer, torch.cat(out, 1)

    layer, y = fill([64, 50, 16, 5, 5, 10])
    for b in range(B):
        want = layer.want(x[b])
        # roundings to bf16 of qkv, the turned rows, the attention and its weights: 5 of half a step each at most, and y's own
        assert float((y[b].double() - want).norm() / want.norm()) < 6 * 2.0 ** -8
    _, one = fill([64, 50] + [1] * 36)
    assert torch.equal(bits(one.contiguous()), bits(y.contiguous()))


@pytest.mark.parametrize("window,sinks,batch,prompt", [(0, 0, 3, 200), (64, 4, 2, 90), (0, 0, 1, 5)])
def test_the_example_emits_the_tokens_of_decoding_one_at_a_time(window, sinks, batch, prompt):
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location("attention_step", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model = ex.Model(vocab=64, width=512, heads=4, kv_heads=2, window=window, sinks=sinks)
    tokens = torch.randint(0, 64, (batch, prompt), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    runs = []
    for drafts in (0, 3):
        d = ex.Decoder(model, batch, prompt + 4 * 40, drafts)
        d.prompt(tokens)
        runs.append(d.generate(40)[0])
    assert runs[0] == runs[1] and g.qmv_device_error() == 0
