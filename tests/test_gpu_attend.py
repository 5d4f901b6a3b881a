"""qmv_attend_run against its formula in 64 bits: lengths, masks, pages, strides, and what it leaves alone."""

import math

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


class Problem:
    """Sequences with the given new tokens and keys; a cache in the given order, pages shuffled, unused entries -1."""

    def __init__(self, new, keys, heads=8, kv=2, D=128, page=16, seed=0, order="tokens", pad=0, sharp=1.0, tail=0, spare=1, junk=math.nan):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.keys, self.heads, self.kv, self.D, self.page, self.order = new, keys, heads, kv, D, page, order
        B, self.T = len(new), sum(new) + tail
        self.most = max(1, max(-(-k // page) for k in keys)) + 1
        need = [-(-k // page) for k in keys]
        self.pages = max(1, sum(need)) + spare
        perm = torch.randperm(self.pages, generator=gen)
        self.table = torch.full((B, self.most), -1, dtype=torch.int32)
        k = torch.full((self.pages, page, kv, D), junk, dtype=torch.bfloat16)
        v = k.clone()
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            for i in range(need[b]):
                rows = min(page, keys[b] - i * page)
                for c in (k, v):
                    c[perm[at + i], :rows] = torch.randn(rows, kv, D, generator=gen).bfloat16()
            at += need[b]
        self.k, self.v = k, v
        self.start = [sum(new[:b]) for b in range(B + 1)]
        self.q = (torch.randn(self.T, heads, D, generator=gen) * sharp).bfloat16()
        self.ld = heads * D + pad

    def device(self):
        def cache(c):
            return (c if self.order == "tokens" else c.transpose(1, 2)).contiguous().cuda()
        q = torch.zeros(self.T, self.ld, dtype=torch.bfloat16)
        q[:, :self.heads * self.D] = self.q.flatten(1)
        return dict(q=q.cuda(), k=cache(self.k), v=cache(self.v), table=self.table.cuda(), start=torch.tensor(self.start, dtype=torch.int32).cuda(),
                    keys=torch.tensor(self.keys, dtype=torch.int32).cuda())

    def strides(self):
        n = self.page * self.kv * self.D
        if self.order == "tokens":
            return dict(page_stride=n, token_stride=self.kv * self.D, head_stride=self.D)
        return dict(page_stride=n, token_stride=self.D, head_stride=self.page * self.D)

    def run(self, d=None, window=0, sinks=0, scale=None, max_new=None, **kw):
        d = d or self.device()
        out = torch.full((self.T, self.ld), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.heads), 7.0, device="cuda")
        g.qmv_attend_run(d["q"], d["k"], d["v"], d["table"], d["start"], d["keys"], out, lse, len(self.new), self.T, max_new or max(max(self.new), 1),
                         self.heads, self.kv, self.D, self.page, self.pages, self.most, scale=scale, window=window, sinks=sinks, ld_q=self.ld,
                         ld_out=self.ld, **self.strides(), **kw)
        torch.cuda.synchronize()
        assert g.qmv_device_error() == 0
        assert (out[:, self.heads * self.D:] == 7.0).all(), "columns behind a row's heads are left alone"
        return out[:, :self.heads * self.D].view(self.T, self.heads, self.D).cpu(), lse.cpu()

    def want(self, window=0, sinks=0, scale=None, max_new=None):
        # (what no query may see is not a number: the formula leaves it out before it counts)
        return ref.attend(self.q.double(), self.k.double(), self.v.double(), self.table, self.start, self.keys, self.kv,
                          self.D ** -0.5 if scale is None else scale, window, sinks, max_new)

    def check(self, got, **kw):
        out, lse = got[0].double(), got[1].double()
        y, z, oe, le = self.want(**kw)
        left = torch.isnan(z)
        assert (lse[left] == 7.0).all() and (out[left] == 7.0).all(), "rows of no sequence are left as they were"
        none = z == -math.inf
        assert (lse[none] == -math.inf).all() and (out[none] == 0).all()
        fine = ~left & ~none
        assert torch.isfinite(out[fine]).all() and torch.isfinite(lse[fine]).all()
        assert ((out - y).abs()[fine] <= oe[fine] + 1e-30).all(), float(((out - y).abs()[fine] / (oe[fine] + 1e-30)).max())
        assert ((lse - z).abs()[fine] <= le[fine]).all(), float(((lse - z).abs()[fine] / le[fine]).max())


def bits(a):
    return a.view(torch.int16) if a.dtype == torch.bfloat16 else a.view(torch.int32)


def same(a, b):
    return all(torch.equal(bits(x.contiguous()), bits(y.contiguous())) for x, y in zip(a, b))


SHAPES = [(8, 2, 128), (5, 1, 128), (16, 8, 256), (3, 3, 64), (8, 1, 64), (64, 1, 128), (40, 8, 128), (10, 2, 256)]


@pytest.mark.parametrize("heads,kv,D", SHAPES)
@pytest.mark.parametrize("new,keys", [
    ([1], [1]), ([1], [2]), ([1, 1, 1], [127, 128, 129]), ([2, 1, 5], [511, 512, 516]), ([1, 3], [255, 1030]), ([16, 7, 1], [16, 700, 2000]), ([13], [1500]),
])
def test_few_tokens(heads, kv, D, new, keys):
    p = Problem(new, keys, heads, kv, D, page=16, seed=heads + sum(keys))
    p.check(p.run())


@pytest.mark.parametrize("heads,kv,D", SHAPES)
@pytest.mark.parametrize("new,keys", [([17], [17]), ([130], [130]), ([40, 300], [200, 300]), ([256, 1, 20], [300, 900, 21]), ([129, 64], [1400, 64])])
def test_prompts(heads, kv, D, new, keys):
    p = Problem(new, keys, heads, kv, D, page=32, seed=heads + sum(keys))
    p.check(p.run())


@pytest.mark.parametrize("heads,kv,D", [(24, 8, 256), (4, 4, 256), (16, 2, 128), (6, 2, 64)])
@pytest.mark.parametrize("new,keys", [([29], [3323]), ([17, 100, 5, 33], [5000, 2100, 3000, 1100])])
def test_prompts_in_pieces(heads, kv, D, new, keys):
    """Few rows over many keys: their tiles in several pieces, which end at other tiles each."""
    p = Problem(new, keys, heads, kv, D, page=16, seed=heads + sum(keys), sharp=2.0)
    d = p.device()
    got = p.run(d)
    p.check(got)
    for _ in range(3):
        assert same(p.run(d), got)


@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 96, 128, 200, 256, 1000])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_pages(page, order):
    p = Problem([1, 4, 30], [333, 1029, 450], 6, 2, 128, page=page, order=order, seed=page, pad=8)
    p.check(p.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 4), (64, 0), (100, 3), (128, 130), (129, 128), (700, 0), (700, 64), (5000, 4), (1 << 30, 1 << 30)])
def test_windows(D, window, sinks):
    p = Problem([1, 5, 16, 90, 200], [900, 2000, 16, 90, 1300], 4, 2, D, page=16, seed=window)
    p.check(p.run(window=window, sinks=sinks), window=window, sinks=sinks)


def test_pages_behind_the_window_are_not_needed():
    """Entries of pages that no query sees may be anything."""
    p = Problem([1, 3, 40], [900, 2000, 1500], 4, 2, 128, page=16, seed=1)
    want = p.run(window=100, sinks=20)
    for b, (n, keys) in enumerate(zip(p.new, p.keys)):
        low = keys - n - 100 + 1
        for i in range(2, low // 16):
            p.k[p.table[b, i]] = math.nan
            p.v[p.table[b, i]] = math.nan
            p.table[b, i] = (1 << 31) - 1 if i % 2 else -5
    assert same(p.run(window=100, sinks=20), want)


def test_bad_pages_are_not_seen():
    p = Problem([1, 3, 40], [300, 1200, 1100], 4, 2, 128, page=16, seed=2)
    p.table[0, 3], p.table[1, 20], p.table[1, 74], p.table[2, 5], p.table[2, 6] = -1, p.pages, 1 << 30, -(1 << 31), p.pages + 3
    p.check(p.run())
    p.table[0, :] = -1
    p.check(p.run())


@pytest.mark.parametrize("new,keys", [([0], [0]), ([0, 0], [50, 0]), ([1, 0, 2, 0, 30, 1], [0, 77, 1, 0, 29, 64]), ([4], [2]), ([40], [3])])
def test_empty_sequences_and_rows_that_see_nothing(new, keys):
    p = Problem(new, keys, 4, 2, 128, tail=3, seed=3)
    p.check(p.run())


def test_rows_of_no_sequence():
    p = Problem([3, 20], [100, 300], 4, 2, 64, tail=5, seed=4)
    d = p.device()
    d["start"] = torch.tensor([2, 5, 25], dtype=torch.int32).cuda()
    p.start = [2, 5, 25]
    p.check(p.run(d))


def test_more_rows_than_max_new():
    for new, most in (([5, 2], 3), ([40, 2], 20)):
        p = Problem(new, [100, 50], 4, 2, 128, seed=5)
        p.check(p.run(max_new=most), max_new=most)


def test_without_q_start():
    p = Problem([3, 3, 3], [100, 400, 3], 4, 2, 128, seed=6)
    want = p.run()
    d = p.device()
    d["start"] = None
    assert same(p.run(d), want)


@pytest.mark.parametrize("sharp,scale", [(30.0, None), (1.0, 0.0), (1.0, -0.2), (200.0, 1.0), (1e-3, 1e-3)])
@pytest.mark.parametrize("new", [1, 40])
def test_sharp_and_flat_scores(sharp, scale, new):
    """Scores that lie thousands apart, all alike, of the other sign."""
    p = Problem([new], [1200], 4, 2, 128, seed=7, sharp=sharp)
    p.check(p.run(scale=scale), scale=scale)


@pytest.mark.parametrize("new", [1, 5, 40])
def test_scores_that_rise_and_fall(new):
    """The largest score far behind many small ones, or far before."""
    for at in (0, 130, 260, 700, 1190 - new):
        p = Problem([new], [1200], 2, 1, 128, seed=8)
        p.q[:] = p.q[0, 0]
        page, place = int(p.table[0, at // 16]), at % 16
        p.k[page, place, 0] = (p.q[0, 0].float() * 4).bfloat16()
        p.check(p.run())


@pytest.mark.parametrize("junk", [math.nan, math.inf, -3.3e38])
def test_what_is_not_seen_has_no_influence(junk):
    """Every unused place of the cache, and the rest of each last page."""
    a = Problem([1, 3, 16, 60], [130, 517, 40, 77], 8, 2, 128, seed=9, junk=junk)
    b = Problem([1, 3, 16, 60], [130, 517, 40, 77], 8, 2, 128, seed=9, junk=0.0)
    assert same(a.run(), b.run())
    a.check(a.run())


def test_a_token_does_not_depend_on_the_others():
    """Bit for bit: one token alone, drafted with others, in a batch, in another place, over other pages."""
    for heads, kv, D in ((10, 2, 128), (16, 8, 256), (8, 1, 64)):
        keys, n = [700, 1537, 40], [16, 5, 7]
        p = Problem(n, keys, heads, kv, D, seed=10)
        out, lse = p.run()
        out_w, lse_w = p.run(window=200, sinks=4)
        for b in range(3):
            for i in range(n[b]):
                one = Problem([1], [keys[b] - n[b] + i + 1], heads, kv, D, seed=11)
                one.k, one.v, one.pages, one.most = p.k, p.v, p.pages, p.most
                one.table = p.table[b:b + 1].clone()
                one.q = p.q[p.start[b] + i:p.start[b] + i + 1]
                t = p.start[b] + i
                assert same(one.run(), (out[t:t + 1], lse[t:t + 1])), (b, i)
                assert same(one.run(window=200, sinks=4), (out_w[t:t + 1], lse_w[t:t + 1])), (b, i)


def test_calls_repeat():
    p = Problem([1, 9, 200, 33], [3000, 2000, 1900, 33], 8, 2, 128, seed=12)
    d = p.device()
    want = p.run(d)
    for _ in range(5):
        assert same(p.run(d), want)


def test_workspaces_streams_and_graphs():
    p = Problem([1, 4, 30], [700, 1500, 900], 8, 2, 128, seed=13)
    d = p.device()
    want = p.run(d)
    size = g.qmv_attend_workspace_size(3, p.T, 30, 8, 2, 128, p.page, p.most)
    ws = torch.full((size + 64,), 0xff, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert same(p.run(d, workspace=ws, workspace_bytes=size, stream=s), want)
    assert (ws[size:] == 0xff).all()
    with pytest.raises(g.QmvError) as e:
        p.run(d, workspace=ws, workspace_bytes=size - 1)
    assert e.value.code == 8
    out = torch.zeros(p.T, p.ld, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(p.T, 8, device="cuda")

    def call(ws):
        g.qmv_attend_run(d["q"], d["k"], d["v"], d["table"], d["start"], d["keys"], out, lse, 3, p.T, 30, 8, 2, 128, p.page, p.pages, p.most,
                         workspace=ws, workspace_bytes=size)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:  # two graphs of one workspace, one after the other
        with torch.cuda.graph(graph):
            call(ws)
    for graph in graphs + graphs:
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same((out.view(want[0].shape).cpu(), lse.cpu()), want)
    # lengths that change between replays
    d["keys"].copy_(torch.tensor([350, 1200, 40], dtype=torch.int32))
    p.keys = [350, 1200, 40]
    graphs[0].replay()
    torch.cuda.synchronize()
    p.check((out.view(want[0].shape).cpu(), lse.cpu()))


def test_two_calls_at_once():
    """Two streams with a workspace each."""
    a, b = Problem([1] * 6, [2000] * 6, seed=14), Problem([5] * 3, [3000, 100, 1111], seed=15)
    da, db = a.device(), b.device()
    wa, wb = a.run(da), b.run(db)
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for p, d in ((a, da), (b, db)):
        size = g.qmv_attend_workspace_size(len(p.new), p.T, max(p.new), 8, 2, 128, p.page, p.most)
        outs.append((torch.zeros(p.T, p.ld, dtype=torch.bfloat16, device="cuda"), torch.zeros(p.T, 8, device="cuda"),
                     torch.zeros(size, dtype=torch.uint8, device="cuda"), size))
    torch.cuda.synchronize()
    for _ in range(20):
        for (p, d), s, (o, l, ws, size) in zip(((a, da), (b, db)), streams, outs):
            g.qmv_attend_run(d["q"], d["k"], d["v"], d["table"], d["start"], d["keys"], o, l, len(p.new), p.T, max(p.new), 8, 2, 128, p.page, p.pages, p.most,
                             workspace=ws, workspace_bytes=size, stream=s)
    torch.cuda.synchronize()
    for p, w, (o, l, _, _) in ((a, wa, outs[0]), (b, wb, outs[1])):
        assert same((o.view(w[0].shape).cpu(), l.cpu()), w)


def test_a_cache_past_2_to_the_31():
    """Offsets of more than 32 bits: the sequence's pages lie at the end of a cache of 6 GB."""
    heads, kv, D, page = 4, 2, 128, 64
    p = Problem([2, 20], [500, 300], heads, kv, D, page=page, seed=16)
    want = p.run()
    pages = (3 << 31) // (2 * page * kv * D) + 50
    d = p.device()
    for name in ("k", "v"):
        big = torch.zeros(pages, page, kv, D, dtype=torch.bfloat16, device="cuda")
        big[-p.pages:] = d[name]
        d[name] = big
    shift = pages - p.pages
    d["table"] = torch.where(d["table"] >= 0, d["table"] + shift, d["table"])
    p.pages = pages
    assert same(p.run(d), want)
