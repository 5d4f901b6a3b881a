"""Cases, plain forms and 64-bit values of the operators of an attention layer in a quantized model's step.

Between the quantized projections of a layer's queries, keys and values and that
of its output stand two operators:

* ``rope``: norms of each head's query and key, rotation by position (one axis, or
  several for images and video), and the new keys and values put into a paged cache.
* ``attend``: the new tokens' queries over the paged cache, causal, optionally with
  a sliding window and a few first tokens that stay visible.

A cache is [pages, page_size, kv_heads, head_dim] in bf16, keys and values apart; a
sequence's pages are listed in its row of the page table, in any order.
"""

import math
import random

import torch

own = False

_EPS = 1e-6


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one decoded token, heads of the 27B-class stack's projections (5120 and 1024 wide): latency
        dict(name="rope one token", op="rope", T=1, heads=40, kv_heads=8, dim=128, rot=128, axes=1, f32=False, plus_one=False, norm=True, pairs="halves", page=16, far=9000),
        # a full verify width straight from fp32 projections, part of each head rotated, neighbours as pairs
        dict(name="rope verify of 13", op="rope", T=13, heads=16, kv_heads=8, dim=256, rot=64, axes=1, f32=True, plus_one=True, norm=True, pairs="neighbours", page=32, far=131072),
        # a prompt with an image: time, height and width have their own frequencies
        dict(name="rope image prompt", op="rope", T=1155, heads=32, kv_heads=4, dim=128, rot=128, axes=3, f32=False, plus_one=False, norm=True, pairs="halves", page=64, far=40000),
        # a large batch of prompts
        dict(name="rope prompts", op="rope", T=16384, heads=40, kv_heads=8, dim=128, rot=128, axes=1, f32=False, plus_one=False, norm=True, pairs="halves", page=64, far=16384),
        # one decoded token of one request: latency
        dict(name="attend one token", op="attend", B=1, new=1, ctx=4100, heads=40, kv_heads=8, dim=128, page=16, window=0, sinks=0),
        # drafts of five tokens, four requests, large heads
        dict(name="attend drafts of 5", op="attend", B=4, new=5, ctx=9000, heads=16, kv_heads=8, dim=256, page=32, window=0, sinks=0),
        # a window layer's decode step: far fewer keys than the cache holds
        dict(name="attend window decode", op="attend", B=32, new=1, ctx=30000, heads=40, kv_heads=8, dim=128, page=64, window=1024, sinks=4),
        # a decode step of a large batch: the cache is what is read
        dict(name="attend batch decode", op="attend", B=64, new=1, ctx=8192, heads=40, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a full verify width over a long context
        dict(name="attend 13 long", op="attend", B=1, new=13, ctx=131000, heads=32, kv_heads=4, dim=128, page=128, window=0, sinks=0),
        # chunks of two prompts over what is cached already, an odd page size
        dict(name="attend chunk", op="attend", B=2, new=512, ctx=16500, heads=40, kv_heads=8, dim=128, page=24, window=0, sinks=0),
        # a batch of whole prompts of different lengths
        dict(name="attend prompts", op="attend", B=6, new=8192, ctx=8192, heads=40, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a long prompt through a window layer
        dict(name="attend window prompt", op="attend", B=1, new=8000, ctx=12000, heads=16, kv_heads=8, dim=256, page=64, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128, 200])
    if rng.random() < 0.35:
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return dict(op="rope", T=_log(rng, 1, 16384), heads=heads, kv_heads=kv, dim=dim, rot=rot, axes=axes, f32=rng.random() < 0.3, plus_one=rng.random() < 0.3,
                    norm=rng.random() < 0.8, pairs=rng.choice(["halves", "halves", "neighbours"]), page=page, far=_log(rng, 1000, 1000000))
    kind = rng.choice(["one", "drafts", "drafts", "chunk", "chunk"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 100, 4096), rng.choice([0, 1, 4, 64]))])
    if kind == "chunk":
        B, new = rng.randint(1, 6), _log(rng, 17, 4096)
        ctx = new + _log(rng, 1, 24000)
    else:
        new = 1 if kind == "one" else rng.randint(2, 16)
        B = _log(rng, 1, 64)
        ctx = new + _log(rng, 30, min(131072, 600000 // B))
    return dict(op="attend", B=B, new=new, ctx=ctx, heads=heads, kv_heads=kv, dim=dim, page=page, window=window, sinks=sinks)


# --------------------------------------------------------------- the inputs --
def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence, by the case alone."""
    rng = random.Random("%d %d %d %d" % (c["B"], c["new"], c["ctx"], c["page"]))
    new, ctx = [], []
    for b in range(c["B"]):
        whole = b == 0 or c["new"] == 1
        n = c["new"] if whole else rng.randint(1, c["new"]) if c["new"] <= 16 else _log(rng, max(1, c["new"] // 16), c["new"])
        old = c["ctx"] - c["new"]
        new.append(n)
        ctx.append(n + (old if b == 0 else rng.randint(old // 2, old)))
    return new, ctx


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    gen = _gen(seed)
    c = case
    s = dict(case=c)
    H, KV, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    if c["op"] == "rope":
        T = c["T"]
        x = torch.randn((T, (H + 2 * KV) * D), generator=gen, device="cuda") * 1.5
        s["qkv"] = x if c["f32"] else x.to(torch.bfloat16)
        shift = 0.0 if c["plus_one"] else 1.0
        for k in ("q_norm", "k_norm"):
            s[k] = (torch.randn((D,), generator=gen, device="cuda") * 0.2 + shift).to(torch.bfloat16) if c["norm"] else None
        first = int(torch.randint(0, max(1, c["far"] - T), (1,), generator=gen, device="cuda"))
        at = torch.arange(T, device="cuda", dtype=torch.int32) + first
        if c["axes"] > 1:  # rows of an image: one time, its rows and columns
            side = max(1, math.isqrt(T))
            at = torch.stack([at // (side * side) * side, at // side % side + first, at % side + first][:c["axes"]])
        s["positions"] = at.reshape(c["axes"], T).to(torch.int32).contiguous()
        half = c["rot"] // 2
        s["inv_freq"] = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
        s["axis"] = (torch.arange(half, device="cuda") * c["axes"] // half).to(torch.uint8) if c["axes"] > 1 else None
        pages = -(-T // P) + 3
        s["pages"] = pages
        s["slots"] = torch.randperm(pages * P, generator=gen, device="cuda")[:T] if T <= 64 else (
            torch.randperm(pages, generator=gen, device="cuda")[:, None] * P + torch.arange(P, device="cuda")).flatten()[:T]
        s["slots"] = s["slots"].to(torch.int64).contiguous()
        s["q"] = torch.zeros((T, H, D), device="cuda", dtype=torch.bfloat16)
        for k in ("k_cache", "v_cache"):
            s[k] = torch.randn((pages, P, KV, D), generator=gen, device="cuda").to(torch.bfloat16)
        return s
    new, ctx = _lengths(c)
    B, T = c["B"], sum(new)
    most = -(-max(ctx) // P)
    need = [-(-n // P) for n in ctx]
    pages = sum(need)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, most), -1, device="cuda", dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"], s["pages"], s["most"] = table, pages, most
    s["new"], s["ctx"] = new, ctx
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    s["q_start"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
    s["kv_len"] = torch.tensor(ctx, device="cuda", dtype=torch.int32)
    # normed keys; queries of sharper and of flatter heads; a direction that all queries share and first tokens have
    common = torch.randn((KV, D), generator=gen, device="cuda")
    s["k_cache"] = torch.randn((pages, P, KV, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["v_cache"] = torch.randn((pages, P, KV, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    for b in range(B):
        s["k_cache"][int(table[b, 0]), 0] = (2 * common).to(torch.bfloat16)
    sharp = torch.rand((H, 1), generator=gen, device="cuda") * 2 + 0.7
    q = torch.randn((T, H, D), generator=gen, device="cuda") * sharp + 0.3 * common.repeat_interleave(H // KV, 0)
    s["queries"] = q.to(torch.bfloat16)
    s["out"] = torch.zeros((T, H, D), device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.zeros((T, H), device="cuda", dtype=torch.float32)
    return s


# ----------------------------------------------------------- the operators --
def _normed(x, weight, plus_one):
    if weight is None:
        return x
    w = weight.float() + (1.0 if plus_one else 0.0)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w


def _rope(s):
    c = s["case"]
    T, H, KV, D, rot = c["T"], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].float().view(T, H + 2 * KV, D)
    pos = s["positions"].double()  # angles of far positions lose their fraction in 32 bits
    pos = pos[0].unsqueeze(1) if s["axis"] is None else pos[s["axis"].long()].T
    angle = pos * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)

    def turned(v):
        r = v[..., :rot]
        if c["pairs"] == "halves":
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([r, v[..., rot:]], -1)

    s["q"].copy_(turned(_normed(x[:, :H], s["q_norm"], c["plus_one"])))
    for name, rows in (("k_cache", turned(_normed(x[:, H:H + KV], s["k_norm"], c["plus_one"]))), ("v_cache", x[:, H + KV:])):
        s[name].view(-1, KV, D)[s["slots"]] = rows.to(torch.bfloat16)
    return s["q"], s["k_cache"], s["v_cache"]


def _attend_rows(s, seqs, rows, pos, keys):
    """Rows [b, m] of the new tokens, at positions pos (-1: none), of the sequences seqs, over the key positions keys [b, w] (-1: none)."""
    c = s["case"]
    H, KV, D = c["heads"], c["kv_heads"], c["dim"]
    b, m, w = len(seqs), rows.shape[1], keys.shape[1]
    page = s["table"][seqs].gather(1, keys.clamp_min(0) // c["page"]).long()
    k, v = (s[x][page, keys.clamp_min(0) % c["page"]].float().permute(0, 2, 1, 3).reshape(b * KV, w, D) for x in ("k_cache", "v_cache"))
    q = s["queries"][rows].float().view(b, m, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(b * KV, -1, D)
    score = (torch.bmm(q, k.transpose(1, 2)) / math.sqrt(D)).view(b, KV, m, H // KV, w)
    key, at = keys.unsqueeze(1), pos.unsqueeze(2)
    seen = (key >= 0) & (key <= at)
    if c["window"]:
        seen &= (key > at - c["window"]) | (key < c["sinks"])
    score.masked_fill_(~seen.view(b, 1, m, 1, w), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(b * KV, -1, w), v).view(b, KV, m, H // KV, D) / total
    lse = (top + torch.log(total)).squeeze(-1)
    real = pos >= 0
    s["out"][rows[real]] = o.permute(0, 2, 1, 3, 4).reshape(b, m, H, D)[real].to(torch.bfloat16)
    s["lse"][rows[real]] = lse.permute(0, 2, 1, 3).reshape(b, m, H)[real]


def _attend(s):
    c = s["case"]
    W, S = c["window"], c["sinks"]
    start, length = s["q_start"].long(), s["kv_len"].long()
    if c["new"] <= 16:  # all sequences at once, padded to the longest
        new = (start[1:] - start[:-1]).unsqueeze(1)
        step = torch.arange(c["new"], device="cuda")
        length = length.unsqueeze(1)
        pos = torch.where(step < new, length - new + step, -1)
        rows = torch.where(step < new, start[:-1].unsqueeze(1) + step, 0)
        wide = max(s["ctx"])
        if W and wide > W + S + c["new"]:
            tail = length - (W + c["new"]) + torch.arange(W + c["new"], device="cuda")
            keys = torch.cat([torch.arange(S, device="cuda").expand(c["B"], S), torch.where(tail >= S, tail, -1)], 1)
        else:
            keys = torch.arange(wide, device="cuda").expand(c["B"], wide)
        _attend_rows(s, torch.arange(c["B"], device="cuda"), rows, pos, torch.where(keys < length, keys, -1))
        return s["out"], s["lse"]
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["ctx"])):  # prompts: blocks of tokens over the keys that any of them sees
        step = min(1024, max(1, (1 << 30) // (c["heads"] * L)))
        for t in range(0, n, step):
            m, first = min(step, n - t), L - n + t
            low = max(0, first - W + 1) if W else 0
            keys = torch.cat([torch.arange(min(S if W else 0, low), device="cuda"), torch.arange(low, first + m, device="cuda")])
            block = torch.arange(m, device="cuda").unsqueeze(0)
            _attend_rows(s, torch.tensor([b], device="cuda"), at + t + block, first + block, keys.unsqueeze(0))
        at += n
    return s["out"], s["lse"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _rope, "attend": _attend}[c["op"]](s)
    import group_quantized_mat_gb300 as g
    if c["op"] == "rope":
        flags = (g.ROPE_F32_IN if c["f32"] else 0) | (g.ROPE_NEIGHBOURS if c["pairs"] == "neighbours" else 0) | (g.ROPE_NORM_PLUS_ONE if c["plus_one"] else 0)
        g.qmv_rope_run(s["qkv"], s["q_norm"], s["k_norm"], s["positions"], s["inv_freq"], s["axis"], s["slots"], s["q"], s["k_cache"], s["v_cache"],
                       c["T"], c["heads"], c["kv_heads"], c["dim"], c["rot"], c["page"], s["pages"], axes=c["axes"], eps=_EPS, flags=flags)
        return s["q"], s["k_cache"], s["v_cache"]
    g.qmv_attend_run(s["queries"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"], s["out"], s["lse"], c["B"], len(s["queries"]), c["new"],
                     c["heads"], c["kv_heads"], c["dim"], c["page"], s["pages"], s["most"], window=c["window"], sinks=c["sinks"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------- bounds --
def _visible(first, last, window, sinks):
    """Keys that the query positions first .. last see, summed over the positions, and how many different ones."""
    if not window:
        return (first + 1 + last + 1) * (last - first + 1) // 2, last + 1
    pairs = sum(min(p + 1, window) + max(0, min(sinks, p + 1 - window)) for p in range(first, last + 1))
    low = max(0, first - window + 1)
    return pairs, last + 1 - low + min(sinks, low)


def work(case):
    c = case
    H, KV, D = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "rope":
        T = c["T"]
        return {"bytes": T * (H + 2 * KV) * D * ((4 if c["f32"] else 2) + 2) + T * (8 + 4 * c["axes"]),
                "flops": T * (H + KV) * (D * (4 if c["norm"] else 0) + 3 * c["rot"])}
    nbytes = flops = 0
    for n, L in zip(*_lengths(c)):
        pairs, keys = _visible(L - n, L - 1, c["window"], c["sinks"])
        nbytes += keys * KV * D * 4 + n * H * (4 * D + 4) + 4 * (-(-L // c["page"]))
        flops += 4 * pairs * H * D
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------- values in 64 bits --
def _exact_rope(s):
    c = s["case"]
    T, H, KV, D, half = c["T"], c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    heads = s["qkv"].double().reshape(T, -1, D).clone()
    for lo, hi, w in ((0, H, s["q_norm"]), (H, H + KV, s["k_norm"])):
        if w is not None:
            part = heads[:, lo:hi]
            size = (part.pow(2).sum(-1, keepdim=True) / D + _EPS).sqrt()
            heads[:, lo:hi] = part / size * (w.double() + int(c["plus_one"]))
    both = heads[:, :H + KV]
    for i in range(half):
        a, b = (i, i + half) if c["pairs"] == "halves" else (2 * i, 2 * i + 1)
        pos = s["positions"][0 if s["axis"] is None else int(s["axis"][i])].double()
        turn = torch.polar(torch.ones_like(pos), pos * float(s["inv_freq"][i]))
        z = torch.complex(both[:, :, a], both[:, :, b]) * turn.unsqueeze(-1)
        both[:, :, a], both[:, :, b] = z.real, z.imag
    out = [heads[:, :H]]
    for name, lo in (("k_cache", H), ("v_cache", H + KV)):
        cache = s[name].double()
        page, place = s["slots"] // c["page"], s["slots"] % c["page"]
        cache[page, place] = heads[:, lo:lo + KV]
        out.append(cache)
    return tuple(out)


def _exact_attend(s):
    c = s["case"]
    H, KV, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros((len(s["queries"]), H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["ctx"])):
        where = torch.arange(L, device="cuda")
        page, place = s["table"][b].long()[where // P], where % P
        for h in range(H):
            k, v = (s[x][page, place, h * KV // H].double() for x in ("k_cache", "v_cache"))
            for t in range(0, n, 2048):
                rows = slice(at + t, at + min(t + 2048, n))
                mine = torch.arange(L - n, L, device="cuda")[t:t + 2048]
                away = mine.unsqueeze(1) - where
                hidden = away < 0
                if c["window"]:
                    hidden |= (away >= c["window"]) & (where >= c["sinks"])
                z = (s["queries"][rows, h].double() @ k.mT / D ** 0.5).masked_fill(hidden, -math.inf)
                lse[rows, h] = torch.logsumexp(z, -1)
                out[rows, h] = torch.softmax(z, -1) @ v
        at += n
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend}[case["op"]](s)
