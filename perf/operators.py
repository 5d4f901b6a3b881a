"""Cases, plain forms and 64-bit values of the operators of a quantized decode step.

Three operators stand next to the group-quantized mat-vec in one step of
speculative decoding, in which a few drafted tokens go through a model at once:

* ``lora``: a group-quantized projection shared by all tokens, plus each token's
  own low-rank adapter: y = W x + scale_a B_a (A_a x).
* ``moe``: a whole mixture-of-experts layer whose experts are group-quantized:
  router, top-k, gate/up products, activation, down product, weighted sum.
* ``verify``: the drafted tokens against the target's probabilities, from given
  random numbers: accepted prefix, the token after it, log-probabilities.

Quantized weights are packed words, element 0 in the low bits, with one bf16
scale and one bf16 bias for each group along K.
"""

import math

import torch

own = False

_VERIFY_TINY = 1.1754943508222875e-38  # least race time, the smallest normal number


# ---------------------------------------------------------------- the cases --
def listed():
    return [
        # one decoded token through a key/value-sized projection with its adapter: latency
        dict(name="lora one token", op="lora", M=1, N=1024, K=5120, bits=4, group=64, adapters=4, rank=16, none=0.0),
        # four drafted tokens of one request mix through an up projection
        dict(name="lora draft of 4", op="lora", M=4, N=15360, K=3840, bits=4, group=64, adapters=8, rank=16, none=0.25),
        # a full verify width through the long-K down projection, odd rank
        dict(name="lora 13 long K", op="lora", M=13, N=3840, K=15360, bits=4, group=128, adapters=16, rank=27, none=0.2),
        # a batch of requests, 2-bit weights, higher rank
        dict(name="lora batch of 64", op="lora", M=64, N=17408, K=5120, bits=2, group=64, adapters=12, rank=64, none=0.1),
        # one token, many small experts
        dict(name="moe one token", op="moe", M=1, K=2048, inter=768, experts=64, top_k=8, bits=4, group=64, act="silu", renorm=True),
        # a draft of five tokens, few larger experts, 2-bit
        dict(name="moe draft of 5", op="moe", M=5, K=3840, inter=1920, experts=8, top_k=2, bits=2, group=128, act="gelu", renorm=False),
        # a full verify width over many experts: nearly all of them are read
        dict(name="moe 16 many experts", op="moe", M=16, K=2048, inter=768, experts=128, top_k=8, bits=4, group=64, act="silu", renorm=True),
        # a small batch over larger experts
        dict(name="moe batch of 48", op="moe", M=48, K=5120, inter=1280, experts=32, top_k=4, bits=4, group=128, act="silu", renorm=True),
        # one request, three drafted tokens, a small vocabulary
        dict(name="verify one request", op="verify", B=1, S=3, V=32000, pad=0, dtype="bf16", draft=True, greedy=0.0),
        # eight requests, fp32 logits, an odd vocabulary whose rows are not aligned
        dict(name="verify 8 odd f32", op="verify", B=8, S=4, V=50257, pad=0, dtype="f32", draft=True, greedy=0.25),
        # drafts without probabilities (looked up, not sampled), padded rows
        dict(name="verify 24 looked up", op="verify", B=24, S=12, V=101001, pad=23, dtype="bf16", draft=False, greedy=0.5),
        # a large batch over a large vocabulary
        dict(name="verify 64 large", op="verify", B=64, S=7, V=131072, pad=0, dtype="bf16", draft=True, greedy=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, unit, lo, hi):
    """A multiple of unit between lo and hi, spread over its logarithm; not of three units, so that it splits unevenly over most tilings."""
    n = _log(rng, -(-lo // unit), hi // unit)
    return unit * (n if n % 3 else n - 1 if n > 3 else n + 1)


def draw(rng):
    op = rng.choice(["lora", "moe", "verify"])
    bits, group = rng.choice([4, 4, 2]), rng.choice([64, 128])
    if op == "lora":
        return dict(op=op, M=_log(rng, 1, 64), N=_size(rng, 1, 250, 17408), K=_size(rng, group, 512, 15360), bits=bits, group=group,
                    adapters=rng.randint(1, 16), rank=rng.choice([4, 8, 16, 32, 64, rng.randint(1, 64)]), none=rng.choice([0.0, 0.25, 0.9]))
    if op == "moe":
        experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
        K, inter = _size(rng, group, 512, 5120), _size(rng, group, 256, 1920)
        return dict(op=op, M=_log(rng, 1, 48), K=K, inter=inter, experts=experts, top_k=rng.randint(1, min(8, experts)), bits=bits, group=group,
                    act=rng.choice(["silu", "gelu"]), renorm=rng.random() < 0.7)
    return dict(op=op, B=_log(rng, 1, 48), S=rng.randint(1, 9), V=_size(rng, 1, 1000, 131072), pad=rng.choice([0, 0, 5, 64]),
                dtype=rng.choice(["bf16", "bf16", "f32"]), draft=rng.random() < 0.75, greedy=rng.choice([0.0, 0.0, 0.3, 1.0]))


# --------------------------------------------------------------- the inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantized(shape, K, bits, group, gen):
    """Packed words, scales and biases of a checkpoint's matrix [*shape, K]: fields uniform, weights about 0.05 in size."""
    w = torch.randint(-(1 << 31), 1 << 31, (*shape, K * bits // 32), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    s = (torch.rand((*shape, K // group), generator=gen, device="cuda") * 0.019 + 0.001).to(torch.bfloat16)
    b = (torch.randn(s.shape, generator=gen, device="cuda") * 1e-3 - (1 << (bits - 1)) * s.float()).to(torch.bfloat16)
    return w, s, b


def prepare(case, seed):
    gen = _gen(seed)
    c = case
    s = dict(case=c)
    if c["op"] == "lora":
        M, N, K, L, R = c["M"], c["N"], c["K"], c["adapters"], c["rank"]
        s["w"], s["scales"], s["biases"] = _quantized((N,), K, c["bits"], c["group"], gen)
        s["x"] = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
        s["a"] = (torch.randn((L, R, K), generator=gen, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (torch.randn((L, N, R), generator=gen, device="cuda") * 0.5).to(torch.bfloat16)
        ids = torch.randint(0, L, (M,), generator=gen, device="cuda", dtype=torch.int32)
        off = torch.rand((M,), generator=gen, device="cuda") < c["none"]
        s["ids"] = torch.where(off, torch.full_like(ids, -1), ids)
        s["alpha"] = torch.rand((L,), generator=gen, device="cuda") * 1.5 + 0.5
        s["y"] = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
    elif c["op"] == "moe":
        M, K, I, E = c["M"], c["K"], c["inter"], c["experts"]
        s["gu"] = _quantized((E, 2 * I), K, c["bits"], c["group"], gen)
        s["dn"] = _quantized((E, K), I, c["bits"], c["group"], gen)
        s["x"] = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
        s["router"] = (torch.randn((E, K), generator=gen, device="cuda") * (1.5 / math.sqrt(K))).to(torch.bfloat16)
        s["y"] = torch.empty((M, K), device="cuda", dtype=torch.bfloat16)
        s["ids"] = torch.empty((M, c["top_k"]), device="cuda", dtype=torch.int32)
        s["weights"] = torch.empty((M, c["top_k"]), device="cuda", dtype=torch.float32)
    else:
        B, S, V = c["B"], c["S"], c["V"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        ld = V + c["pad"]
        # logits of a language model: a wide bulk and a few tokens that stand out; the draft's are near the target's
        base = torch.randn((B, S + 1, ld), generator=gen, device="cuda") * 2.0
        peak = torch.randint(0, V, (B, S + 1, 8), generator=gen, device="cuda")
        base.scatter_add_(2, peak, torch.rand(peak.shape, generator=gen, device="cuda") * 6.0 + 8.0)
        masked = torch.rand((ld,), generator=gen, device="cuda") < 0.02  # tokens that the request's grammar forbids
        base.masked_fill_(masked, -math.inf)
        s["target"] = base.to(dt)
        near = base[:, :S] + torch.randn((B, S, ld), generator=gen, device="cuda") * 0.7
        del base
        s["draft"] = near.to(dt) if c["draft"] else None
        race = torch.empty((B, S, ld), device="cuda").exponential_(generator=gen).clamp_min_(_VERIFY_TINY)
        s["tokens"] = (torch.softmax(near.to(dt)[..., :V].float(), -1) / race[..., :V]).argmax(-1).to(torch.int32)
        del near, race
        s["len"] = torch.randint(0, S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32).clamp_min((S + 1) // 2) if B > 1 else torch.full((B,), S, device="cuda", dtype=torch.int32)
        t = torch.rand((B,), generator=gen, device="cuda") * 0.6 + 0.6
        s["temperature"] = torch.where(torch.rand((B,), generator=gen, device="cuda") < c["greedy"], torch.zeros_like(t), t)
        s["uniform"] = torch.rand((B, S), generator=gen, device="cuda")
        s["noise"] = torch.empty((B, V), device="cuda").exponential_(generator=gen)
        s["out_tokens"] = torch.empty((B, S + 1), device="cuda", dtype=torch.int32)
        s["accepted"] = torch.empty((B,), device="cuda", dtype=torch.int32)
        s["logprob"] = torch.empty((B, S + 1), device="cuda", dtype=torch.float32)
    return s


# ----------------------------------------------------------- the operators --
def _fields(w, bits):
    """Packed words [..., W] -> fields [..., W * 32 / bits] as fp32."""
    shifts = torch.arange(0, 32, bits, device=w.device, dtype=torch.int32)
    return ((w.unsqueeze(-1) >> shifts) & ((1 << bits) - 1)).flatten(-2).float()


def _matrix(w, s, b, bits):
    """The fp32 matrix of packed words with a scale and a bias for each group."""
    q = _fields(w, bits).unflatten(-1, (s.shape[-1], -1))
    return (q * s.float().unsqueeze(-1) + b.float().unsqueeze(-1)).flatten(-2)


def _lora(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ _matrix(s["w"], s["scales"], s["biases"], c["bits"]).T
    ids = s["ids"].long().clamp_min(0)
    v = torch.einsum("mrk,mk->mr", s["a"][ids].float(), x)
    d = torch.einsum("mnr,mr->mn", s["b"][ids].float(), v) * s["alpha"][ids].unsqueeze(-1)
    return (y + torch.where(s["ids"].unsqueeze(-1) >= 0, d, torch.zeros_like(d))).to(torch.bfloat16)


def _moe(s):
    c = s["case"]
    x = s["x"].float()
    M, E, k, I, bits = c["M"], c["experts"], c["top_k"], c["inter"], c["bits"]
    logits = x @ s["router"].float().T
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = order.values[:, :k], order.indices[:, :k]
    weights = torch.softmax(top, -1) if c["renorm"] else torch.softmax(logits, -1).gather(1, ids)
    # the experts computed: one for each (token, choice) while those are fewer, else all of them
    pairs = M * k < E
    used = ids.flatten() if pairs else torch.arange(E, device=x.device)
    share = torch.zeros((M, len(used)), device=x.device)
    col = torch.arange(M * k, device=x.device).view(M, k) if pairs else ids
    share.scatter_(1, col, weights)
    gu = _matrix(s["gu"][0][used], s["gu"][1][used], s["gu"][2][used], bits)
    h = torch.matmul(x, gu.transpose(1, 2))
    del gu
    gate, up = h[..., :I], h[..., I:]
    act = gate * torch.sigmoid(gate) if c["act"] == "silu" else 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)))
    dn = _matrix(s["dn"][0][used], s["dn"][1][used], s["dn"][2][used], bits)
    y = torch.matmul(act * up * share.T.unsqueeze(-1), dn.transpose(1, 2)).sum(0)
    return y.to(torch.bfloat16), ids.to(torch.int32), weights


def _first_max(v):
    """The index of the largest value in the last dimension, the lowest where several are equal."""
    n = v.shape[-1]
    at = torch.arange(n, device=v.device)
    return torch.where(v == v.amax(-1, keepdim=True), at, torch.full_like(at, n)).amin(-1)


def _verify(s):
    c = s["case"]
    B, S, V = c["B"], c["S"], c["V"]
    greedy = s["temperature"] == 0
    inv = (1.0 / torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"])).view(B, 1, 1)
    at = torch.arange(S + 1, device="cuda")
    drafted = s["tokens"].long()

    def soft(logits):
        t = logits[..., :V].float()
        z = (t - t.amax(-1, keepdim=True)) * inv
        e = torch.exp(z)
        total = e.sum(-1, keepdim=True)
        return z, e / total, total

    z, p, total = soft(s["target"])
    q = soft(s["draft"])[1] if c["draft"] else torch.zeros_like(p[:, :S]).scatter_(2, drafted.unsqueeze(-1), 1.0)
    pt, qt = p[:, :S].gather(2, drafted.unsqueeze(-1)).squeeze(-1), q.gather(2, drafted.unsqueeze(-1)).squeeze(-1)
    best = _first_max(s["target"][..., :V].float())
    ok = torch.where(greedy.unsqueeze(-1), best[:, :S] == drafted, s["uniform"] * qt < pt)
    ok &= at[:S] < s["len"].unsqueeze(-1)
    n = ok.long().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    row = p[b, n]
    less = torch.where((n < s["len"]).unsqueeze(-1), q[b, n.clamp_max(S - 1)], torch.zeros_like(row))
    rest = (row - less).clamp_min(0)
    rest = torch.where((rest > 0).any(-1, keepdim=True), rest, row)
    last = torch.where(greedy, best[b, n], _first_max(rest / s["noise"].clamp_min(_VERIFY_TINY)))
    draft = torch.cat([drafted, drafted[:, :1]], 1)
    out = torch.where(at < n.unsqueeze(-1), draft, torch.where(at == n.unsqueeze(-1), last.unsqueeze(-1), torch.full_like(draft, -1)))
    lp = z.gather(2, out.clamp_min(0).unsqueeze(-1)).squeeze(-1) - torch.log(total.squeeze(-1))
    return out.to(torch.int32), n.to(torch.int32), torch.where(out >= 0, lp, torch.zeros_like(lp))


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"lora": _lora, "moe": _moe, "verify": _verify}[c["op"]](s)
    import group_quantized_mat_gb300 as g
    if c["op"] == "lora":
        g.qmv_lora_run(s["w"], s["scales"], s["biases"], s["x"], s["a"], s["b"], s["ids"], s["alpha"], s["y"],
                       c["M"], c["N"], c["K"], c["bits"], c["group"], c["adapters"], c["rank"])
        return s["y"]
    if c["op"] == "moe":
        flags = (g.MOE_GELU if c["act"] == "gelu" else 0) | (0 if c["renorm"] else g.MOE_SOFTMAX_ALL)
        g.qmv_moe_run(s["x"], s["router"], *s["gu"], *s["dn"], s["y"], s["ids"], s["weights"],
                      c["M"], c["K"], c["inter"], c["experts"], c["top_k"], c["bits"], c["group"], flags=flags)
        return s["y"], s["ids"], s["weights"]
    ld = c["V"] + c["pad"]
    g.qmv_verify_run(s["target"], s["draft"], s["tokens"], s["len"], s["temperature"], s["uniform"], s["noise"],
                     s["out_tokens"], s["accepted"], s["logprob"], c["B"], c["S"], c["V"],
                     ld_target=ld, ld_draft=ld, ld_noise=c["V"], flags=g.VERIFY_F32_LOGITS if c["dtype"] == "f32" else 0)
    return s["out_tokens"], s["accepted"], s["logprob"]


# ------------------------------------------------------------------- bounds --
def _packed(rows, K, c):
    return rows * K * c["bits"] / 8 + 4 * rows * (K // c["group"])


def work(case):
    c = case
    if c["op"] == "lora":
        M, N, K, L, R = c["M"], c["N"], c["K"], c["adapters"], c["rank"]
        with_adapter = M * (1 - c["none"])
        seen = L * (1 - (1 - 1 / L) ** with_adapter)
        return {"bytes": _packed(N, K, c) + 2 * M * (K + N) + seen * 2 * R * (K + N), "flops": 2 * M * N * K + 2 * with_adapter * R * (K + N)}
    if c["op"] == "moe":
        M, K, I, E, k = c["M"], c["K"], c["inter"], c["experts"], c["top_k"]
        seen = E * (1 - (1 - k / E) ** M)
        return {"bytes": seen * (_packed(2 * I, K, c) + _packed(K, I, c)) + 2 * E * K + 4 * M * K + 8 * M * k, "flops": 2 * M * k * 3 * K * I + 2 * M * E * K}
    size = 2 if c["dtype"] == "bf16" else 4
    warm = 1 - c["greedy"]
    rows = c["B"] * (c["S"] + 1 + (c["S"] * warm if c["draft"] else 0))
    # a maximum, a difference, a scale, an exponential and a sum for each logit; noise for the row that is sampled
    return {"bytes": rows * c["V"] * size + c["B"] * c["V"] * 4 * warm + 12 * c["B"] * (c["S"] + 1), "flops": rows * c["V"] * 5 + c["B"] * c["V"] * 6 * warm}


# ------------------------------------------------------- values in 64 bits --
def _wide(w, s, b, bits, group):
    """The matrix in 64 bits, from the words' bytes: the fields of a byte are its `bits`-wide digits, the lowest first."""
    digits = w.contiguous().view(torch.uint8).to(torch.int64)
    cols = []
    for _ in range(8 // bits):
        cols.append(digits % (1 << bits))
        digits = digits // (1 << bits)
    q = torch.stack(cols, -1).reshape(w.shape[0], -1).double()
    return q * s.double().repeat_interleave(group, 1) + b.double().repeat_interleave(group, 1)


def _exact_lora(s):
    c = s["case"]
    x = s["x"].double()
    y = x @ _wide(s["w"], s["scales"], s["biases"], c["bits"], c["group"]).mT
    for m, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            y[m] += float(s["alpha"][a]) * (s["b"][a].double() @ (s["a"][a].double() @ x[m]))
    return y


def _exact_moe(s):
    c = s["case"]
    x = s["x"].double()
    M, K, I, k = c["M"], c["K"], c["inter"], c["top_k"]
    logits = (x @ s["router"].double().mT).cpu()
    y = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    weights = torch.zeros((M, k), dtype=torch.float64)
    members = {}
    for m in range(M):
        row = logits[m].tolist()
        ids = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        top = max(row)
        mass = [math.exp(row[e] - top) for e in ids]
        whole = sum(mass) if c["renorm"] else sum(math.exp(v - top) for v in row)
        for j, e in enumerate(ids):
            weights[m, j] = mass[j] / whole
            members.setdefault(e, []).append((m, mass[j] / whole))
    for e, tokens in members.items():
        at = torch.tensor([m for m, _ in tokens], device="cuda")
        h = x[at] @ _wide(*(t[e] for t in s["gu"]), c["bits"], c["group"]).mT
        gate, up = h[:, :I], h[:, I:]
        if c["act"] == "silu":
            act = gate / (1 + torch.exp(-gate))
        else:
            act = gate / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)))
        d = (act * up) @ _wide(*(t[e] for t in s["dn"]), c["bits"], c["group"]).mT
        y.index_add_(0, at, d * torch.tensor([w for _, w in tokens], dtype=torch.float64, device="cuda").unsqueeze(-1))
    return y, None, weights


def _exact_verify(s):
    """The log-probabilities of the emitted tokens; the tokens themselves are whole numbers."""
    c = s["case"]
    B, S, V = c["B"], c["S"], c["V"]
    logprob = torch.zeros((B, S + 1), dtype=torch.float64)
    temps, lens = s["temperature"].double().tolist(), s["len"].tolist()
    for b in range(B):
        t = temps[b] if temps[b] > 0 else 1.0
        lp = torch.log_softmax(s["target"][b, :, :V].double() / t, -1)
        lq = torch.log_softmax(s["draft"][b, :, :V].double() / t, -1) if c["draft"] else None
        for i in range(S + 1):
            drafted = int(s["tokens"][b, i]) if i < lens[b] else None
            if temps[b] == 0:
                last = int((lp[i] == lp[i].max()).nonzero()[0])
                take = drafted == last
            else:
                p = lp[i].exp()
                q = torch.zeros_like(p)
                if drafted is not None:
                    if lq is None:
                        q[drafted] = 1.0
                    else:
                        q = lq[i].exp()
                take = drafted is not None and float(s["uniform"][b, i]) * float(q[drafted]) < float(p[drafted])
                if not take:
                    rest = (p - q).clamp_min(0)
                    last = int(((rest if bool((rest > 0).any()) else p) / s["noise"][b].double().clamp_min(_VERIFY_TINY)).argmax())
            logprob[b, i] = lp[i, drafted if take else last]
            if not take:
                break
    return None, None, logprob


def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "moe": _exact_moe, "verify": _exact_verify}[case["op"]](s)
