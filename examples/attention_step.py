"""A decode loop through an attention layer with a paged cache, on a toy model.

    python examples/attention_step.py [--batch 4] [--prompt 300] [--tokens 48] [--drafts 4] [--window 0] [--sinks 0]

One layer: quantized projections of queries, keys and values (qmv_run), their norms,
rotation and the write to the cache (qmv_rope_run), attention over the cache
(qmv_attend_run) and the quantized output projection; then a vocabulary projection. The
weights are random. Prompts go in chunks of at most 256 rows; after them each step takes
the last token and `drafts` drafted ones (here: the tokens that followed last time the
last token was seen) and keeps the accepted ones (qmv_verify_run, greedy). A refused draft's
keys stay in the cache behind the sequence's length, where nothing reads them until they
are written over. The step is captured in a CUDA graph.

The emitted tokens are those of decoding one token at a time, bit for bit: no operator's
result for a token depends on the tokens drafted with it. That holds for up to 16 tokens
of a sequence in a step, the last one and 15 drafted ones, and for caches with room for as
many keys (qmv_attend_run); a step takes 256 rows in all (qmv_run).
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import group_quantized_mat_gb300 as g  # noqa: E402

BITS, GROUP = 4, 64


def packed(rows, cols, gen, size=0.4):
    w = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols * BITS // 32), dtype=torch.int32, device="cuda", generator=gen)
    s = (torch.rand((rows, cols // GROUP), device="cuda", generator=gen) + 0.5) * size / cols ** 0.5
    return w, s.bfloat16(), (s * -7.5).bfloat16()


class Model:
    def __init__(self, vocab=4096, width=1024, heads=8, kv_heads=2, head_dim=128, window=0, sinks=0, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.vocab, self.width, self.heads, self.kv_heads, self.head_dim = vocab, width, heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        self.embed = torch.randn(vocab, width, device="cuda", generator=gen).bfloat16()
        self.qkv = packed((heads + 2 * kv_heads) * head_dim, width, gen)
        self.out = packed(width, heads * head_dim, gen)
        self.head = packed(vocab, width, gen)
        self.q_norm, self.k_norm = ((torch.rand(head_dim, device="cuda", generator=gen) + 0.5).bfloat16() for _ in range(2))
        half = head_dim // 2
        self.inv_freq = (10000.0 ** (-torch.arange(half, device="cuda") / half)).float()


class Decoder:
    """`batch` sequences of up to `room` tokens, `drafts` drafted ones a step."""

    def __init__(self, model, batch, room, drafts, page=16):
        if not 0 <= drafts < g.QMV_TILE_M:
            raise ValueError(f"{drafts} drafted tokens: 0 to {g.QMV_TILE_M - 1}, as those of more are not bit for bit those of single tokens")
        if not 1 <= batch * (drafts + 1) <= g.QMV_MAX_M:
            raise ValueError(f"{batch} sequences of {drafts + 1} tokens a step: 1 to {g.QMV_MAX_M} rows")
        self.model, self.B, self.S, self.page = model, batch, drafts, page
        self.per = -(-(room + g.QMV_TILE_M) // page)  # (whatever `drafts` is: sums are divided by the room)
        self.pages = batch * self.per
        shape = (self.pages, page, model.kv_heads, model.head_dim)
        self.k, self.v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.randperm(self.pages, device="cuda").int().view(batch, self.per)
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")  # tokens whose keys are cached for good
        self.last = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.after = torch.zeros(batch, model.vocab, dtype=torch.int32, device="cuda")  # the token seen after each
        self.tokens = torch.empty(batch, drafts + 1, dtype=torch.int32, device="cuda")
        self.accepted = torch.empty(batch, dtype=torch.int32, device="cuda")
        self.zeros, self.ones = torch.zeros(batch, max(drafts, 1), device="cuda"), torch.ones(batch, model.vocab, device="cuda")
        self.graph = None

    def layer(self, tokens):
        """The rows [batch, n] of tokens at the sequences' ends, through the layer; their keys go behind `length`."""
        m, (B, n) = self.model, tokens.shape
        M, h, kv, D = B * n, m.heads, m.kv_heads, m.head_dim
        wide = (h + 2 * kv) * D
        empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        x, both, q, a, y = m.embed[tokens.reshape(-1).long()], empty(M, wide), empty(M, h, D), empty(M, h, D), empty(M, m.width)
        at = self.length[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
        slots = self.table.long().gather(1, at.long() // self.page) * self.page + at % self.page
        g.qmv_run(*m.qkv, x, both, M, wide, m.width, BITS, GROUP)
        g.qmv_rope_run(both, m.q_norm, m.k_norm, at.reshape(1, M).contiguous(), m.inv_freq, None, slots.reshape(M).contiguous(), q, self.k, self.v,
                       M, h, kv, D, D, self.page, self.pages)
        g.qmv_attend_run(q, self.k, self.v, self.table, None, self.length + n, a, None, B, M, n, h, kv, D, self.page, self.pages, self.per,
                         window=m.window, sinks=m.sinks)
        g.qmv_run(*m.out, a, y, M, m.width, h * D, BITS, GROUP)
        return x + y

    def prompt(self, tokens):
        """All but the last of the tokens [batch, n] into the cache, in chunks."""
        step = 256 // self.B
        for t in range(0, tokens.shape[1] - 1, step):
            chunk = tokens[:, t:min(t + step, tokens.shape[1] - 1)]
            self.layer(chunk)
            self.length += chunk.shape[1]
        self.last.copy_(tokens[:, -1])

    def step(self):
        m, B, S = self.model, self.B, self.S
        drafted, token = [], self.last
        for _ in range(S):
            token = self.after.gather(1, token[:, None].long())[:, 0]
            drafted.append(token)
        drafted = torch.stack(drafted, 1) if S else None
        x = self.layer(torch.cat([self.last[:, None], drafted], 1) if S else self.last[:, None])
        logits = torch.empty(B, S + 1, m.vocab, dtype=torch.bfloat16, device="cuda")
        g.qmv_run(*m.head, x, logits, B * (S + 1), m.vocab, m.width, BITS, GROUP)
        g.qmv_verify_run(logits, None, drafted, None, self.zeros[:, 0].contiguous(), self.zeros if S else None, self.ones, self.tokens, self.accepted, None, B, S,
                         m.vocab)
        before = torch.cat([self.last[:, None], self.tokens[:, :-1]], 1)
        real = self.tokens >= 0
        self.after.scatter_(1, torch.where(real, before, self.last[:, None]).long(), torch.where(real, self.tokens, self.tokens[:, :1]))
        self.length += self.accepted + 1
        self.last.copy_(self.tokens.gather(1, self.accepted.long()[:, None])[:, 0])

    def generate(self, count):
        """At least `count` tokens for each sequence, and the steps it took."""
        out, steps = [[] for _ in range(self.B)], 0
        while min(map(len, out)) < count:
            if steps == 0:
                self.step()  # the first step runs as it is: workspaces are made
            else:
                if self.graph is None:
                    torch.cuda.synchronize()
                    self.graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(self.graph):
                        self.step()
                self.graph.replay()
            steps += 1
            for b, row in enumerate(self.tokens.tolist()):
                out[b] += [t for t in row if t >= 0]
        return [o[:count] for o in out], steps


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("batch", 4), ("prompt", 300), ("tokens", 48), ("drafts", 4), ("window", 0), ("sinks", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    model = Model(window=a.window, sinks=a.sinks)
    tokens = torch.randint(0, model.vocab, (a.batch, a.prompt), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    for drafts in (0, a.drafts):
        d = Decoder(model, a.batch, a.prompt + (a.drafts + 1) * a.tokens, drafts)
        d.prompt(tokens)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        _, steps = d.generate(a.tokens)
        torch.cuda.synchronize()
        print(f"{drafts} drafted tokens: {a.tokens / steps:.2f} tokens a step, {(time.perf_counter() - t0) / steps * 1e6:.0f} us a step")
    assert g.qmv_device_error() == 0


if __name__ == "__main__":
    main()
