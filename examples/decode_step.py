"""Speculative decoding with the operators of a decode step, on a toy model.

    python examples/decode_step.py [--tokens 64] [--drafts 4] [--batch 4] [--temperature 0.8]

The model has no attention: the next token depends on the current one, through a
mixture-of-experts layer and a vocabulary projection that every request sees
through its own low-rank adapter. Its weights are random. The drafts come from
the same projection without the layer and the adapter, one token at a time; then
one pass takes all drafted tokens of all requests through the layer
(qmv_moe_run), the adapted projection (qmv_lora_run) and the verification
(qmv_verify_run). The step allocates nothing and is captured in a CUDA graph.

At temperature 0 the emitted tokens are those of decoding one token at a time, bit
for bit: no operator's result for a token depends on the other tokens of its call.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import group_quantized_mat_gb300 as g  # noqa: E402

BITS, GROUP = 4, 64


def packed(rows, cols, scale, gen):
    """Random weights of a group-quantized matrix: words, scales, biases."""
    w = torch.randint(-2 ** 31, 2 ** 31 - 1, (*rows, cols * BITS // 32), dtype=torch.int32, device="cuda", generator=gen)
    s = (torch.rand((*rows, cols // GROUP), device="cuda", generator=gen) + 0.5) * scale
    return w, s.bfloat16(), (s * -7.5).bfloat16()


class Model:
    def __init__(self, vocab=8192, width=1024, inter=512, experts=16, top_k=4, adapters=3, rank=16, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        randn = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
        self.vocab, self.width, self.inter, self.experts, self.top_k = vocab, width, inter, experts, top_k
        self.adapters, self.rank = adapters, rank
        self.embed = randn(vocab, width).bfloat16()
        self.router = (randn(experts, width) / width ** 0.5).bfloat16()
        self.gate_up = packed((experts, 2 * inter), width, 0.2 / width ** 0.5, gen)
        self.down = packed((experts, width), inter, 0.1 / inter ** 0.5, gen)
        self.head = packed((vocab,), width, 0.4 / width ** 0.5, gen)
        self.lora_a = (randn(adapters, rank, width) / width ** 0.5).bfloat16()
        self.lora_b = (randn(adapters, vocab, rank) / rank ** 0.5).bfloat16()
        self.lora_scale = torch.full((adapters,), 0.5, device="cuda")


class Decoder:
    """`batch` requests, each with its adapter (negative: none), up to `drafts` drafted tokens a step."""

    def __init__(self, model, batch, drafts, adapter, temperature, seed=1):
        m, self.model, self.B, self.S = model, model, batch, drafts
        M = self.M = batch * (drafts + 1)
        empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        self.adapter = torch.as_tensor(adapter, dtype=torch.int32, device="cuda").repeat_interleave(drafts + 1)
        self.temperature = torch.full((batch,), float(temperature), device="cuda")
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.last = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.drafted = empty(batch, max(drafts, 1), dtype=torch.int32)
        self.draft_x = empty(batch, m.width, dtype=torch.bfloat16)
        self.draft_logits = empty(max(drafts, 1), batch, m.vocab, dtype=torch.bfloat16)
        self.draft_rows = empty(batch, max(drafts, 1), m.vocab, dtype=torch.bfloat16)
        self.x = empty(M, m.width, dtype=torch.bfloat16)
        self.layer = empty(M, m.width, dtype=torch.bfloat16)
        self.logits = empty(batch, drafts + 1, m.vocab, dtype=torch.bfloat16)
        self.uniform = empty(batch, max(drafts, 1))
        self.noise = empty(drafts + 1, batch, m.vocab)
        self.tokens = empty(batch, drafts + 1, dtype=torch.int32)
        self.accepted = empty(batch, dtype=torch.int32)
        self.logprob = empty(batch, drafts + 1)
        self.bytes = max(g.qmv_workspace_size(batch, m.vocab, m.width, BITS, GROUP),
                         g.qmv_moe_workspace_size(M, m.width, m.inter, m.experts, m.top_k, BITS, GROUP),
                         g.qmv_lora_workspace_size(M, m.vocab, m.width, BITS, GROUP, m.rank),
                         g.qmv_verify_workspace_size(batch, drafts, m.vocab), 16)
        self.workspace = empty(self.bytes, dtype=torch.uint8)
        self.graph = None

    def draft(self):
        """Drafted tokens, sampled one after the other from the projection alone."""
        m, token = self.model, self.last
        for i in range(self.S):
            torch.index_select(m.embed, 0, token, out=self.draft_x)
            g.qmv_run_ex(*m.head, self.draft_x, self.draft_logits[i], self.B, m.vocab, m.width, BITS, GROUP, self.workspace, self.bytes)
            logits = self.draft_logits[i].float()
            t = self.temperature[:, None]
            race = torch.softmax(logits / t.clamp_min(1e-6), -1) / self.noise[i]
            token = torch.where(t[:, 0] > 0, race.argmax(-1), logits.argmax(-1)).int()
            self.drafted[:, i] = token
        self.draft_rows.copy_(self.draft_logits.transpose(0, 1))

    def verify(self):
        """One pass of the model over the last token and the drafts, and what is kept of them."""
        m, B, S, M = self.model, self.B, self.S, self.M
        tokens = torch.cat([self.last[:, None], self.drafted[:, :S]], 1).reshape(-1)
        torch.index_select(m.embed, 0, tokens, out=self.x)
        g.qmv_moe_run(self.x, m.router, *m.gate_up, *m.down, self.layer, None, None, M, m.width, m.inter, m.experts, m.top_k,
                      BITS, GROUP, self.workspace, self.bytes)
        self.layer.add_(self.x)
        g.qmv_lora_run(*m.head, self.layer, m.lora_a, m.lora_b, self.adapter, m.lora_scale, self.logits, M, m.vocab, m.width,
                       BITS, GROUP, m.adapters, m.rank, self.workspace, self.bytes)
        g.qmv_verify_run(self.logits, self.draft_rows if S else None, self.drafted if S else None, None, self.temperature,
                         self.uniform if S else None, self.noise[S], self.tokens, self.accepted, self.logprob, B, S, m.vocab,
                         workspace=self.workspace, workspace_bytes=self.bytes)
        self.last.copy_(self.tokens.gather(1, self.accepted.long()[:, None])[:, 0])

    def step(self):
        """One step; its results stay in tokens, accepted and logprob until the next."""
        self.uniform.uniform_(generator=self.gen)
        self.noise.exponential_(generator=self.gen)
        if self.graph is None:
            last = self.last.clone()
            self.draft()  # the first step runs once as it is: libraries set themselves up
            self.verify()
            self.last.copy_(last)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.draft()
                self.verify()
        self.graph.replay()

    def generate(self, first, count):
        """At least `count` tokens for each request after `first`; also the steps it took."""
        self.last.copy_(torch.as_tensor(first, dtype=torch.int32))
        out, steps = [[] for _ in range(self.B)], 0
        while min(map(len, out)) < count:
            self.step()
            steps += 1
            for b, row in enumerate(self.tokens.tolist()):
                out[b] += [t for t in row if t >= 0]
        return out, steps


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    model = Model()
    adapter = [b % (model.adapters + 1) - 1 for b in range(a.batch)]
    first = list(range(1, a.batch + 1))
    for drafts in (0, a.drafts):
        d = Decoder(model, a.batch, drafts, adapter, a.temperature)
        d.generate(first, 2)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        out, steps = d.generate(first, a.tokens)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        made = sum(map(len, out))
        print(f"{drafts} drafted tokens: {made / steps / a.batch:.2f} tokens a step and request, {took / steps * 1e6:.0f} us a step")
    assert g.qmv_device_error() == 0


if __name__ == "__main__":
    main()
