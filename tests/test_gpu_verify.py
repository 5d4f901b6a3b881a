"""qmv_verify_run on the GPU against the 64-bit rule. Tokens are compared where
no decision lies within 1e-5 of its boundary (fp32 cannot settle those)."""

import math

import numpy as np
import pytest
import torch

import group_quantized_mat_gb300 as g
import operators_reference as ref
from gpu_helpers import dev

pytestmark = pytest.mark.gpu
BIG = {"bf16": 3.3895313892515355e38, "f32": 3.4028234663852886e38}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    g.load()


class Batch:
    def __init__(self, B, S, V, dtype="bf16", pad=0, draft=True, greedy=0.0, seed=0, lens=None, spread=2.5):
        rng = np.random.default_rng(seed)
        self.B, self.S, self.V, self.ld, self.dtype = B, S, V, V + pad, dtype
        t = rng.standard_normal((B, S + 1, self.ld)) * spread
        self.target = self.round(t)
        self.draft = self.round(t[:, :S] + rng.standard_normal((B, S, self.ld)) * 0.8) if draft and S else None
        near = t[:, :S, :V] + rng.gumbel(size=(B, S, V))
        self.tokens = np.argmax(near, -1).astype(np.int32).reshape(B, S)
        self.lens = np.asarray(rng.integers(0, S + 1, B) if lens is None else lens, dtype=np.int32)
        self.temp = np.where(rng.random(B) < greedy, 0.0, rng.uniform(0.5, 1.5, B)).astype(np.float32)
        self.uniform = rng.random((B, S)).astype(np.float32)
        self.noise = rng.exponential(size=(B, self.ld)).astype(np.float32)

    def round(self, a):
        return ref.bf(ref.to_bf16(a)) if self.dtype == "bf16" else np.asarray(a, dtype=np.float32).astype(np.float64)

    def logits(self, a):
        if a is None:
            return None
        return dev(ref.to_bf16(a)) if self.dtype == "bf16" else torch.from_numpy(a.astype(np.float32)).cuda()

    def run(self, shift=0, logprob=True, lens=True, temp=True, **kw):
        """``shift``: elements by which the logits' storage is off a 16-byte boundary."""
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()

        def off(t):
            if t is None or not shift:
                return t
            flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
            flat[shift:] = t.flatten()
            return flat[shift:]
        out = torch.full((self.B + 1, self.S + 1), -7, dtype=torch.int32, device="cuda")
        acc = torch.full((self.B + 1,), -7, dtype=torch.int32, device="cuda")
        lp = torch.full((self.B + 1, self.S + 1), 7.0, device="cuda") if logprob else None
        g.qmv_verify_run(off(self.logits(self.target)), off(self.logits(self.draft)), f(self.tokens) if self.S else None,
                         f(self.lens) if lens else None, f(self.temp) if temp else None, f(self.uniform) if self.S else None,
                         f(self.noise), out, acc, lp, self.B, self.S, self.V, ld_target=self.ld, ld_draft=self.ld,
                         ld_noise=self.ld, flags=g.VERIFY_F32_LOGITS if self.dtype == "f32" else 0, **kw)
        torch.cuda.synchronize()
        assert (out[-1] == -7).all() and acc[-1] == -7 and (lp is None or (lp[-1] == 7).all())
        return out[:-1].cpu().numpy(), acc[:-1].cpu().numpy(), None if lp is None else lp[:-1].cpu().numpy()

    def expect(self):
        V = self.V
        return ref.verify(self.target[..., :V], None if self.draft is None else self.draft[..., :V], self.tokens, self.lens,
                          self.temp.astype(np.float64), self.uniform.astype(np.float64), self.noise[:, :V].astype(np.float64),
                          BIG[self.dtype])

    def check(self, **kw):
        tok, acc, lp, close = self.expect()
        got, gacc, glp = self.run(**kw)
        keep = ~close
        assert keep.sum() >= max(1, 0.9 * self.B), "too many undecided sequences"
        assert np.array_equal(got[keep], tok[keep]) and np.array_equal(gacc[keep], acc[keep])
        # z = (l - max) / T and a sum of exponentials of fp32 size: |z| <= 100 here, a few roundings each
        fin = np.isfinite(lp[keep])
        assert np.array_equal(np.isfinite(glp[keep]), fin)
        assert np.all(np.abs(glp[keep][fin] - lp[keep][fin]) <= 2e-6 * (4 + np.abs(lp[keep][fin])))
        return got, gacc, glp


SHAPES = [
    (1, 0, 1), (1, 1, 1), (2, 1, 2), (1, 3, 7), (3, 2, 255), (2, 4, 256), (5, 5, 1000), (1, 7, 4097), (4, 1, 8191),
    (2, 3, 32000), (1, 15, 2051), (9, 0, 513), (1, 63, 129), (1, 2, 131072), (40, 3, 77),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,S,V", SHAPES)
def test_verify_matches_the_rule(B, S, V, dtype):
    Batch(B, S, V, dtype, seed=B + S + V).check()


@pytest.mark.parametrize("dtype,pad,shift", [("bf16", 1, 0), ("bf16", 3, 1), ("bf16", 8, 5), ("f32", 1, 0), ("f32", 2, 3), ("f32", 4, 1)])
@pytest.mark.parametrize("draft", [True, False])
def test_rows_off_any_alignment(dtype, pad, shift, draft):
    Batch(3, 3, 1237, dtype, pad=pad, draft=draft, seed=11).check(shift=shift)


@pytest.mark.parametrize("greedy", [0.5, 1.0])
@pytest.mark.parametrize("draft", [True, False])
def test_greedy_sequences(greedy, draft):
    b = Batch(12, 5, 3001, greedy=greedy, draft=draft, seed=12, spread=1.0, lens=[5] * 12)
    # make most drafts right, so that prefixes of every length occur
    best = np.argmax(b.target[:, :5], -1)
    rng = np.random.default_rng(1)
    b.tokens = np.where(rng.random(best.shape) < 0.8, best, b.tokens).astype(np.int32)
    _, acc, _ = b.check()
    assert len(set(acc.tolist())) > 2


def test_greedy_takes_the_lowest_of_equal_logits():
    b = Batch(2, 1, 5000, greedy=1.0, seed=13, lens=[1, 1])
    b.target[:, :, [4999, 17, 1800]] = 20.0
    b.tokens[:] = [[17], [1800]]
    out, acc, _ = b.check()
    assert out[0].tolist() == [17, 17] and out[1].tolist() == [17, -1] and acc.tolist() == [1, 0]


def test_equal_rows_always_accept():
    """Where draft and target rows are the same every token is accepted, and the last is sampled from the target."""
    b = Batch(6, 4, 900, seed=14, lens=[4] * 6)
    b.draft = b.target[:, :4].copy()
    b.uniform[:] = 1.0 - 2.0 ** -24
    _, acc, _ = b.run()
    assert (acc == 4).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_infinities_and_nan(dtype):
    b = Batch(8, 2, 700, dtype, seed=15, lens=[2] * 8, greedy=0.0)
    b.target[:, :, ::3] = -math.inf              # forbidden tokens
    b.target[0, :, 5:] = math.nan                # nearly all
    b.draft[1, :, 7] = math.nan
    b.target[2, :, 100] = math.inf               # certain
    b.target[3, :, :] = -math.inf                # nothing is left
    b.target[4, 0, :] = math.nan
    b.target[5, :, 101:] = -BIG[dtype]           # a mask of the type's lowest value
    b.draft[6] = -math.inf                       # a draft row without mass: q = 0
    b.target[7, 0, :] = -math.inf
    b.target[7, 0, 11] = 3.0
    b.tokens[7, 0] = 11
    b.tokens[2, :] = 100
    out, acc, lp = b.check()
    assert out[3, 0] == -1 and lp[3, 0] == -math.inf and acc[3] == 0
    assert out[2, 0] == 100 and acc[7] >= 1


def test_greedy_masks():
    b = Batch(3, 2, 300, seed=16, lens=[2] * 3, greedy=1.0)
    b.target[0] = -math.inf
    b.target[1, 0, :299] = math.nan
    b.tokens[1, 0] = 299
    b.target[2, 1, :] = -math.inf
    b.tokens[2, 0] = int(np.argmax(b.target[2, 0]))
    out, acc, _ = b.check()
    assert out[0].tolist() == [-1, -1, -1] and acc.tolist()[0] == 0 and acc[1] >= 1 and out[2, 1] == -1


def test_tokens_outside_the_vocabulary_are_refused():
    b = Batch(4, 2, 64, seed=17, lens=[2] * 4)
    b.tokens[:, 0] = [-1, 64, 2 ** 31 - 1, -2 ** 31]
    _, acc, _ = b.check()
    assert (acc == 0).all()
    b.draft = None
    b.check()


def test_lengths_outside_the_range_are_taken_into_it():
    b = Batch(4, 3, 64, seed=18, lens=[-4, 0, 3, 99])
    b.check()


def test_defaults():
    """No lengths: all drafts count. No temperature: 1. No logprob."""
    b = Batch(3, 3, 500, seed=19, lens=[3] * 3)
    b.temp[:] = 1.0
    want = b.run()
    got = b.run(lens=False, temp=False, logprob=False)
    assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])


def test_noise_of_zero_wins():
    b = Batch(2, 0, 300, seed=20)
    b.noise[0, 77] = 0.0
    b.noise[1, 5] = 1e-42
    out, _, _ = b.check()
    assert out[0, 0] == 77 and out[1, 0] == 5


def test_emitted_tokens_follow_the_target():
    """The first emitted token over many draws has the target's distribution (chi-square over 6 tokens, 4000 draws)."""
    B, V = 4000, 6
    b = Batch(B, 1, V, "f32", seed=21, lens=[1] * B)
    b.target[:] = b.target[0]
    b.draft[:] = b.draft[0]
    b.temp[:] = 1.0
    q = np.exp(b.draft[0, 0] - b.draft[0, 0].max())
    q /= q.sum()
    b.tokens[:, 0] = np.random.default_rng(2).choice(V, B, p=q)
    p = np.exp(b.target[0, 0] - b.target[0, 0].max())
    p /= p.sum()
    out, _, _ = b.run()
    seen = np.bincount(out[:, 0], minlength=V)
    chi = ((seen - B * p) ** 2 / (B * p)).sum()
    assert chi < 25, chi  # 5 degrees of freedom: beyond 25 with probability 1.4e-4, and the seed is fixed


def test_own_workspace_stream_and_graph():
    b = Batch(5, 4, 6000, seed=22)
    want = b.run()
    need = g.qmv_verify_workspace_size(5, 4, 6000)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            got = b.run(workspace=ws, workspace_bytes=need, stream=st)
            assert all(np.array_equal(x, y) for x, y in zip(want, got))
    assert torch.isnan(ws[need // 4:]).all(), "wrote past the workspace"
    with pytest.raises(g.QmvError) as e:
        b.run(workspace=ws, workspace_bytes=need - 1)
    assert e.value.code == 8
