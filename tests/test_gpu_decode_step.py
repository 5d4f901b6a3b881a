"""The operators of a decode step together, as examples/decode_step.py runs them."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from group_quantized_mat_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("drafts,batch", [(1, 1), (3, 2), (4, 5)])
def test_drafting_does_not_change_greedy_tokens(ex, drafts, batch):
    model = ex.Model(vocab=2000, width=512, inter=192, experts=6, top_k=2)
    adapter = [b % 4 - 1 for b in range(batch)]
    first = list(range(3, 3 + batch))
    plain, _ = ex.Decoder(model, batch, 0, adapter, 0.0).generate(first, 24)
    drafted, steps = ex.Decoder(model, batch, drafts, adapter, 0.0).generate(first, 24)
    assert [t[:24] for t in plain] == [t[:24] for t in drafted]
    assert ex.g.qmv_device_error() == 0


def test_sampled_tokens_are_drafts_and_one_more(ex):
    model = ex.Model(vocab=1500, width=256, inter=128, experts=4, top_k=2, adapters=2, rank=5)
    d = ex.Decoder(model, 3, 4, [0, -1, 1], 0.7)
    d.last.copy_(torch.tensor([5, 6, 7]))
    some = 0
    for _ in range(12):
        d.step()
        drafted, tokens, accepted = d.drafted.tolist(), d.tokens.tolist(), d.accepted.tolist()
        some += sum(accepted)
        for b in range(3):
            n = accepted[b]
            assert tokens[b][:n] == drafted[b][:n] and tokens[b][n + 1:] == [-1] * (4 - n)
            assert 0 <= tokens[b][n] < 1500 and d.last[b].item() == tokens[b][n]
        assert torch.isfinite(d.logprob).all()
    assert some > 0
