"""What examples/attention_step.py refuses, and that its decoders of one room divide sums alike."""

import importlib.util
import os
import sys

import pytest
import torch

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_step", EXAMPLE)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch,drafts", [(1, 16), (4, 40), (1, -1), (0, 3), (257, 0), (64, 4), (17, 15)])
def test_steps_that_would_not_be_exact_or_not_run(example, batch, drafts):
    with pytest.raises(ValueError, match="tokens"):
        example.Decoder(None, batch, 100, drafts)


@pytest.mark.gpu
def test_as_many_drafts_and_sequences_as_there_may_be(example):
    model = example.Model(vocab=64, width=512, heads=4, kv_heads=2)
    for batch, prompt, most in ((2, 70, 15), (51, 5, 4)):
        tokens = torch.randint(0, 64, (batch, prompt), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
        runs = []
        for drafts in (0, most):
            d = example.Decoder(model, batch, prompt + (most + 1) * 20, drafts)
            runs.append((d.per, d.prompt(tokens), d.generate(20)[0]))
        assert runs[0] == runs[1]
    d = example.Decoder(model, 256, 40, 0)  # a chunk of one token each
    d.prompt(torch.zeros(256, 3, dtype=torch.int32, device="cuda"))
    assert len(d.generate(2)[0]) == 256


@pytest.mark.gpu
def test_the_command_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["attention_step.py", "--batch", "3", "--prompt", "40", "--tokens", "8", "--drafts", "3", "--window", "16", "--sinks", "2"])
    example.main()
    assert capsys.readouterr().out.count("tokens a step") == 2
