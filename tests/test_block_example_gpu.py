"""The example block (``examples/gated_delta_block.py``): its loss falls, and a prefill followed
by one-token steps gives the logits of the whole sequence at once (bf16 activations through two
blocks, each rounding 2^-9: 3e-2 of the logits' norm)."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_delta_block",
                                                  os.path.join(ROOT, "examples", "gated_delta_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
def test_training_lowers_the_loss(example):
    torch.manual_seed(0)
    losses = example.train(example.Model().cuda(), steps=25)
    assert all(x == x for x in losses)
    assert sum(losses[-3:]) / 3 < 0.9 * losses[0], losses


@pytest.mark.gpu
def test_serving_equals_the_whole_sequence(example):
    torch.manual_seed(1)
    net = example.Model().cuda()
    gen = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, 64, (n,), generator=gen) for n in (1, 40, 130)]
    tokens, logits = example.serve(net, prompts, 6)
    for p, t, got in zip(prompts, tokens, logits):
        full = torch.cat([p.cuda(), t[:-1]])
        cu = torch.tensor([0, len(full)], dtype=torch.int32, device="cuda")
        with torch.no_grad():
            want = net(full, cu)[len(p) - 1:]
        assert float((got - want).float().norm() / want.float().norm()) <= 3e-2
