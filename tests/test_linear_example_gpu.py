"""The example block of linear attention (``examples/linear_attention_block.py``): its operators together,
as they would be used. It trains and serves; a block's output and gradients are those of the fp64
definitions; a prefill followed by one-token steps gives the logits of the whole sequence at once.

Bars: bf16 activations are rounded (2^-9 rms of a value at most) after the norm, the projection, the norm of
q and k, the recurrence, the gated norm and the output, 6 times, and as often again on the way back; the
parts that a gradient passes add up as their squares, sqrt(12) 2^-9 = 7e-3, and the products of q and k
weigh them twice: 3e-2 of a gradient's norm. Two blocks' logits: 3e-2 (as for the gated delta block)."""
import copy
import importlib
import math

import pytest
import torch

from oracle import block as definition

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    return importlib.import_module("examples.linear_attention_block")


def test_it_trains(example):
    torch.manual_seed(0)
    net = example.Model().cuda()
    before = [p.detach().clone() for p in net.parameters()]
    losses = example.train(net, steps=3)
    assert all(math.isfinite(x) for x in losses)
    assert all(not torch.equal(a, b) for a, b in zip(before, net.parameters()))


def plain_block(b, x, residual, cu, positions):
    """The block from the definitions, in fp64 on its parameters' copies."""
    y, r = definition.residual_norm(x, b.norm, residual, b.scale, 1e-6)
    q, k, v, gate = ((y @ b.proj.weight.T).chunk(4, -1)[i].unflatten(-1, (b.heads, b.d)) for i in range(4))
    q, k = (definition.head_norm_rope(t, w, positions, b.freqs, 1e-6, False) for t, w in ((q, b.q_norm), (k, b.k_norm)))
    o, _ = definition.dla(q, k, v, -b.rate.exp(), None, cu)
    return definition.gated_norm(o, gate, b.out_norm, 1e-6, "silu").flatten(1) @ b.out.weight.T, r


def test_block_gradients(example):
    torch.manual_seed(1)
    lengths = [70, 1, 0, 130]
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    net = example.Block(128, 4, 64, 32).cuda()
    with torch.no_grad():
        for w in (net.norm, net.q_norm, net.k_norm, net.out_norm):
            w += 0.2 * torch.randn_like(w)
    ref = copy.deepcopy(net).cpu().double()
    n = cu[-1]
    x, res = (torch.randn(n, 128, device="cuda").bfloat16().requires_grad_(True) for _ in range(2))
    dy, dr = (torch.randn(n, 128, device="cuda").bfloat16() for _ in range(2))
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    at = example.token_positions(offsets, n)
    assert at.tolist() == [t for length in lengths for t in range(length)]
    out, stream = net(x, res, offsets, at)
    torch.autograd.backward((out, stream), (dy, dr))
    xs = [t.detach().cpu().double().requires_grad_(True) for t in (x, res)]
    want, want_stream = plain_block(ref, *xs, cu, at.cpu())
    torch.autograd.backward((want, want_stream), (dy.cpu().double(), dr.cpu().double()))
    pairs = [("out", out, want), ("x", x.grad, xs[0].grad), ("residual", res.grad, xs[1].grad)]
    pairs += [(name, p.grad, q.grad) for (name, p), q in zip(net.named_parameters(), ref.parameters())]
    for name, a, b in pairs:
        e = float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())
        assert e <= 3e-2, f"{name}: {e:.1e}"


def test_serving_equals_the_whole_sequence(example):
    torch.manual_seed(2)
    net = example.Model().cuda()
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, 64, (n,), generator=gen) for n in (1, 40, 130)]
    tokens, logits = example.serve(net, prompts, 6)
    for p, t, got in zip(prompts, tokens, logits):
        full = torch.cat([p.cuda(), t[:-1]])
        cu = torch.tensor([0, len(full)], dtype=torch.int32, device="cuda")
        with torch.no_grad():
            want = net(full, cu)[len(p) - 1:]
        assert float((got - want).float().norm() / want.float().norm()) <= 3e-2
