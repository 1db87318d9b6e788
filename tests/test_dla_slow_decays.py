"""Linear attention with decays near none, g from log(1 - 2^-11) to -1e-6 at every token and slopes
down to 1e-8: rates of retention and lightning layers, whose memories are as long as the sequence.
An error of the rate, however small beside 1, is the same at every token and adds up over the memory.

The reference is a chunked fp64 form, held to the recurrence of ``oracle.block`` on the CPU. Bars: those of
``tests/test_dla_gpu.py``, per head. What a long memory adds to them is each tile's rounding of the state,
2^-24 at most and random in sign: sqrt(1024) 2^-24 = 2e-6 over 64K tokens at most, of which its root mean
square is a third.
"""
import math

import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from oracle import block
from tests.test_dla_gpu import BF, DEV, FP, Inputs, backward, bar, forward, rel

RATES = [math.log1p(-2.0 ** -11), -1e-4, -3.7e-5, -1e-6]
SLOPES = [-1e-5 * 2.0 ** (-h / 4) for h in range(32)]
F64 = torch.float64


def chunked(q, k, v, g, h0, scale):
    """One sequence in fp64, chunk by chunk of 64 tokens (zeros past its end), g [N, H]."""
    n, hv, c = v.shape[0], v.shape[1], 64
    more = -n % c
    group = hv // q.shape[1]

    def split(x):
        x = torch.cat((x, x.new_zeros(more, *x.shape[1:])))
        return x.unflatten(0, (-1, c)).movedim(2, 1)  # [chunks, H, 64, ...]

    q, k = (split(x.repeat_interleave(group, 1)) for x in (q, k))
    v, g = split(v), split(g).cumsum(-1)
    low = torch.ones(c, c, dtype=torch.bool, device=q.device).tril()
    pair = torch.where(low, (g[..., :, None] - g[..., None, :]), -math.inf).exp()
    add = ((g[..., -1:] - g).exp()[..., None] * k).mT @ v
    whole = g[..., -1].exp()[..., None, None]
    S, starts = h0[0], []
    for i in range(q.shape[0]):
        starts.append(S)
        S = whole[i] * S + add[i]
    out = (g.exp()[..., None] * q) @ torch.stack(starts) + (pair * (q @ k.mT)) @ v
    return scale * out.movedim(1, 2).flatten(0, 1)[:n], S[None]


def gradients(xs, scale, dout, dhf):
    xs = [x.clone().requires_grad_(True) for x in xs]
    out, end = chunked(*xs, scale)
    return torch.autograd.grad((out * dout).sum() + (end * dhf).sum(), xs)


def test_the_chunked_form_is_the_recurrence():
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, dtype=F64)  # noqa: E731
    q, k, v, g, h0 = r(150, 2, 5), r(150, 2, 5), r(150, 4, 3), -0.1 * r(150, 4).abs(), r(1, 4, 5, 3)
    dout, dhf = r(150, 4, 3), r(1, 4, 5, 3)
    got = chunked(q, k, v, g, h0, 0.3) + gradients((q, k, v, g, h0), 0.3, dout, dhf)
    want = block.dla(q, k, v, g, h0, [0, 150], 0.3) + block.dla_grads(q, k, v, g, h0, [0, 150], dout, dhf, 0.3)
    assert all(torch.allclose(a, b, atol=1e-10) for a, b in zip(got, want))


def inputs(n, hk, dk, dv, dtype, rates, per_head, seed):
    x = Inputs([n], hk, len(rates), dk, dv, dtype, seed=seed)
    rates = torch.tensor(rates, device=DEV)
    x.g = rates if per_head else rates.expand(n, len(rates)).contiguous()
    return x


def each_head(name, got, want, heads, dtype, head_axis):
    for h in range(heads):
        a, b = got.select(head_axis, h), want.select(head_axis, h)
        assert rel(a, b) <= bar(got, dtype), f"{name}, head {h}: {rel(a, b):.2e}"


def check(x, grads=True):
    xs = x.f64(DEV)
    scale, hv = x.q.shape[2] ** -0.5, x.v.shape[1]
    out, end = forward(x)
    want = chunked(*xs[:3], xs[3].expand(x.v.shape[:2]), xs[4], scale)
    each_head("out", out, want[0], hv, x.dtype, 1)
    each_head("h_final", end, want[1], hv, x.dtype, 1)
    if not grads:
        return
    got = backward(x)
    want = gradients((*xs[:3], xs[3].expand(x.v.shape[:2]), xs[4]), scale, x.dout.double(), x.dhf.double())
    for i, (name, a, b) in enumerate(zip(("dq", "dk", "dv", "dg", "dh0"), got, want)):
        if name == "dg" and x.g.dim() == 1:  # the terms cancel: of the sum of their sizes
            err = (a.double() - b.sum(0)).abs() / b.abs().sum(0)
            assert float(err.max()) <= bar(a, x.dtype), f"dg: {err}"
        else:
            each_head(name, a, b, a.shape[1], x.dtype, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,hk,dk,dv", [(8192, 2, 64, 64), (8192, 4, 128, 128), (8191, 1, 33, 72), (65536, 1, 64, 32)])
def test_constant_rates(n, hk, dk, dv, dtype, per_head):
    check(inputs(n, hk, dk, dv, dtype, RATES, per_head, seed=n + dk))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [FP, BF])
def test_slopes_of_many_heads(dtype):
    """Memories far longer than the sequence, all heads whole in one walk or cut."""
    check(inputs(65536, 8, 64, 64, dtype, SLOPES, True, seed=1), grads=False)
    check(inputs(16384, 8, 64, 64, dtype, SLOPES, True, seed=2))


@pytest.mark.gpu
def test_ragged_slow_decays():
    """Rates that differ from token to token, a fifth of the tokens without any, several sequences."""
    lengths = [3000, 0, 1, 8192, 515]
    x = Inputs(lengths, 2, 4, 64, 128, BF, seed=3)
    gen = torch.Generator().manual_seed(4)
    g = -(10.0 ** (-7 + 4 * torch.rand(sum(lengths), 4, generator=gen)))
    g[torch.rand(g.shape, generator=gen) < 0.2] = 0.0
    x.g = g.to(DEV)
    out, end = forward(x)
    grads = backward(x)
    for i, (a, b) in enumerate(zip(x.cu_host[:-1], x.cu_host[1:])):
        if a == b:
            continue
        xs = [t[a:b].double() for t in (x.q, x.k, x.v, x.g)] + [x.h0[i:i + 1].double()]
        want = chunked(*xs, 8.0 ** -1) + gradients(xs, 8.0 ** -1, x.dout[a:b].double(), x.dhf[i:i + 1].double())
        got = (out[a:b], end[i:i + 1], *[t[a:b] for t in grads[:4]], grads[4][i:i + 1])
        for name, y, ref in zip(("out", "h_final", "dq", "dk", "dv", "dg", "dh0"), got, want):
            if name != "dg" or b - a > 1:  # of one token dg is a single sum that may cancel
                assert rel(y, ref) <= bar(y, BF), f"{name} of sequence {i}: {rel(y, ref):.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [FP, BF])
def test_many_steps(dtype):
    """4096 tokens one by one. A step rounds the state twice, 2^-24 at most and random in sign: sqrt(2 4096) 2^-24 =
    5.4e-6 at most, whatever the rate; a rate rounded beside 1, by up to 2^-25 a step and always the same
    way, is off by ten times as much."""
    n = 4096
    x = inputs(n, 2, 64, 64, dtype, RATES, True, seed=5)
    xs = x.f64(DEV)
    want, end = chunked(*xs[:3], xs[3].expand(x.v.shape[:2]), xs[4], 0.125)
    pool = x.h0.clone()
    out = torch.cat([kda.dla_step(x.q[t:t + 1], x.k[t:t + 1], x.v[t:t + 1], x.g, pool) for t in range(n)])
    for h in range(4):
        assert rel(pool[:, h], end[:, h]) <= 5.4e-6, f"state, head {h}: {rel(pool[:, h], end[:, h]):.2e}"
        assert rel(out[:, h], want[:, h]) <= (5.4e-6 if dtype == FP else 2.0 ** -8 + 5.4e-6)


@pytest.mark.gpu
def test_a_step_keeps_an_infinity():
    x = inputs(1, 1, 64, 64, FP, [0.0, -1e-6, -1e-3, -3.0], True, seed=6)
    pool = x.h0.clone()
    pool[0, :, 5, 7], pool[0, :, 9, 11] = math.inf, -math.inf
    kda.dla_step(x.q, x.k, x.v, x.g, pool)
    assert bool((pool[0, :, 5, 7] == math.inf).all()) and bool((pool[0, :, 9, 11] == -math.inf).all())
    assert int(torch.isfinite(pool).sum()) == pool.numel() - 8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("at", [1000, 4097, 8191])
def test_a_decay_that_is_nan_shows_through_segments(dtype, at):
    """Few heads, so that the sequence is cut: every token from the NaN's on, of its head alone, and the
    gradient of the starting state."""
    x = inputs(8192, 2, 64, 64, dtype, RATES[:2], False, seed=7)
    ref, grads = forward(x), backward(x)
    x.g[at, 1] = float("nan")
    got, back = forward(x), backward(x)
    chunk = at // 128 * 128
    assert bool(torch.isnan(got[0][at:, 1]).all()) and bool(torch.isnan(got[1][0, 1]).all())
    assert bool(torch.isnan(back[0][at:, 1]).all()) and bool(torch.isnan(back[4][0, 1]).all())
    assert torch.equal(got[0][:chunk, 1], ref[0][:chunk, 1])
    for a, b in zip((got[0], back[0], back[1], back[2], back[3]), (ref[0], *grads[:4])):
        assert torch.equal(a[:, 0], b[:, 0])
    assert torch.equal(got[1][0, 0], ref[1][0, 0]) and torch.equal(back[4][0, 0], grads[4][0, 0])


@pytest.mark.gpu
def test_strong_decays_after_slow_ones_through_segments():
    """A segment whose sum of exponents passes any that fp32 holds, and resets, beside heads that keep all."""
    x = inputs(8192, 2, 64, 64, BF, RATES, False, seed=8)
    x.g[1000:3000, 0] = -60.0
    x.g[4000, 1] = -math.inf
    x.g[5000:, 2] = -200.0
    xs = x.f64(DEV)
    xs[3] = xs[3].clamp(min=-300.0)
    out, end = forward(x)
    want = chunked(*xs[:3], xs[3], xs[4], 0.125)
    each_head("out", out, want[0], 4, BF, 1)
    each_head("h_final", end, want[1], 4, BF, 1)
    got = backward(x)
    ref = gradients((*xs[:3], xs[3], xs[4]), 0.125, x.dout.double(), x.dhf.double())
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dh0"), got, ref):
        assert rel(a, b) <= bar(a, BF), f"{name}: {rel(a, b):.2e}"
