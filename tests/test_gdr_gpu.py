"""GPU parity of the gated delta rule with one decay per head (``kda_gdr_chunk_fwd``,
``kda_gdr_chunk_bwd``, ``kda_gdr_step``) against the fp64 recurrence on the same inputs.

Bars on the rel-L2 error, from the number formats:
  bf16 results   one rounding to bf16 has 2^-9 = 2.0e-3 rms at most; the output's operands S
                 and P are rounded to bf16 once more, the gradients' pair weights likewise, on
                 parts of the result each: 4e-3
  fp32 results of bf16 inputs   operands in two bf16 parts keep 2^-17 each, through a product
                 of two and a chain of four products: 2e-5
  fp32 results of fp32 inputs   three parts keep 2^-24; the tensor cores' fp32 sums drop bits
                 below 2^-23 of the running sum, about 50 times a chunk: 6e-6
  one token      fp32 arithmetic throughout, sums of 128 terms: 1e-6
"""
import numpy as np
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from oracle import block
from tests.gpu_helpers import assert_finite, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def bar(t, dtype):
    return 4e-3 if t.dtype == BF else 2e-5 if dtype == BF else 6e-6


class Inputs:
    def __init__(self, lengths, hk, hv, dk, dv, dtype, seed=0, h0=True, decay=1.0):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        n = sum(lengths)
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
        k = r(n, hk, dk)
        self.q, self.k = unit(r(n, hk, dk)).to(DEV, dtype), unit(k + 0.5 * k.roll(1, 0)).to(DEV, dtype)
        self.v = r(n, hv, dv).to(DEV, dtype)
        # the decay's range over heads: from nearly none to strong
        self.g = (-decay * r(n, hv).abs() * torch.logspace(-2, 0.5, hv)).to(DEV)
        self.beta = torch.sigmoid(r(n, hv)).to(DEV)
        self.h0 = (0.3 * r(len(lengths), hv, dk, dv)).to(DEV) if h0 else None
        self.cu_host = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        self.cu = torch.tensor(self.cu_host, dtype=torch.int32, device=DEV)
        self.dout = r(n, hv, dv).to(DEV, dtype)
        self.dhf = (0.3 * r(len(lengths), hv, dk, dv)).to(DEV) if h0 else None
        self.dtype = dtype

    @property
    def args(self):
        return self.q, self.k, self.v, self.g, self.beta, self.h0, self.cu

    def f64(self):
        return [block.f64(t) for t in (self.q, self.k, self.v, self.g, self.beta, self.h0)]


def forward(x):
    out, end = kda.gdr_chunk_fwd(*x.args)
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    return out, end


def check_forward(x):
    out, end = forward(x)
    assert_finite(out, end)
    want = block.gdr(*x.f64(), x.cu_host)
    for got, ref in zip((out, end), want):
        e = rel_l2(got.double().cpu().numpy(), ref.numpy())
        assert e <= bar(got, x.dtype), f"{e:.2e}"


def check_backward(x, dhf=True):
    got = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf if dhf else None)
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    assert_finite(*got)
    want = block.gdr_grads(*x.f64(), x.cu_host, block.f64(x.dout), block.f64(x.dhf) if dhf else None)
    for name, a, ref in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want):
        e = rel_l2(a.double().cpu().numpy(), ref.numpy())
        assert e <= bar(a, x.dtype), f"{name}: {e:.2e}"


SHAPES = [([1], 1, 1, 128, 128), ([2], 2, 2, 64, 64), ([63], 1, 2, 128, 64), ([64], 2, 2, 128, 128),
          ([65], 1, 3, 64, 128), ([200], 2, 4, 128, 128), ([0, 1, 130, 0, 64, 17], 2, 2, 128, 128),
          ([5, 0, 66], 1, 4, 33, 31), ([100], 3, 3, 96, 112), ([70, 129], 2, 2, 40, 72), ([3], 1, 1, 1, 1),
          ([90], 1, 2, 65, 33), ([140], 2, 2, 8, 128)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", SHAPES)
def test_forward(lengths, hk, hv, dk, dv, dtype):
    check_forward(Inputs(lengths, hk, hv, dk, dv, dtype, seed=len(lengths) + dk))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", SHAPES)
def test_backward(lengths, hk, hv, dk, dv, dtype):
    check_backward(Inputs(lengths, hk, hv, dk, dv, dtype, seed=len(lengths) + dk))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_without_states(dtype):
    x = Inputs([77, 64], 2, 4, 128, 128, dtype, seed=3, h0=False)
    check_forward(x)
    check_backward(x, dhf=False)
    out, end = kda.gdr_chunk_fwd(*x.args, output_final_state=False)
    assert end is None and torch.equal(out, forward(x)[0])


def test_many_chunks_take_the_two_plane_backward():
    """A bf16 backward of many (token, head) pairs carries two planes."""
    check_backward(Inputs([700, 333], 16, 64, 32, 32, BF, seed=5))


def wide(hv):
    """Sequences of 65536 (token, head) pairs and a few, where the bf16 backward carries two planes.
    Too many for the host's recurrence: the same one runs on the device, in fp64."""
    n = 65536 // hv + 5
    return [n - 131, 0, 1, 130]


def check_wide(x):
    got = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    assert_finite(*got)
    f64 = [t.double() for t in (x.q, x.k, x.v, x.g, x.beta, x.h0)]
    want = block.gdr_grads(*f64, x.cu_host, x.dout.double(), x.dhf.double())
    for name, a, ref in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want):
        e = float((a.double() - ref).norm() / ref.norm())
        assert e <= bar(a, x.dtype), f"{name}: {e:.2e}"


@pytest.mark.parametrize("hk,hv,dk,dv", [(64, 128, 128, 128), (128, 128, 128, 72), (16, 96, 100, 40), (64, 192, 72, 8),
                                         (64, 128, 64, 128), (8, 128, 16, 24), (48, 96, 33, 31), (16, 288, 128, 16)])
def test_two_plane_backward(hk, hv, dk, dv):
    """One to eighteen value heads a key head, one to eight slices of value channels, padded
    channels, rows that a tensor copy cannot fetch."""
    check_wide(Inputs(wide(hv), hk, hv, dk, dv, BF, seed=dk + dv))


def test_two_plane_backward_with_resets_and_slices():
    x = Inputs(wide(128), 32, 128, 128, 64, BF, seed=6)
    x.g[:, 0] = 0.0
    for t in (0, 63, 64, 100, 383, 385, 387, 450):
        x.g[t, 2] = -float("inf")
    x.beta[10:20] = 0.0
    check_wide(x)
    ref = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    assert float(ref[3][x.g == -float("inf")].abs().max()) == 0.0
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf), ref))
    for q, k, v in slices(x):
        grads = kda.gdr_chunk_bwd(q, k, v, x.g, x.beta, x.h0, x.cu, x.dout, x.dhf)
        assert all(torch.equal(a, b) for a, b in zip(grads, ref))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_decays_of_every_size(dtype):
    """No decay, decays far below fp32's range, -inf (a new document) at a chunk's first, middle
    and last token; beta 0 and 2."""
    x = Inputs([150, 70], 1, 4, 64, 64, dtype, seed=7)
    x.g[:, 0] = 0.0
    x.g[::7, 1] = -300.0
    for t in (0, 63, 64, 100, 149, 151):
        x.g[t, 2] = -float("inf")
    x.g[:, 3] = -50.0
    x.beta[10:20] = 0.0
    x.beta[30:40, 1] = 2.0
    check_forward(x)
    check_backward(x)
    dg = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)[3]
    assert float(dg[torch.isinf(x.g)].abs().max()) == 0.0


def test_equal_keys_keep_the_inverse_exact():
    """Every key of a chunk the same, beta 1: the off-diagonal of I + A is all ones."""
    x = Inputs([128], 1, 2, 64, 64, FP, seed=8)
    x.k[:] = x.k[0]
    x.beta.fill_(1.0)
    x.g.fill_(-0.01)
    check_forward(x)
    check_backward(x)


def slices(x):
    """The same inputs as slices of one wide projection, and that at an odd offset."""
    for lead in (8, 3):
        n = x.q.shape[0]
        parts = [t.reshape(n, -1) for t in (x.q, x.k, x.v)]
        wide = torch.full((n, lead + sum(p.shape[1] for p in parts) + 5), float("nan"), device=DEV, dtype=x.dtype)
        views, at = [], lead
        for t, p in zip((x.q, x.k, x.v), parts):
            wide[:, at:at + p.shape[1]] = p
            views.append(wide[:, at:at + p.shape[1]].unflatten(1, t.shape[1:]))
            at += p.shape[1]
        yield views


@pytest.mark.parametrize("dtype", [FP, BF])
def test_slices_of_a_projection_give_the_same_bits(dtype):
    x = Inputs([130, 9], 2, 4, 128, 64, dtype, seed=11)
    ref, ref_b = forward(x), kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    state = x.h0.repeat_interleave(70, 0)[:139].contiguous()
    ref_s = kda.gdr_step(x.q, x.k, x.v, x.g, x.beta, state.clone())
    for q, k, v in slices(x):
        got = kda.gdr_chunk_fwd(q, k, v, x.g, x.beta, x.h0, x.cu)
        grads = kda.gdr_chunk_bwd(q, k, v, x.g, x.beta, x.h0, x.cu, x.dout, x.dhf)
        assert all(torch.equal(a, b) for a, b in zip((*got, *grads), (*ref, *ref_b)))
        assert torch.equal(kda.gdr_step(q, k, v, x.g, x.beta, state.clone()), ref_s)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_packing_cutting_and_repeating_change_no_bit(dtype):
    """A sequence's result does not depend on its neighbours; a sequence cut at a multiple of
    64 tokens continues from its state; the same call gives the same bits."""
    lengths = [192, 1, 75]
    x = Inputs(lengths, 2, 4, 128, 128, dtype, seed=13)
    out, end = forward(x)
    again = forward(x)
    assert torch.equal(out, again[0]) and torch.equal(end, again[1])
    for n, (a, b) in enumerate(zip(x.cu_host[:-1], x.cu_host[1:])):
        o, e = kda.gdr_chunk_fwd(x.q[a:b], x.k[a:b], x.v[a:b], x.g[a:b], x.beta[a:b], x.h0[n:n + 1])
        assert torch.equal(o, out[a:b]) and torch.equal(e[0], end[n])
    o1, e1 = kda.gdr_chunk_fwd(x.q[:128], x.k[:128], x.v[:128], x.g[:128], x.beta[:128], x.h0[:1])
    o2, e2 = kda.gdr_chunk_fwd(x.q[128:192], x.k[128:192], x.v[128:192], x.g[128:192], x.beta[128:192], e1)
    assert torch.equal(torch.cat([o1, o2]), out[:192]) and torch.equal(e2[0], end[0])
    g1, g2 = (kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))


def test_a_nan_stays_in_its_sequence():
    x = Inputs([100, 100, 37], 1, 2, 128, 128, BF, seed=17)
    clean, grads = forward(x), kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    for t in (x.q, x.k, x.v, x.g, x.beta, x.dout):
        t[100:200] = float("nan")
    out, end = forward(x)
    bad = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    keep = torch.tensor([*range(100), *range(200, 237)], device=DEV)
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(end[::2], clean[1][::2])
    for a, b in zip(bad[:5], grads[:5]):
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(bad[5][::2], grads[5][::2])
    assert bool(torch.isnan(out[100:200]).all()) and bool(torch.isnan(end[1]).all())


@pytest.mark.parametrize("dtype", [FP, BF])
def test_no_token(dtype):
    x = Inputs([0, 0], 1, 2, 64, 64, dtype, seed=19)
    out, end = forward(x)
    assert out.shape == (0, 2, 64) and torch.equal(end, x.h0)
    assert torch.equal(kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)[5], x.dhf)
    y = Inputs([0], 1, 2, 64, 64, dtype, seed=19, h0=False)
    assert float(forward(y)[1].abs().max()) == 0.0


def test_gradients_are_differences_of_the_forward():
    """fp32, step 2e-2 along a random direction: the difference's rounding is ~1e-6 of the loss
    over the step, its truncation (h^2 / 6) f''' ~ 1e-4; bar 2e-3 of |grad| |direction|."""
    x = Inputs([90, 40], 1, 2, 32, 32, FP, seed=23)
    grads = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    gen = torch.Generator().manual_seed(1)
    tensors = [x.q, x.k, x.v, x.g, x.beta, x.h0]

    def loss(ts):
        out, end = kda.gdr_chunk_fwd(*ts, x.cu)
        return float((out.double() * x.dout).sum() + (end.double() * x.dhf).sum())

    for i, (t, grad) in enumerate(zip(tensors, grads)):
        d = torch.randn(t.shape, generator=gen).to(DEV)
        d /= d.norm()
        h = 2e-2
        hi, lo = (loss([u + s * h * d if j == i else u for j, u in enumerate(tensors)]) for s in (1, -1))
        got, want = float((grad * d).sum()), (hi - lo) / (2 * h)
        assert abs(got - want) <= 2e-3 * float(grad.norm()), (i, got, want)


def test_another_stream():
    """Inputs made on a side stream, the call on that stream: ordered behind them."""
    side = torch.cuda.Stream()
    x = Inputs([300], 2, 2, 128, 128, BF, seed=29)
    ref = forward(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q, k, v = (t.clone() for t in (x.q, x.k, x.v))
        got = kda.gdr_chunk_fwd(q, k, v, x.g, x.beta, x.h0, x.cu)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_offsets_beyond_32_bits():
    """v and out of 2.2e9 elements: the last sequence equals the same one alone."""
    n, tail, hv, d = 1_080_000, 150, 16, 128
    x = Inputs([tail], 1, hv, d, d, BF, seed=31, h0=False)
    k = torch.zeros((n, 1, d), device=DEV, dtype=BF)
    k[..., 0] = 1.0
    v = torch.zeros((n, hv, d), device=DEV, dtype=BF)
    g, beta = torch.full((n, hv), -0.1, device=DEV), torch.full((n, hv), 0.5, device=DEV)
    q = k.clone()
    for big, small in ((q, x.q), (k, x.k), (v, x.v), (g, x.g), (beta, x.beta)):
        big[n - tail:] = small
    cu = torch.tensor([0, n - tail, n], dtype=torch.int32, device=DEV)
    out, end = kda.gdr_chunk_fwd(q, k, v, g, beta, None, cu)
    ref, ref_end = forward(x)
    assert out.numel() > 2 ** 31
    assert torch.equal(out[n - tail:], ref) and torch.equal(end[1], ref_end[0])
    assert float(out[:n - tail].abs().max()) == 0.0


# ---------------------------------------------------------------- one token

@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("B,hk,hv,dk,dv", [(1, 16, 32, 128, 128), (5, 2, 6, 64, 128), (40, 4, 8, 128, 128),
                                           (3, 1, 1, 1, 1), (4, 1, 3, 33, 31), (2, 2, 2, 128, 72)])
def test_step(B, hk, hv, dk, dv, dtype):
    x = Inputs([1] * B, hk, hv, dk, dv, dtype, seed=B + dk)
    pool = torch.randn((B + 3, hv, dk, dv), generator=torch.Generator().manual_seed(2)).to(DEV)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(3))[:B].to(DEV, torch.int32)
    pool[slots.long()] = x.h0
    before = pool.clone()
    out = kda.gdr_step(x.q, x.k, x.v, x.g, x.beta, pool, slots)
    torch.cuda.synchronize()
    want, end = block.gdr(*x.f64(), x.cu_host)
    assert rel_l2(out.double().cpu().numpy(), want.numpy()) <= (4e-3 if dtype == BF else 1e-6)
    assert rel_l2(pool[slots.long()].double().cpu().numpy(), end.numpy()) <= 1e-6
    others = torch.ones(B + 3, dtype=torch.bool, device=DEV)
    others[slots.long()] = False
    assert torch.equal(pool[others], before[others])


def test_step_padded_rows_touch_nothing():
    x = Inputs([1] * 6, 1, 2, 64, 64, BF, seed=37)
    pool = torch.randn((4, 2, 64, 64), device=DEV)
    before = pool.clone()
    slots = torch.tensor([2, -1, 4, 0, 1 << 30, -(1 << 31)], dtype=torch.int32, device=DEV)
    out = kda.gdr_step(x.q, x.k, x.v, x.g, x.beta, pool, slots)
    rows = [1, 2, 4, 5]
    assert float(out[rows].abs().max()) == 0.0 and float(out[[0, 3]].abs().min(dim=-1).values.max()) > 0
    assert torch.equal(pool[[1, 3]], before[[1, 3]])
    assert not torch.equal(pool[0], before[0]) and not torch.equal(pool[2], before[2])


@pytest.mark.parametrize("dtype", [FP, BF])
def test_steps_continue_a_prefill(dtype):
    x = Inputs([70], 2, 4, 128, 128, dtype, seed=41)
    full, end = forward(x)
    out, state = kda.gdr_chunk_fwd(x.q[:60], x.k[:60], x.v[:60], x.g[:60], x.beta[:60], x.h0)
    outs = [out]
    for t in range(60, 70):
        outs.append(kda.gdr_step(x.q[t:t + 1], x.k[t:t + 1], x.v[t:t + 1], x.g[t:t + 1], x.beta[t:t + 1], state))
    # both sides carry their own error against the recurrence
    assert rel_l2(torch.cat(outs).double().cpu().numpy(), full.double().cpu().numpy()) <= 2 * bar(full, dtype)
    assert rel_l2(state.cpu().numpy(), end.cpu().numpy()) <= 2 * bar(end, dtype)


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses():
    x = Inputs([64], 1, 2, 64, 64, BF, seed=43)
    q, k, v, g, beta, h0, cu = x.args
    bad = [(q[:, :, :32], k, v, g, beta, h0, cu), (q, k.float(), v, g, beta, h0, cu), (q, k, v, g.double(), beta, h0, cu),
           (q, k, v, g, beta[:, :1], h0, cu), (q, k, v, g, beta, h0.half(), cu), (q, k, v, g, beta, h0, cu.long()),
           (q.transpose(0, 2), k, v, g, beta, h0, cu), (q.half(), k.half(), v.half(), g, beta, h0, cu),
           (q, k, v.flip(0).expand(64, 2, 64)[:, :, ::2], g, beta, h0, cu), (q[0], k[0], v[0], g, beta, h0, cu),
           (q, k, v, g, beta, h0[:0], cu)]
    for args in bad:
        with pytest.raises(ValueError):
            kda.gdr_chunk_fwd(*args)
        with pytest.raises(ValueError):
            kda.gdr_chunk_bwd(*args, x.dout)
    with pytest.raises(ValueError):
        kda.gdr_chunk_bwd(*x.args, x.dout.float())
    with pytest.raises(kda.KDAError):
        kda.gdr_chunk_fwd(*x.args, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.gdr_chunk_fwd(*x.args, h_final=x.h0)      # an output over an input
    with pytest.raises(ValueError):
        kda.gdr_step(q, k, v, g, beta, torch.zeros((64, 2, 64, 32), device=DEV))
    with pytest.raises(ValueError):
        kda.gdr_step(q, k, v, g, beta, torch.zeros((64, 2, 64, 64), device=DEV), torch.zeros(64, device=DEV))
    y = Inputs([4], 1, 1, 160, 16, BF, seed=1)
    with pytest.raises(kda.KDAError):
        kda.gdr_chunk_fwd(*y.args)


# ---------------------------------------------------------------- one rounding in a bf16 result

def rounded_once(got, ref):
    """A bf16 result against the definition's value rounded to bf16: apart only where the value
    before its rounding, off by d, falls on the other side of a boundary. That happens to d / ulp
    of the values, each then an ulp off, an ulp up to 2^-7 of the value: the mean square of the
    difference is up to d ulp = 2e-5 2^-7 (d as for the fp32 results), its root 4e-4."""
    e = rel_l2(got.double().cpu().numpy(), ref.to(BF).double().numpy())
    assert e <= 4e-4, f"{e:.2e}"


ROUNDED = [([1], 1, 1, 128, 128), ([200], 2, 4, 128, 128), ([0, 1, 130, 0, 64, 17], 2, 2, 128, 128),
           ([5, 0, 66], 1, 4, 33, 31), ([100], 3, 3, 96, 112), ([90], 1, 2, 65, 33), ([140], 2, 2, 8, 128),
           ([700, 333], 4, 8, 64, 64)]


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", ROUNDED)
def test_forward_output_is_rounded_once(lengths, hk, hv, dk, dv):
    x = Inputs(lengths, hk, hv, dk, dv, BF, seed=len(lengths) + dk)
    rounded_once(forward(x)[0], block.gdr(*x.f64(), x.cu_host)[0])


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", ROUNDED)
def test_gradients_are_rounded_once(lengths, hk, hv, dk, dv):
    x = Inputs(lengths, hk, hv, dk, dv, BF, seed=len(lengths) + dk)
    got = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    want = block.gdr_grads(*x.f64(), x.cu_host, block.f64(x.dout), block.f64(x.dhf))
    for a, ref in zip(got[:3], want):
        rounded_once(a, ref)


@pytest.mark.parametrize("hk,hv,dk,dv", [(64, 128, 128, 128), (16, 96, 100, 40), (8, 128, 16, 24)])
def test_gradients_of_many_pairs_are_rounded_once(hk, hv, dk, dv):
    x = Inputs(wide(hv), hk, hv, dk, dv, BF, seed=dk + dv)
    got = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    f64 = [t.double() for t in (x.q, x.k, x.v, x.g, x.beta, x.h0)]
    want = block.gdr_grads(*f64, x.cu_host, x.dout.double(), x.dhf.double())
    for a, ref in zip(got[:3], want):
        rounded_once(a, ref.cpu())


@pytest.mark.parametrize("lengths,hk,hv", [([9000], 1, 1), ([5000, 4100], 1, 2)])
def test_long_sequences_of_few_heads(lengths, hk, hv):
    """Two planes over a hundred chunks of one sequence and more, few heads: the norm of a gradient
    is made up by its tokens alone."""
    x = Inputs(lengths, hk, hv, 64, 64, BF, seed=hv)
    check_forward(x)
    check_wide(x)


def test_one_sequence_in_a_graph():
    """Without offsets a call can be captured; the replay computes on what its inputs hold then."""
    x = Inputs([150], 1, 2, 64, 64, BF, seed=47)
    args = (x.q, x.k, x.v, x.g, x.beta, x.h0)

    def both():
        return (*kda.gdr_chunk_fwd(*args), *kda.gdr_chunk_bwd(*args, None, x.dout, x.dhf))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = both()
    torch.cuda.synchronize()
    x.v.copy_(x.v.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, both()))
    assert kda.read_device_flags() == 0


# ---------------------------------------------------------------- many sequences

def many(n):
    """Empty and short sequences, every fiftieth of more than a chunk."""
    return [70 if i % 50 == 7 else (1, 0, 3, 2, 5)[i % 5] for i in range(n)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n", [300, 1024, 1100])
def test_many_sequences(n, dtype):
    """More sequences than a chain has threads, and than any rule of the launch order looks at."""
    x = Inputs(many(n), 1, 2, 16, 16, dtype, seed=n)
    check_forward(x)
    check_backward(x)


def test_packed_gradients_are_as_accurate_as_the_call():
    """A sequence alone (three planes) and packed beyond 8192 (token, head) pairs (two): each within
    its bar, so apart by two bars at most."""
    x = Inputs([90, 2100], 2, 4, 64, 64, BF, seed=53)
    packed = kda.gdr_chunk_bwd(*x.args, x.dout, x.dhf)
    alone = kda.gdr_chunk_bwd(x.q[:90], x.k[:90], x.v[:90], x.g[:90], x.beta[:90], x.h0[:1], None, x.dout[:90],
                              x.dhf[:1])
    for a, b in zip(packed, alone):
        a = a[:len(b)]
        assert rel_l2(a.double().cpu().numpy(), b.double().cpu().numpy()) <= 2 * bar(a, BF)


@pytest.mark.parametrize("n", [2, 63, 64, 65])
def test_launch_order_changes_no_bit(n):
    """Up to 64 sequences the longest chains are launched first, beyond in order."""
    x = Inputs([1 + (i * 37) % 130 for i in range(n)], 1, 1, 32, 32, BF, seed=n)
    out, end = forward(x)
    for i in range(0, n, 9):
        a, b = x.cu_host[i], x.cu_host[i + 1]
        o, e = kda.gdr_chunk_fwd(x.q[a:b], x.k[a:b], x.v[a:b], x.g[a:b], x.beta[a:b], x.h0[i:i + 1])
        assert torch.equal(o, out[a:b]) and torch.equal(e[0], end[i])
    check_backward(x)


def test_many_short_sequences_cost_what_they_hold():
    """A chain's choice of its sequence may not grow with the square of their number: 1024 sequences
    of 16 tokens take less than four times what 1025 do (they took fifteen times)."""
    times = []
    for n in (1024, 1025):
        x = Inputs([16] * n, 4, 8, 64, 64, BF, seed=59, h0=False)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(6):
            start.record()
            kda.gdr_chunk_fwd(*x.args, output_final_state=False)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        times.append(best)
    assert times[0] < 4 * times[1], times
