"""GPU parity of linear attention with one decay per head (``kda_dla_chunk_fwd``,
``kda_dla_chunk_bwd``, ``kda_dla_step``) against the fp64 recurrence on the same inputs.

Bars on the rel-L2 error, from the number formats:
  bf16 results   the definition's rounded once: half a step is 2^-8 of a value at most; the operands in
                 two bf16 parts add half a step of half a step each, 2^-16: 2^-8 + 2^-14
  fp32 results of bf16 inputs   operands in two parts are off by 2^-16 at most and 2^-18 in the root mean
                 square, through products of up to four of them and sums of 256 terms in fp32, dg
                 through sums over a chunk's rows and columns: 2e-5
  fp32 results of fp32 inputs   sums of up to 256 terms, each addition 2^-24, random in sign, and the
                 exponentials' 2^-22: 6e-6
  one token      fp32 arithmetic throughout, sums of 128 terms: 1e-6
A gradient of one decay per head is a sum over tokens whose terms cancel: its bar is of the sum of the
terms' sizes.
"""
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from oracle import block
from tests.gpu_helpers import assert_finite

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
INF = float("inf")


def bar(t, dtype):
    return 2.0 ** -8 + 2.0 ** -14 if t.dtype == BF else 2e-5 if dtype == BF else 6e-6


def rel(got, want):
    got, want = got.double().cpu(), want.cpu()
    e, n = float((got - want).norm()), float(want.norm())
    return e / n if n > 0 else e


class Inputs:
    def __init__(self, lengths, hk, hv, dk, dv, dtype, seed=0, h0=True, decay=1.0, per_head=False):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        n = sum(lengths)
        k = r(n, hk, dk)
        self.q, self.k = r(n, hk, dk).to(DEV, dtype), (k + 0.5 * k.roll(1, 0)).to(DEV, dtype)
        self.v = r(n, hv, dv).to(DEV, dtype)
        # the decay's range over heads: from nearly none to strong
        rates = torch.logspace(-2, 0.5, hv)
        self.g = (-decay * (rates if per_head else r(n, hv).abs() * rates)).to(DEV)
        self.h0 = r(len(lengths), hv, dk, dv).to(DEV) if h0 else None
        self.cu_host = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        self.cu = torch.tensor(self.cu_host, dtype=torch.int32, device=DEV)
        self.dout = r(n, hv, dv).to(DEV, dtype)
        self.dhf = r(len(lengths), hv, dk, dv).to(DEV) if h0 else None
        self.dtype = dtype

    @property
    def args(self):
        return self.q, self.k, self.v, self.g, self.h0, self.cu

    def f64(self, where="cpu"):
        return [None if t is None else t.to(where, torch.float64) for t in (self.q, self.k, self.v, self.g, self.h0)]


def forward(x, **kw):
    out, end = kda.dla_chunk_fwd(*x.args, **kw)
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    return out, end


def backward(x, dhf=True, **kw):
    got = kda.dla_chunk_bwd(*x.args, x.dout, x.dhf if dhf else None, **kw)
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    return got


def check_forward(x, where="cpu", **kw):
    got = forward(x, **kw)
    assert_finite(*got)
    want = block.dla(*x.f64(where), x.cu_host, **kw)
    for name, a, ref in zip(("out", "h_final"), got, want):
        assert rel(a, ref) <= bar(a, x.dtype), f"{name}: {rel(a, ref):.2e}"


def check_backward(x, dhf=True, where="cpu", **kw):
    got = backward(x, dhf, **kw)
    assert_finite(*got)
    q, k, v, g, h0 = x.f64(where)
    rates = g.expand(v.shape[:2]).clone()
    f = lambda t: None if t is None else t.to(where, torch.float64)  # noqa: E731
    want = list(block.dla_grads(q, k, v, rates, h0, x.cu_host, f(x.dout), f(x.dhf) if dhf else None, **kw))
    if g.dim() == 1:
        terms, err = want[3].abs().sum(0).cpu(), (got[3].double().cpu() - want[3].sum(0).cpu()).abs()
        # 2^-126: a decay below e^-200 acts as none at all, and its gradient as 0, below fp32's range
        assert bool((err <= bar(got[3], x.dtype) * terms + 2.0 ** -126).all()), f"dg: {err / terms}"
        want[3] = want[3].sum(0)
        got = list(got)
        got[3] = want[3]
    for name, a, ref in zip(("dq", "dk", "dv", "dg", "dh0"), got, want):
        assert rel(a, ref) <= bar(a, x.dtype), f"{name}: {rel(a, ref):.2e}"


SHAPES = [([1], 1, 1, 128, 128), ([2], 2, 2, 64, 64), ([63], 1, 2, 128, 64), ([64], 2, 2, 128, 128),
          ([65], 1, 3, 64, 128), ([128], 1, 1, 128, 128), ([129, 127], 2, 2, 128, 128), ([200], 2, 4, 128, 128),
          ([0, 1, 130, 0, 64, 17], 2, 2, 128, 128), ([5, 0, 66], 1, 4, 33, 31), ([100], 3, 3, 96, 112),
          ([70, 129], 2, 2, 40, 72), ([3], 1, 1, 1, 1), ([90], 1, 2, 65, 33), ([140], 2, 2, 8, 128),
          ([257], 1, 8, 128, 64), ([300], 2, 6, 72, 100)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", SHAPES)
def test_forward(lengths, hk, hv, dk, dv, dtype):
    check_forward(Inputs(lengths, hk, hv, dk, dv, dtype, seed=len(lengths) + dk))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", SHAPES)
def test_backward(lengths, hk, hv, dk, dv, dtype):
    check_backward(Inputs(lengths, hk, hv, dk, dv, dtype, seed=len(lengths) + dk))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lengths,hk,hv,dk,dv", [([150], 2, 2, 128, 128), ([0, 65, 1, 200], 1, 4, 64, 72)])
def test_one_decay_per_head(lengths, hk, hv, dk, dv, dtype):
    x = Inputs(lengths, hk, hv, dk, dv, dtype, seed=4, per_head=True)
    check_forward(x)
    check_backward(x)
    # the same as that decay at every token
    out, end = forward(x)
    grads = backward(x)
    x.g = x.g.expand(x.v.shape[:2]).contiguous()
    assert all(torch.equal(a, b) for a, b in zip((out, end), forward(x)))
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(grads, backward(x))) if i != 3)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_without_states(dtype):
    x = Inputs([77, 64], 2, 4, 128, 128, dtype, seed=3, h0=False)
    check_forward(x)
    check_backward(x, dhf=False)
    out, end = kda.dla_chunk_fwd(*x.args, output_final_state=False)
    assert end is None and torch.equal(out, forward(x)[0])
    got, without = backward(x, dhf=False), backward(x, dhf=False, want_dg=False, want_dh0=False)
    assert without[3] is None and without[4] is None
    assert all(torch.equal(a, b) for a, b in zip(got[:3], without[:3]))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_a_given_scale(dtype):
    x = Inputs([90], 1, 2, 64, 64, dtype, seed=6)
    check_forward(x, scale=1.0)
    check_backward(x, scale=-0.3)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_decays_of_every_size(dtype):
    """No decay, decays far below fp32's range, -inf (a new document) at a chunk's first, middle
    and last token."""
    x = Inputs([290, 70], 1, 4, 64, 64, dtype, seed=7)
    x.g[:, 0] = 0.0
    x.g[::7, 1] = -300.0
    for t in (0, 63, 64, 100, 127, 128, 255, 256, 289, 291):
        x.g[t, 2] = -INF
    x.g[:, 3] = -50.0
    check_forward(x)
    check_backward(x)
    dg = backward(x)[3]
    assert float(dg[torch.isinf(x.g)].abs().max()) == 0.0
    x.g = torch.tensor([0.0, -INF, -300.0, -1e-4], device=DEV)
    check_forward(x)
    check_backward(x)
    assert float(backward(x)[3][1:3].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("g", [0.0, -1e-3])
def test_long_memories(g, dtype):
    """Sequences of many segments whose first token still counts at the last one; few heads, so that
    a sequence is cut into as many segments as there are."""
    x = Inputs([3001, 0, 1111], 1, 2, 128, 64, dtype, seed=8, h0=True)
    x.q *= 0.25
    x.g[:] = g
    x.g[2000] = -INF
    check_forward(x, DEV)
    check_backward(x, where=DEV)


@pytest.mark.parametrize("hk,hv,dk,dv", [(16, 16, 128, 128), (8, 32, 64, 64), (40, 40, 96, 40)])
def test_many_heads(hk, hv, dk, dv):
    x = Inputs([1500, 1, 333], hk, hv, dk, dv, BF, seed=9, per_head=hk == 8)
    check_forward(x, DEV)
    check_backward(x, where=DEV)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_many_sequences(dtype):
    lengths = [(7 * i) % 90 for i in range(150)]
    x = Inputs(lengths, 2, 4, 64, 128, dtype, seed=10)
    check_forward(x, DEV)
    check_backward(x, where=DEV)


def rounded_once(got, ref):
    """A bf16 result against the definition's value rounded to bf16: apart only where the value
    before its rounding, off by d, falls on the other side of a boundary. That happens to d / ulp
    of the values, each then an ulp off, an ulp up to 2^-7 of the value: the mean square of the
    difference is up to d ulp = 2e-5 2^-7 (d as for the fp32 results), its root 4e-4."""
    e = rel(got, ref.to(BF).double())
    assert e <= 4e-4, f"{e:.2e}"


@pytest.mark.parametrize("lengths,hk,hv,dk,dv", [
    ([1], 1, 1, 128, 128), ([200], 2, 4, 128, 128), ([0, 1, 130, 0, 64, 17], 2, 2, 128, 128), ([5, 0, 66], 1, 4, 33, 31),
    ([100], 3, 3, 96, 112), ([140], 2, 2, 8, 128), ([700, 333], 4, 8, 64, 64), ([2500], 1, 1, 128, 128),
    ([900, 1], 16, 16, 128, 64)])
def test_bf16_results_are_rounded_once(lengths, hk, hv, dk, dv):
    x = Inputs(lengths, hk, hv, dk, dv, BF, seed=len(lengths) + dk)
    xs = x.f64(DEV)
    want = (block.dla(*xs, x.cu_host)[0],) + block.dla_grads(*xs, x.cu_host, x.dout.double(), x.dhf.double())[:3]
    for a, ref in zip((forward(x)[0],) + backward(x)[:3], want):
        rounded_once(a, ref)


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


@pytest.mark.parametrize("lengths,dk,dv", [([130, 70], 128, 64), ([130, 70], 33, 31), ([40], 64, 31), ([1100], 33, 128)])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_slices_of_a_projection_give_the_same_bits(dtype, lengths, dk, dv):
    x = Inputs(lengths, 2, 4, dk, dv, dtype, seed=11)
    ref, grads = forward(x), backward(x)
    for q, k, v in slices(x):
        got = kda.dla_chunk_fwd(q, k, v, x.g, x.h0, x.cu)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        got = kda.dla_chunk_bwd(q, k, v, x.g, x.h0, x.cu, x.dout, x.dhf)
        assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_repeating_changes_no_bit_and_cutting_little(dtype):
    x = Inputs([900], 2, 4, 128, 128, dtype, seed=12)
    ref, grads = forward(x), backward(x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(forward(x), ref))
        assert all(torch.equal(a, b) for a, b in zip(backward(x), grads))
    cut = 333
    one = torch.tensor([0, cut], dtype=torch.int32, device=DEV)
    two = torch.tensor([0, 900 - cut], dtype=torch.int32, device=DEV)
    a, mid = kda.dla_chunk_fwd(x.q[:cut], x.k[:cut], x.v[:cut], x.g[:cut], x.h0, one)
    b, end = kda.dla_chunk_fwd(x.q[cut:], x.k[cut:], x.v[cut:], x.g[cut:], mid, two)
    # both sides round once: twice the bar
    assert rel(torch.cat((a, b)), ref[0].double()) <= 2 * bar(a, dtype) and rel(end, ref[1].double()) <= 2 * bar(end, dtype)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_a_nan_stays_in_its_sequence(dtype):
    lengths = [100, 30, 150, 64]
    x = Inputs(lengths, 2, 2, 128, 128, dtype, seed=13)
    ref, grads = forward(x), backward(x)
    for t in (x.q, x.k, x.v, x.dout):
        t[110] = float("nan")  # in the second sequence
    x.h0[1, 0, 3] = INF
    out, end = forward(x)
    got = backward(x)
    for a, b in [(out, ref[0])] + list(zip(got[:4], grads[:4])):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[130:], b[130:])
    for a, b in ((end, ref[1]), (got[4], grads[4])):
        assert torch.equal(a[[0, 2, 3]], b[[0, 2, 3]])
    assert bool(torch.isnan(out[110:130]).any())


@pytest.mark.parametrize("dtype", [FP, BF])
def test_a_decay_that_is_nan_shows(dtype):
    """It reaches the tokens from its own on, of its head and sequence alone."""
    x = Inputs([100, 230, 40], 2, 2, 128, 128, dtype, seed=25)
    ref, grads = forward(x), backward(x)
    x.g[150, 1] = float("nan")
    out, end = forward(x)
    got = backward(x)
    assert bool(torch.isnan(out[150:330, 1]).all()) and bool(torch.isnan(end[1, 1]).all())
    assert bool(torch.isnan(got[0][150:330, 1]).all()) and bool(torch.isnan(got[4][1, 1]).all())
    for a, b in [(out, ref[0])] + list(zip(got[:4], grads[:4])):
        assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[:100], b[:100]) and torch.equal(a[330:], b[330:])
    for a, b in ((end, ref[1]), (got[4], grads[4])):
        assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 0], b[1, 0])


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("hk", [4, 1])
def test_tokens_behind_the_last_sequence(hk, dtype, per_head):
    """Buffers with more tokens than the sequences: those change nothing, their results are not written."""
    lengths, n, more = [130, 0, 77], 207, 93
    x = Inputs(lengths, hk, 4, 128, 64, dtype, seed=26, per_head=per_head)
    y = Inputs([n + more], hk, 4, 128, 64, dtype, seed=27, per_head=per_head)
    for name in ("q", "k", "v", "dout") + (() if per_head else ("g",)):
        getattr(y, name)[:n] = getattr(x, name)
        getattr(y, name)[n:] = float("nan")
    g = x.g if per_head else y.g
    lib, stream = kda.load_library(), torch.cuda.current_stream().cuda_stream
    sizes = (n + more, 3, hk, 4, 128, 64, {FP: 0, BF: 1}[dtype])
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
    ins = (y.q.data_ptr(), y.k.data_ptr(), y.v.data_ptr(), hk * 128, hk * 128, 256, g.data_ptr(), 0 if per_head else 4,
           x.h0.data_ptr(), x.cu.data_ptr(), 128 ** -0.5)
    for t in (y.q, y.k, y.v):
        assert t.is_contiguous()
    out, end = torch.full_like(y.v, 7.0), torch.empty_like(x.h0)
    assert lib.kda_dla_chunk_fwd(*ins, out.data_ptr(), end.data_ptr(), ws.data_ptr(), ws.numel(), *sizes, stream) == 0
    ref = forward(x)  # the same chunks in the same order: the same bits
    assert torch.equal(out[:n], ref[0]) and torch.equal(end, ref[1]) and bool((out[n:] == 7).all())
    dq, dk, dv = torch.full_like(y.q, 7.0), torch.full_like(y.k, 7.0), torch.full_like(y.v, 7.0)
    dg, dh0 = torch.full_like(g, 7.0), torch.empty_like(x.h0)
    assert lib.kda_dla_chunk_bwd(*ins, y.dout.data_ptr(), x.dhf.data_ptr(), *[t.data_ptr() for t in (dq, dk, dv, dg, dh0)],
                                 ws.data_ptr(), ws.numel(), *sizes, stream) == 0
    grads = backward(x)
    for a, b in zip((dq, dk, dv, dg, dh0), grads):
        if a.shape[0] == n + more:
            assert bool((a[n:] == 7).all())
            a = a[:n]
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_no_token(dtype):
    x = Inputs([0, 0], 2, 2, 64, 64, dtype, seed=14)
    out, end = forward(x)
    assert out.shape == (0, 2, 64) and torch.equal(end, x.h0)
    grads = backward(x)
    assert grads[0].numel() == 0 and torch.equal(grads[4], x.dhf)
    x.g = torch.full((2,), -0.1, device=DEV)
    assert torch.equal(backward(x)[3], torch.zeros(2, device=DEV))
    x = Inputs([], 2, 2, 64, 64, dtype, seed=14, h0=False, per_head=True)
    out, end = forward(x)
    assert out.shape == (0, 2, 64) and end.shape == (0, 2, 64, 64)
    assert torch.equal(backward(x)[3], torch.zeros(2, device=DEV))


def test_gradients_are_differences_of_the_forward():
    """The kernel's gradients against differences of the kernel's forward pass, fp32. The loss is
    linear in q, v and h0, so that a step of any size is exact up to the forward's rounding (6e-6 of
    out's norm, taken twice, over a change of 0.1 of it); k likewise; g by its own small step, whose
    square adds 1e-3."""
    x = Inputs([90, 41], 2, 4, 64, 48, FP, seed=15)
    gen = torch.Generator().manual_seed(16)

    def loss():
        out, end = forward(x)
        return float((out.double() * x.dout.double()).sum() + (end.double() * x.dhf.double()).sum())

    grads = backward(x)
    for name, gr in zip(("q", "k", "v", "g", "h0"), grads):
        t = getattr(x, name)
        d = torch.randn(t.shape, generator=gen).to(DEV) * (t.abs() if name == "g" else 1.0)
        step = 0.02 if name == "g" else 0.5
        up, down = t + step * d, t - step * d
        setattr(x, name, up)
        a = loss()
        setattr(x, name, down)
        b = loss()
        setattr(x, name, t)
        got, want = (a - b) / (2 * step), float((gr.double() * d.double()).sum())
        assert abs(got - want) <= 3e-3 * float(gr.double().norm() * d.double().norm()), name


def test_another_stream_and_a_callers_workspace():
    x = Inputs([700, 80], 4, 4, 128, 128, BF, seed=17)
    ref, grads = forward(x), backward(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device=DEV)  # NaNs wherever it is not written
        out = torch.full_like(x.v, float("nan"))
        got = kda.dla_chunk_fwd(*x.args, out=out, workspace=ws)
        back = kda.dla_chunk_bwd(*x.args, x.dout, x.dhf, workspace=ws)
    s.synchronize()
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(torch.equal(a, b) for a, b in zip(back, grads))


@pytest.mark.parametrize("dk", [128, 33])
def test_two_calls_at_once(dk):
    """Calls on two streams share nothing, whichever of them a kernel of the other's follows."""
    xs = [Inputs([600, 90], 4, 4, dk, 128, BF, seed=28), Inputs([20, 700], 4, 4, dk, 128, BF, seed=29)]
    ref = [(*forward(x), *backward(x)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append((*kda.dla_chunk_fwd(*x.args), *kda.dla_chunk_bwd(*x.args, x.dout, x.dhf)))
    torch.cuda.synchronize()
    assert kda.read_device_flags() == 0
    for want, calls in zip(ref, got):
        for call in calls:
            assert all(torch.equal(a, b) for a, b in zip(call, want))


def test_in_a_graph():
    x = Inputs([300, 50], 2, 4, 128, 64, BF, seed=18)
    state = torch.zeros(3, 4, 128, 64, device=DEV)
    kda.dla_chunk_fwd(*x.args), backward(x), kda.dla_step(x.q[:3], x.k[:3], x.v[:3], x.g[:3], state)
    state.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, end = kda.dla_chunk_fwd(*x.args)
        grads = kda.dla_chunk_bwd(*x.args, x.dout, x.dhf)
        one = kda.dla_chunk_fwd(x.q, x.k, x.v, x.g)[0]
        kda.dla_step(x.q[:3], x.k[:3], x.v[:3], x.g[:3], state)
    for seed in (18, 19):
        y = Inputs([300, 50], 2, 4, 128, 64, BF, seed=seed)
        for n in ("q", "k", "v", "g", "h0", "dout", "dhf"):
            getattr(x, n).copy_(getattr(y, n))
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, back = forward(y), backward(y)
        assert all(torch.equal(a, b) for a, b in zip((out, end), want))
        assert all(torch.equal(a, b) for a, b in zip(grads, back))
        assert torch.equal(one, kda.dla_chunk_fwd(y.q, y.k, y.v, y.g)[0])
        again = torch.zeros_like(state)
        kda.dla_step(y.q[:3], y.k[:3], y.v[:3], y.g[:3], again)
        assert torch.equal(state, again)


def test_offsets_beyond_32_bits():
    """Tokens so far apart that their offsets pass 2^32 bytes and 2^31 elements."""
    n, stride = 260, 1 << 23
    x = Inputs([n], 1, 1, 128, 128, BF, seed=20, h0=False)
    ref, grads = forward(x), backward(x, dhf=False)
    wide = torch.empty(n * stride, dtype=BF, device=DEV).view(n, stride)
    views = []
    for i, t in enumerate((x.q, x.k, x.v)):
        wide[:, 128 * i:128 * i + 128] = t.view(n, 128)
        views.append(wide[:, 128 * i:128 * i + 128].unflatten(1, (1, 128)))
    assert wide.numel() > 1 << 31
    got = kda.dla_chunk_fwd(*views, x.g, None, x.cu)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    got = kda.dla_chunk_bwd(*views, x.g, None, x.cu, x.dout)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


# ---------------------------------------------------------------- one token

STEPS = [(1, 1, 1, 128, 128), (1, 32, 32, 128, 128), (5, 2, 4, 64, 64), (9, 2, 2, 40, 72), (3, 1, 3, 33, 31),
         (64, 4, 4, 128, 64), (7, 1, 2, 1, 1), (130, 2, 2, 96, 124), (4, 2, 2, 128, 125), (6, 1, 1, 8, 4)]


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("B,hk,hv,dk,dv", STEPS)
def test_step(B, hk, hv, dk, dv, dtype, per_head):
    x = Inputs([1] * B, hk, hv, dk, dv, dtype, seed=B + dk, per_head=per_head)
    gen = torch.Generator().manual_seed(B)
    slots = torch.randperm(B + 3, generator=gen)[:B].to(DEV, torch.int32)
    pool = torch.randn(B + 3, hv, dk, dv, generator=gen).to(DEV)
    before = pool.clone()
    x.h0 = pool[slots.long()].clone()
    out = kda.dla_step(x.q, x.k, x.v, x.g, pool, slots)
    torch.cuda.synchronize()
    want, end = block.dla(*x.f64(), x.cu_host)
    assert rel(out, want) <= (1e-6 if dtype == FP else 2.0 ** -8) and rel(pool[slots.long()], end) <= 1e-6
    rest = torch.ones(B + 3, dtype=torch.bool, device=DEV)
    rest[slots.long()] = False
    assert torch.equal(pool[rest], before[rest])
    own = x.h0.clone()
    assert torch.equal(kda.dla_step(x.q, x.k, x.v, x.g, own), out) and torch.equal(own, pool[slots.long()])


def test_step_padded_rows_touch_nothing():
    x = Inputs([1] * 6, 2, 4, 64, 64, BF, seed=21)
    pool = torch.randn(4, 4, 64, 64, device=DEV)
    before = pool.clone()
    slots = torch.tensor([-1, 2, 4, 0, -2147483648, 2147483647], dtype=torch.int32, device=DEV)
    x.q[0] = x.v[2] = float("nan")
    out = kda.dla_step(x.q, x.k, x.v, x.g, pool, slots)
    assert float(out[[0, 2, 4, 5]].abs().max()) == 0.0 and torch.equal(pool[[1, 3]], before[[1, 3]])
    assert not torch.equal(pool[2], before[2]) and bool(torch.isfinite(out).all())


def test_step_reset_forgets():
    x = Inputs([1] * 2, 1, 2, 64, 64, FP, seed=22)
    x.g[0] = -INF
    pool = torch.randn(2, 2, 64, 64, device=DEV)
    pool[0, 0, 3] = float("nan")
    kda.dla_step(x.q, x.k, x.v, x.g, pool)
    for h in range(2):
        assert torch.equal(pool[0, h], x.k[0, 0][:, None] * x.v[0, h][None])


@pytest.mark.parametrize("dtype", [FP, BF])
def test_steps_continue_a_prefill(dtype):
    x = Inputs([80], 2, 4, 64, 128, dtype, seed=23)
    out, end = forward(x)
    cu = torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    head, state = kda.dla_chunk_fwd(x.q[:70], x.k[:70], x.v[:70], x.g[:70], x.h0, cu)
    rows = [kda.dla_step(x.q[t:t + 1], x.k[t:t + 1], x.v[t:t + 1], x.g[t:t + 1], state) for t in range(70, 80)]
    # both sides round once: twice the bar
    assert rel(torch.cat(rows), out[70:].double()) <= 2 * bar(out, dtype)
    assert rel(state, end.double()) <= 2 * bar(end, dtype)


def test_binding_refuses():
    x = Inputs([40], 1, 2, 64, 64, BF, seed=24)
    with pytest.raises(ValueError):
        kda.dla_chunk_fwd(x.q.half(), x.k.half(), x.v.half(), x.g)
    with pytest.raises(ValueError):
        kda.dla_chunk_fwd(x.q, x.k, x.v, x.g.cpu())
    with pytest.raises(kda.KDAError):
        kda.dla_chunk_fwd(*x.args, scale=INF)
    with pytest.raises(kda.KDAError):
        kda.dla_chunk_fwd(*x.args, out=x.v)
    with pytest.raises(kda.KDAError):
        kda.dla_chunk_fwd(*x.args, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.dla_step(x.q, x.k, x.v, x.g, torch.zeros(3, 2, 64, 64, device=DEV))
    big = Inputs([4], 1, 1, 130, 8, BF)
    with pytest.raises(kda.KDAError):
        kda.dla_chunk_fwd(*big.args)
