"""GPU parity of the norm of queries and keys with the position rotation (``kda_qk_norm_rope_fwd``,
``kda_qk_norm_rope_bwd``) against the fp64 definition on the same inputs.

Bars: every operation is fp32 (sums of up to 256 terms, 2^-24 each; the angle to 2^-25 of a turn, so
1.9e-7 of a pair's size): 6e-7 of a result's norm, the weights' gradients, sums over all rows, 2e-6;
bf16 results are rounded once, half a step, 2^-8 of a value at most. dx = c (t - n mean(t n)) is a
difference of terms rounded to 2^-24 each, and with few channels both are far larger than it (one channel:
n^2 = 1 - eps / x^2, so dx is 1e-6 of its terms): its bar is of the norm of c t, which dx, its projection,
never exceeds."""
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from oracle import block
from tests.gpu_helpers import assert_finite

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def bar(t):
    return 2.0 ** -8 if t.dtype == BF else 2e-6 if t.dim() == 1 else 6e-7


def rel(got, want, of=None):
    got = got.double().cpu()
    e, n = float((got - want).norm()), float((want if of is None else of).norm())
    return e / n if n > 0 else e


class Inputs:
    def __init__(self, n, hq, hk, d, rot, dtype, seed=0, wide=torch.int32, positions=None):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.q, self.k = (3 * r(n, hq, d)).to(DEV, dtype), (0.1 * r(n, hk, d)).to(DEV, dtype)
        self.wq, self.wk = r(d).to(DEV), r(d).to(DEV)
        self.dq, self.dk = r(n, hq, d).to(DEV, dtype), r(n, hk, d).to(DEV, dtype)
        pos = torch.randint(0, 1 << 20, (n,), generator=gen) if positions is None else positions
        self.pos = pos.to(DEV, wide)
        self.freqs = kda.rotary_frequencies(rot)

    @property
    def args(self):
        return self.q, self.k, self.wq, self.wk, self.pos, self.freqs


def check(x, interleaved=False, eps=1e-6):
    kw = dict(eps=eps, interleaved=interleaved)
    out = kda.qk_norm_rope_fwd(*x.args, **kw)
    grads = kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args, **kw)
    torch.cuda.synchronize()
    assert_finite(*out, *grads)
    f = block.f64
    pos, freqs = x.pos.cpu(), x.freqs.cpu()
    for i, (a, w, dy) in enumerate(((x.q, x.wq, x.dq), (x.k, x.wk, x.dk))):
        want = block.head_norm_rope(f(a), f(w), pos, freqs, eps, interleaved)
        assert rel(out[i], want) <= bar(out[i]), f"y {rel(out[i], want):.2e}"
        dx, dw = block.head_norm_rope_grads(f(dy), f(a), f(w), pos, freqs, eps, interleaved)
        # c t: dy turned back, times weight and c
        ones, back = torch.ones(x.q.shape[2], dtype=torch.float64), -pos.to(torch.int64)
        size = f(dy).square().mean(-1, keepdim=True).sqrt()
        t = size * block.head_norm_rope(f(dy), ones, back, freqs, 0.0, interleaved) * f(w)
        t = t / torch.sqrt(f(a).square().mean(-1, keepdim=True) + eps)
        e = rel(grads[i], dx, t)
        assert e <= bar(grads[i]), f"dx {e:.2e}"
        assert rel(grads[2 + i], dw) <= bar(grads[2 + i]), f"dw {rel(grads[2 + i], dw):.2e}"
    return out, grads


SHAPES = [(1, 1, 1, 128, 128), (1, 32, 8, 128, 64), (5, 2, 2, 64, 64), (33, 3, 1, 100, 50), (7, 4, 4, 80, 20),
          (130, 7, 1, 256, 128), (17, 1, 5, 256, 256), (9, 2, 2, 8, 8), (3, 1, 1, 1, 0), (12, 2, 3, 33, 32),
          (40, 32, 32, 128, 0), (20, 5, 2, 128, 48), (600, 16, 4, 72, 72), (11, 2, 1, 2, 2), (5, 300, 300, 16, 8),
          (50, 4, 2, 100, 100), (21, 3, 3, 100, 0), (70, 2, 4, 36, 20), (9, 5, 1, 252, 124), (6, 1, 1, 4, 4), (19, 2, 2, 20, 6)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,hq,hk,d,rot", SHAPES)
def test_parity(n, hq, hk, d, rot, dtype, interleaved):
    check(Inputs(n, hq, hk, d, rot, dtype, seed=n + d), interleaved)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_many_tokens(dtype):
    """More token blocks than the backward pass has CTAs."""
    check(Inputs(20011, 4, 2, 64, 32, dtype, seed=1))


def test_positions_of_every_size_and_sign():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -7, 1 << 20])
    a, _ = check(Inputs(8, 2, 2, 64, 64, FP, seed=2, positions=pos))
    b, _ = check(Inputs(8, 2, 2, 64, 64, FP, seed=2, positions=pos, wide=torch.int64))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # beyond int32: the fp64 product of the definition rounds its angle to 2^-52 of 3e10
    check(Inputs(2, 2, 2, 64, 64, FP, seed=3, positions=torch.tensor([3 * 10 ** 10, -5 * 10 ** 9]), wide=torch.int64))


def test_turning_back_is_the_inverse():
    x = Inputs(50, 2, 2, 128, 128, FP, seed=4)
    ones = torch.ones(128, device=DEV)
    y, z = kda.qk_norm_rope_fwd(x.q, x.k, ones, ones, x.pos, x.freqs)
    back, _ = kda.qk_norm_rope_fwd(y, z, ones, ones, -x.pos, x.freqs)
    plain, _ = kda.qk_norm_rope_fwd(x.q, x.k, ones, ones)
    assert rel(back, plain.double().cpu()) <= 2e-6


def test_without_rotation():
    x = Inputs(50, 4, 2, 128, 0, BF, seed=5)
    a = kda.qk_norm_rope_fwd(*x.args)
    b = kda.qk_norm_rope_fwd(x.q, x.k, x.wq, x.wk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args), kda.qk_norm_rope_bwd(x.dq, x.dk, x.q, x.k, x.wq, x.wk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lead,tail", [(8, 16), (3, 2)])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_slices_of_a_projection(lead, tail, dtype, interleaved):
    """Aligned slices give the same bits; at odd offsets the sums run in another order."""
    x = Inputs(70, 4, 2, 64, 64, dtype, seed=6)
    out, grads = check(x, interleaved)
    n = 70
    wide = torch.full((n, lead + 6 * 64 + tail), float("nan"), device=DEV, dtype=dtype)
    dwide = wide.clone()
    for w, a, b in ((wide, x.q, x.k), (dwide, x.dq, x.dk)):
        w[:, lead:lead + 256], w[:, lead + 256:lead + 384] = a.flatten(1), b.flatten(1)
    q, k, dq, dk = (w[:, lead + o:lead + o + s].unflatten(1, (-1, 64)) for w in (wide, dwide)
                    for o, s in ((0, 256), (256, 128)))
    kw = dict(interleaved=interleaved)
    got = kda.qk_norm_rope_fwd(q, k, *x.args[2:], **kw), kda.qk_norm_rope_bwd(dq, dk, q, k, *x.args[2:], **kw)
    for a, b in zip(got[0] + got[1], out + grads):
        assert torch.equal(a, b) if lead == 8 else rel(a, b.double().cpu()) <= 2 * bar(a)


def test_rows_of_zeros_and_of_large_and_small_values():
    x = Inputs(6, 2, 2, 64, 64, FP, seed=7)
    x.q[0] = 0.0
    x.q[1] *= 1e15
    x.q[2] *= 1e-15
    x.k[3] *= 1e-3
    check(x)
    assert float(kda.qk_norm_rope_fwd(*x.args)[0][0].abs().max()) == 0.0


def test_a_nan_stays_in_its_row():
    x = Inputs(40, 3, 2, 128, 64, BF, seed=8)
    ref = kda.qk_norm_rope_fwd(*x.args)
    grads = kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    x.q[17, 1, 5] = float("nan")
    x.k[3, 0, 0] = float("inf")
    got, back = kda.qk_norm_rope_fwd(*x.args), kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    for a, b, (t, h) in zip(got + back[:2], ref + grads[:2], ((17, 1), (3, 0)) * 2):
        assert bool(torch.isnan(a[t, h]).any())
        a[t, h] = b[t, h]
        assert torch.equal(a, b)


def test_no_token():
    x = Inputs(0, 2, 1, 64, 32, BF)
    q, k = kda.qk_norm_rope_fwd(*x.args)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    grads = kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    assert grads[0].numel() == 0 and float(grads[2].abs().max()) == 0.0 and float(grads[3].abs().max()) == 0.0


def test_another_stream_a_graph_and_given_outputs():
    x = Inputs(300, 4, 2, 128, 64, BF, seed=9)
    ref, grads = kda.qk_norm_rope_fwd(*x.args), kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    qo, ko = torch.empty_like(x.q), torch.empty_like(x.k)
    with torch.cuda.graph(graph):
        got = kda.qk_norm_rope_fwd(*x.args, q_out=qo, k_out=ko)
        back = kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args, workspace=ws)
    assert got[0] is qo and got[1] is ko
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + back, ref + grads))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, back = kda.qk_norm_rope_fwd(*x.args), kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + back, ref + grads))


def test_offsets_beyond_32_bits():
    n, stride = 260, 1 << 23
    x = Inputs(n, 1, 1, 128, 128, BF, seed=10)
    ref, grads = kda.qk_norm_rope_fwd(*x.args), kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args)
    wide = torch.empty(n * stride, dtype=BF, device=DEV).view(n, stride)
    q, k, dq, dk = (wide[:, 128 * i:128 * i + 128].unflatten(1, (1, 128)) for i in range(4))
    for a, b in ((q, x.q), (k, x.k), (dq, x.dq), (dk, x.dk)):
        a.copy_(b)
    got, back = kda.qk_norm_rope_fwd(q, k, *x.args[2:]), kda.qk_norm_rope_bwd(dq, dk, q, k, *x.args[2:])
    assert all(torch.equal(a, b) for a, b in zip(got + back, ref + grads))


def test_binding_refuses():
    x = Inputs(4, 2, 1, 64, 32, BF)
    with pytest.raises(ValueError):
        kda.qk_norm_rope_fwd(x.q.half(), x.k.half(), x.wq, x.wk)
    with pytest.raises(ValueError):
        kda.qk_norm_rope_fwd(x.q, x.k, x.wq, x.wk.cpu())
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope_fwd(*x.args, eps=0.0)
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope_fwd(*x.args, q_out=x.q)
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope_bwd(x.dq, x.dk, *x.args, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))
    wide = torch.zeros(2, 1, 300, device=DEV)
    with pytest.raises(kda.KDAError):
        kda.qk_norm_rope_fwd(wide, wide, torch.ones(300, device=DEV), torch.ones(300, device=DEV))
