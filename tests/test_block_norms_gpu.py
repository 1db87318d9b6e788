"""GPU parity of the residual norm and the gated norm, forward and backward, against their fp64
definitions on the same inputs.

Bars on the rel-L2 error: bf16 results are held to the definition's value rounded to bf16, from
which an fp32 value can only differ next to a rounding boundary: 2.1e-3; fp32 results come from fp32 sums of up to 8192 terms (added pairwise or by a few
threads: below 30 roundings of 2^-24) and a handful of roundings: 2e-6."""
import threading

import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from oracle import block
from tests.gpu_helpers import assert_finite, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32
EPS = 1e-5


def rand(seed, *shape, dtype=FP):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def check(got, want):
    for a, ref in zip(got, want):
        if ref is None:
            assert a is None
            continue
        assert_finite(a)
        if a.dtype == BF:
            ref = ref.to(BF).double()
        e = rel_l2(a.double().cpu().numpy(), ref.numpy())
        assert e <= (2.1e-3 if a.dtype == BF else 2e-6), f"{e:.2e}"


def inside(t, lead, tail):
    """The rows of ``t`` inside wider rows, NaN around them."""
    flat = t.reshape(t.shape[0], -1)
    wide = torch.full((t.shape[0], lead + flat.shape[1] + tail), float("nan"), device=DEV, dtype=t.dtype)
    wide[:, lead:lead + flat.shape[1]] = flat
    return wide[:, lead:lead + flat.shape[1]].unflatten(1, t.shape[1:]) if t.dim() > 2 else wide[:, lead:lead + flat.shape[1]]


SIZES = [(1, 4096), (3, 1), (5, 7), (2, 8), (9, 255), (4, 256), (6, 264), (3, 513), (700, 1024), (2, 1025),
         (7, 4104), (2, 8192), (3, 12000), (2, 32768), (1000, 40)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("with_residual,with_scale", [(True, True), (True, False), (False, True), (False, False)])
def test_residual_norm(n, d, with_residual, with_scale, dtype):
    x, res = rand(1, n, d, dtype=dtype), rand(2, n, d, dtype=dtype) if with_residual else None
    w, sc = 1 + 0.2 * rand(3, d), 0.5 + 0.2 * rand(4, d) if with_scale else None
    y, r = kda.residual_norm_fwd(x, w, res, sc, eps=EPS)
    check((y, r), block.residual_norm(block.f64(x), block.f64(w), block.f64(res), block.f64(sc), EPS))
    assert (r is x) == (not with_residual and not with_scale)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("with_dr,with_scale", [(True, True), (True, False), (False, True)])
def test_residual_norm_backward(n, d, with_dr, with_scale, dtype):
    if d < 8 and not with_dr:
        pytest.skip("at one channel the norm's own gradient is a difference of equal numbers")
    r, dy, x = rand(1, n, d, dtype=dtype), rand(2, n, d, dtype=dtype), rand(3, n, d, dtype=dtype)
    dr = rand(4, n, d, dtype=dtype) if with_dr else None
    w, sc = 1 + 0.2 * rand(5, d), 0.5 + 0.2 * rand(6, d) if with_scale else None
    got = kda.residual_norm_bwd(dy, r, w, dr, x if with_scale else None, sc, eps=EPS)
    want = block.residual_norm_grads(block.f64(dy), block.f64(r), block.f64(w), block.f64(dr), block.f64(x),
                                     block.f64(sc), EPS)
    check(got, want)
    again = kda.residual_norm_bwd(dy, r, w, dr, x if with_scale else None, sc, eps=EPS)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lead,tail", [(8, 8), (3, 2)])
def test_residual_norm_of_slices(lead, tail, dtype):
    n, d = 37, 520
    x, res, dy, dr = (rand(i, n, d, dtype=dtype) for i in range(4))
    w, sc = 1 + 0.2 * rand(5, d), 0.5 + 0.2 * rand(6, d)
    a = kda.residual_norm_fwd(inside(x, lead, tail), w, inside(res, lead, tail), sc, eps=EPS)
    check(a, block.residual_norm(block.f64(x), block.f64(w), block.f64(res), block.f64(sc), EPS))
    g = kda.residual_norm_bwd(inside(dy, lead, tail), inside(res, lead, tail), w, inside(dr, lead, tail),
                              inside(x, lead, tail), sc, eps=EPS)
    check(g, block.residual_norm_grads(block.f64(dy), block.f64(res), block.f64(w), block.f64(dr), block.f64(x),
                                       block.f64(sc), EPS))


def test_residual_norm_edge_rows():
    """A row of zeros, one of large and one of tiny values; NaN and inf stay in their row."""
    d = 96
    x = rand(1, 6, d)
    x[0], x[1], x[2] = 0.0, x[1] * 1e15, x[2] * 1e-15
    x[3, 5], x[4, 7] = float("nan"), float("inf")
    w = 1 + 0.2 * rand(2, d)
    y, _ = kda.residual_norm_fwd(x, w, eps=EPS)
    ok = [0, 1, 2, 5]
    check((y[ok],), block.residual_norm(block.f64(x[ok]), block.f64(w), None, None, EPS)[:1])
    assert float(y[0].abs().max()) == 0.0
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4, 7]))


def test_norms_of_no_row():
    w = torch.ones(16, device=DEV)
    x, z = torch.zeros((0, 16), device=DEV), torch.zeros((0, 2, 16), device=DEV)
    y, r = kda.residual_norm_fwd(x, w, x)
    assert y.shape == (0, 16) and r.shape == (0, 16)
    _, _, dw, ds = kda.residual_norm_bwd(x, x, w, None, x, w)
    assert float(dw.abs().max()) == 0.0 and float(ds.abs().max()) == 0.0
    assert kda.gated_norm_fwd(z, z, w).shape == (0, 2, 16)
    assert float(kda.gated_norm_bwd(z, z, z, w)[2].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
@pytest.mark.parametrize("n,h,d", [(1, 1, 128), (3, 32, 128), (130, 5, 64), (7, 3, 100), (2, 31, 256), (9, 2, 33),
                                   (5, 4, 1), (2, 1, 8), (400, 7, 31)])
def test_gated_norm(n, h, d, activation, dtype):
    x, z, dy = (rand(i, n, h, d, dtype=dtype) for i in range(3))
    z = z * 4
    w = 1 + 0.2 * rand(5, d)
    y = kda.gated_norm_fwd(x, z, w, eps=EPS, activation=activation)
    f = [block.f64(t) for t in (x, z, w)]
    check((y,), (block.gated_norm(*f, EPS, activation),))
    got = kda.gated_norm_bwd(dy, x, z, w, eps=EPS, activation=activation)
    want = block.gated_norm_grads(block.f64(dy), *f, EPS, activation)
    # at one channel dx is a difference of equal numbers: nothing is left of it to compare
    check(got if d > 1 else got[1:], want if d > 1 else want[1:])
    again = kda.gated_norm_bwd(dy, x, z, w, eps=EPS, activation=activation)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("lead,tail", [(16, 8), (1, 3)])
def test_gated_norm_of_slices(lead, tail, dtype):
    x, z, dy = (rand(i, 21, 3, 40, dtype=dtype) for i in range(3))
    w = 1 + 0.2 * rand(5, 40)
    a = kda.gated_norm_fwd(inside(x, lead, tail), inside(z, lead, tail), w, eps=EPS, activation="silu")
    f = [block.f64(t) for t in (x, z, w)]
    check((a,), (block.gated_norm(*f, EPS, "silu"),))
    g = kda.gated_norm_bwd(inside(dy, lead, tail), inside(x, lead, tail), inside(z, lead, tail), w, eps=EPS,
                           activation="silu")
    check(g, block.gated_norm_grads(block.f64(dy), *f, EPS, "silu"))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gated_norm_saturated_gates(dtype):
    """Gates far out on both sides: the sigmoid ends at 0 and 1, nothing overflows."""
    x = rand(1, 4, 2, 64, dtype=dtype)
    z = torch.full((4, 2, 64), 200.0, device=DEV, dtype=dtype)
    z[2:] = -200.0
    w = torch.ones(64, device=DEV)
    for act in ("sigmoid", "silu"):
        y = kda.gated_norm_fwd(x, z, w, eps=EPS, activation=act)
        dx, dz, dw = kda.gated_norm_bwd(x, x, z, w, eps=EPS, activation=act)
        assert_finite(y, dx, dz, dw)
        assert float(y[2:].abs().max()) == 0.0 and float(dx[2:].abs().max()) == 0.0


def test_residual_norm_offsets_beyond_32_bits():
    n, d = 2_200_000, 1024
    x = torch.zeros((n, d), device=DEV, dtype=BF)
    x[-3:] = rand(1, 3, d, dtype=BF)
    w = 1 + 0.2 * rand(2, d)
    y, _ = kda.residual_norm_fwd(x, w, eps=EPS)
    assert torch.equal(y[-3:], kda.residual_norm_fwd(x[-3:].clone(), w, eps=EPS)[0])
    dx, _, _, _ = kda.residual_norm_bwd(x, x, w, eps=EPS)
    assert torch.equal(dx[-3:], kda.residual_norm_bwd(x[-3:].clone(), x[-3:].clone(), w, eps=EPS)[0])


def test_binding_refuses():
    x, w = rand(1, 4, 16), torch.ones(16, device=DEV)
    z = rand(2, 4, 2, 16)
    for call in (lambda: kda.residual_norm_fwd(x, w[:8]), lambda: kda.residual_norm_fwd(x.half(), w),
                 lambda: kda.residual_norm_fwd(x, w, x[:2]), lambda: kda.residual_norm_fwd(x.T, w[:4]),
                 lambda: kda.residual_norm_fwd(x, w.double()), lambda: kda.residual_norm_bwd(x, x, w, scale=w),
                 lambda: kda.residual_norm_bwd(x.to(BF), x, w), lambda: kda.gated_norm_fwd(z, z[:, :1], w),
                 lambda: kda.gated_norm_fwd(z, z, w, activation="tanh"), lambda: kda.gated_norm_fwd(x, x, w),
                 lambda: kda.gated_norm_fwd(z.transpose(0, 1), z.transpose(0, 1), w),
                 lambda: kda.gated_norm_bwd(z, z, z, w[:3])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(kda.KDAError):
        kda.residual_norm_fwd(x, w, eps=0.0)
    with pytest.raises(kda.KDAError):
        kda.residual_norm_fwd(x, w, x, out=x)


# ---------------------------------------------------------------- more rows than a launch holds at once

@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d", [(1901, 2048), (701, 4096), (333, 8192), (5003, 264), (9001, 96), (1301, 1003)])
@pytest.mark.parametrize("with_dr,with_scale", [(True, True), (False, False)])
def test_residual_norm_backward_walks_over_rows(n, d, with_dr, with_scale, dtype):
    r, dy, x = rand(1, n, d, dtype=dtype), rand(2, n, d, dtype=dtype), rand(3, n, d, dtype=dtype)
    dr = rand(4, n, d, dtype=dtype) if with_dr else None
    w, sc = 1 + 0.2 * rand(5, d), 0.5 + 0.2 * rand(6, d) if with_scale else None
    got = kda.residual_norm_bwd(dy, r, w, dr, x if with_scale else None, sc, eps=EPS)
    check(got, block.residual_norm_grads(block.f64(dy), block.f64(r), block.f64(w), block.f64(dr), block.f64(x),
                                         block.f64(sc), EPS))
    # a row does not depend on the ones a thread has handled before it
    part = slice(n - 7, n)
    last = kda.residual_norm_bwd(dy[part], r[part], w, None if dr is None else dr[part],
                                 x[part] if with_scale else None, sc, eps=EPS)
    assert torch.equal(last[1], got[1][part])


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,h,d", [(1301, 32, 128), (2003, 16, 64), (1001, 31, 100), (4001, 5, 256), (9001, 7, 24)])
def test_gated_norm_walks_over_rows(n, h, d, dtype):
    x, z, dy = (rand(i, n, h, d, dtype=dtype) for i in range(3))
    w = 1 + 0.2 * rand(4, d)
    y = kda.gated_norm_fwd(x, z, w, eps=EPS, activation="silu")
    check((y,), (block.gated_norm(block.f64(x), block.f64(z), block.f64(w), EPS, "silu"),))
    got = kda.gated_norm_bwd(dy, x, z, w, eps=EPS, activation="silu")
    check(got, block.gated_norm_grads(block.f64(dy), block.f64(x), block.f64(z), block.f64(w), EPS, "silu"))
    part = slice(n - 3, n)
    assert torch.equal(kda.gated_norm_fwd(x[part], z[part], w, eps=EPS, activation="silu"), y[part])
    last = kda.gated_norm_bwd(dy[part], x[part], z[part], w, eps=EPS, activation="silu")
    assert torch.equal(last[0], got[0][part]) and torch.equal(last[1], got[1][part])


def test_threads_of_different_widths_keep_their_shared_memory():
    """Threads run one kernel at two widths, whose launches take 192 and 164 KB of shared memory,
    straight through the C entry: none takes another's away, so no launch is refused."""
    lib = kda.load_library()
    calls, keep = [], []
    for i in range(4):
        d = (8192, 4608)[i % 2]
        x, dy, w, s = rand(i, 2, d), rand(i + 4, 2, d), rand(i + 8, d), rand(i + 12, d)
        dx, dres, dw, ds = (torch.empty_like(t) for t in (x, x, w, w))
        need = lib.kda_residual_norm_bwd_workspace_bytes(2, d, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        stream = torch.cuda.Stream()
        keep.append((x, dy, w, s, dx, dres, dw, ds, ws, stream))
        p = [t.data_ptr() for t in keep[-1][:9]]
        calls.append((p[1], d, None, 0, p[0], d, p[0], d, p[3], p[2], p[4], p[5], p[7], p[6], p[8], need, 2, d,
                      1e-5, 0, stream.cuda_stream))
    torch.cuda.synchronize()
    failures = []

    def run(args):
        failures.extend(status for status in (lib.kda_residual_norm_bwd(*args) for _ in range(10000)) if status)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, (len(failures), failures[0])


@pytest.mark.parametrize("dtype,bar", [(FP, 4e-6), (BF, 2 ** -7)])
@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
def test_gradient_of_a_closing_gate(activation, dtype, bar):
    """The sigmoid's derivative falls to 1e-7 at z = +-16: every value of dgate keeps its own relative
    accuracy. fp32: the exponential's and the quotient's roundings, those of the row's sum of 64
    squares and a dozen products, 2^-24 each: 4e-6. bf16: an ulp, against the rounded definition."""
    n, d = 66, 64
    x, dy = rand(1, n, 2, d, dtype=dtype), rand(2, n, 2, d, dtype=dtype)
    z = torch.linspace(-16, 16, n * 2 * d, device=DEV).view(n, 2, d).to(dtype)
    w = 1 + 0.2 * rand(3, d)
    if activation == "silu":
        z = z[z[:, 0, 0] > -1]  # further down its derivative crosses zero
        x, dy = x[:len(z)], dy[:len(z)]
    got = kda.gated_norm_bwd(dy, x, z, w, eps=EPS, activation=activation)[1]
    want = block.gated_norm_grads(block.f64(dy), block.f64(x), block.f64(z), block.f64(w), EPS, activation)[1]
    if dtype == BF:
        want = want.to(BF).double()
    off = (got.double().cpu() - want).abs() / want.abs().clamp_min(1e-30)
    assert float(off.max()) <= bar, f"{float(off.max()):.2e}"


@pytest.mark.parametrize("dtype", [FP, BF])
def test_a_nan_gate_stays_in_its_row(dtype):
    x, z, dy = (rand(i, 5, 2, 64, dtype=dtype) for i in range(3))
    w = 1 + 0.2 * rand(5, 64)
    clean = kda.gated_norm_bwd(dy, x, z, w, eps=EPS)
    z[2, 1, 7] = float("nan")
    dx, dz, dw = kda.gated_norm_bwd(dy, x, z, w, eps=EPS)
    assert bool(torch.isnan(dx[2, 1]).all()) and bool(torch.isnan(dz[2, 1, 7])) and bool(torch.isnan(dw[7]))
    keep = torch.ones(5, 2, dtype=torch.bool, device=DEV)
    keep[2, 1] = False
    assert torch.equal(dx[keep], clean[0][keep]) and torch.equal(dz[keep], clean[1][keep])
