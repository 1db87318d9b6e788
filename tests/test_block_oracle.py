"""The fp64 definitions in ``oracle.block`` (CPU): the recurrence against unrolled transition
matrices and closed forms, every gradient against central differences.

Differences use a step of 1e-5 in fp64: truncation ~1e-10, cancellation ~1e-11 of the values,
so 1e-6 of the gradient's scale is a safe bar."""
import pytest
import torch

from oracle import block

torch.set_num_threads(4)


def inputs(lengths, hk, hv, dk, dv, seed=0, h0=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    n = sum(lengths)
    k = r(n, hk, dk)
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    return (r(n, hk, dk) / dk ** 0.5, k / k.norm(dim=-1, keepdim=True), r(n, hv, dv), -r(n, hv).abs(),
            torch.sigmoid(r(n, hv)), 0.5 * r(len(lengths), hv, dk, dv) if h0 else None, cu)


def test_recurrence_is_the_product_of_transition_matrices():
    q, k, v, g, beta, h0, cu = inputs([5], 1, 2, 3, 4)
    out, end = block.gdr(q, k, v, g, beta, h0, cu)
    for h in range(2):
        S = h0[0, h]
        for t in range(5):
            kt = k[t, 0][:, None]
            S = (torch.eye(3, dtype=torch.float64) - beta[t, h] * kt @ kt.T) @ (g[t, h].exp() * S) \
                + beta[t, h] * kt @ v[t, h][None]
            assert torch.allclose(out[t, h], 3 ** -0.5 * (S.T @ q[t, 0]), atol=1e-13)
        assert torch.allclose(end[0, h], S, atol=1e-13)


def test_infinite_decay_forgets_everything():
    q, k, v, g, beta, h0, cu = inputs([6], 1, 1, 3, 4)
    g[3] = -float("inf")
    out, end = block.gdr(q, k, v, g, beta, h0, cu)
    tail, tail_end = block.gdr(q[3:], k[3:], v[3:], g[3:], beta[3:], None, [0, 3])
    assert torch.equal(out[3:], tail) and torch.equal(end, tail_end)


def differences(f, xs, i, direction, h=1e-5):
    hi, lo = list(xs), list(xs)
    hi[i] = xs[i] + h * direction
    lo[i] = xs[i] - h * direction
    return (f(*hi) - f(*lo)) / (2 * h)


def check_gradients(f, xs, grads, seed=0):
    gen = torch.Generator().manual_seed(seed)
    for i, (x, g) in enumerate(zip(xs, grads)):
        if x is None or g is None or x.numel() == 0:
            continue
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        got, want = float((g * d).sum()), float(differences(f, xs, i, d))
        assert abs(got - want) <= 1e-6 * max(1.0, float(g.norm() * d.norm())), i


@pytest.mark.parametrize("lengths,hk,hv", [([7], 1, 1), ([3, 0, 4], 2, 4)])
def test_recurrence_gradients_are_differences(lengths, hk, hv):
    q, k, v, g, beta, h0, cu = inputs(lengths, hk, hv, 4, 3)
    gen = torch.Generator().manual_seed(9)
    dout = torch.randn(v.shape, generator=gen, dtype=torch.float64)
    dhf = torch.randn(h0.shape, generator=gen, dtype=torch.float64)

    def loss(*xs):
        out, end = block.gdr(*xs, cu)
        return (out * dout).sum() + (end * dhf).sum()

    check_gradients(loss, (q, k, v, g, beta, h0), block.gdr_grads(q, k, v, g, beta, h0, cu, dout, dhf))


@pytest.mark.parametrize("scaled", [True, False])
def test_residual_norm_gradients_are_differences(scaled):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, res, dy, dr = r(4, 6), r(6), r(4, 6), r(4, 6), r(4, 6)
    sc = r(6) if scaled else None

    def loss(x, res, w, sc):
        y, out = block.residual_norm(x, w, res, sc, 1e-3)
        return (y * dy).sum() + (out * dr).sum()

    _, rr = block.residual_norm(x, w, res, sc, 1e-3)
    check_gradients(loss, (x, res, w, sc), block.residual_norm_grads(dy, rr, w, dr, x, sc, 1e-3))


@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
def test_gated_norm_gradients_are_differences(activation):
    gen = torch.Generator().manual_seed(4)
    x, z, dy = (torch.randn(3, 2, 5, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.randn(5, generator=gen, dtype=torch.float64)
    check_gradients(lambda x, z, w: (block.gated_norm(x, z, w, 1e-3, activation) * dy).sum(), (x, z, w),
                    block.gated_norm_grads(dy, x, z, w, 1e-3, activation))
