"""The fp64 definitions of linear attention with one decay per head and of the norm of queries and
keys with the position rotation in ``oracle.block`` (CPU): closed forms, and every gradient against
central differences (step 1e-5 in fp64, bar 1e-6 of the gradient's scale)."""
import pytest
import torch

from oracle import block
from tests.test_block_oracle import check_gradients, inputs

torch.set_num_threads(4)
F64 = torch.float64


def linear(lengths, hk, hv, dk, dv, h0=True, per_head=False):
    q, k, v, g, _, h, cu = inputs(lengths, hk, hv, dk, dv, h0=h0)
    return q, k, v, (g[0] if per_head else g), h, cu


@pytest.mark.parametrize("per_head", [False, True])
def test_output_is_the_decayed_sum_over_the_past(per_head):
    q, k, v, g, h0, cu = linear([4, 3], 1, 2, 3, 5, per_head=per_head)
    out, end = block.dla(q, k, v, g, h0, cu, scale=0.7)
    rates = g.expand(7, 2)
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        for h in range(2):
            for t in range(a, b):
                want = rates[a:t + 1, h].sum().exp() * (h0[n, h].T @ q[t, 0])
                for j in range(a, t + 1):
                    want = want + rates[j + 1:t + 1, h].sum().exp() * (q[t, 0] @ k[j, 0]) * v[j, h]
                assert torch.allclose(out[t, h], 0.7 * want, atol=1e-13)
            want = rates[a:b, h].sum().exp() * h0[n, h]
            for j in range(a, b):
                want = want + rates[j + 1:b, h].sum().exp() * torch.outer(k[j, 0], v[j, h])
            assert torch.allclose(end[n, h], want, atol=1e-13)


def test_infinite_decay_starts_anew():
    q, k, v, g, h0, cu = linear([6], 1, 1, 3, 4)
    g[3] = -float("inf")
    out, end = block.dla(q, k, v, g, h0, cu)
    tail, tail_end = block.dla(q[3:], k[3:], v[3:], g[3:], None, [0, 3])
    assert torch.equal(out[3:], tail) and torch.equal(end, tail_end)


@pytest.mark.parametrize("per_head", [False, True])
def test_gradients_are_differences(per_head):
    q, k, v, g, h0, cu = linear([5, 0, 3], 2, 4, 3, 4, per_head=per_head)
    gen = torch.Generator().manual_seed(1)
    dout = torch.randn(v.shape, generator=gen, dtype=F64)
    dhf = torch.randn(h0.shape, generator=gen, dtype=F64)

    def loss(*xs):
        out, end = block.dla(*xs, cu)
        return float((out * dout).sum() + (end * dhf).sum())

    check_gradients(loss, (q, k, v, g, h0), block.dla_grads(q, k, v, g, h0, cu, dout, dhf))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_relative_positions(interleaved):
    gen = torch.Generator().manual_seed(2)
    q, k = torch.randn(2, 1, 1, 8, generator=gen, dtype=F64)
    w, f = torch.ones(8, dtype=F64), torch.tensor([1.0, 0.3, 0.01, 2e-3], dtype=F64)

    def dot(m, n):
        a, b = (block.head_norm_rope(x, w, torch.tensor([p]), f, 1e-6, interleaved) for x, p in ((q, m), (k, n)))
        return float((a * b).sum())

    assert abs(dot(5, 2) - dot(1003, 1000)) < 1e-12
    assert abs(dot(7, 7) - dot(0, 0)) < 1e-12 and abs(dot(5, 2) - dot(5, 3)) > 1e-6


def test_pairs_of_both_orders_are_the_same_turns():
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn(3, 2, 10, generator=gen, dtype=F64), torch.randn(10, generator=gen, dtype=F64)
    f, pos = torch.tensor([1.0, 0.1, 0.01], dtype=F64), torch.tensor([0, -4, 9])
    order = torch.tensor([0, 2, 4, 1, 3, 5, 6, 7, 8, 9])  # halves from pairs
    a = block.head_norm_rope(x, w, pos, f, 1e-6, True)
    b = block.head_norm_rope(x[..., order], w[order], pos, f, 1e-6, False)
    assert torch.allclose(a[..., order], b, atol=1e-14)
    c = torch.complex(*(block.head_norm_rope(x, w, pos, None, 1e-6, True)[..., i:6:2].contiguous() for i in (0, 1)))
    c = c * torch.polar(torch.ones(3, 1, 3, dtype=F64), (pos[:, None] * f)[:, None])
    assert torch.allclose(a[..., 0:6:2], c.real, atol=1e-14) and torch.allclose(a[..., 1:6:2], c.imag, atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation_gradients_are_differences(interleaved):
    gen = torch.Generator().manual_seed(4)
    x, dy = torch.randn(2, 3, 2, 10, generator=gen, dtype=F64)
    w, f, pos = torch.randn(10, generator=gen, dtype=F64), torch.tensor([1.0, 0.1], dtype=F64), torch.tensor([2, 0, 70])
    check_gradients(lambda *xs: float((block.head_norm_rope(*xs, pos, f, 1e-6, interleaved) * dy).sum()), (x, w),
                    block.head_norm_rope_grads(dy, x, w, pos, f, 1e-6, interleaved))
