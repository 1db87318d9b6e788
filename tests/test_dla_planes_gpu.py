"""What linear attention of bf16 inputs keeps of an operand that is not one: values times their
tokens' decays, seen by themselves. A key of a single 1 puts them into a row of the state."""
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def tokens(n, heads, dk, dv, seed):
    gen = torch.Generator().manual_seed(seed)
    one = torch.zeros(n, heads, dk)
    one[0, :, 0] = 1.0
    v = torch.randn(n, heads, dv, generator=gen)
    g = -2.0 * torch.rand(n, heads, generator=gen)
    return one.to(DEV, BF), v.to(DEV, BF), g.to(DEV)


def largest(got, want):
    return float(((got.double() - want) / want).abs().max())


@pytest.mark.parametrize("dv", [128, 64, 40])
def test_values_of_the_forward_in_two_parts(dv):
    """A decay's first two bf16 parts leave 2^-17 of it. The product with the first, in [2^e, 2^(e+1)), is off by
    2^(e-8) at most when it is rounded, and that with the second is below 2^(e-7): their sum, below 2^(e-6), is
    off by 2^(e-15). The decay itself is the product of two exponentials, off by 2^-22 each, and is rounded:
    2^-15 + 2^-17 + 2^-20 in all, and a little for second orders: 2^-15 + 2^-16."""
    k, v, g = tokens(3, 64, 128, dv, seed=dv)
    v[1:] = 0.0
    end = kda.dla_chunk_fwd(k, k, v, g)[1]
    want = (g[1] + g[2].double()).exp()[:, None] * v[0].double()
    assert largest(end[0, :, 0], want) <= 2.0 ** -15 + 2.0 ** -16


@pytest.mark.parametrize("dv", [128, 64, 40])
def test_values_of_the_walks_in_three_parts(dv):
    """Three parts leave 2^-26. The decay is the product of two exponentials, off by 2^-22 each; its roundings with
    the scale are 2^-24 each, and the sum in tensor memory drops what is below its last place, 2^-23: 2^-20."""
    q, do, g = tokens(1, 64, 128, dv, seed=dv + 1)
    k = torch.zeros_like(q)
    dh0 = kda.dla_chunk_bwd(q, k, do, g, None, None, do, scale=0.7)[4]
    want = 0.7 * g[0].double().exp()[:, None] * do[0].double()
    assert largest(dh0[0, :, 0], want) <= 2.0 ** -20

