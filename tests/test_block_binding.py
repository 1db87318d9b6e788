"""Checks of the block operators' Python binding on the host: the calls run up to their checks
with CPU tensors (device index -1) and no library, so whatever passes them fails the test."""
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from chunked_linear_attention_kda_gb300 import block


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(block, "_start", lambda t, what: (None, 0, -1))


def inputs(n, m, hk=1, hv=2, d=8):
    """q, k, g and beta of n tokens, v of m."""
    return (torch.zeros(n, hk, d), torch.zeros(n, hk, d), torch.zeros(m, hv, d), torch.zeros(n, hv),
            torch.zeros(n, hv))


@pytest.mark.parametrize("m", [0, 5, 11])
@pytest.mark.parametrize("strided", [False, True])
def test_values_of_another_length_are_refused(on_host, m, strided):
    q, k, v, g, beta = inputs(8, m)
    if strided:
        q = torch.zeros(8, 1, 16)[..., :8]
    state = torch.zeros(11, 2, 8, 8)
    for call in (lambda: kda.gdr_chunk_fwd(q, k, v, g, beta, None, torch.tensor([0, 8], dtype=torch.int32)),
                 lambda: kda.gdr_chunk_bwd(q, k, v, g, beta, None, torch.tensor([0, 8], dtype=torch.int32),
                                           torch.zeros(8, 2, 8)),
                 lambda: kda.gdr_step(q, k, v, g, beta, state),
                 lambda: kda.gdr_step(q, k, v, g, beta, state, out=torch.zeros_like(v))):
        with pytest.raises(ValueError, match="v must be"):
            call()
