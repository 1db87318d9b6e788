"""Checks of the block operators' Python binding on the host: the calls run up to their checks
with CPU tensors (device index -1) and no library, so whatever passes them fails the test."""
import os
import subprocess
import sys

import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from chunked_linear_attention_kda_gb300 import block


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(block, "_start", lambda t, what: (None, 0, -1))
    monkeypatch.setattr(block, "_empty", lambda shape, dtype, dev: torch.empty(shape, dtype=dtype))


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


def calls_with_a_workspace(workspace, dev="cpu"):
    q, k, v, g, beta = (t.to(dev) for t in inputs(8, 8))
    cu = torch.tensor([0, 8], dtype=torch.int32, device=dev)
    x, w = torch.ones(4, 16, device=dev), torch.ones(16, device=dev)
    z = torch.ones(4, 2, 16, device=dev)
    return (lambda: kda.gdr_chunk_fwd(q, k, v, g, beta, None, cu, workspace=workspace),
            lambda: kda.gdr_chunk_bwd(q, k, v, g, beta, None, cu, torch.zeros_like(v), workspace=workspace),
            lambda: kda.residual_norm_bwd(x, x, w, workspace=workspace),
            lambda: kda.gated_norm_bwd(z, z, z, w, workspace=workspace))


def test_a_workspace_with_gaps_is_refused(on_host):
    # expanded, it spans a byte of the 16 MB that it counts; cut out, more than it counts
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 20)[::2]):
        for call in calls_with_a_workspace(bad):
            with pytest.raises(ValueError, match="workspace"):
                call()


@pytest.mark.gpu
def test_a_workspace_on_another_device_is_refused():
    for call in calls_with_a_workspace(torch.zeros(1 << 24, dtype=torch.uint8), "cuda"):
        with pytest.raises(ValueError, match="workspace"):
            call()
    for call in calls_with_a_workspace(torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"), "cuda"):
        call()


class OnDevice:
    """What _start reads of a CUDA tensor."""
    is_cuda, dtype = True, torch.float32

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_a_device_that_is_not_current_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(block, "_current", lambda: 0, raising=False)
    monkeypatch.setattr(block, "_stream", lambda dev: 7)
    monkeypatch.setattr(kda, "_lib", object())
    assert block._start(OnDevice(0), "gdr_step")[1:] == (7, 0)
    with pytest.raises(ValueError, match="current device"):
        block._start(OnDevice(1), "gdr_step")


def test_the_package_imports_without_torch():
    """Its calls need torch; building the library and reading its symbols do not."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import chunked_linear_attention_kda_gb300 as kda\n"
            "from chunked_linear_attention_kda_gb300 import build\n"
            "assert kda.library_path() and 'gdr_step' in dir(kda) and not hasattr(kda, 'nothing')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], cwd=root, check=True)


def test_every_public_name_is_there():
    for name in kda.__all__:
        assert getattr(kda, name) is not None
    assert kda.block is block and kda.gdr_step is block.gdr_step
