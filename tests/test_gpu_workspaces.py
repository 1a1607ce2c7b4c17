"""Calls whose inputs are refused on the device, with workspaces that hold anything."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vfa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fill", [0xff, 0x80, 0x7f])
def test_refused_lengths_with_any_workspace(vfa, d, fill):
    """The prefill takes items by a counter of the workspace: refused lengths leave no items, so
    the counter must not be what the workspace held (negative numbers read ahead of the list)."""
    q = torch.ones(128, 2, d, device="cuda", dtype=torch.bfloat16)
    cq = torch.tensor([0, 100, 90], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 64, 128], dtype=torch.int32, device="cuda")
    for window in (-1, 9):
        out = torch.full_like(q, 7.0)
        ws = vfa.alloc_workspace(2, 128, 128, 2, d).fill_(fill)
        vfa.varlen_fwd(q, q, q, cq, ck, 128, 0.1, 1, out=out, workspace=ws, window_left=window)
        assert vfa.read_status(ws) == vfa.VFA_ERR_BAD_SEQLENS
        assert (out == 7.0).all()
