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


def test_workspaces_of_a_call_belong_to_its_stream(vfa, monkeypatch):
    """A call on a stream of its own makes its workspace there: the block is handed out again behind
    the kernels that still use it, not to what runs beside them."""
    made = []
    for name in ("alloc_workspace", "alloc_bwd_workspace"):
        def alloc(*args, plain=getattr(vfa, name), **kw):
            made.append(torch.cuda.current_stream())
            return plain(*args, **kw)
        monkeypatch.setattr(vfa, name, alloc)
    q = torch.ones(70, 2, 64, device="cuda", dtype=torch.bfloat16)
    q8 = torch.full((70, 2, 64), 0x30, device="cuda", dtype=torch.uint8)
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, None):
        want = [stream or torch.cuda.current_stream()]
        out, lse = vfa.varlen_fwd(q, q, q, cu, cu, 70, 0.1, 1, stream=stream)
        vfa.varlen_fwd_fp8(q8, q8, q, cu, cu, 70, 0.1, 1.0, 1.0, 1, stream=stream)
        vfa.varlen_bwd(q, q, q, out, q, lse, cu, cu, 0.1, 1, stream=stream)
        vfa.varlen_bwd(q, q, q, out, q, lse, cu, cu, 0.1, 1, window_left=9, sink_tokens=2, stream=stream)
        assert made == 4 * want
        made.clear()
    torch.cuda.synchronize()
