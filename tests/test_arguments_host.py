"""Arguments of the packed forward and backward that are refused before any work, without a GPU:
the tensors here have shapes, types and a device, but no memory."""
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from variable_length_flashattention_gb300 import vfa

T, TK, H, HKV, D, B = 6, 8, 4, 2, 64, 2
STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class Never:
        def __getattr__(self, name):
            def call(*args):
                raise AssertionError(f"{name}: a call that should have been refused reached the library")
            return call

    monkeypatch.setattr(vfa, "_lib", Never())
    monkeypatch.setattr(vfa, "lib", Never)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")             # addresses of tensors without memory
        yield


def _t(*shape, dtype=torch.bfloat16, device="cuda:0"):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


def _inputs(fp8=False):
    x = torch.uint8 if fp8 else torch.bfloat16
    cu = [_t(B + 1, dtype=torch.int32) for _ in range(2)]
    return [_t(T, H, D, dtype=x), _t(TK, HKV, D, dtype=x), _t(TK, HKV, D)], cu


def _fwd(qkv, cu, out=None, lse=None, workspace=None, most=T, causal=1, **kw):
    return vfa.varlen_fwd(*qkv, *cu, most, 0.1, causal, _t(T, H, D) if out is None else out,
                          _t(T, H, dtype=torch.float32) if lse is None else lse,
                          _t(1 << 16, dtype=torch.uint8) if workspace is None else workspace, STREAM, **kw)


def _fp8(qkv, cu, out=None, lse=None, workspace=None, most=T, causal=1, **kw):
    return vfa.varlen_fwd_fp8(*qkv, *cu, most, 0.1, 1.0, 1.0, causal, _t(T, H, D) if out is None else out,
                              _t(T, H, dtype=torch.float32) if lse is None else lse,
                              _t(1 << 16, dtype=torch.uint8) if workspace is None else workspace, STREAM, **kw)


def _noalloc(qkv, cu, out=None, lse=None, workspace=None, most=T, causal=1, **kw):
    return vfa.varlen_fwd_noalloc(*qkv, *cu, most, 0.1, causal, _t(T, H, D) if out is None else out,
                                  _t(T, H, dtype=torch.float32) if lse is None else lse, workspace, STREAM, **kw)


def _bwd(qkv, cu, out=None, lse=None, workspace=None, causal=1, dout=None, dq=None, dk=None, dv=None, **kw):
    give = lambda t, *shape: _t(*shape) if t is None else t
    return vfa.varlen_bwd(*qkv, give(out, T, H, D), give(dout, T, H, D),
                          _t(T, H, dtype=torch.float32) if lse is None else lse, *cu, 0.1, causal,
                          dq=give(dq, T, H, D), dk=give(dk, TK, HKV, D), dv=give(dv, TK, HKV, D),
                          workspace=_t(1 << 16, dtype=torch.uint8) if workspace is None else workspace,
                          stream=STREAM, **kw)


CALLS = [(_fwd, False), (_fp8, True), (_noalloc, False), (_bwd, False)]


@pytest.mark.parametrize("call,fp8", CALLS)
def test_tensors_that_do_not_fit_each_other(call, fp8):
    qkv, cu = _inputs(fp8)
    x = qkv[0].dtype
    f32, i32 = torch.float32, torch.int32
    for word, change in (
            ("out", dict(out=_t(T - 1, H, D))), ("out", dict(out=_t(T, D, H))),
            ("out", dict(out=_t(T, H, D, dtype=f32))),
            ("lse", dict(lse=_t(T, H - 1, dtype=f32))), ("lse", dict(lse=_t(T * H, dtype=f32))),
            ("lse", dict(lse=_t(T, H))), ("CUDA", dict(lse=_t(T, H, dtype=f32, device="cpu"))),
            ("CUDA", dict(out=_t(T, H, D, device="cpu")))):
        with pytest.raises(ValueError, match=word):
            call(qkv, cu, **change)
    for i, t in ((0, _t(T, H, D + 8, dtype=x)), (0, _t(T, 3, D, dtype=x)), (0, _t(T * H, D, dtype=x)),
                 (1, _t(TK, HKV, 2 * D, dtype=x)), (2, _t(TK - 1, HKV, D)), (1, _t(TK, 0, D, dtype=x))):
        bad = list(qkv)
        bad[i] = t
        if t.shape[1] == 0:
            bad[2] = _t(TK, 0, D)
        with pytest.raises(ValueError, match="heads"):
            call(bad, cu)
    for i in range(3):
        bad = list(qkv)
        bad[i] = _t(*qkv[i].shape, dtype=qkv[i].dtype, device="cpu")
        with pytest.raises(ValueError, match="CUDA"):
            call(bad, cu)
    for bad in ([cu[0], _t(B, dtype=i32)], [_t(B + 2, dtype=i32), cu[1]]):
        with pytest.raises(ValueError, match="same length"):
            call(qkv, bad)


@pytest.mark.parametrize("call,fp8", [c for c in CALLS if c[0] is not _noalloc])
def test_workspaces_elsewhere(call, fp8):
    qkv, cu = _inputs(fp8)
    for word, ws in (("CUDA", _t(1 << 16, dtype=torch.uint8, device="cpu")),
                     ("contiguous", _t(2, dtype=torch.uint8)[:1].expand(1 << 16))):
        with pytest.raises(ValueError, match=word):
            call(qkv, cu, workspace=ws)


@pytest.mark.parametrize("call,fp8", CALLS)
def test_tensors_of_another_device_than_the_current_one(monkeypatch, call, fp8):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        call(*_inputs(fp8))


def test_gradients_that_do_not_fit():
    qkv, cu = _inputs()
    for word, change in (("dq", dict(dq=_t(T - 1, H, D))), ("dk", dict(dk=_t(T, HKV, D))),
                         ("dk", dict(dk=_t(TK, H, D))), ("dv", dict(dv=_t(TK, HKV, D, dtype=torch.float16))),
                         ("dv", dict(dv=_t(TK, HKV))), ("dout", dict(dout=_t(T + 1, H, D)))):
        with pytest.raises(ValueError, match=word):
            _bwd(qkv, cu, **change)


@pytest.mark.parametrize("call,fp8", CALLS)
def test_numbers_past_32_bits(call, fp8):
    """A window larger than anything is refused, not cut to the 0 that its low bits are."""
    qkv, cu = _inputs(fp8)
    changes = [dict(window_left=1 << 32), dict(window_left=(1 << 32) - 1), dict(window_left=-(1 << 32)),
               dict(causal=(1 << 32) + 1)]
    changes += [dict(most=(1 << 32) + T)] if call is not _bwd else []
    changes += [dict(sink_tokens=1 << 32)] if call in (_fwd, _bwd) else []
    for change in changes:
        with pytest.raises(ValueError, match="32 bits"):
            call(qkv, cu, **change)


@pytest.mark.parametrize("call,fp8", CALLS)
def test_sizes_past_32_bits(call, fp8):
    qkv, cu = _inputs(fp8)
    qkv[0] = _t((1 << 32) + T, H, D, dtype=qkv[0].dtype)
    with pytest.raises(ValueError, match="32 bits"):
        call(qkv, cu)


@pytest.mark.parametrize("call,fp8", CALLS)
def test_tensors_of_a_machine_without_a_gpu(monkeypatch, call, fp8):
    def none():
        raise RuntimeError("no driver")

    monkeypatch.setattr(torch._C, "_cuda_getDevice", none)
    monkeypatch.setattr(torch.cuda, "current_device", none)
    qkv, cu = _inputs(fp8)
    qkv[0] = _t(T, H, D, dtype=qkv[0].dtype, device="cpu")
    with pytest.raises(ValueError, match="q8? must be a CUDA tensor"):
        call(qkv, cu)
