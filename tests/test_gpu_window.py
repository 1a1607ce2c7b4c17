"""GPU parity of attention with a window and sinks, forward and backward, with the 64-bit
definitions.

Forward, per element (u = 2^-23 for a product of bf16 values added up in the tensor core's
fp32, eps / 2 of bf16 = 2^-8):
  scores: a chain of at most D additions, the scale and the subtraction of the reference: the
    exponent is off by at most dx = (D + 16) u max_j sum|q k| scale;
  p: e^dx - 1, 2^-20 for ex2, and half a bf16 step, 2^-8; l the same without bf16;
  out: (2 (e^dx - 1) + 2^-8 + n u + 2^-19) sum p|v| / l, and its own rounding 2^-8 |out|;
  lse: dx + n u + 2^-19 + 2^-22 |lse|.
Backward: the first-order bound of tests/bwd_error_model.py under this mask.
"""
import numpy as np
import pytest
import torch

import bwd_error_model
import oracle.bounded as O
from helpers import FLT_MAX
from variable_length_flashattention_gb300 import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module")
def vfa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


def _case(lq, lk, hq, hkv, d, seed, scale=None):
    c = W.make_varlen("window", lq, lk, hq, d, True, 1.0, seed, scale)
    gen = torch.Generator().manual_seed(seed + 1)
    c.k, c.v = (W.bf16_normal((c.total_k, hkv, d), 1.0, gen) for _ in range(2))
    return c


def _nan_like(t):
    return torch.full_like(t.view(torch.int16), 0x7FC0).view(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _dev(c):
    return [t.cuda() for t in (c.q, c.k, c.v, torch.from_numpy(c.cu_seqlens_q),
                               torch.from_numpy(c.cu_seqlens_k))]


def _forward(vfa, c, causal, window, sinks):
    q, k, v, cq, ck = _dev(c)
    out = _nan_like(q)
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    ws = vfa.alloc_workspace(c.batch, c.total_q, c.total_k, c.num_heads, c.head_dim)
    vfa.varlen_fwd(q, k, v, cq, ck, c.max_seqlen_q, c.softmax_scale, causal, out=out, lse=lse,
                   workspace=ws, window_left=window, sink_tokens=sinks)
    assert vfa.read_status(ws) == 0
    return out, lse


def _check_forward(c, causal, window, sinks, out, lse):
    ref, rlse, dot, absv = O.varlen_fwd(_f64(c.q), _f64(c.k), _f64(c.v), c.cu_seqlens_q,
                                        c.cu_seqlens_k, c.softmax_scale, causal, window, sinks)
    n = max(c.lengths_k + [1])
    dx = (c.head_dim + 16) * U * dot
    got, glse = _f64(out), _f64(lse)
    assert np.all(np.isfinite(got)) and np.all(np.isfinite(glse))
    bound = (2 * np.expm1(dx) + 2.0 ** -8 + n * U + 2.0 ** -19)[..., None] * absv + \
        2.0 ** -8 * np.abs(ref) + 1e-30
    assert np.all(np.abs(got - ref) <= bound), (np.abs(got - ref) / bound).max()
    empty = rlse == -FLT_MAX
    assert np.all(glse[empty] == np.float32(-FLT_MAX)) and np.all(got[empty] == 0)
    lbound = dx + n * U + 2.0 ** -19 + 2.0 ** -22 * np.abs(rlse)
    assert np.all((np.abs(glse - rlse) <= lbound)[~empty])


# lengths of none and one, tiles that end inside, sinks that reach into the window, past it
# and over tile borders; queries past the keys (causal 1) and before them (causal 2)
LENGTHS = [([1, 0, 5, 129], [1, 3, 0, 129]), ([300], [300]), ([257, 64], [511, 64]),
           ([400, 130], [90, 17]), ([40, 200], [700, 33])]
MASKS = [(0, 1), (1, 4), (31, 64), (63, 65), (100, 128), (128, 129), (200, 300), (5, 1 << 30),
         (2 ** 31 - 1, 3)]


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 2, 2), (256, 3, 1)])
@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("causal", [1, 2])
def test_forward(vfa, d, hq, hkv, window, sinks, causal):
    for i, (lq, lk) in enumerate(LENGTHS):
        c = _case(lq, lk, hq, hkv, d, seed=17 * i + d)
        _check_forward(c, causal, window, sinks, *_forward(vfa, c, causal, window, sinks))


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 2, 2), (256, 3, 1)])
@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("causal", [1, 2])
def test_backward(vfa, monkeypatch, d, hq, hkv, window, sinks, causal):
    monkeypatch.setattr(bwd_error_model, "_visible",
                        lambda a, b, cz, w: torch.from_numpy(O.visible(a, b, cz, w, sinks)))
    for i, (lq, lk) in enumerate(LENGTHS):
        c = _case(lq, lk, hq, hkv, d, seed=31 * i + d)
        _check_backward(vfa, c, causal, window, sinks)


def _backward(vfa, c, causal, window, sinks, dout):
    out, lse = _forward(vfa, c, causal, window, sinks)
    q, k, v, cq, ck = _dev(c)
    dq, dk, dv = _nan_like(q), _nan_like(k), _nan_like(v)
    *_, ws = vfa.varlen_bwd(q, k, v, out, dout.cuda(), lse, cq, ck, c.softmax_scale, causal,
                            window_left=window, dq=dq, dk=dk, dv=dv, sink_tokens=sinks)
    assert vfa.read_status(ws) == 0
    return dq, dk, dv


def _check_backward(vfa, c, causal, window, sinks):
    dout = W.upstream_grad(c, 3)
    got = _backward(vfa, c, causal, window, sinks, dout)
    ref = O.varlen_bwd(_f64(c.q), _f64(c.k), _f64(c.v), _f64(dout), c.cu_seqlens_q,
                       c.cu_seqlens_k, c.softmax_scale, causal, window, sinks)
    mags = bwd_error_model.magnitudes(c, dout, causal, window, c.k.shape[1])
    for name, g, r, m in zip(("dq", "dk", "dv"), got, ref, mags):
        bwd_error_model.check_grad(_f64(g), r, m, name)


def test_backward_cuts_long_sink_tiles(vfa, monkeypatch):
    """Enough queries for the sinks' tiles to be cut into chunks, in sequences that differ."""
    window, sinks = 40, 130
    monkeypatch.setattr(bwd_error_model, "_visible",
                        lambda a, b, cz, w: torch.from_numpy(O.visible(a, b, cz, w, sinks)))
    for d, hq, hkv in ((64, 8, 1), (128, 4, 1), (256, 2, 1)):
        c = _case([900, 3, 1500, 0, 700], [900, 3, 1500, 5, 700], hq, hkv, d, seed=d)
        _check_backward(vfa, c, 1, window, sinks)


def test_backward_is_the_same_every_time(vfa):
    c = _case([2000, 100], [2000, 100], 8, 2, 128, seed=5)
    dout = W.upstream_grad(c, 1)
    a, b = (_backward(vfa, c, 1, 64, 4, dout) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_without_sinks_or_window_nothing_changes(vfa, d):
    """No sinks, or no window: the bits of the plain forward and backward."""
    c = _case([300, 77], [300, 77], 4, 2, d, seed=d)
    q, k, v, cq, ck = _dev(c)
    dout = W.upstream_grad(c, 1).cuda()

    def run(**kw):
        out, lse = vfa.varlen_fwd(q, k, v, cq, ck, 300, c.softmax_scale, 1, **kw)
        return (out, lse, *vfa.varlen_bwd(q, k, v, out, dout, lse, cq, ck, c.softmax_scale, 1, **kw)[:3])

    for a, b in ((run(), run(sink_tokens=5)), (run(window_left=20), run(window_left=20, sink_tokens=0))):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_sinks_over_everything_are_a_causal_mask(vfa):
    c = _case([700, 129], [700, 129], 4, 4, 128, seed=9)
    out, lse = _forward(vfa, c, 1, 3, 700)
    _check_forward(c, 1, -1, 0, out, lse)


def test_scale_of_zero_and_large_logits(vfa):
    c = _case([200], [200], 2, 1, 64, seed=11, scale=0.0)
    _check_forward(c, 1, 20, 4, *_forward(vfa, c, 1, 20, 4))
    c = _case([200], [200], 2, 1, 128, seed=12, scale=1.0)
    _check_forward(c, 1, 20, 4, *_forward(vfa, c, 1, 20, 4))


def test_bad_sequence_lengths_write_nothing(vfa):
    c = _case([64, 64], [64, 64], 2, 2, 64, seed=1)
    q, k, v, _, ck = _dev(c)
    cq = torch.tensor([0, 100, 90], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = vfa.alloc_workspace(2, 128, 128, 2, 64)
    vfa.varlen_fwd(q, k, v, cq, ck, 128, 0.1, 1, out=out, workspace=ws, window_left=9, sink_tokens=2)
    assert vfa.read_status(ws) == vfa.VFA_ERR_BAD_SEQLENS and (out == 7.0).all()
    bws = vfa.alloc_bwd_workspace(2, 128, 2, 64, sink_tokens=2)
    dq = torch.full_like(q, 7.0)
    lse = torch.zeros(128, 2, device="cuda")
    _, dk, dv, _ = vfa.varlen_bwd(q, k, v, out, out, lse, cq, ck, 0.1, 1, window_left=9, dq=dq,
                                  dk=torch.full_like(k, 7.0), dv=torch.full_like(k, 7.0),
                                  workspace=bws, sink_tokens=2)
    assert vfa.read_status(bws) == vfa.VFA_ERR_BAD_SEQLENS
    assert all((t == 7.0).all() for t in (dq, dk, dv))


def test_training_step_in_a_graph(vfa):
    c = _case([513, 40], [513, 40], 4, 2, 128, seed=21)
    q, k, v, cq, ck = _dev(c)
    dout = W.upstream_grad(c, 2).cuda()
    ws = vfa.alloc_workspace(2, c.total_q, c.total_k, 4, 128)
    bws = vfa.alloc_bwd_workspace(2, c.total_q, 4, 128, sink_tokens=7)

    def step():
        out, lse = vfa.varlen_fwd(q, k, v, cq, ck, 513, c.softmax_scale, 1, workspace=ws,
                                  window_left=100, sink_tokens=7)
        return (out, lse, *vfa.varlen_bwd(q, k, v, out, dout, lse, cq, ck, c.softmax_scale, 1,
                                          window_left=100, workspace=bws, sink_tokens=7)[:3])

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_results_at_any_allowed_address(vfa, d):
    """An output at a multiple of 16 bytes that is none of 32: the same bits, and nothing around it."""
    c = _case([200, 0, 129], [200, 5, 129], 4, 2, d, 21)
    q, k, v, cq, ck = _dev(c)
    want, lse = vfa.varlen_fwd(q, k, v, cq, ck, c.max_seqlen_q, c.softmax_scale, 1, window_left=40, sink_tokens=3)
    flat = torch.full((q.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:-8].view(q.shape)
    assert out.data_ptr() % 32 == 16
    _, lse2 = vfa.varlen_fwd(q, k, v, cq, ck, c.max_seqlen_q, c.softmax_scale, 1, window_left=40, sink_tokens=3,
                             out=out)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    assert (flat[:8] == 7.0).all() and (flat[-8:] == 7.0).all()


@pytest.mark.parametrize("sinks", [0, 4])
def test_backward_calls_in_a_row_share_a_workspace(vfa, sinks):
    """Each call's first kernels start behind all of the call before, which reads the same scratch."""
    cases = []
    for seed, lens in ((31, [700, 300]), (32, [64, 0, 900])):
        c = _case(lens, lens, 4, 2, 64, seed)
        q, k, v, cq, ck = _dev(c)
        out, lse = vfa.varlen_fwd(q, k, v, cq, ck, c.max_seqlen_q, c.softmax_scale, 1, window_left=100,
                                  sink_tokens=sinks)
        cases.append((q, k, v, out, torch.randn_like(q), lse, cq, ck, c.softmax_scale, 1))
    want = [vfa.varlen_bwd(*a, window_left=100, sink_tokens=sinks)[:3] for a in cases]
    torch.cuda.synchronize()
    ws = vfa.alloc_bwd_workspace(3, 1000, 4, 64, sink_tokens=sinks)
    got = [[torch.empty_like(t) for t in w] for w in want]
    for _ in range(20):
        for a, g in zip(cases, got):
            vfa.varlen_bwd(*a, window_left=100, sink_tokens=sinks, dq=g[0], dk=g[1], dv=g[2], workspace=ws)
    assert vfa.read_status(ws) == 0
    assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window,sinks", [(2, -1, 0), (2, 30, 0), (2, 30, 3), (1, 30, 0), (0, -1, 0)])
@pytest.mark.parametrize("value", [-float("inf"), float("inf")])
def test_backward_of_rows_that_see_nothing(vfa, d, causal, window, sinks, value):
    """What a logsumexp of nothing is elsewhere is no less than -FLT_MAX here: zero gradients."""
    c = _case([300, 64, 40], [130, 64, 0], 4, 2, d, seed=d)
    q, k, v, cq, ck = _dev(c)
    out, lse = _forward(vfa, c, causal, window, sinks)
    empty = lse == -FLT_MAX
    assert empty.any() and not empty.all()
    dout = W.upstream_grad(c, 5).cuda()

    def grads(lse):
        *g, ws = vfa.varlen_bwd(q, k, v, out, dout, lse, cq, ck, c.softmax_scale, causal, window_left=window,
                                sink_tokens=sinks)
        assert vfa.read_status(ws) == 0
        return g

    want, got = grads(lse), grads(torch.where(empty, value, lse))
    assert all(t.isfinite().all() for t in want) and not want[0][empty].any()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
