"""GPU parity of qk_norm_rope and its backward against the 64-bit definitions.

Tolerances, per element, from the roundings (u32 = 2^-24, bf16 half step 2^-8):
  forward: bf16 rounding of the result, 2^-8 |y|, plus fp32 work on the pair.  The mean square
    is a sum of 16 fmas and at most 4 shuffle adds (21 roundings incl. the mean), halved by the
    root; rsqrtf is within 2 ulp (4 u32); x r w 2 roundings; the sine and cosine within 2 ulp
    (4 u32) plus an angle error of pi (2^-25 + 2^-32) < 4 u32; product and fma 2.  Together
    below 11 + 4 + 2 + 8 + 2 < 32 u32 of |n_a| + |n_b|.
  dx: 2^-8 |dx| plus, on r (|u| + |x| r^2 mean|u x|) with u from the rotated pair: rotation
    10 u32, w and products 4, r three times 15, the mean 21, the difference 2: below 96 u32.
  dweight: sums of N = tokens * heads terms in chains of at most N + 64 additions, each term
    within 32 u32: (N + 96) u32 sum |g x r| (with |g| the pair's magnitude).
"""
import math

import numpy as np
import pytest
import torch

import oracle.serving as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def vfa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


def _case(T, Hq, Hkv, D, R, axes, norm, seed=0, maxpos=5000, strided=True, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    width = (Hq + 2 * Hkv) * D
    qkv = (torch.randn(T, width, generator=g) * sigma).bfloat16()
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(-maxpos, maxpos, (axes, T), generator=g, dtype=torch.int32)
    f = [10000.0 ** (-2 * i / max(R, 1)) for i in range(R // 2)]
    ax = [i % axes for i in range(R // 2)]
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    dy = [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv)]
    return dict(qkv=qkv, q=q, k=k, pos=pos, f=f, ax=ax, w=w, dy=dy, D=D, Hq=Hq, Hkv=Hkv, T=T)


def _dev(c):
    qkv = c["qkv"].cuda()
    T, D, Hq, Hkv = c["T"], c["D"], c["Hq"], c["Hkv"]
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    if c["q"].is_contiguous() and T > 1:
        q, k = q.contiguous(), k.contiguous()
    return q, k, c["pos"].cuda(), [None if w is None else w.cuda() for w in c["w"]]


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _amp(x, R, inter):
    """|first| + |second| of each pair, |x| outside."""
    a = np.abs(x).copy()
    n = R // 2
    if n:
        i, j = O._pairs(n, inter)
        s = a[..., i] + a[..., j]
        a[..., i] = s
        a[..., j] = s
    return a


def _check_fwd(c, got, inter, eps):
    for x, w, y in ((c["q"], c["w"][0], got[0]), (c["k"], c["w"][1], got[1])):
        ref = O.norm_rope(_f64(x), c["pos"].numpy(), c["f"], c["ax"], _f64(w), eps, inter)
        amp = _amp(O.norm(_f64(x), _f64(w), eps), 2 * len(c["f"]), inter)
        err = np.abs(_f64(y) - ref)
        tol = 2.0 ** -8 * np.abs(ref) + 32 * U * amp * (1 + 2.0 ** -8)
        assert np.isfinite(err).all() and (err <= tol).all(), float((err - tol).max())


SHAPES = [
    (1, 1, 1, 64, 64, 1, True, False), (3, 2, 1, 128, 128, 1, True, True),
    (7, 5, 5, 64, 48, 3, True, True), (130, 7, 1, 256, 256, 2, True, False),
    (33, 32, 8, 128, 16, 4, True, False), (257, 3, 3, 128, 128, 1, False, False),
    (64, 28, 4, 128, 64, 1, False, True), (19, 9, 3, 256, 48, 1, True, True),
    (12, 4, 2, 64, 0, 1, True, False), (5000, 2, 1, 64, 32, 2, True, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,axes,norm,inter", SHAPES)
def test_forward(vfa, T, Hq, Hkv, D, R, axes, norm, inter):
    c = _case(T, Hq, Hkv, D, R, axes, norm, seed=T)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], c["ax"]) if R else None
    got = vfa.qk_norm_rope(q, k, pos if R else None, table, w[0], w[1], eps=1e-5,
                           interleaved=inter)
    _check_fwd(c, got, inter, 1e-5)


@pytest.mark.parametrize("T,Hq,Hkv,D,R,axes,norm,inter", SHAPES)
def test_backward(vfa, T, Hq, Hkv, D, R, axes, norm, inter):
    c = _case(T, Hq, Hkv, D, R, axes, norm, seed=T + 1)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], c["ax"]) if R else None
    dy = [t.cuda() for t in c["dy"]]
    eps = 1e-5
    got = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos if R else None, table, w[0], w[1], eps=eps,
                               interleaved=inter)
    for i, x in enumerate((c["q"], c["k"])):
        x, y, wt = _f64(x), _f64(c["dy"][i]), _f64(c["w"][i])
        dx, dw = O.norm_rope_bwd(x, y, c["pos"].numpy(), c["f"], c["ax"], wt, eps, inter)
        g = _amp(y, R, inter)
        if wt is None:
            amp = g
            assert got[2 + i] is None
        else:
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            u = g * np.abs(wt)
            amp = r * (u + np.abs(x) * r * r * (u * np.abs(x)).mean(-1, keepdims=True))
            tol = (T * x.shape[1] + 96) * U * (g * np.abs(x) * r).sum((0, 1))
            assert (np.abs(_f64(got[2 + i]) - dw) <= tol).all()
        err = np.abs(_f64(got[i]) - dx)
        tol = 2.0 ** -8 * np.abs(dx) + 96 * U * amp * (1 + 2.0 ** -8)
        assert np.isfinite(err).all() and (err <= tol).all(), float((err - tol).max())
    again = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos if R else None, table, w[0], w[1],
                                 eps=eps, interleaved=inter)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)          # fixed order of the sums


def test_far_positions_and_extremes(vfa):
    """Positions up to the ends of int32 turn exactly as in 64 bits."""
    c = _case(8, 2, 1, 64, 64, 1, False)
    c["pos"] = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567890, 2 ** 24 + 1, -999999937]],
                            dtype=torch.int32)
    q, k, pos, _ = _dev(c)
    # frequencies that 64-bit angles hold to 2^-53 * 2^31 * f: keep the check's own error small
    c["f"] = [2.0 ** -i for i in range(32)]
    got = vfa.qk_norm_rope(q, k, pos, vfa.rope_table(c["f"]), None, None)
    for x, y in ((c["q"], got[0]), (c["k"], got[1])):
        ref = O.norm_rope(_f64(x), c["pos"].numpy(), c["f"], [0] * 32, None, 0, False)
        err = np.abs(_f64(y) - ref)
        # + the 64-bit angle's own rounding of 2 pi multiples, 2^31 * 2^-53
        tol = 2.0 ** -8 * np.abs(ref) + (32 * U + 2.0 ** -21) * _amp(_f64(x), 64, False) * (1 + 2.0 ** -8)
        assert (err <= tol).all(), float((err - tol).max())


def test_small_and_large_values(vfa):
    """eps matters for tiny rows; zero rows give zeros and zero gradients, no NaN."""
    c = _case(6, 2, 2, 64, 32, 1, True, sigma=1e-3)
    for t in (c["q"], c["k"]):
        t[2] = 0
        t[3] *= 1e6
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], c["ax"])
    got = vfa.qk_norm_rope(q, k, pos, table, w[0], w[1], eps=1e-6)
    _check_fwd(c, got, False, 1e-6)
    assert (got[0][2] == 0).all()
    dy = [t.cuda() for t in c["dy"]]
    r = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, w[0], w[1], eps=1e-6)
    assert all(torch.isfinite(t.float()).all() for t in r)


def test_in_place_and_strided_outputs(vfa):
    c = _case(37, 6, 2, 128, 128, 1, True)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], c["ax"])
    want = vfa.qk_norm_rope(q, k, pos, table, w[0], w[1])
    joint = torch.full((37, (6 + 2 + 2) * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    qo, ko = joint[:, :768].view(37, 6, 128), joint[:, 768:1024].view(37, 2, 128)
    vfa.qk_norm_rope(q, k, pos, table, w[0], w[1], q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert (joint[:, 1024:] == 7.0).all()
    dy = [t.cuda() for t in c["dy"]]
    ref = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, w[0], w[1])
    got = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, w[0], w[1], dq=dy[0], dk=dy[1])
    assert got[0] is dy[0] and all(torch.equal(a, b) for a, b in zip(ref, got))
    vfa.qk_norm_rope(q, k, pos, table, w[0], w[1], q_out=q, k_out=k)      # over its inputs
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_token_strides_past_32_bits(vfa):
    """Tokens 2^30 elements apart: the packed case's bits, in place, forward and backward."""
    T, H, D = 4, 3, 128
    c = _case(T, H, H, D, 64, 1, True, seed=8, strided=False)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"])
    dy = [d.cuda() for d in c["dy"]]
    want = vfa.qk_norm_rope(q, k, pos, table, *w)
    wantb = vfa.qk_norm_rope_bwd(q, k, *dy, pos, table, *w)
    buf = torch.empty((T - 1 << 30) + 4 * H * D, dtype=torch.bfloat16, device="cuda")
    far = [buf.as_strided((T, H, D), (1 << 30, D, 1), i * H * D) for i in range(4)]
    for x, f in zip((q, k, *dy), far):
        f.copy_(x)
    gotb = vfa.qk_norm_rope_bwd(*far, pos, table, *w, dq=far[2], dk=far[3])
    got = vfa.qk_norm_rope(far[0], far[1], pos, table, *w, q_out=far[0], k_out=far[1])
    for a, b in zip((*want, *wantb), (*got, *gotb)):
        assert torch.equal(a, b)


def test_no_tokens(vfa):
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    table = vfa.rope_table([1.0] * 8)
    a, b = vfa.qk_norm_rope(q, q, pos, table, w, w)
    assert a.shape == (0, 4, 64)
    r = vfa.qk_norm_rope_bwd(q, q, q, q, pos, table, w, w, dq_weight=w * 5, dk_weight=w * 5)
    assert (r[2] == 0).all() and (r[3] == 0).all()


def test_one_weight_only_and_axis_clamp(vfa):
    c = _case(9, 2, 2, 64, 64, 1, True)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], [3] * 32)          # an axis past the positions' reads the last
    got = vfa.qk_norm_rope(q, k, pos, table, None, w[1])
    c["w"][0] = None
    _check_fwd(c, got, False, 1e-6)
    dy = [t.cuda() for t in c["dy"]]
    r = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, None, w[1])
    assert r[2] is None and r[3] is not None


def test_captured_backward_beside_an_eager_one(vfa):
    """A graph replay on another stream, and an eager call between, give the eager results."""
    c = _case(301, 4, 2, 128, 128, 1, True)
    q, k, pos, w = _dev(c)
    table = vfa.rope_table(c["f"], c["ax"])
    dy = [t.cuda() for t in c["dy"]]
    eager = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, w[0], w[1])
    ws = vfa.alloc_qk_norm_rope_bwd_workspace(128)
    outs = [torch.zeros_like(t) for t in eager]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, table, w[0], w[1], dq=outs[0],
                                 dk=outs[1], dq_weight=outs[2], dk_weight=outs[3], workspace=ws)
        for _ in range(2):
            for t in outs:
                t.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, outs))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 3), (5, 7), (3, 1), (8, 2)])
def test_backward_without_eps(vfa, D, Hq, Hkv):
    """eps = 0 and head counts that leave lanes of a warp's turn without a head: the rows have a
    norm, so every gradient is an ordinary number (tolerances as above)."""
    T, R = 41, 32
    c = _case(T, Hq, Hkv, D, R, 1, True, seed=D + Hq)
    q, k, pos, w = _dev(c)
    dy = [t.cuda() for t in c["dy"]]
    got = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, vfa.rope_table(c["f"]), w[0], w[1], eps=0.0)
    for i, x in enumerate((c["q"], c["k"])):
        x, y, wt = _f64(x), _f64(c["dy"][i]), _f64(c["w"][i])
        dx, dw = O.norm_rope_bwd(x, y, c["pos"].numpy(), c["f"], c["ax"], wt, 0.0, False)
        g = _amp(y, R, False)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True))
        u = g * np.abs(wt)
        amp = r * (u + np.abs(x) * r * r * (u * np.abs(x)).mean(-1, keepdims=True))
        tol = (T * x.shape[1] + 96) * U * (g * np.abs(x) * r).sum((0, 1))
        assert (np.abs(_f64(got[2 + i]) - dw) <= tol).all(), got[2 + i]
        tol = 2.0 ** -8 * np.abs(dx) + 96 * U * amp * (1 + 2.0 ** -8)
        assert (np.abs(_f64(got[i]) - dx) <= tol).all()


@pytest.mark.parametrize("T,H,D", [(20000, 8, 64), (30001, 1, 128), (6000, 12, 256)])
def test_weight_gradients_are_summed_as_a_tree(vfa, T, H, D):
    """The sums of dweight run over lanes, warps and CTAs side by side.  A lane adds one term per
    turn of its warp: with four warps in four CTAs of every SM, each taking whole tokens, at most
    ceil(T / (16 SMs)) tokens of ceil(H / (512 / D)) turns; then log2(512 / D) <= 3 exchanges, 4
    warps, ceil(4 SMs / 32) CTAs per slice and 5 exchanges of the slices.  A term is within 32 u32
    (above), so the error is at most (depth + 32) u32 sum |g x r|, far below the chain of all
    T * H terms."""
    c = _case(T, H, H, D, 32, 1, True, seed=T)
    q, k, pos, w = _dev(c)
    dy = [t.cuda() for t in c["dy"]]
    got = vfa.qk_norm_rope_bwd(q, k, dy[0], dy[1], pos, vfa.rope_table(c["f"]), w[0], w[1])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T >= 32 * sms                                   # (fewer tokens: their heads are shared)
    depth = -(-T // (16 * sms)) * -(-H * D // 512) + 3 + 4 + -(-4 * sms // 32) + 5
    for i, x in enumerate((c["q"], c["k"])):
        x, y, wt = _f64(x), _f64(c["dy"][i]), _f64(c["w"][i])
        _, dw = O.norm_rope_bwd(x, y, c["pos"].numpy(), c["f"], c["ax"], wt, 1e-6, False)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        tol = (depth + 32) * U * (_amp(y, 32, False) * np.abs(x) * r).sum((0, 1))
        assert (np.abs(_f64(got[2 + i]) - dw) <= tol).all()
