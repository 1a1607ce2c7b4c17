"""GPU parity of the 4-bit paged cache (write, gather, decode) with the 64-bit definitions.

Write and gather are exact.  Decode, per element:
  scores: the products of f16 operands are exact in fp32; a chain of at most D + 8 additions,
    the multiplication by the scale and the subtraction of the maximum give an error of the
    exponent of at most dx = (D + 16) u32 sum|q k| scale (+ 2 u32 |x| inside it);
  p: e^dx - 1, 2^-21 for ex2, and half an f16 step, 2^-11 of p; l the same without f16;
  small p: 2^10 p is held in f16, whose values below 2^-14 are 2^-24 apart, so half a step is
    2^-25 / 2^10 = 2^-35 absolute for every key, relative to a reference weight that is at most
    the largest one (the reference maximum never exceeds the true one): 2^-35 sum |v| / l;
  out: (2 (e^dx - 1) + 2^-11 + n u32 + 2^-20) sum p |v| / l + 2^-35 sum |v| / l + 2^-8 |out|;
  lse: dx + (n u32 + 2^-20) + 2^-22 |lse| for the logarithm and the final product.
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


def _tables(lens, rng, extra=3, spare=2):
    nb = [-(-n // 16) for n in lens]
    cap = max(max(nb), 1) + spare
    blocks = sum(nb) + extra
    perm = rng.permutation(blocks)
    t = np.full((len(lens), cap), -1, dtype=np.int32)     # unused entries are no pages
    at = 0
    for i, n in enumerate(nb):
        t[i, :n] = perm[at:at + n]
        at += n
    return t, blocks


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _write_case(lens, starts, Hkv, D, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    ends = [a + n for a, n in zip(starts, lens)]
    tables, blocks = _tables(ends, rng)
    total = sum(lens)
    kv = torch.from_numpy(rng.standard_normal((total + 3, 2 * Hkv * D)) *
                          scale * np.exp(rng.uniform(-3, 3, (total + 3, 1)))).bfloat16()
    cu = np.concatenate(([0], np.cumsum(lens)))
    return tables, blocks, kv, cu, total


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,starts,Hkv,dk,dv", [
    ([1], [0], 1, 1.0, 1.0), ([5, 0, 17, 1, 33], [3, 2, 0, 15, 31], 3, 0.125, 2.0),
    ([64], [7], 8, 2.0 ** -6, 2.0 ** 4), ([1, 1, 1, 1, 1], [0, 15, 16, 31, 40], 5, 1.0, 0.5)])
def test_write_and_gather_are_exact(vfa, D, lens, starts, Hkv, dk, dv):
    tables, blocks, kv, cu, total = _write_case(lens, starts, Hkv, D, seed=D + len(lens))
    # three rows past the end are padding: NaN there, and they must not be read or written
    kv[total:] = float("nan")
    x = kv.cuda()
    k, v = x[:, :Hkv * D].view(-1, Hkv, D), x[:, Hkv * D:].view(-1, Hkv, D)
    rng = np.random.default_rng(0)
    before = rng.integers(0, 256, (blocks, Hkv, 18 * D), dtype=np.uint8)
    pool = torch.from_numpy(before.copy()).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_i32(tables), _i32(cu), _i32(starts))
    vfa.kv4_write(k, v, pool, *args, dk, dv, status=status)
    want = before.copy()
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    for s in range(len(lens)):
        for i in range(lens[s]):
            p = starts[s] + i
            O.write_token(want, tables[s, p // 16], p % 16, kn[cu[s] + i], vn[cu[s] + i], dk, dv)
    got = pool.cpu().numpy()
    # a negative value that rounds to zero may keep its sign: compare values, and all other bytes
    pk, pv = O.page_values(got, dk, dv)
    wk, wv = O.page_values(want, dk, dv)
    assert np.array_equal(pk, wk, equal_nan=True) and np.array_equal(pv, wv, equal_nan=True)
    assert np.array_equal(got[..., 16 * D:], want[..., 16 * D:])
    untouched = np.setdiff1d(np.arange(blocks), tables[tables >= 0])
    assert np.array_equal(got[untouched], before[untouched])
    ko = torch.full((total + 3, Hkv, D), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 4.0)
    vfa.kv4_gather(pool, *args, total + 3, dk, dv, k_out=ko, v_out=vo, status=status)
    assert vfa.read_status(status) == 0
    for o, x64, ds, pad in ((ko, kn, dk, 3.0), (vo, vn, dv, 4.0)):
        ref = O.dequantise(*O.quantise(x64[:total], ds), ds)
        assert np.array_equal(o[:total].double().cpu().numpy(), ref)
        assert (o[total:] == pad).all()


def test_quantiser_borders(vfa):
    """Every midpoint of the two formats, both signs, exact ties and their bf16 neighbours."""
    D, rows = 64, []
    for sb in (1, 2, 5, 8, 15, 56, 60, 63, 119, 126):            # subnormal, ordinary, largest
        s = float(O.e4m3_value(sb))
        mids = [s * (a + b) / 2 for a, b in zip(O.E2M1[:-1], O.E2M1[1:])]
        base = torch.tensor([6 * s] + mids + [-m for m in mids] + [0.0]).bfloat16()
        for step in (-1, 0, 1):
            r = base.clone()
            bits = r[1:15].view(torch.int16)
            r[1:15] = (bits + step).view(torch.bfloat16)
            rows.append(r)
    for lo, hi in zip(range(0, 126), range(1, 127)):              # ties of the scale itself
        m = (float(O.e4m3_value(lo)) + float(O.e4m3_value(hi))) / 2 * 6
        for step in (-1, 0, 1):
            r = torch.zeros(16).bfloat16()
            t = torch.tensor([m]).bfloat16()
            r[0] = (t.view(torch.int16) + step).view(torch.bfloat16)[0]
            r[1] = -r[0] / 3
            rows.append(r)
    rows.append(torch.full((16,), 3e38).bfloat16())               # far past the largest scale
    rows.append(torch.full((16,), 1e-38).bfloat16())              # far below the smallest
    while len(rows) % 4:
        rows.append(torch.zeros(16).bfloat16())
    x = torch.stack(rows).view(-1, 1, D)
    n = x.shape[0]
    for ds in (1.0, 2.0 ** -5, 2.0 ** 7):
        xs = (x.float() * ds).bfloat16()
        d = xs.cuda()
        pool = vfa.alloc_kv4_pool(-(-n // 16), 1, D)
        args = (_i32(np.arange(pool.shape[0])[None]), _i32([0, n]), _i32([0]))
        vfa.kv4_write(d, d, pool, *args, ds, ds)
        k, v = vfa.kv4_gather(pool, *args, n, ds, ds)
        ref = O.dequantise(*O.quantise(xs.double().numpy(), ds), ds)
        assert np.array_equal(k.double().cpu().numpy(), ref)
        assert np.array_equal(v.double().cpu().numpy(), ref)


# ------------------------------------------------------------------ decode

def _decode_case(lens, Hq, Hkv, D, seed, dk=0.25, dv=0.5, qscale=1.0):
    rng = np.random.default_rng(seed)
    tables, blocks = _tables(lens, rng)
    # pages of random codes and plausible scales; unused rows and pages hold NaN scales
    pool = rng.integers(0, 256, (blocks, Hkv, 18 * D), dtype=np.uint8)
    pool[..., 16 * D:] = rng.integers(40, 64, (blocks, Hkv, 2 * D))
    used = np.zeros((blocks, 16), bool)
    for s, n in enumerate(lens):
        for t in range(n):
            used[tables[s, t // 16], t % 16] = True
    for b, t in np.argwhere(~used):
        for g in range(0, D, 16):
            pool[b, :, O.k_scale_byte(t, g, D)] = 0x7f
            pool[b, :, O.v_scale_byte(t, g, D)] = 0xff
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)) * qscale).bfloat16()
    return q, pool, tables, np.asarray(lens, np.int32), dk, dv


def _bounds(ref, n):
    out, lse, absdot, absv, allv = ref
    D = out.shape[-1]
    dx = (D + 16) * U * absdot
    p = 2 * np.expm1(dx) + 2.0 ** -11 + n[:, None] * U + 2.0 ** -20
    return p[..., None] * absv + 2.0 ** -35 * allv + 2.0 ** -8 * np.abs(out) + 1e-30, \
        dx + n[:, None] * U + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(lse == -O.FLT_MAX, 0, lse))


def _check_decode(got, case, scale=None):
    q, pool, tables, n, dk, dv = case
    ref = O.kv4_decode(q.double().numpy(), pool, tables, n, dk, dv, scale)
    bo, bl = _bounds(ref, n)
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    assert np.isfinite(out).all()
    empty = n == 0
    assert (out[empty] == 0).all() and (lse[empty] == -O.FLT_MAX).all()
    assert (np.abs(out - ref[0]) <= bo).all(), float((np.abs(out - ref[0]) - bo).max())
    assert (np.abs(lse - ref[1])[~empty] <= bl[~empty]).all(), float((np.abs(lse - ref[1]) - bl)[~empty].max())


def _run(vfa, case, **kw):
    q, pool, tables, n, dk, dv = case
    return vfa.kv4_decode(q.cuda(), torch.from_numpy(pool).cuda(), _i32(tables), _i32(n), dk, dv, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (32, 8), (7, 1), (6, 2), (40, 8), (16, 1),
                                    (33, 3)])
def test_decode_heads(vfa, D, Hq, Hkv):
    case = _decode_case([1, 16, 0, 17, 130, 333], Hq, Hkv, D, seed=Hq * D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(vfa, case, status=status)
    assert vfa.read_status(status) == 0
    _check_decode(got, case)


@pytest.mark.parametrize("lens", [
    [1], [0], [0, 0, 0], [15], [16], [129], [9000], [1, 5000, 2], [128] * 40,
    list(range(0, 300)), [4000, 0, 0, 1, 1, 3999, 0], [2047, 2048, 2049, 127, 128, 129]])
def test_decode_lengths(vfa, lens):
    """Runs that begin and end inside, at, and over the sequences' borders."""
    case = _decode_case(lens, 4, 2, 64, seed=len(lens) + sum(lens))
    ws = vfa.alloc_kv4_decode_workspace(len(lens), 4, 2, 64)
    first = _run(vfa, case, workspace=ws)
    _check_decode(first, case)
    assert (ws[-len(lens) * 2 * 4:] == 0).all()           # the tickets
    second = _run(vfa, case, workspace=ws)                # the workspace serves again
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


@pytest.mark.parametrize("qscale,scale", [(1e-6, 0.0), (200.0, 0.0), (1.0, 1e-3), (1.0, 2.0),
                                          (1e30, 1e-30), (1e-30, 1e30)])
def test_decode_scales(vfa, qscale, scale):
    """Flat and peaked softmaxes; query magnitudes far outside f16's range."""
    case = _decode_case([700, 40, 3], 6, 2, 128, seed=5, qscale=qscale)
    _check_decode(_run(vfa, case, softmax_scale=scale), case, scale if scale > 0 else None)


@pytest.mark.parametrize("lens", [[40], [9000, 3, 700]])
@pytest.mark.parametrize("exponent", [12, 24, 40, 90])
def test_decode_huge_logits(vfa, lens, exponent):
    """Logits far apart and past 2^24, where their fp32 neighbours are whole units apart: the
    largest take all the weight, equal ones share it.

    q has one element and the keys multiples of 1/2 there, so the accumulators are exact and a
    difference is 0 or at least 2^11 / sqrt(64) * log2(e) > 360: the other weights are below
    2^-360.  Equal weights are equal numbers, so the mean over c of them is off by (c + 2) u32
    and ex2's 2^-20 of sum |v| / c and the bf16 rounding; lse by four roundings, 2^-22 of itself,
    and 2^-20 for the logarithm.
    """
    D, Hq = 64, 3
    q, pool, tables, n, dk, dv = _decode_case(lens, Hq, 1, D, seed=exponent)
    pool[..., 16 * D:] = 0x38                             # every scale 1.0
    q[:] = 0
    q[:, 0, 7], q[:, 1, 7], q[:, 2, 7] = 2.0 ** exponent, -2.0 ** exponent, 1.5 * 2.0 ** exponent
    got = _run(vfa, (q, pool, tables, n, 1.0, 1.0))
    for s, m in enumerate(lens):
        k, v = (a[:, 0].reshape(-1, D)[:m]
                for a in O.page_values(pool[tables[s, :-(-m // 16)]], 1.0, 1.0))
        for h in range(Hq):
            x = k[:, 7] * float(q[s, h, 7]) / math.sqrt(D)
            top = x == x.max()
            c = int(top.sum())
            ref = v[top].mean(0)
            tol = ((c + 2) * U + 2.0 ** -20) * np.abs(v[top]).mean(0) + 2.0 ** -8 * np.abs(ref) + 1e-30
            assert (np.abs(got[0][s, h].double().cpu().numpy() - ref) <= tol).all()
            want = x.max() + math.log(c)
            assert abs(float(got[1][s, h]) - want) <= 2.0 ** -22 * abs(want) + 2.0 ** -20


def test_decode_many_small_weights(vfa):
    """One strong key among thousands of weak ones whose weights add up: none are lost to f16."""
    lens = [16384]
    q, pool, tables, n, dk, dv = _decode_case(lens, 1, 1, 64, seed=1)
    D = 64
    pool[..., :8 * D] = 0x22                              # every code 1.0
    pool[..., 16 * D:] = 0x38                             # every scale 1.0
    # token 0: all K codes 6 (0x77) -> a score 5 * 64 / 8 * |q| above the others
    pool[tables[0, 0], 0, :D // 2] = 0x77
    q[:] = 0.25                                           # scores 10 ln-units apart
    case = (q, pool, tables, n, 1.0, 1.0)
    _check_decode(_run(vfa, case), case)


def test_decode_keeps_bad_numbers_where_they_are(vfa):
    """NaN and infinity in one query head, a NaN scale in one sequence's pages: the heads of the
    same tile and the other sequences, some in the same CTA, are right."""
    case = _decode_case([700, 3, 40, 9, 2500], 8, 2, 64, seed=11)
    q, pool, tables, n, dk, dv = case
    bad_q, bad_pool = q.clone(), pool.copy()
    bad_q[1, 5, 7] = float("nan")
    bad_q[4, 0] = float("inf")
    bad_q[4, 1, 3] = float("-inf")
    bad_pool[tables[2, 1], 1, O.v_scale_byte(3, 16, 64)] = 0x7f
    bad_pool[tables[2, 1], 1, O.k_scale_byte(4, 0, 64)] = 0xff
    got = _run(vfa, (bad_q, bad_pool, tables, n, dk, dv))
    hit = np.zeros((5, 8), bool)
    hit[1, 5] = hit[4, :2] = hit[2, 4:] = True
    ref = O.kv4_decode(q.double().numpy(), pool, tables, n, dk, dv)
    bo, bl = _bounds(ref, n)
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    assert (np.abs(out - ref[0]) <= bo)[~hit].all() and (np.abs(lse - ref[1]) <= bl)[~hit].all()
    assert np.isnan(out[hit]).any(-1).all() and not np.isfinite(lse[hit]).any()


def test_decode_refuses_bad_pages(vfa):
    """A bad count or page id: status set, that sequence's rows as they were, the others right."""
    case = _decode_case([100, 3000, 50, 20, 64], 4, 2, 128, seed=2)
    q, pool, tables, n, dk, dv = case
    bad_t, bad_n = tables.copy(), n.copy()
    bad_t[1, 100] = pool.shape[0]
    bad_t[3, 1] = -1
    bad_n[4] = tables.shape[1] * 16 + 1
    bad_n[2] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 4), 9.0, device="cuda")
    ws = vfa.alloc_kv4_decode_workspace(5, 4, 2, 128)
    got = vfa.kv4_decode(q.cuda(), torch.from_numpy(pool).cuda(), _i32(bad_t), _i32(bad_n), dk, dv,
                         out=out, lse=lse, status=status, workspace=ws)
    assert vfa.read_status(status) == vfa.VFA_ERR_BAD_BLOCK
    assert (out[1:] == 9.0).all() and (lse[1:] == 9.0).all()
    one = (q[:1], pool, tables[:1], n[:1], dk, dv)
    _check_decode((got[0][:1], got[1][:1]), one)
    status.zero_()
    again = _run(vfa, case, workspace=ws, status=status)  # the workspace is still good
    assert vfa.read_status(status) == 0
    _check_decode(again, case)


def test_write_and_gather_skip_bad_places(vfa):
    D, Hkv = 64, 2
    tables, blocks, kv, cu, total = _write_case([20, 4, 9], [0, 0, 0], Hkv, D, seed=1)
    x = kv[:total].cuda()
    k, v = x[:, :Hkv * D].view(-1, Hkv, D), x[:, Hkv * D:].view(-1, Hkv, D)
    bad = tables.copy()
    bad[0, 1] = blocks
    pool = vfa.alloc_kv4_pool(blocks, Hkv, D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = _i32([0, tables.shape[1] * 16 - 2, 0])       # sequence 1 runs past its row
    # (its in-range tokens fall on entries that hold no page)
    vfa.kv4_write(k, v, pool, _i32(bad), _i32(cu), starts, status=status)
    assert vfa.read_status(status) == vfa.VFA_ERR_BAD_BLOCK
    status.zero_()
    ko, vo = (torch.full((total, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    vfa.kv4_gather(pool, _i32(bad), _i32(cu), starts, total, k_out=ko, v_out=vo, status=status)
    assert vfa.read_status(status) == vfa.VFA_ERR_BAD_BLOCK
    ref = O.dequantise(*O.quantise(k.double().cpu().numpy(), 1.0), 1.0)
    got = ko.double().cpu().numpy()
    ok = np.r_[0:16, 24:33]
    assert np.array_equal(got[ok], ref[ok])
    assert (got[16:24] == 5.0).all()
    for bad_cu in ([0, 25, 20, total], [1, 20, 24, total], [0, 20, 24, total + 1]):
        status.zero_()
        vfa.kv4_write(k, v, pool, _i32(tables), _i32(bad_cu), _i32([0, 0, 0]), status=status)
        assert vfa.read_status(status) in (vfa.VFA_ERR_BAD_SEQLENS, vfa.VFA_ERR_BAD_BLOCK)


def test_decode_captured_twice_with_one_workspace(vfa):
    """Two graphs that share a workspace, replayed in turn on one side stream."""
    a = _decode_case([3000, 1, 77], 8, 2, 128, seed=3)
    b = _decode_case([5, 2500, 900], 8, 2, 128, seed=4)
    ws = vfa.alloc_kv4_decode_workspace(3, 8, 2, 128)
    s = torch.cuda.Stream()
    dev, outs, graphs = [], [], []
    for q, pool, tables, n, dk, dv in (a, b):
        d = (q.cuda(), torch.from_numpy(pool).cuda(), _i32(tables), _i32(n))
        dev.append(d)
        outs.append((torch.zeros_like(d[0]), torch.zeros(3, 8, device="cuda")))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for d, o in zip(dev, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                vfa.kv4_decode(*d, 0.25, 0.5, out=o[0], lse=o[1], workspace=ws)
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    _check_decode(outs[0], a)
    _check_decode(outs[1], b)


def test_one_workspace_for_smaller_batches(vfa):
    """A workspace made for the largest batch serves the smaller ones between."""
    big = _decode_case([3000, 1, 77, 900, 2500, 40, 0, 129, 4000], 8, 2, 128, seed=6)
    ws = vfa.alloc_kv4_decode_workspace(9, 8, 2, 128)
    for n in (9, 2, 5, 1, 9, 3, 9):
        q, pool, tables, lens, dk, dv = big
        case = (q[:n], pool, tables[:n], lens[:n], dk, dv)
        _check_decode(_run(vfa, case, workspace=ws), case)


def test_offsets_past_32_bits(vfa):
    """Pages beyond 4 GiB of the pool."""
    D, Hkv = 256, 8
    page = Hkv * 18 * D
    blocks = (1 << 32) // page + 40
    pool = torch.zeros(blocks, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    tables = np.array([[blocks - 1, blocks - 3, 0]], np.int32)
    rng = np.random.default_rng(0)
    n = 40
    kv = torch.from_numpy(rng.standard_normal((n, 2, Hkv, D))).bfloat16()
    k, v = kv[:, 0].contiguous(), kv[:, 1].contiguous()
    vfa.kv4_write(k.cuda(), v.cuda(), pool, _i32(tables), _i32([0, n]), _i32([0]))
    small = pool[[blocks - 1, blocks - 3, 0]].cpu().numpy()
    q = torch.from_numpy(rng.standard_normal((1, Hkv, D))).bfloat16()
    got = vfa.kv4_decode(q.cuda(), pool, _i32(tables), _i32([n]))
    _check_decode(got, (q, small, np.array([[0, 1, 2]], np.int32), np.array([n], np.int32), 1.0, 1.0))
    kk, _ = vfa.kv4_gather(pool, _i32(tables), _i32([0, n]), _i32([0]), n)
    assert np.array_equal(kk.double().cpu().numpy(),
                          O.dequantise(*O.quantise(k.double().numpy(), 1.0), 1.0))


@pytest.mark.parametrize("exponent,scale,dk", [(100, 2.0 ** 100, 1.0), (0, 3e38, 2.0 ** 64),
                                               (120, 0.0, 2.0 ** 40)])
def test_decode_scale_past_fp32(vfa, exponent, scale, dk):
    """Logits whose scale passes the largest fp32: they are finite numbers in the definition, the
    largest takes all the weight (equal ones share it), and lse is past fp32 with its sign.

    Exactly as in test_decode_huge_logits: accumulators are exact, different ones are at least
    1/2 apart in units of the largest element of q, so all other weights are zero; the mean over
    the c largest is off by (c + 2) u32 and ex2's 2^-20 of sum |v| / c and the bf16 rounding.
    """
    D, lens = 64, [40, 3, 900]
    q, pool, tables, n, _, _ = _decode_case(lens, 2, 1, D, seed=exponent)
    pool[..., 16 * D:] = 0x38                             # every scale 1.0
    q[:] = 0
    q[:, 0, 7], q[:, 1, 7] = 2.0 ** exponent, -1.5 * 2.0 ** exponent
    got = vfa.kv4_decode(q.cuda(), torch.from_numpy(pool).cuda(), _i32(tables), _i32(n), dk, 1.0, scale)
    for s, m in enumerate(lens):
        k, v = (a[:, 0].reshape(-1, D)[:m]
                for a in O.page_values(pool[tables[s, :-(-m // 16)]], 1.0, 1.0))
        for h in range(2):
            x = k[:, 7] * float(q[s, h, 7])
            top = x == x.max()
            ref = v[top].mean(0)
            c = int(top.sum())
            tol = ((c + 2) * U + 2.0 ** -20) * np.abs(v[top]).mean(0) + 2.0 ** -8 * np.abs(ref) + 1e-30
            assert (np.abs(got[0][s, h].double().cpu().numpy() - ref) <= tol).all(), (s, h)
            if x.max() != 0:
                assert float(got[1][s, h]) == math.copysign(math.inf, x.max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (32, 1), (66, 2)])
def test_decode_several_head_chunks(vfa, D, Hq, Hkv):
    """More query heads per kv head than one CTA takes, the last chunk of them almost empty."""
    case = _decode_case([1, 16, 0, 17, 130, 333], Hq, Hkv, D, seed=Hq * D)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(vfa, case, status=status)
    assert vfa.read_status(status) == 0
    _check_decode(got, case)


@pytest.mark.parametrize("Hq,Hkv,D", [(34, 1, 64), (20, 1, 128), (40, 2, 128), (11, 1, 256)])
def test_decode_head_chunks_over_several_runs(vfa, Hq, Hkv, D):
    """Long sequences cut into runs, with several head chunks per kv head: every chunk has
    partial states and tickets of its own, and the workspace serves again."""
    case = _decode_case([6000, 3, 700, 0, 2500], Hq, Hkv, D, seed=Hq)
    ws = vfa.alloc_kv4_decode_workspace(5, Hq, Hkv, D)
    per = 8 if D == 256 else 16
    rows = Hkv * -(-(Hq // Hkv) // per)
    first = _run(vfa, case, workspace=ws)
    _check_decode(first, case)
    assert (ws[-5 * rows * 4:] == 0).all()                # the tickets
    second = _run(vfa, case, workspace=ws)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


def test_bad_cu_seqlens_are_recorded_as_such(vfa):
    """Every token these prefix sums place has a page, so nothing else can be recorded."""
    D, Hkv, total = 64, 2, 33
    x = torch.randn(total, Hkv, D).bfloat16().cuda()
    pool = vfa.alloc_kv4_pool(12, Hkv, D)
    tables = _i32(np.arange(12).reshape(3, 4))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu in ([0, 25, 20, total], [1, 20, 24, total], [0, 20, 24, total + 1], [-1, 20, 24, total]):
        for call in (lambda: vfa.kv4_write(x, x, pool, tables, _i32(cu), _i32([0, 0, 0]), status=status),
                     lambda: vfa.kv4_gather(pool, tables, _i32(cu), _i32([0, 0, 0]), total,
                                            status=status)):
            status.zero_()
            call()
            assert vfa.read_status(status) == vfa.VFA_ERR_BAD_SEQLENS, cu
