"""GPU parity of the operators of a bounded cache with the 64-bit definitions: one-launch paged
decode, accumulated key weights, eviction and truncation.

Decode, per element (u = 2^-23 for bf16 products added up in the tensor core's fp32):
  scores: the exponent is off by at most dx = (D + 16) u max_j sum|q k| scale;
  p: e^dx - 1, 2^-20 for ex2, and half a bf16 step, 2^-8; l the same without bf16;
  out: (2 (e^dx - 1) + 2^-8 + n u + 2^-19) sum p|v| / l, and its own rounding 2^-8 |out|;
  lse: dx + n u + 2^-19 + 2^-22 |lse|;
  weights: (2 (e^dx - 1) + n u + 2^-19) of what is added, and a rounding 2^-24 of the sum per
  addition (one per query head).
Key weights of a prompt: the exponent is off by dx' = (D + 16) u max sum|q k| scale + 2^-22 |lse|
(the product with log2 e), a sum of m terms by m u more.
Eviction and truncation are exact.
"""
import numpy as np
import pytest
import torch

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


def _f64(t):
    return t.double().cpu().numpy()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _tables(lens, rng, extra=3, spare=2):
    nb = [-(-n // 16) for n in lens]
    cap = max(max(nb), 1) + spare
    t = np.full((len(lens), cap), -1, dtype=np.int32)     # unused entries are no pages
    perm, at = rng.permutation(sum(nb) + extra), 0
    for i, n in enumerate(nb):
        t[i, :n] = perm[at:at + n]
        at += n
    return t, sum(nb) + extra


def _cache(lens, hkv, d, seed, scale=1.0):
    """Pools whose unused slots hold NaN, and the tables."""
    rng = np.random.default_rng(seed)
    tables, blocks = _tables(lens, rng)
    pools = []
    for _ in range(2):
        p = np.full((blocks, 16, hkv, d), np.nan)
        for s, n in enumerate(lens):
            for j in range(n):
                p[tables[s, j // 16], j % 16] = rng.standard_normal((hkv, d)) * scale
        pools.append(torch.from_numpy(p).bfloat16())
    return pools[0], pools[1], tables, rng


def _check_decode(c, lens, window, sinks, scale, got, weights=None):
    q, k, v, tables = c
    out, lse = got[:2]
    zero = lambda t: np.nan_to_num(_f64(t))
    sc = scale if scale > 0 else 1 / np.sqrt(q.shape[2])
    ref, rlse, dot, absv, rw = O.paged_decode(_f64(q), zero(k), zero(v), tables, lens, window, sinks,
                                              float(np.float32(sc)))
    n, d = max(list(lens) + [1]), q.shape[2]
    dx = (d + 16) * U * dot
    g, gl = _f64(out), _f64(lse)
    bound = (2 * np.expm1(dx) + 2.0 ** -8 + n * U + 2.0 ** -19)[..., None] * absv + \
        2.0 ** -8 * np.abs(ref) + 1e-30
    assert np.all(np.abs(g - ref) <= bound), np.nanmax(np.abs(g - ref) / bound)
    empty = rlse == -FLT_MAX
    assert np.all(gl[empty] == np.float32(-FLT_MAX)) and np.all(g[empty] == 0)
    assert np.all((np.abs(gl - rlse) <= dx + n * U + 2.0 ** -19 + 2.0 ** -22 * np.abs(rlse))[~empty])
    if weights is None:
        return
    before, after, old = (_f64(x) for x in weights)
    hkv = rw.shape[1]
    worst = (2 * np.expm1(dx) + n * U + 2.0 ** -19).reshape(len(lens), hkv, -1).max(-1)[..., None]
    seen = rw > 0
    group = q.shape[1] // hkv
    want = before + rw
    assert np.all((np.abs(after - want) <= worst * rw + (group + 1) * 2.0 ** -24 * np.abs(want))[seen])
    # slots that nobody sees stay as they were; a visible weight may underflow to nothing
    untouched = (after == old) | (after == before)
    assert np.all(untouched[~seen])
    hidden = np.ones(seen.shape, bool)
    for s, m in enumerate(lens):
        for j in range(m):
            hidden[s, :, j] = not (window < 0 or j >= m - 1 - window or j < sinks)
    assert np.all((after == old)[hidden])


LENS = [[1], [5, 0, 17, 1, 33, 16], [300, 2, 129, 64], [700]]
WINDOWS = [(-1, 0), (0, 0), (0, 1), (7, 3), (15, 16), (16, 17), (33, 40), (100, 4), (5000, 2)]


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (128, 8, 2), (256, 3, 1), (64, 9, 1), (128, 20, 2),
                                      (256, 16, 2)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_decode(vfa, d, hq, hkv, window, sinks):
    for i, lens in enumerate(LENS):
        k, v, tables, rng = _cache(lens, hkv, d, seed=i + d)
        q = torch.from_numpy(rng.standard_normal((len(lens), hq, d))).bfloat16()
        args = (q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(lens))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        plain = vfa.paged_decode(*args, window, sinks, status=status)
        w = torch.rand(len(lens), hkv, 16 * tables.shape[1], device="cuda")
        old = torch.full_like(w, 3.0)
        w_out = old.clone()
        got = vfa.paged_decode(*args, window, sinks, key_weights=w, key_weights_out=w_out, status=status)
        assert vfa.read_status(status) == 0
        _check_decode((q, k, v, tables), lens, window, sinks, 0.0, got, (w, w_out, old))
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
        same = w.clone()
        vfa.paged_decode(*args, window, sinks, key_weights=same, status=status)
        assert torch.equal(same, torch.where(w_out == 3.0, w, w_out))


def test_decode_of_many_and_of_long_sequences(vfa):
    """Runs that hold many sequences, and sequences cut into many runs, by one workspace."""
    ws = vfa.alloc_paged_decode_workspace(300, 8, 2, 128, capacity=400)
    for lens, window, sinks in (([6000], -1, 0), (list(range(300)), -1, 0), ([5000, 1, 6111], 4000, 20),
                                ([3] * 300, 1, 1), ([6000], -1, 0)):
        k, v, tables, rng = _cache(lens, 2, 128, seed=len(lens))
        q = torch.from_numpy(rng.standard_normal((len(lens), 8, 128))).bfloat16()
        args = (q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(lens))
        w = torch.zeros(len(lens), 2, 16 * tables.shape[1], device="cuda")
        got = vfa.paged_decode(*args, window, sinks, key_weights=w, workspace=ws)
        _check_decode((q, k, v, tables), lens, window, sinks, 0.0, got,
                      (torch.zeros_like(w), w, torch.zeros_like(w)))
        again = vfa.paged_decode(*args, window, sinks, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("group", [65, 72, 130])
def test_decode_weights_of_many_query_heads(vfa, group):
    """More query heads of a kv head than their sums wait in shared memory for."""
    lens = [100, 1, 33]
    k, v, tables, rng = _cache(lens, 2, 64, seed=group)
    q = torch.from_numpy(rng.standard_normal((3, 2 * group, 64))).bfloat16()
    w = torch.rand(3, 2, 16 * tables.shape[1], device="cuda")
    old, w_out = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    got = vfa.paged_decode(q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(lens), 60, 3, key_weights=w,
                           key_weights_out=w_out)
    _check_decode((q, k, v, tables), lens, 60, 3, 0.0, got, (w, w_out, old))


def test_decode_workspace_between_calls_of_all_kinds(vfa):
    """One workspace for many short sequences, for few with long rows and key weights, and again: what
    the one leaves there is never what the other counts with."""
    cases = []
    for lens, weights in (([400 + 7 * i for i in range(40)], False), ([5000], True), ([1300, 9], True),
                          ([60] * 300, True), ([100] * 60, False)):
        k, v, tables, rng = _cache(lens, 2, 64, seed=len(lens))
        q = torch.from_numpy(rng.standard_normal((len(lens), 8, 64))).bfloat16()
        cases.append(((q, k, v, tables), lens, weights))
    size = max(vfa.alloc_paged_decode_workspace(len(lens), 8, 2, 64, c[3].shape[1] if weights else 0).numel()
               for c, lens, weights in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for (q, k, v, tables), lens, weights in cases + cases[::-1]:
        args = (q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(lens))
        w = torch.zeros(len(lens), 2, 16 * tables.shape[1], device="cuda")
        # (the bytes a call asks for, and all there are)
        need = vfa.alloc_paged_decode_workspace(len(lens), 8, 2, 64, tables.shape[1] if weights else 0).numel()
        for n in (need, size):
            nan = torch.full_like(args[0], float("nan"))
            got = vfa.paged_decode(*args, key_weights=w if weights else None, workspace=ws[:n], out=nan)
            _check_decode((q, k, v, tables), lens, -1, 0, 0.0, got)


@pytest.mark.parametrize("scale", [1e-30, 0.01, 1.0, 30.0])
def test_decode_scales(vfa, scale):
    lens = [200, 31]
    k, v, tables, rng = _cache(lens, 2, 128, seed=3, scale=2.0)
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)) * 2).bfloat16()
    got = vfa.paged_decode(q.cuda(), k.cuda(), v.cuda(), _i32(tables), _i32(lens), 100, 4,
                           softmax_scale=scale)
    _check_decode((q, k, v, tables), lens, 100, 4, scale, got)


def test_decode_matches_the_last_row_of_a_prompt(vfa):
    """What the forward with the same mask says of the last token, and the step form without one."""
    lens = [130, 77]
    k, v, tables, rng = _cache(lens, 2, 64, seed=5)
    q = torch.from_numpy(rng.standard_normal((2, 4, 64))).bfloat16().cuda()
    kc, vc = k.cuda(), v.cuda()
    out, lse = vfa.paged_decode(q, kc, vc, _i32(tables), _i32(lens), 20, 3)
    rows = [torch.cat([p[tables[s, j // 16], j % 16][None] for j in range(lens[s])]) for p in (kc, vc)
            for s in range(2)]
    cu = _i32([0, 130, 207])
    o2, l2 = vfa.varlen_fwd(q, torch.cat(rows[:2]), torch.cat(rows[2:]), _i32([0, 1, 2]), cu, 1, 0.125,
                            2, window_left=20, sink_tokens=3)
    assert (out.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * vc[~vc.isnan()].abs().max()
    assert (lse - l2).abs().max() < 1e-5


def test_decode_bad_pages_and_counts(vfa):
    lens = [40, 100, 33, 64]
    k, v, tables, rng = _cache(lens, 2, 64, seed=7)
    q = torch.from_numpy(rng.standard_normal((4, 4, 64))).bfloat16().cuda()
    good = vfa.paged_decode(q, k.cuda(), v.cuda(), _i32(tables), _i32(lens), 30, 2)
    tables[1, 5], tables[3, 3] = k.shape[0], -5
    tables[2, 1] = 1 << 30                       # between the sinks and the window: not read
    lens[0] = 16 * tables.shape[1] + 1
    out, lse = torch.full_like(q, 7.0), torch.full((4, 4), 7.0, device="cuda")
    w = torch.full((4, 2, 16 * tables.shape[1]), 7.0, device="cuda")
    ws = vfa.alloc_paged_decode_workspace(4, 4, 2, 64, capacity=tables.shape[1])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens[2] = 64
    tables[2, 3] = tables[2, 2] = tables[2, 0]
    for _ in range(2):                           # the tickets are left as they have to be
        vfa.paged_decode(q, k.cuda(), v.cuda(), _i32(tables), _i32(lens), 30, 2, key_weights=w, out=out,
                         lse=lse, workspace=ws, status=status)
    assert vfa.read_status(status) == vfa.VFA_ERR_BAD_BLOCK
    for s in (0, 1, 3):
        assert (out[s] == 7.0).all() and (lse[s] == 7.0).all() and (w[s] == 7.0).all()
    assert (out[2] != 7.0).any() and good[0].shape == out.shape


# ------------------------------------------------------------------ key weights of prompts

def _prompt(lq, lk, hq, hkv, d, seed):
    c = W.make_varlen("prompt", lq, lk, hq, d, True, 1.0, seed)
    c.k = W.bf16_normal((c.total_k, hkv, d), 1.0, torch.Generator().manual_seed(seed + 1))
    return c


def _key_weights(vfa, c, hkv, causal, window, sinks, extra=5):
    rng = np.random.default_rng(c.total_q)
    zero = np.zeros(c.k.shape)
    _, lse, _, _ = O.varlen_fwd(_f64(c.q), _f64(c.k), zero, c.cu_seqlens_q, c.cu_seqlens_k,
                                c.softmax_scale, causal, window, sinks)
    lse32 = torch.from_numpy(lse).float()
    w = torch.from_numpy(rng.random((c.batch, hkv, max(c.lengths_k) + extra))).float()
    old = torch.full_like(w, 9.0).cuda()
    ws = vfa.alloc_key_weights_workspace(c.batch, c.total_q, c.total_k, c.max_seqlen_q, c.num_heads)
    args = (c.q.cuda(), c.k.cuda(), lse32.cuda(), torch.from_numpy(c.cu_seqlens_q).cuda(),
            torch.from_numpy(c.cu_seqlens_k).cuda(), c.max_seqlen_q, c.softmax_scale, causal, w.cuda())
    got = vfa.varlen_key_weights(*args, window_left=window, sink_tokens=sinks, key_weights_out=old,
                                 workspace=ws)
    assert vfa.read_status(ws) == 0 and got is old
    again = vfa.varlen_key_weights(*args, window_left=window, sink_tokens=sinks, workspace=ws)
    want, dot = O.key_weights(_f64(c.q), _f64(c.k), _f64(lse32), c.cu_seqlens_q, c.cu_seqlens_k,
                              c.softmax_scale, causal, window, sinks, _f64(w))
    g, w64 = _f64(got), _f64(w)
    for b, n in enumerate(c.lengths_k):
        assert np.all(g[b, :, n:] == 9.0) and np.all(_f64(again)[b, :, n:] == w64[b, :, n:])
        m = c.lengths_q[b] * c.num_heads // hkv + 2
        live = np.abs(lse[lse != -FLT_MAX]).max() if (lse != -FLT_MAX).any() else 0.0
        dx = (c.head_dim + 16) * U * dot[b, :, :n] + 2.0 ** -22 * live
        bound = (np.expm1(dx) + m * U + 2.0 ** -19) * (want - w64)[b, :, :n] + 2.0 ** -23 * want[b, :, :n]
        err = np.abs(g[b, :, :n] - want[b, :, :n])
        assert np.all(err <= bound), (err / bound).max()
        assert np.array_equal(g[b, :, :n], _f64(again)[b, :, :n])


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 2, 2), (256, 3, 1)])
@pytest.mark.parametrize("causal,window,sinks", [(0, -1, 0), (1, -1, 0), (2, -1, 3), (1, 0, 0), (2, 31, 65),
                                                 (1, 200, 130), (2, 128, 4)])
def test_key_weights(vfa, d, hq, hkv, causal, window, sinks):
    for i, (lq, lk) in enumerate([([1, 0, 5, 129], [1, 3, 0, 129]), ([300], [300]), ([257, 64], [511, 64]),
                                  ([400, 130], [90, 17]), ([40, 200], [700, 33])]):
        _key_weights(vfa, _prompt(lq, lk, hq, hkv, d, 7 * i + d), hkv, causal, window, sinks)


def test_key_weights_of_many_blocks(vfa):
    """Units of several chunks, and enough of them for long chunks."""
    _key_weights(vfa, _prompt([2300, 1100], [2300, 1100], 2, 1, 64, 1), 1, 1, -1, 0)
    _key_weights(vfa, _prompt([1500], [1500], 64, 8, 64, 2), 8, 1, -1, 0)


@pytest.mark.parametrize("scale", [0.0, 1e-45, 1e-30, 1.0])
@pytest.mark.parametrize("d,causal,window,sinks", [(64, 1, -1, 0), (128, 0, -1, 0), (128, 2, 31, 65),
                                                   (256, 1, 40, 3)])
def test_key_weights_scales(vfa, d, causal, window, sinks, scale):
    """Also a scale of zero: every key that a query sees gets the same weight, hidden ones none."""
    c = _prompt([257, 64, 5], [511, 64, 9], 4, 2, d, 11)
    c.softmax_scale = scale
    _key_weights(vfa, c, 2, causal, window, sinks)


def test_key_weights_of_hidden_queries_that_are_no_numbers(vfa):
    """A query that is NaN, or whose lse is, changes the keys that it sees and no others."""
    for d, bad_q, value in ((64, True, np.nan), (128, False, np.nan), (256, False, np.nan),
                            (128, False, np.inf), (64, False, -np.inf)):
        c = _prompt([300, 70], [300, 70], 2, 1, d, d)
        cq = torch.from_numpy(c.cu_seqlens_q).cuda()
        lse = torch.full((370, 2), 3.0, device="cuda")
        q, k = c.q.cuda(), c.k.cuda()
        call = lambda: vfa.varlen_key_weights(q, k, lse, cq, cq, 300, c.softmax_scale, 1,
                                              torch.zeros(2, 1, 300, device="cuda"), window_left=40,
                                              sink_tokens=3)
        good = call()
        if bad_q:
            q[200] = value
        else:
            lse[200] = value
        got = call()
        sees = torch.zeros_like(good, dtype=torch.bool)
        sees[0, 0, :3] = sees[0, 0, 160:201] = True
        assert torch.equal(got[~sees], good[~sees])
        if value != value:
            assert got[sees].isnan().all()


def test_key_weights_sum_to_the_queries(vfa):
    """With the forward's own lse every query spends a weight of one per head."""
    c = _prompt([700, 90], [700, 90], 8, 2, 128, 3)
    c.v = W.bf16_normal(c.k.shape, 1.0, torch.Generator().manual_seed(4))
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    cq = torch.from_numpy(c.cu_seqlens_q).cuda()
    _, lse = vfa.varlen_fwd(q, k, v, cq, cq, 700, c.softmax_scale, 1, window_left=64, sink_tokens=4)
    w = vfa.varlen_key_weights(q, k, lse, cq, cq, 700, c.softmax_scale, 1,
                               torch.zeros(2, 2, 700, device="cuda"), window_left=64, sink_tokens=4)
    assert np.allclose(_f64(w).sum(-1), [[2800, 2800], [360, 360]], rtol=1e-5)


def test_key_weights_by_one_workspace(vfa):
    """A workspace for the largest call, whose chunks are long ones, in smaller ones of either length of
    chunk and of longer chunks still; none writes past the bytes it asks for.  Against sums over
    every query in 64 bits, for some of the keys."""
    hq, hkv, d, scale = 8, 2, 64, 0.125
    calls = [([140000], [19700]), ([9000, 20000], [12000, 7700]), ([300, 5], [19456, 3]), ([140000], [700]),
             ([2000], [2000]), ([17, 0, 129], [400, 3, 129])]
    ws = vfa.alloc_key_weights_workspace(3, 140000, 19700, 140000, hq)
    for i, (lq, lk) in enumerate(calls + calls[::-1]):
        gen = torch.Generator(device="cuda").manual_seed(i)
        q, k = (torch.randn(sum(n), h, d, device="cuda", generator=gen).bfloat16() for n, h in ((lq, hq), (lk, hkv)))
        lse = 11.0 + torch.rand(sum(lq), hq, device="cuda", generator=gen)
        cq, ck = W.cu_seqlens(lq), W.cu_seqlens(lk)
        need = vfa.lib().vfa_varlen_key_weights_workspace_bytes(len(lq), sum(lq), sum(lk), max(lq), hq)
        assert need <= ws.numel()
        ws.fill_(0xff)
        got = vfa.varlen_key_weights(q, k, lse, _i32(cq), _i32(ck), max(lq), scale, 0,
                                     torch.zeros(len(lq), hkv, max(lk), device="cuda"), workspace=ws[:need])
        assert vfa.read_status(ws) == 0 and (ws[need:] == 0xff).all()
        for b in range(len(lq)):
            at = torch.randint(0, lk[b], (40,), device="cuda", generator=gen)
            for h in range(hkv):
                qb = q[cq[b]:cq[b + 1], 4 * h:4 * h + 4].double().reshape(-1, d)
                kb = k[ck[b] + at, h].double()
                x = qb @ kb.T * scale
                p = torch.exp(x - lse[cq[b]:cq[b + 1], 4 * h:4 * h + 4].double().reshape(-1, 1)).sum(0)
                dx = (d + 16) * U * float((qb.abs() @ kb.abs().T).amax() if len(qb) else 0) * scale + 2.0 ** -22 * 12
                bound = (np.expm1(dx) + (len(qb) + 2) * U + 2.0 ** -19) * p
                assert ((got[b, h, at].double() - p).abs() <= bound).all()


def test_key_weights_refuse_bad_lengths(vfa):
    c = _prompt([64, 64], [64, 64], 2, 2, 64, 1)
    q, k = c.q.cuda(), c.k.cuda()
    lse = torch.zeros(128, 2, device="cuda")
    w = torch.full((2, 2, 64), 7.0, device="cuda")
    good = torch.from_numpy(c.cu_seqlens_q).cuda()
    for cq, ck, most, row in ((_i32([0, 100, 90]), good, 128, w), (good, _i32([0, -5, 128]), 128, w),
                              (good, good, 63, w), (good, good, 64, w[:, :, :63].contiguous())):
        ws = vfa.alloc_key_weights_workspace(2, 128, 128, most, 2).fill_(0xff)
        vfa.varlen_key_weights(q, k, lse, cq, ck, most, 0.1, 1, row, workspace=ws)
        assert vfa.read_status(ws) == vfa.VFA_ERR_BAD_SEQLENS and (row == 7.0).all()


# ------------------------------------------------------------------ eviction, truncation

def _evict_case(lens, hkv, d, seed, known=None, gone=None, spare=2):
    rng = np.random.default_rng(seed)
    tables, blocks = _tables(lens, rng, spare=spare)
    refs = np.zeros(blocks, dtype=np.int32)
    for s, n in enumerate(lens):
        refs[tables[s, :-(-n // 16)]] = 1
    rows = (len(lens), hkv, 16 * tables.shape[1])
    pools = [torch.from_numpy(rng.standard_normal((blocks, 16, hkv, d))).bfloat16() for _ in range(2)]
    # few values: ties everywhere
    weights = rng.integers(0, 5, rows).astype(np.float32) * rng.choice([1.0, -1.0, 0.0], rows)
    known = [0] * len(lens) if known is None else known
    gone = [0] * len(lens) if gone is None else gone
    positions = np.full(rows, -7, dtype=np.int32)
    for s in range(len(lens)):
        for h in range(hkv):
            positions[s, h, :known[s]] = rng.permutation(known[s] + gone[s])[:known[s]]
    history = np.stack((known, gone), 1).astype(np.int32)
    return pools, refs, tables, weights.astype(np.float32), positions, history


def _check_evict(vfa, case, lens, budgets, sinks, recent, in_place):
    (k, v), refs, tables, weights, positions, history = case
    kept, hist, moves, state, refused = O.evict(refs, tables, lens, budgets, weights.astype(np.float64),
                                                positions, history, sinks, recent)
    pools = [k.cuda(), v.cuda()]
    w, p, h = torch.from_numpy(weights).cuda(), _i32(positions), _i32(history)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = {}
    if not in_place:
        outs = {"key_weights_out": torch.full_like(w, 11.0), "positions_out": torch.full_like(p, 11),
                "history_out": torch.full_like(h, 11)}
    got = vfa.cache_evict(*pools, _i32(refs), _i32(tables), _i32(lens), _i32(budgets), w, p, h, sinks,
                          recent, status=status, **outs)
    assert vfa.read_status(status) == (vfa.VFA_ERR_BAD_BLOCK if refused else 0)
    assert np.array_equal(got.cpu().numpy(), kept)
    ow, op, oh = (outs[x] if outs else y for x, y in
                  (("key_weights_out", w), ("positions_out", p), ("history_out", h)))
    assert np.array_equal(oh.cpu().numpy(), hist)
    want_pools = [x.clone() for x in (k, v)]
    for s, hd, frm, to in moves:
        for x, src in zip(want_pools, (k, v)):
            x[tables[s, to // 16], to % 16, hd] = src[tables[s, frm // 16], frm % 16, hd]
    assert all(torch.equal(a.cpu(), b) for a, b in zip(pools, want_pools))
    want_w = weights.copy() if in_place else np.full(weights.shape, 11.0)
    want_p = positions.copy() if in_place else np.full(positions.shape, 11)
    for (s, hd), (ww, pp) in state.items():
        b = kept[s]
        want_w[s, hd, :b], want_p[s, hd, :b] = ww, pp
        want_w[s, hd, b:lens[s]] = 0
    assert np.array_equal(ow.cpu().numpy(), want_w) and np.array_equal(op.cpu().numpy(), want_p)
    return got


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 2), (256, 1)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (1, 5), (4, 100), (1000, 1000)])
def test_evict(vfa, in_place, d, hkv, sinks, recent):
    lens = [1, 0, 17, 40, 300, 64, 33]
    for budgets in ([0] * 7, [1] * 7, [16, 3, 16, 16, 150, 63, 32], [-1, 5, 17, 39, 299, 400, 31]):
        _check_evict(vfa, _evict_case(lens, hkv, d, sum(budgets) + d), lens, budgets, sinks, recent,
                     in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_again(vfa, in_place):
    """Rows that were cut before: stored positions, in no order, and tokens appended since."""
    lens = [50, 300, 31, 129]
    case = _evict_case(lens, 2, 64, 3, known=[40, 200, 31, 0], gone=[7, 1000, 3, 0], spare=1)
    _check_evict(vfa, case, lens, [30, 128, 20, 100], 4, 16, in_place)


def test_evict_long_rows(vfa):
    lens = [5000, 2049, 1024]
    _check_evict(vfa, _evict_case(lens, 2, 64, 4), lens, [1000, 2048, 100], 4, 64, True)


@pytest.mark.parametrize("budgets", [[20000, 10000, 60000], [32999, 30001, 35001], [1, 0, 40000]])
def test_evict_rows_past_shared_memory(vfa, budgets):
    """More slots than the CTAs of a cluster keep the keys of: they wait where the lists of moves go."""
    lens = [33000, 40000, 70001]
    case = _evict_case(lens, 1, 64, 8, known=[0, 39000, 500], gone=[0, 5, 77])
    _check_evict(vfa, case, lens, budgets, 4, 100, True)


def test_evict_orders_every_float(vfa):
    lens = [64]
    case = _evict_case(lens, 1, 64, 5)
    special = [np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0, np.nextafter(np.float32(1), 2)]
    case[3][0, 0, :64] = np.resize(np.array(special, dtype=np.float32), 64)
    for b in (1, 7, 8, 20, 33, 50):
        _check_evict(vfa, case, lens, [b], 0, 0, True)
    # NaN counts as the largest
    case[3][0, 0, 40:43] = [np.nan, -np.nan, np.inf]
    w = torch.from_numpy(case[3]).cuda()
    h, p = _i32(case[5]), _i32(case[4])
    vfa.cache_evict(case[0][0].cuda(), case[0][1].cuda(), _i32(case[1]), _i32(case[2]), _i32(lens), _i32([2]),
                    w, p, h)
    assert sorted(p[0, 0, :2].tolist()) == [40, 41]


def test_evict_positions_that_name_too_many(vfa):
    lens = [64, 64]
    case = list(_evict_case(lens, 2, 64, 6, known=[64, 64], gone=[5, 5]))
    case[4][0] = 0                               # every token of row 0 says it is the first
    _check_evict(vfa, case, lens, [20, 20], 3, 4, True)


def test_evict_refuses_shared_and_bad_pages(vfa):
    lens = [64, 64, 64, 64, 64, 64]
    case = list(_evict_case(lens, 2, 64, 7))
    refs, tables = case[1], case[2]
    refs[tables[0, 0]] = 2                       # written by a cut to 20
    refs[tables[1, 3]] = 2                       # only read by it
    tables[2, 1], tables[3, 3] = -1, len(refs)
    refs[tables[4, 0]] = 2                       # not written where nothing goes
    _check_evict(vfa, case, lens, [20, 20, 20, 20, 64, 20], 0, 0, False)
    case[5][5] = (65, 0)                         # more positions than tokens
    _check_evict(vfa, case, lens, [20, 20, 20, 20, 64, 20], 0, 0, True)


@pytest.mark.parametrize("in_place", [True, False])
def test_truncate(vfa, in_place):
    tables = np.array([[0, 1, 2, 9], [1, 3, -1, 9], [4, 5, 6, 7], [4, -1, 99, 8], [8, 8, 8, 8]], dtype=np.int32)
    refs = np.array([1, 2, 1, 1, 2, 1, 1, 1, 0, 1], dtype=np.int32)
    counts = [40, 20, 64, 60, 65]
    for new in ([16, 17, 0, 16, 3], [31, 3, 64, 5, -1], [40, 21, 33, 0, 0], [-1, -9, 1, 48, 10]):
        want_r, want_c, bad = O.truncate(refs, tables, counts, new, 16)
        r, c = _i32(refs), _i32(counts)
        outs = {} if in_place else {"refcounts_out": torch.full_like(r, 7), "token_counts_out": c.clone()}
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        vfa.pages_truncate(r, _i32(tables), c, _i32(new), 16, status=status, **outs)
        assert np.array_equal((r if in_place else outs["refcounts_out"]).cpu().numpy(), want_r)
        assert np.array_equal((c if in_place else outs["token_counts_out"]).cpu().numpy(), want_c)
        assert vfa.read_status(status) == (vfa.VFA_ERR_BAD_BLOCK if bad else 0)


def test_truncate_many_rows(vfa):
    """More rows and pages than one CTA takes."""
    rng = np.random.default_rng(3)
    S, cap, blocks = 1200, 40, 30000
    counts = rng.integers(0, 16 * cap + 1, S)
    tables = rng.integers(0, blocks, (S, cap)).astype(np.int32)
    refs = np.zeros(blocks, dtype=np.int32)
    for s in range(S):
        np.add.at(refs, tables[s, :-(-counts[s] // 16)], 1)
    new = np.minimum(counts, rng.integers(-1, 16 * cap, S))
    want_r, want_c, bad = O.truncate(refs, tables, counts, new, 16)
    for in_place in (True, False):
        r, c = _i32(refs), _i32(counts)
        outs = {} if in_place else {"refcounts_out": torch.full_like(r, 7), "token_counts_out": c.clone()}
        vfa.pages_truncate(r, _i32(tables), c, _i32(new), 16, **outs)
        assert np.array_equal((r if in_place else outs["refcounts_out"]).cpu().numpy(), want_r)
        assert np.array_equal((c if in_place else outs["token_counts_out"]).cpu().numpy(), want_c)


# ------------------------------------------------------------------ together

def test_a_bounded_cache_in_use(vfa):
    """Prompts, their key weights, cut to a budget; then steps that append, attend, count the weights
    and cut again: against a cache that is kept as plain lists."""
    rng = np.random.default_rng(1)
    d, hq, hkv, cap, budget, sinks, recent = 64, 4, 2, 12, 60, 2, 10
    lens = [150, 37, 101]
    S, blocks = len(lens), 40
    dev = "cuda"
    refs = torch.zeros(blocks, dtype=torch.int32, device=dev)
    tables = torch.full((S, cap), -1, dtype=torch.int32, device=dev)
    counts, status = _i32([0] * S), _i32([0])
    pws = vfa.alloc_pages_workspace(blocks, S)
    pools = [torch.full((blocks, 16, hkv, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    weights = torch.zeros(S, hkv, 16 * cap, device=dev)
    positions = torch.zeros(S, hkv, 16 * cap, dtype=torch.int32, device=dev)
    history = torch.zeros(S, 2, dtype=torch.int32, device=dev)
    budgets = _i32([budget] * S)
    T = sum(lens)
    q, k, v = (torch.from_numpy(rng.standard_normal((T, h, d))).bfloat16() for h in (hq, hkv, hkv))
    cu = W.cu_seqlens(lens)
    vfa.pages_extend(refs, tables, counts, _i32(lens), 16, pws, status=status)

    def put(s, slot, kk, vv):
        page = tables[s, slot // 16]
        pools[0][page, slot % 16], pools[1][page, slot % 16] = kk.cuda(), vv.cuda()

    cache = [[[] for _ in range(hkv)] for _ in range(S)]    # slots: position, k, v, weight
    for s in range(S):
        for j in range(lens[s]):
            put(s, j, k[cu[s] + j], v[cu[s] + j])
    out, lse = vfa.varlen_fwd(q.cuda(), k.cuda(), v.cuda(), _i32(cu), _i32(cu), max(lens), d ** -0.5, 1)
    vfa.varlen_key_weights(q.cuda(), k.cuda(), lse, _i32(cu), _i32(cu), max(lens), d ** -0.5, 1, weights)
    want, _ = O.key_weights(_f64(q), _f64(k), _f64(lse), cu, cu, d ** -0.5, 1, -1, 0,
                            np.zeros(weights.shape))
    assert np.allclose(_f64(weights), want, rtol=1e-4, atol=1e-6)
    w_now = _f64(weights)                        # ties aside, cuts go by what the device holds
    for s in range(S):
        for h in range(hkv):
            for j in range(lens[s]):
                cache[s][h].append([j, _f64(k[cu[s] + j, h]), _f64(v[cu[s] + j, h])])
    seen = list(lens)

    def cut():
        w_now = _f64(weights)
        n_now = counts.tolist()
        kept = vfa.cache_evict(*pools, refs, tables, counts, budgets, weights, positions, history, sinks,
                               recent, status=status)
        vfa.pages_truncate(refs, tables, counts, kept, 16, status=status)
        for s in range(S):
            n = n_now[s]
            b = min(n, budget)
            for h in range(hkv):
                c = cache[s][h]
                safe = lambda x: x[0] < sinks or x[0] >= seen[s] - recent
                order = sorted(range(n), key=lambda j: (not safe(c[j]), -w_now[s, h, j], j))
                keep = set(order[:b])
                movers = [j for j in range(b, n) if j in keep]
                for to, frm in zip([j for j in range(b) if j not in keep], movers):
                    c[to] = c[frm]
                del c[b:]
                assert positions[s, h, :b].tolist() == [x[0] for x in c]
        assert counts.tolist() == [min(n, budget) for n in n_now]
        assert int(refs.sum()) == sum(-(-n // 16) for n in counts.tolist())

    cut()
    for step in range(40):
        vfa.pages_extend(refs, tables, counts, _i32([1] * S), 16, pws, status=status)
        nq, nk, nv = (torch.from_numpy(rng.standard_normal((S, h, d))).bfloat16() for h in (hq, hkv, hkv))
        for s in range(S):
            put(s, int(counts[s]) - 1, nk[s], nv[s])
            for h in range(hkv):
                cache[s][h].append([seen[s], _f64(nk[s, h]), _f64(nv[s, h])])
            seen[s] += 1
        before = _f64(weights)
        out, _ = vfa.paged_decode(nq.cuda(), *pools, tables, counts, key_weights=weights, status=status)
        for s in range(S):
            for h in range(hq):
                c = cache[s][h // 2]
                x = np.stack([e[1] for e in c]) @ _f64(nq[s, h]) * d ** -0.5
                p = np.exp(x - x.max())
                ref = p @ np.stack([e[2] for e in c]) / p.sum()
                assert np.abs(_f64(out[s, h]) - ref).max() < 0.04      # 2^-8 (sum p|v| + |out|), |v| < 5
        grown = _f64(weights) - before
        assert np.allclose(grown.sum(-1), hq // hkv, rtol=1e-4)
        if step % 13 == 12:
            cut()
    assert vfa.read_status(status) == 0


def test_steps_in_a_graph_and_on_another_stream(vfa):
    """A step of decode with weights, eviction and truncation captured and replayed, and the same
    calls on a stream of their own."""
    lens = [300, 64, 129]
    (k, v), refs, tables, weights, positions, history = _evict_case(lens, 2, 128, 9)
    rng = np.random.default_rng(2)
    q = torch.from_numpy(rng.standard_normal((3, 8, 128))).bfloat16().cuda()
    start = [k.cuda(), v.cuda(), _i32(refs), _i32(lens), torch.from_numpy(np.abs(weights)).cuda(),
             _i32(positions), _i32(history)]
    state = [t.clone() for t in start]
    t, b = _i32(tables), _i32([100, 64, 100])
    ws = vfa.alloc_paged_decode_workspace(3, 8, 2, 128, capacity=tables.shape[1])
    ews = vfa.alloc_evict_workspace(3, 2, tables.shape[1])

    def step(stream=None):
        kp, vp, r, c, w, p, h = state
        out, lse = vfa.paged_decode(q, kp, vp, t, c, key_weights=w, workspace=ws, stream=stream)
        kept = vfa.cache_evict(kp, vp, r, t, c, b, w, p, h, 2, 20, workspace=ews, stream=stream)
        vfa.pages_truncate(r, t, c, kept, 16, stream=stream)
        return out, lse

    def reset():
        for x, y in zip(state, start):
            x.copy_(y)

    want_out = [x.clone() for x in step()]
    want = [x.clone() for x in state]
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, state))
    assert all(torch.equal(a, c) for a, c in zip(want_out, got))
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, state))
        assert all(torch.equal(a, c) for a, c in zip(want_out, got))


def test_offsets_past_32_bits(vfa):
    """Pages past 2^32 bytes of a pool, and slots past 2^31 of all rows: as in a small cache."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    hkv, d, lens, shift, cap = 2, 64, [40, 0, 3, 0, 100], 1_200_000, 1 << 24
    k, v, tables, rng = _cache(lens, hkv, d, seed=11)
    q = torch.from_numpy(rng.standard_normal((5, 4, d))).bfloat16().cuda()
    blocks = k.shape[0]
    results = []
    for far in (False, True):
        t = _i32(tables)
        pools = [x.cuda() for x in (k, v)]
        refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        if far:
            pools = [torch.zeros(shift + blocks, 16, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for x, y in zip(pools, (k, v)):
                x[shift:] = y.cuda()
            refs = torch.zeros(shift + blocks, dtype=torch.int32, device="cuda")
            t = torch.full((5, cap), -1, dtype=torch.int32, device="cuda")
            t[:, :tables.shape[1]] = torch.where(_i32(tables) < 0, -1, _i32(tables) + shift)
        refs[-blocks:] = 1
        rows = (5, hkv, 16 * t.shape[1])
        w = torch.zeros(rows, device="cuda")
        p = torch.zeros(rows, dtype=torch.int32, device="cuda")
        h = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
        n = _i32(lens)
        out, lse = vfa.paged_decode(q, *pools, t, n, key_weights=w)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kept = vfa.cache_evict(*pools, refs, t, n, _i32([16, 0, 2, 5, 70]), w, p, h, 2, 8, status=status)
        vfa.pages_truncate(refs, t, n, kept, 16, status=status)
        assert vfa.read_status(status) == 0
        results.append((out, lse, kept, h, n, w[:, :, :112].clone(), p[:, :, :112].clone(), refs[-blocks:].clone(),
                        *(x[-blocks:].nan_to_num() for x in pools)))
        assert not w[:, :, 112:].any() and not p[:, :, 112:].any()
        del pools, w, p, t, refs
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*results))
