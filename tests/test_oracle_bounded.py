"""The 64-bit definitions of the bounded cache's operators against each other and against
differences (CPU)."""
import numpy as np
import pytest

import oracle
import oracle.bounded as O


def _inputs(lq, lk, hq, hkv, d, seed):
    rng = np.random.default_rng(seed)
    cu = lambda x: np.concatenate(([0], np.cumsum(x)))
    q, do = (rng.standard_normal((sum(lq), hq, d)) for _ in range(2))
    k, v = (rng.standard_normal((sum(lk), hkv, d)) for _ in range(2))
    return q, k, v, do, cu(lq), cu(lk)


@pytest.mark.parametrize("causal", [1, 2])
@pytest.mark.parametrize("window,sinks", [(-1, 5), (3, 0), (0, 1), (2, 4), (100, 3)])
def test_mask(causal, window, sinks):
    for lq, lk in ((5, 9), (9, 5), (1, 1), (7, 7)):
        m = O.visible(lq, lk, causal, window, sinks)
        off = lk - lq if causal == 2 else 0
        for i in range(lq):
            want = {j for j in range(lk) if j <= i + off}
            if window >= 0:
                want = {j for j in want if j >= i + off - window} | {j for j in want if j < sinks}
            assert set(np.flatnonzero(m[i])) == want


def test_forward_without_sinks_is_the_other_oracle():
    import torch
    q, k, v, _, cq, ck = _inputs([5, 0, 33], [7, 2, 33], 2, 2, 64, 0)
    t = [torch.from_numpy(x).bfloat16() for x in (q, k, v)]
    ref, lse, _ = oracle.varlen_fwd(*t, cq.astype(np.int32), ck.astype(np.int32), 2, 64, 0.3, 1,
                                    window_left=4)
    got, glse, _, _ = O.varlen_fwd(*(x.double().numpy() for x in t), cq, ck, 0.3, 1, 4, 0)
    assert np.allclose(got, ref, atol=1e-12) and np.allclose(glse, lse, atol=1e-12)


@pytest.mark.parametrize("causal,window,sinks", [(1, 3, 2), (2, 2, 3), (1, 0, 1)])
def test_gradients_against_differences(causal, window, sinks):
    args = _inputs([6, 4], [8, 4], 4, 2, 3, 1)
    q, k, v, do, cq, ck = args
    loss = lambda: float((do * O.varlen_fwd(q, k, v, cq, ck, 0.7, causal, window, sinks)[0]).sum())
    grads = O.varlen_bwd(q, k, v, do, cq, ck, 0.7, causal, window, sinks)
    rng, h = np.random.default_rng(2), 1e-5
    for x, g in zip((q, k, v), grads):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in x.shape)
            old = x[at]
            x[at] = old + h
            up = loss()
            x[at] = old - h
            down = loss()
            x[at] = old
            assert abs((up - down) / (2 * h) - g[at]) < 1e-8


def test_key_weights_are_the_column_sums():
    q, k, v, _, cq, ck = _inputs([6, 4], [8, 4], 4, 2, 3, 3)
    _, lse, _, _ = O.varlen_fwd(q, k, v, cq, ck, 0.7, 2, 3, 1)
    w, _ = O.key_weights(q, k, lse, cq, ck, 0.7, 2, 3, 1, np.zeros((2, 2, 9)))
    assert np.allclose(w.sum(-1), [[12, 12], [8, 8]])        # a row's weights sum to one


def test_decode_is_the_last_row():
    rng = np.random.default_rng(4)
    d, hq, hkv, n, page = 4, 4, 2, 37, 16
    pools = [rng.standard_normal((5, page, hkv, d)) for _ in range(2)]
    table = np.array([[3, 0, 4]])
    q = rng.standard_normal((n, hq, d))
    k, v = (p[table[0]].reshape(-1, hkv, d)[:n] for p in pools)
    cu = [0, n]
    ref, lse, _, _ = O.varlen_fwd(q, k, v, cu, cu, 0.5, 1, 9, 2)
    out, l2, _, _, got = O.paged_decode(q[-1:], *pools, table, [n], 9, 2, 0.5)
    assert np.allclose(out[0], ref[-1]) and np.allclose(l2[0], lse[-1])
    assert np.allclose(got.sum(-1), hq // hkv) and (got[0, :, 2:27] == 0).all()


def test_evict_keeps_what_it_says():
    w = np.array([[[5., 1., 9., 9., 0., 7., 3., 2.]]])
    kept, hist, moves, state, bad = O.evict([1], np.array([[0]]), [8], [5], w,
                                            np.zeros((1, 1, 16), int), [[0, 0]], 1, 2)
    # slot 0 (sink), 6 and 7 (recent), then 9 and 9
    assert kept[0] == 5 and list(hist[0]) == [5, 3] and not bad
    assert moves == [(0, 0, 6, 1), (0, 0, 7, 4)]
    assert list(state[0, 0][1]) == [0, 6, 2, 3, 7]
    # a second eviction knows where its tokens came from
    pos = np.zeros((1, 1, 16), int)
    pos[0, 0, :5] = state[0, 0][1]
    w2 = np.array([[[1., 1., 5., 1., 1., 1.]]])
    kept, hist, moves, state, bad = O.evict([1], np.array([[0]]), [6], [3], w2, pos, hist, 1, 1)
    assert list(state[0, 0][1]) == [0, 8, 2] and list(hist[0]) == [3, 6]


def test_truncate():
    tables = np.array([[0, 1, 2], [1, 3, -1]])
    refs, counts, bad = O.truncate([1, 2, 1, 1], tables, [40, 20], [16, 17], 16)
    assert list(refs) == [1, 1, 0, 1] and list(counts) == [16, 17] and not bad
    refs, counts, bad = O.truncate([1, 2, 1, 1], tables, [40, 20], [31, 3], 16)
    assert list(counts) == [40, 20] and bad == [0, 1]
