"""Oracle of the operators of a bounded cache -- TEST INFRASTRUCTURE ONLY.

Plain 64-bit statements of attention with a window and sinks (forward and
gradients), one-token decode over a paged cache, the accumulated weights of
keys, eviction by them, and truncation.  No code is shared with the library.
"""
from __future__ import annotations

import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def visible(lq, lk, causal, window_left, sink_tokens):
    """bool [lq, lk]: which keys a query sees (local positions)."""
    off = lk - lq if causal == 2 else 0
    i, j = np.arange(lq)[:, None] + off, np.arange(lk)[None, :]
    out = np.ones((lq, lk), dtype=bool)
    if causal:
        out &= j <= i
        if window_left >= 0:
            out &= (j >= i - window_left) | (j < sink_tokens)
    return out


def _sequences(cu_q, cu_k):
    for b in range(len(cu_q) - 1):
        yield b, slice(int(cu_q[b]), int(cu_q[b + 1])), slice(int(cu_k[b]), int(cu_k[b + 1]))


def varlen_fwd(q, k, v, cu_q, cu_k, scale, causal, window_left, sink_tokens):
    """(out, lse, sum |q k| scale of the worst visible key per row, sum p |v|) in float64."""
    hq, hkv = q.shape[1], k.shape[1]
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, dot = np.full(q.shape[:2], -FLT_MAX), np.zeros(q.shape[:2])
    for _, sq, sk in _sequences(cu_q, cu_k):
        vis = visible(sq.stop - sq.start, sk.stop - sk.start, causal, window_left, sink_tokens)
        for h in range(hq):
            kh = h // (hq // hkv)
            x = q[sq, h] @ k[sk, kh].T * scale
            a = np.abs(q[sq, h]) @ np.abs(k[sk, kh]).T * scale
            for i in range(x.shape[0]):
                js = np.flatnonzero(vis[i])
                if not len(js):
                    continue
                m = x[i, js].max()
                p = np.exp(x[i, js] - m)
                lse[sq.start + i, h] = m + math.log(p.sum())
                out[sq.start + i, h] = p @ v[sk, kh][js] / p.sum()
                absv[sq.start + i, h] = p @ np.abs(v[sk, kh][js]) / p.sum()
                dot[sq.start + i, h] = a[i, js].max()
    return out, lse, dot, absv


def varlen_bwd(q, k, v, dout, cu_q, cu_k, scale, causal, window_left, sink_tokens):
    """(dq, dk, dv): the derivative of sum(dout * out)."""
    hq, hkv = q.shape[1], k.shape[1]
    out, lse, _, _ = varlen_fwd(q, k, v, cu_q, cu_k, scale, causal, window_left, sink_tokens)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for _, sq, sk in _sequences(cu_q, cu_k):
        vis = visible(sq.stop - sq.start, sk.stop - sk.start, causal, window_left, sink_tokens)
        for h in range(hq):
            kh = h // (hq // hkv)
            x = q[sq, h] @ k[sk, kh].T * scale
            p = np.where(vis, np.exp(np.where(vis, x - lse[sq, h][:, None], 0.0)), 0.0)
            dp = dout[sq, h] @ v[sk, kh].T
            ds = p * (dp - (dout[sq, h] * out[sq, h]).sum(-1, keepdims=True))
            dv[sk, kh] += p.T @ dout[sq, h]
            dq[sq, h] = ds @ k[sk, kh] * scale
            dk[sk, kh] += ds.T @ q[sq, h] * scale
    return dq, dk, dv


def key_weights(q, k, lse, cu_q, cu_k, scale, causal, window_left, sink_tokens, weights):
    """(weights + what each key got, sum |q k| scale of the worst pair of every key)."""
    hq, hkv = q.shape[1], k.shape[1]
    out, dot = weights.copy(), np.zeros(weights.shape)
    for b, sq, sk in _sequences(cu_q, cu_k):
        vis = visible(sq.stop - sq.start, sk.stop - sk.start, causal, window_left, sink_tokens)
        if not vis.size:
            continue
        n = sk.stop - sk.start
        for h in range(hq):
            kh = h // (hq // hkv)
            x = q[sq, h] @ k[sk, kh].T * scale
            a = np.abs(q[sq, h]) @ np.abs(k[sk, kh]).T * scale
            p = np.where(vis, np.exp(np.where(vis, x - lse[sq, h][:, None], 0.0)), 0.0)
            out[b, kh, :n] += p.sum(0)
            dot[b, kh, :n] = np.maximum(dot[b, kh, :n], np.where(vis, a, 0.0).max(0))
    return out, dot


def paged_decode(q, k_pool, v_pool, tables, counts, window_left, sink_tokens, scale):
    """(out, lse, worst sum |q k| scale, sum p |v|, weights per kv head and slot)."""
    seqs, hq, d = q.shape
    page, hkv = k_pool.shape[1:3]
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, dot = np.full((seqs, hq), -FLT_MAX), np.zeros((seqs, hq))
    got = np.zeros((seqs, hkv, tables.shape[1] * page))
    for s in range(seqs):
        n = int(counts[s])
        js = [j for j in range(n) if window_left < 0 or j >= n - 1 - window_left or j < sink_tokens]
        if not js:
            continue
        at = np.array([tables[s, j // page] for j in js]), np.array([j % page for j in js])
        for h in range(hq):
            kh = h // (hq // hkv)
            k, v = k_pool[at[0], at[1], kh], v_pool[at[0], at[1], kh]
            x = k @ q[s, h] * scale
            p = np.exp(x - x.max())
            lse[s, h] = x.max() + math.log(p.sum())
            p /= p.sum()
            out[s, h], absv[s, h] = p @ v, p @ np.abs(v)
            dot[s, h] = (np.abs(k) @ np.abs(q[s, h])).max() * scale
            got[s, kh, js] += p
    return out, lse, dot, absv, got


def evict(refcounts, tables, counts, budgets, weights, positions, history, sinks, recent, page=16):
    """What an eviction does, as lists: (kept [S], history [S, 2], moves (s, head, from, to),
    {(s, head): (weights, positions) of its kept slots}, rows that are refused)."""
    seqs, hkv = weights.shape[:2]
    kept, hist = np.array(counts), np.array(history)
    moves, state, refused = [], {}, []
    for s in range(seqs):
        n, known, gone = int(counts[s]), int(history[s][0]), int(history[s][1])
        b = n if budgets[s] < 0 else min(n, int(budgets[s]))
        bad = not 0 <= n <= tables.shape[1] * page or not 0 <= known <= n or gone < 0
        if not bad:
            ids = [int(x) for x in tables[s, :-(-n // page)]]
            bad = any(not 0 <= x < len(refcounts) for x in ids)
            bad = bad or (b < n and any(refcounts[x] != 1 for x in ids[:-(-b // page)]))
        if bad:
            refused.append(s)
            continue
        kept[s], hist[s] = b, (b, gone + n - b)
        first, last = min(sinks, b), min(recent, b - min(sinks, b))
        for h in range(hkv):
            pos = [int(positions[s, h, j]) if j < known else j + gone for j in range(n)]
            safe = [p < first or p >= n + gone - last for p in pos]
            order = sorted(range(n), key=lambda j: (not safe[j], 0.0 if safe[j] else -weights[s, h, j], j))
            keep = set(order[:b])
            src = list(range(b))
            movers = [j for j in range(b, n) if j in keep]
            for to, frm in zip([j for j in range(b) if j not in keep], movers):
                src[to] = frm
                moves.append((s, h, frm, to))
            state[s, h] = (np.array([weights[s, h, j] for j in src]),
                           np.array([pos[j] for j in src], dtype=np.int64))
    return kept, hist, moves, state, refused


def truncate(refcounts, tables, counts, new_counts, page):
    """(refcounts, counts, rows that are refused) after rows shrink to new_counts."""
    refs, out, refused = np.array(refcounts), np.array(counts), []
    for s, (n, m) in enumerate(zip(counts, new_counts)):
        n, m = int(n), int(m)
        if m < 0 or m == n:
            continue
        bad = m > n or not 0 <= n <= tables.shape[1] * page
        ids = [] if bad else [int(x) for x in tables[s, :-(-n // page)]]
        keep = -(-m // page)
        # a page that is cut in two must not be another row's as well
        if bad or (m % page and ids[keep - 1] in range(len(refs)) and refcounts[ids[keep - 1]] > 1):
            refused.append(s)
            continue
        out[s] = m
        for x in ids[keep:]:
            if 0 <= x < len(refs) and refs[x] > 0:
                refs[x] -= 1
            else:
                refused.append(s)
    return refs, out, refused
