"""Plain 64-bit definitions of the operators around attention: query / key norm
and rotation with its gradients, the 4-bit paged cache and attention over it,
and the page operations.  Test infrastructure only, like the rest of this
package; numpy, written from the definitions in include/vfa.h.
"""
from __future__ import annotations

import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)
PAGE = 16


# ------------------------------------------------------------ norm and rotation

def _angles(positions, inv_freq, axes):
    """[tokens, pairs] angles: position of the pair's axis times its frequency."""
    pos = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    return np.stack([pos[a] * f for f, a in zip(inv_freq, axes)], axis=-1) if len(inv_freq) \
        else np.zeros((pos.shape[1], 0))


def _pairs(n, interleaved):
    """Dimension indices of the first and second members of n pairs."""
    i = np.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n)


def rotate(x, positions, inv_freq, axes, interleaved, sign=1.0):
    """x [T, H, D] with its pairs turned by sign * angle."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    if n == 0:
        return y
    phi = sign * _angles(positions, inv_freq, axes)[:, None, :]
    a, b = _pairs(n, interleaved)
    y[..., a] = x[..., a] * np.cos(phi) - x[..., b] * np.sin(phi)
    y[..., b] = x[..., b] * np.cos(phi) + x[..., a] * np.sin(phi)
    return y


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def norm_rope(x, positions, inv_freq, axes, weight, eps, interleaved):
    return rotate(norm(x, weight, eps), positions, inv_freq, axes, interleaved)


def norm_rope_bwd(x, dy, positions, inv_freq, axes, weight, eps, interleaved):
    """(dx, dweight or None)."""
    x = np.asarray(x, np.float64)
    g = rotate(np.asarray(dy, np.float64), positions, inv_freq, axes, interleaved, sign=-1.0)
    if weight is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    u = g * np.asarray(weight, np.float64)
    return r * (u - x * r * r * (u * x).mean(-1, keepdims=True)), dw


# ------------------------------------------------------------ 4-bit cache

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def e4m3_value(code):
    """Value of an E4M3 byte (NaN for 0x7f / 0xff)."""
    code = np.asarray(code, dtype=np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(code & 128, -v, v)


_E4M3_POS = e4m3_value(np.arange(127))


def nearest_even(x, table):
    """Index of the nearest entry of an ascending table, ties to the even index, x above the
    last entry to the last."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantise(x, descale):
    """(codes 0..15 [..., D], scale bytes [..., D / 16]) of x [..., D]."""
    x = np.asarray(x, np.float64) / descale
    g = x.reshape(*x.shape[:-1], -1, 16)
    amax = np.abs(g).max(-1)
    # nearest scale to amax / 6, compared at six times its size (no quotient rounds)
    sb = nearest_even(amax, 6.0 * _E4M3_POS)
    s = _E4M3_POS[sb][..., None]
    mag = np.zeros(g.shape, dtype=np.int64)
    for i in range(7):
        mid = s * ((E2M1[i] + E2M1[i + 1]) / 2)
        mag += (np.abs(g) > mid) | ((np.abs(g) == mid) & (i % 2 == 1))
    mag = np.where(s > 0, mag, 0)
    code = mag + 8 * ((g < 0) & (mag > 0))
    return code.reshape(x.shape), sb


def dequantise(code, scale_byte, descale):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    g = v.reshape(*v.shape[:-1], -1, 16) * e4m3_value(scale_byte)[..., None] * descale
    return g.reshape(v.shape)


def k_code_byte(t, d, D):
    return t * D // 2 + d // 2


def v_code_byte(t, d, D):
    W = min(16, D // 8)
    c = d // W
    return 8 * D + ((t // 8) * (D // (8 * W)) + c // 8) * 32 * W + \
        ((c % 8) * 4 + (t // 2) % 4) * W + (t % 2) * (W // 2) + (d % W) // 2


def k_scale_byte(t, d, D):
    return 16 * D + t * D // 16 + d // 16


def v_scale_byte(t, d, D):
    return 17 * D + ((d // 16) * 4 + (t // 2) % 4) * 4 + t % 2 + 2 * (t // 8)


def write_token(pool, page, row, k, v, descale_k, descale_v):
    """Stores k, v [Hkv, D] at row `row` of page `page` of uint8 pool [blocks, Hkv, 18 D]."""
    D = k.shape[-1]
    for x, ds, code_at, scale_at in ((k, descale_k, k_code_byte, k_scale_byte),
                                     (v, descale_v, v_code_byte, v_scale_byte)):
        code, sb = quantise(x, ds)
        for d in range(D):
            at = code_at(row, d, D)
            shift = 4 * (d % 2)
            pool[page, :, at] = (pool[page, :, at] & (0xf0 >> shift)) | (code[:, d] << shift)
            if d % 16 == 0:
                pool[page, :, scale_at(row, d, D)] = sb[:, d // 16]


def page_values(pool_pages, descale_k, descale_v):
    """K and V values [n, Hkv, 16, D] of uint8 pages [n, Hkv, 18 D]."""
    D = pool_pages.shape[-1] // 18
    t, d = np.arange(PAGE)[:, None], np.arange(D)[None, :]
    out = []
    for ds, code_at, scale_at in ((descale_k, k_code_byte, k_scale_byte),
                                  (descale_v, v_code_byte, v_scale_byte)):
        code = (pool_pages[..., code_at(t, d, D)].astype(np.int64) >> (4 * (d % 2))) & 15
        s = e4m3_value(pool_pages[..., scale_at(t, d, D)])
        out.append(E2M1[code & 7] * np.where(code & 8, -1.0, 1.0) * s * ds)
    return out


def kv4_decode(q, pool, tables, counts, descale_k, descale_v, scale=None):
    """(out, lse, absdot, absv, allv) over q [S, Hq, D]: the attention in 64 bits, and for
    error bounds per row max_j sum_d |q_d k_jd| * scale, sum_j p_j |v_j| and
    sum_j |v_j| / l, with l = sum_j exp(x_j - max x)."""
    q = np.asarray(q, np.float64)
    S, Hq, D = q.shape
    Hkv = pool.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = np.zeros((S, Hq, D))
    lse = np.full((S, Hq), -FLT_MAX)
    absdot = np.zeros((S, Hq))
    absv = np.zeros((S, Hq, D))
    allv = np.zeros((S, Hq, D))
    for s in range(S):
        n = int(counts[s])
        if n == 0:
            continue
        ids = tables[s, :-(-n // PAGE)]
        k, v = page_values(pool[ids], descale_k, descale_v)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            kk = k[:, kh].reshape(-1, D)[:n]
            vv = v[:, kh].reshape(-1, D)[:n]
            x = kk @ q[s, h] * scale
            m = x.max()
            p = np.exp(x - m)
            out[s, h] = p @ vv / p.sum()
            lse[s, h] = m + math.log(p.sum())
            absdot[s, h] = (np.abs(kk) @ np.abs(q[s, h])).max() * scale
            absv[s, h] = p @ np.abs(vv) / p.sum()
            allv[s, h] = np.abs(vv).sum(0) / p.sum()
    return out, lse, absdot, absv, allv


# ------------------------------------------------------------ pages

def _pages(tokens, block_size):
    return -(-tokens // block_size)


def extend(refs, tables, counts, add, block_size):
    """In place; returns False (and changes nothing) if the pages do not suffice."""
    need = [(s, j) for s in range(len(counts))
            for j in range(_pages(counts[s], block_size), _pages(counts[s] + add[s], block_size))]
    free = [i for i in range(len(refs)) if refs[i] <= 0]
    if len(need) > len(free):
        return False
    for (s, j), page in zip(need, free):
        tables[s, j] = page
        refs[page] = 1
    counts += add
    return True


def fork(refs, tables, counts, parents, children, pools, block_size):
    free = [i for i in range(len(refs)) if refs[i] <= 0]
    entries = [(p, c, int(counts[p])) for p, c in zip(parents, children) if p >= 0]
    if sum(1 for _, _, n in entries if n % block_size) > len(free):
        return False
    for p, c, n in entries:
        full = n // block_size
        for j in range(full):
            tables[c, j] = tables[p, j]
            refs[tables[p, j]] += 1
        if n % block_size:
            page = free.pop(0)
            for pool in pools:
                pool[page] = pool[tables[p, full]]
            tables[c, full] = page
            refs[page] = 1
        counts[c] = n
    return True


def free(refs, tables, counts, seqs, block_size):
    for s in seqs:
        if s < 0:
            continue
        for j in range(_pages(counts[s], block_size)):
            refs[tables[s, j]] -= 1
        counts[s] = 0


def compact(refs, tables, counts, pools, block_size):
    """In place; returns the number of used pages."""
    used = [i for i in range(len(refs)) if refs[i] > 0]
    n = len(used)
    src = [i for i in used if i >= n]
    dst = [i for i in range(n) if refs[i] <= 0]
    new = {a: b for a, b in zip(src, dst)}
    for s in range(len(counts)):
        for j in range(_pages(counts[s], block_size)):
            tables[s, j] = new.get(tables[s, j], tables[s, j])
    for a, b in new.items():
        refs[b], refs[a] = refs[a], 0
        for pool in pools:
            pool[b] = pool[a]
    return n
