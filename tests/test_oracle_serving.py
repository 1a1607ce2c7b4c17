"""Pins of the 64-bit definitions in oracle/serving.py (CPU only): torch autograd and complex
products, central differences, torch's E4M3 conversion, torch SDPA, and the page operations'
invariants.  Each pin uses another route than the definition it checks."""
import numpy as np
import pytest
import torch

import oracle.serving as O


def _rand(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,axes", [(64, 64, 1), (64, 48, 3), (128, 16, 2), (64, 0, 1)])
def test_rotation_is_a_complex_product(D, R, axes, interleaved):
    rng = np.random.default_rng(D + R)
    x = _rand(rng, 5, 3, D)
    f = 10000.0 ** (-np.arange(R // 2) / max(R // 2, 1))
    ax = [i % axes for i in range(R // 2)]
    pos = rng.integers(-50, 4000, (axes, 5))
    w = _rand(rng, D)
    y = O.norm_rope(x, pos, f, ax, w, 1e-6, interleaved)
    n = torch.from_numpy(x)
    n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + 1e-6) * torch.from_numpy(w)
    rot = n[..., :R]
    if interleaved:
        z = torch.complex(rot[..., 0::2], rot[..., 1::2])
    else:
        z = torch.complex(rot[..., :R // 2], rot[..., R // 2:])
    ang = torch.tensor([[f[i] * pos[ax[i], t] for i in range(R // 2)] for t in range(5)],
                       dtype=torch.float64).reshape(5, 1, R // 2)
    z = z * torch.polar(torch.ones_like(ang), ang)
    want = n.clone()
    if interleaved:
        want[..., 0:R:2], want[..., 1:R:2] = z.real, z.imag
    else:
        want[..., :R // 2], want[..., R // 2:R] = z.real, z.imag
    assert np.abs(y - want.numpy()).max() < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_match_central_differences(interleaved):
    rng = np.random.default_rng(7)
    D, R = 64, 32
    x, dy, w = _rand(rng, 2, 2, D), _rand(rng, 2, 2, D), _rand(rng, D)
    f, ax = 1.0 / (1 + np.arange(R // 2)), [i % 2 for i in range(R // 2)]
    pos = np.array([[3, 900], [5, 1]])
    loss = lambda x, w: (O.norm_rope(x, pos, f, ax, w, 1e-3, interleaved) * dy).sum()
    dx, dw = O.norm_rope_bwd(x, dy, pos, f, ax, w, 1e-3, interleaved)
    h = 1e-5
    for _ in range(60):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
        j = rng.integers(0, D)
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_e4m3_and_quantiser():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = O.e4m3_value(np.arange(256))
    assert np.array_equal(np.isnan(want), np.isnan(got))
    assert np.array_equal(want[~np.isnan(want)], got[~np.isnan(got)])
    # every value of the format is its own nearest, in every group of a random page
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 64)) * np.exp(rng.uniform(-12, 9, (40, 1)))).astype(np.float32)
    x = torch.from_numpy(x).bfloat16().double().numpy()
    for descale in (1.0, 0.125, 4.0):
        code, sb = O.quantise(x, descale)
        # the scale is torch's conversion of max / 6
        amax = np.abs(x / descale).reshape(40, 4, 16).max(-1) / 6
        t = torch.from_numpy(np.minimum(amax, 448)).float().to(torch.float8_e4m3fn)
        assert np.array_equal(t.view(torch.uint8).numpy(), sb)
        v = O.dequantise(code, sb, descale)
        # no representable neighbour is nearer
        s = O.e4m3_value(sb)[..., None] * descale
        g, vg = x.reshape(40, 4, 16), v.reshape(40, 4, 16)
        live = np.broadcast_to(s > 0, g.shape)
        for cand in O.E2M1:
            for sign in (1, -1):
                assert (np.abs(g - vg) <= np.abs(g - sign * cand * s))[live].all()
        assert np.array_equal(torch.from_numpy(v).bfloat16().double().numpy(), v)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_bytes_are_disjoint(D):
    seen = {}
    for t in range(16):
        for d in range(D):
            for at, nibble in ((O.k_code_byte(t, d, D), d % 2), (O.v_code_byte(t, d, D), d % 2)):
                assert (at, nibble) not in seen
                seen[(at, nibble)] = t
        for d in range(0, D, 16):
            for at in (O.k_scale_byte(t, d, D), O.v_scale_byte(t, d, D)):
                for nibble in (0, 1):
                    assert (at, nibble) not in seen
                    seen[(at, nibble)] = t
    assert len(seen) == 2 * 18 * D and max(a for a, _ in seen) == 18 * D - 1
    # no byte holds parts of two tokens
    assert all(seen[(a, 0)] == seen[(a, 1)] for a, _ in seen)


def test_write_read_decode():
    rng = np.random.default_rng(1)
    D, Hkv, Hq, n = 64, 2, 4, 37
    pool = np.full((5, Hkv, 18 * D), 0xff, dtype=np.uint8)
    k, v, q = _rand(rng, n, Hkv, D), _rand(rng, n, Hkv, D), _rand(rng, 1, Hq, D)
    table = np.array([[3, 0, 4]])
    for t in range(n):
        O.write_token(pool, table[0, t // 16], t % 16, k[t], v[t], 0.25, 0.5)
    pk, pv = O.page_values(pool[table[0]], 0.25, 0.5)
    want = O.dequantise(*O.quantise(k, 0.25), 0.25)
    assert np.array_equal(pk.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:n], want)
    wv = O.dequantise(*O.quantise(v, 0.5), 0.5)
    out, lse, *_ = O.kv4_decode(q, pool, table, [n], 0.25, 0.5)
    rep = lambda x: torch.from_numpy(x).transpose(0, 1).repeat_interleave(Hq // Hkv, 0)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[0])[:, None], rep(want), rep(wv))
    assert np.abs(out[0] - ref[:, 0].numpy()).max() < 1e-12
    x = (torch.from_numpy(q[0])[:, None] @ rep(want).transpose(1, 2))[:, 0] / D ** 0.5
    assert np.abs(lse[0] - torch.logsumexp(x, -1).numpy()).max() < 1e-12


def test_page_operations_keep_every_sequence():
    rng = np.random.default_rng(3)
    blocks, S, cap, bs = 60, 8, 12, 4
    refs = np.zeros(blocks, np.int64)
    tables = np.full((S, cap), -9)
    counts = np.zeros(S, np.int64)
    pool = rng.standard_normal((blocks, 3))
    text = {}                                   # what each row reads

    def read(s):
        return [tuple(pool[tables[s, j]]) for j in range(-(-counts[s] // bs))]

    def listed():
        n = np.zeros(blocks, np.int64)
        for s in range(S):
            for j in range(-(-counts[s] // bs)):
                n[tables[s, j]] += 1
        return n

    assert O.extend(refs, tables, counts, np.array([10, 7, 0, 16, 0, 0, 0, 0]), bs)
    assert np.array_equal(listed(), refs)
    text = {s: read(s) for s in range(S)}
    assert O.fork(refs, tables, counts, [0, 0, 3, -1], [2, 4, 5, 1], [pool], bs)
    for child, parent in ((2, 0), (4, 0), (5, 3)):
        assert read(child) == text[parent] and counts[child] == counts[parent]
    assert tables[2, 2] != tables[0, 2] and tables[2, 1] == tables[0, 1]
    assert np.array_equal(listed(), refs)
    O.free(refs, tables, counts, [0, 0, -1, 3], bs)
    assert np.array_equal(listed(), refs)
    text = {s: read(s) for s in range(S)}
    n = O.compact(refs, tables, counts, [pool], bs)
    assert n == (refs > 0).sum() and (refs[:n] > 0).all() and np.array_equal(listed(), refs)
    assert {s: read(s) for s in range(S)} == text
    before = (refs.copy(), tables.copy(), counts.copy())
    assert not O.extend(refs, tables, counts, np.full(S, 44), bs)
    assert all(np.array_equal(a, b) for a, b in zip(before, (refs, tables, counts)))
