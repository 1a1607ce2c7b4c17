"""The serving and training operators around varlen attention and paged decode,
as cases that can be run and timed.

Four operators: ``qk_norm_rope`` (RMS norm of every query and key head and the
rotation of its position, forward and backward), ``kv4_write`` / ``kv4_gather``
(a paged cache held in 4 bits), ``kv4_decode`` (one-token attention over that
cache) and the page operations (fork, extend, free, compact).  With ``own``
false, ``run`` computes a case in elementary torch operations; with ``own``
true it calls the framework's operators.

Layout of the 4-bit cache, per page of 16 tokens and kv head, 18 * D bytes:
  [0, 8D)    K codes, token-major: dim d of token t in byte t*D/2 + d/2, low
             nibble for even d;
  [8D, 16D)  V codes, token pairs together in runs of W = min(16, D/8) dims:
             with c = d // W the byte is ((t//8) * (D/(8W)) + c//8) * 32W +
             ((c%8)*4 + (t//2)%4) * W + (t%2) * W/2 + (d%W)/2;
  [16D, 17D) K scales, token-major: byte t*D/16 + d/16;
  [17D, 18D) V scales: byte ((d/16)*4 + (t//2)%4) * 4 + t%2 + 2*(t//8).
Codes are E2M1, scales E4M3; a value is descale * scale * code.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16                      # tokens per page of the decode pools


def _dev():
    return torch.device("cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(case):
    """The case's sequence lengths: log-uniform in [lo, hi], the first one hi."""
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    out = [hi]
    for _ in range(case["seqs"] - 1):
        out.append(int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))))
    r.shuffle(out)
    return out


def _vfa():
    from variable_length_flashattention_gb300 import vfa
    return vfa


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of the repository's 64-sequence serving batch, positions far out
        {"name": "rope_step", "op": "rope", "bwd": False, "tokens": 64, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "axes": 1, "inter": False, "norm": True, "maxpos": 1000000},
        # a prompt of the long-tail workload's size with grouped heads
        {"name": "rope_prompt", "op": "rope", "bwd": False, "tokens": 32768, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "axes": 1, "inter": False, "norm": True, "maxpos": 32768},
        # image / video tokens: time, height, width axes, interleaved pairs, part of the head turned
        {"name": "rope_axes_bwd", "op": "rope", "bwd": True, "tokens": 8649, "hq": 8, "hkv": 8,
         "d": 64, "rot": 48, "axes": 3, "inter": True, "norm": True, "maxpos": 4096},
        # the training step of the packed workload's size, an odd token count
        {"name": "rope_train_bwd", "op": "rope", "bwd": True, "tokens": 32749, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "axes": 1, "inter": False, "norm": True, "maxpos": 32768},
        # one new token for each of 64 sequences into the 4-bit cache
        {"name": "store_step", "op": "store", "seqs": 64, "lo": 1, "hi": 1, "lens": 1,
         "start": 8000, "hkv": 8, "d": 128, "dk": -3, "dv": -5},
        # ragged prompts into the 4-bit cache, and back out for a prompt that continues them
        {"name": "store_prompt", "op": "store", "seqs": 24, "lo": 17, "hi": 16384, "lens": 2,
         "start": 1000, "hkv": 8, "d": 128, "dk": -3, "dv": -5},
        # a few short contexts: latency
        {"name": "decode_small", "op": "decode", "seqs": 3, "lo": 150, "hi": 700, "lens": 3,
         "hq": 32, "hkv": 8, "d": 128, "dk": -3, "dv": -5},
        # four long contexts of the long decode workload
        {"name": "decode_long", "op": "decode", "seqs": 4, "lo": 49152, "hi": 65536, "lens": 4,
         "hq": 32, "hkv": 8, "d": 128, "dk": -3, "dv": -5},
        # a serving batch of many sequences with long-tailed contexts
        {"name": "decode_batch", "op": "decode", "seqs": 256, "lo": 16, "hi": 16384, "lens": 6,
         "hq": 32, "hkv": 8, "d": 128, "dk": -3, "dv": -5},
        # four beams of each of two prompts: fork, one token more, free
        {"name": "pages_beam", "op": "fork", "seqs": 2, "lo": 400, "hi": 4001, "lens": 7,
         "forks": 8, "layers": 2, "blocks": 1024, "hkv": 8, "d": 128},
        # samples of many prompts at once over the pools of all layers
        {"name": "pages_sample", "op": "fork", "seqs": 32, "lo": 100, "hi": 8000, "lens": 8,
         "forks": 256, "layers": 16, "blocks": 6000, "hkv": 8, "d": 64},
        # a fragmented pool packed to its low end
        {"name": "pages_pack", "op": "compact", "seqs": 64, "lo": 300, "hi": 2500, "lens": 9,
         "fill": 60, "layers": 8, "hkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "store", "decode", "decode", "fork", "compact"])
    if op == "rope":
        d = rng.choice([64, 128, 256])
        axes = rng.choice([1, 1, 2, 3, 4])
        hkv = rng.choice([1, 2, 3, 4, 5, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7])
        tokens = _log_int(rng, 1, min(32768, 32768 * 40 * 128 // ((hq + hkv) * d)))
        return {"op": op, "bwd": rng.random() < 0.5, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, 48, 16]), "axes": axes,
                "inter": rng.random() < 0.5, "norm": rng.random() < 0.8,
                "maxpos": _log_int(rng, 64, 1000000)}
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "store":
        hi = _log_int(rng, 1, 16384 * 8 * 128 // (hkv * d) // 2)
        return {"op": op, "seqs": rng.randint(1, 24), "lo": 1, "hi": hi,
                "lens": rng.randrange(1 << 30), "start": rng.randrange(5000), "hkv": hkv, "d": d,
                "dk": rng.randint(-6, 2), "dv": rng.randint(-6, 2)}
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(65536, (1 << 18) * 8 * 128 // (hkv * d) // seqs))
        return {"op": op, "seqs": seqs, "lo": 1, "hi": hi, "lens": rng.randrange(1 << 30),
                "hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), "hkv": hkv, "d": d,
                "dk": rng.randint(-6, 2), "dv": rng.randint(-6, 2)}
    layers = rng.randint(1, 8)
    if op == "fork":
        seqs = rng.randint(1, 24)
        hi = _log_int(rng, 20, 4000)
        forks = _log_int(rng, 1, 200)
        need = seqs * (hi // PAGE + 2) + 2 * forks
        return {"op": op, "seqs": seqs, "lo": 10, "hi": hi, "lens": rng.randrange(1 << 30),
                "forks": forks, "layers": layers, "blocks": need + rng.randrange(500),
                "hkv": rng.choice([1, 2, 4]), "d": d}
    return {"op": op, "seqs": rng.randint(1, 64), "lo": 10, "hi": _log_int(rng, 20, 2500),
            "lens": rng.randrange(1 << 30), "fill": rng.randint(15, 95), "layers": layers,
            "hkv": rng.choice([1, 2, 4]), "d": d}


# ------------------------------------------------------------------ the 4-bit format

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _v_byte(d):
    """[16, d] byte of V's code of (token, dim) within the V code area."""
    w = min(16, d // 8)
    t = torch.arange(PAGE, device=_dev())[:, None]
    i = torch.arange(d, device=_dev())[None, :]
    c = i // w
    return (((t // 8) * (d // (8 * w)) + c // 8) * (32 * w) + ((c % 8) * 4 + (t // 2) % 4) * w +
            (t % 2) * (w // 2) + (i % w) // 2)


def _v_scale_byte(d):
    """[16, d/16] byte of V's scale of (token, group) within the V scale area."""
    t = torch.arange(PAGE, device=_dev())[:, None]
    g = torch.arange(d // 16, device=_dev())[None, :]
    return (g * 4 + (t // 2) % 4) * 4 + t % 2 + 2 * (t // 8)


def _quantise(x, log2_descale):
    """(codes uint8 [..., D], scales E4M3 bytes uint8 [..., D/16]) of fp32 x."""
    x = x * (2.0 ** -log2_descale)
    g = x.reshape(*x.shape[:-1], -1, 16)
    s8 = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    a = g.abs()
    code = ((a > 0.25 * s).byte() + (a >= 0.75 * s).byte() + (a > 1.25 * s).byte() +
            (a >= 1.75 * s).byte() + (a > 2.5 * s).byte() + (a >= 3.5 * s).byte() +
            (a > 5.0 * s).byte())
    code = torch.where(s > 0, code, torch.zeros_like(code))
    code = code + ((g < 0) & (code > 0)).byte() * 8
    return code.reshape(x.shape), s8.view(torch.uint8)


def _code_values(codes):
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=_dev())
    return table[codes.int()]


def _pack_pages(kc, ks, vc, vs):
    """Codes [n, 16, D] and scales [n, 16, D/16] of n (page, head) units -> uint8 [n, 18D]."""
    n, _, d = kc.shape
    out = torch.empty(n, 18 * d, dtype=torch.uint8, device=_dev())
    out[:, :8 * d] = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, -1)
    vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).reshape(n, -1)
    out[:, 8 * d + _v_byte(d)[:, 0::2].reshape(-1)] = vb
    out[:, 16 * d:17 * d] = ks.reshape(n, -1)
    out[:, 17 * d + _v_scale_byte(d).reshape(-1)] = vs.reshape(n, -1)
    return out


def _page_values(pages, log2_dk, log2_dv):
    """uint8 [..., 18D] -> fp32 K and V values [..., 16, D]."""
    d = pages.shape[-1] // 18
    lead = pages.shape[:-1]
    kb = pages[..., :8 * d].reshape(*lead, PAGE, d // 2)
    kc = torch.stack((kb & 15, kb >> 4), -1).reshape(*lead, PAGE, d)
    vb = pages[..., 8 * d + _v_byte(d)[:, 0::2].reshape(-1)].reshape(*lead, PAGE, d // 2)
    vc = torch.stack((vb & 15, vb >> 4), -1).reshape(*lead, PAGE, d)
    ks = pages[..., 16 * d:17 * d].contiguous().view(torch.float8_e4m3fn).float()
    vs = pages[..., 17 * d + _v_scale_byte(d).reshape(-1)].contiguous()
    vs = vs.view(torch.float8_e4m3fn).float()
    k = _code_values(kc).reshape(*lead, PAGE, d // 16, 16)
    v = _code_values(vc).reshape(*lead, PAGE, d // 16, 16)
    k = k * (ks.reshape(*lead, PAGE, d // 16, 1) * 2.0 ** log2_dk)
    v = v * (vs.reshape(*lead, PAGE, d // 16, 1) * 2.0 ** log2_dv)
    return k.reshape(*lead, PAGE, d), v.reshape(*lead, PAGE, d)


# ------------------------------------------------------------------ inputs

def _prepare_rope(case, seed):
    g = _gen(seed)
    t, hq, hkv, d, rot, axes = (case[x] for x in ("tokens", "hq", "hkv", "d", "rot", "axes"))
    # q and k are views of one projection's output [tokens, (hq + 2 hkv) * d]
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g, device=_dev()).bfloat16()
    q = qkv[:, :hq * d].view(t, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    pos = torch.randint(0, case["maxpos"], (axes, t), generator=g, device=_dev(),
                        dtype=torch.int32)
    half = rot // 2
    # consecutive sections of the frequencies for the axes
    ax = [i * axes // half for i in range(half)]
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(half)]
    s = {"q": q, "k": k, "pos": pos, "ax": torch.tensor(ax, device=_dev()),
         "freq": torch.tensor(freq, dtype=torch.float64, device=_dev()),
         "qw": None, "kw": None, "eps": 1e-6, "inter": case["inter"], "bwd": case["bwd"]}
    if case["norm"]:
        s["qw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=_dev())
        s["kw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=_dev())
    if case["bwd"]:
        s["dyq"] = torch.randn(t, hq, d, generator=g, device=_dev()).bfloat16()
        s["dyk"] = torch.randn(t, hkv, d, generator=g, device=_dev()).bfloat16()
    if own:
        vfa = _vfa()
        s["table"] = vfa.rope_table(freq, ax, device=_dev())
        if case["bwd"]:
            s["ws"] = vfa.alloc_qk_norm_rope_bwd_workspace(d, device=_dev())
    return s


def _tables(lens, blocks, cap, g):
    perm = torch.randperm(blocks, generator=g, device=_dev()).int()
    tables = torch.zeros(len(lens), cap, dtype=torch.int32, device=_dev())
    at = 0
    for i, n in enumerate(lens):
        nb = -(-n // PAGE)
        tables[i, :nb] = perm[at:at + nb]
        at += nb
    return tables


def _prepare_store(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    r = random.Random(case["lens"] + 1)
    starts = [r.randint(0, case["start"]) for _ in lens]
    ends = [a + n for a, n in zip(starts, lens)]
    total = sum(lens)
    blocks = sum(-(-e // PAGE) for e in ends)
    kv = torch.randn(total, 2 * hkv * d, generator=g, device=_dev()).bfloat16()
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    tables = _tables(ends, blocks, max(-(-e // PAGE) for e in ends), g)
    return {"k": kv[:, :hkv * d].view(total, hkv, d), "v": kv[:, hkv * d:].view(total, hkv, d),
            "pool": torch.zeros(blocks, hkv, 18 * d, dtype=torch.uint8, device=_dev()),
            "tables": tables, "cu": torch.from_numpy(cu).to(_dev()),
            "start": torch.tensor(starts, dtype=torch.int32, device=_dev()),
            "dk": case["dk"], "dv": case["dv"]}


def _prepare_decode(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    blocks = sum(-(-n // PAGE) for n in lens)
    pool = torch.empty(blocks, hkv, 18 * d, dtype=torch.uint8, device=_dev())
    step = max(1, (1 << 25) // (hkv * PAGE * d))
    for b0 in range(0, blocks, step):
        n = min(step, blocks - b0) * hkv
        kc, ks = _quantise(torch.randn(n, PAGE, d, generator=g, device=_dev()), case["dk"])
        vc, vs = _quantise(torch.randn(n, PAGE, d, generator=g, device=_dev()), case["dv"])
        pool[b0:b0 + step] = _pack_pages(kc, ks, vc, vs).view(-1, hkv, 18 * d)
    s = {"q": torch.randn(len(lens), case["hq"], d, generator=g, device=_dev()).bfloat16(),
         "pool": pool, "tables": _tables(lens, blocks, max(-(-n // PAGE) for n in lens), g),
         "counts": torch.tensor(lens, dtype=torch.int32, device=_dev()), "lens": lens,
         "dk": case["dk"], "dv": case["dv"]}
    if own:
        s["ws"] = _vfa().alloc_kv4_decode_workspace(len(lens), case["hq"], hkv, d, device=_dev())
    return s


def _page_pools(case, blocks, g):
    shape = (blocks, PAGE, case["hkv"], case["d"])
    return [torch.randn(shape, generator=g, device=_dev(), dtype=torch.bfloat16)
            for _ in range(2 * case["layers"])]


def _prepare_fork(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    n = case["forks"]
    cap = -(-case["hi"] // PAGE) + 2
    rows = len(lens) + n
    tables = torch.zeros(rows, cap, dtype=torch.int32, device=_dev())
    tables[:len(lens)] = _tables(lens, case["blocks"], cap, g)
    counts = torch.zeros(rows, dtype=torch.int32, device=_dev())
    counts[:len(lens)] = torch.tensor(lens, dtype=torch.int32, device=_dev())
    refs = torch.zeros(case["blocks"], dtype=torch.int32, device=_dev())
    for i, m in enumerate(lens):
        refs[tables[i, :-(-m // PAGE)].long()] = 1
    parents = [i % len(lens) for i in range(n)]
    children = list(range(len(lens), rows))
    add = torch.zeros(rows, dtype=torch.int32, device=_dev())
    add[len(lens):] = 1
    s = {"refs": refs, "tables": tables, "counts": counts, "add": add,
         "parents": torch.tensor(parents, dtype=torch.int32, device=_dev()),
         "children": torch.tensor(children, dtype=torch.int32, device=_dev()),
         # what the plain form's program knows on the host
         "len_list": [lens[p] for p in parents],
         "pools": _page_pools(case, case["blocks"], g)}
    if own:
        s["ws"] = _vfa().alloc_pages_workspace(case["blocks"], rows, n, device=_dev())
    return s


def _prepare_compact(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    used = sum(-(-m // PAGE) for m in lens)
    blocks = max(used, used * 100 // case["fill"])
    cap = -(-case["hi"] // PAGE)
    tables = _tables(lens, blocks, cap, g)
    refs = torch.zeros(blocks, dtype=torch.int32, device=_dev())
    for i, m in enumerate(lens):
        refs[tables[i, :-(-m // PAGE)].long()] = 1
    s = {"refs": refs, "tables": tables, "cap": cap,
         "counts": torch.tensor(lens, dtype=torch.int32, device=_dev()),
         "refs_out": torch.zeros_like(refs), "tables_out": torch.zeros_like(tables),
         "pools": _page_pools(case, blocks, g)}
    if own:
        s["ws"] = _vfa().alloc_pages_workspace(blocks, len(lens), 0, device=_dev())
    return s


def prepare(case, seed):
    s = {"rope": _prepare_rope, "store": _prepare_store, "decode": _prepare_decode,
         "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------ plain forms

def _cos_sin(s):
    a = s["pos"].double()[s["ax"]].T * s["freq"]            # [T, R/2], 64 bits: far positions
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _turn(x, cos, sin, inter):
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _plain_rope(s):
    cos, sin = _cos_sin(s)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        out.append(_turn(x, cos, sin, s["inter"]).bfloat16())
    return out


def _plain_rope_bwd(s):
    cos, sin = _cos_sin(s)
    dxs, dws = [], []
    for x, w, dy in ((s["q"], s["qw"], s["dyq"]), (s["k"], s["kw"], s["dyk"])):
        g = _turn(dy.float(), cos, -sin, s["inter"])
        if w is not None:
            x = x.float()
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
            xn = x * r
            dws.append((g * xn).sum((0, 1), dtype=torch.float64).float())
            u = g * w
            g = r * (u - xn * (u * xn).mean(-1, keepdim=True))
        dxs.append(g.bfloat16())
    return dxs + dws


def _slots(s):
    """(page id, token in the page) of every packed token."""
    cu = s["cu"].long()
    total = s["k"].shape[0]
    t = torch.arange(total, device=_dev())
    seq = torch.searchsorted(cu, t, right=True) - 1
    p = s["start"].long()[seq] + t - cu[seq]
    return s["tables"].long()[seq, p // PAGE], p % PAGE


def _plain_store(s):
    page, row = _slots(s)
    pool, (total, hkv, d) = s["pool"], s["k"].shape
    flat = pool.view(-1)
    base = ((page[:, None] * hkv + torch.arange(hkv, device=_dev())) * (18 * d))[:, :, None]
    vb, vsb = _v_byte(d)[:, 0::2], _v_scale_byte(d)
    half = torch.arange(d // 2, device=_dev())
    grp = torch.arange(d // 16, device=_dev())
    kc, ks = _quantise(s["k"].float(), s["dk"])
    vc, vs = _quantise(s["v"].float(), s["dv"])
    flat[base + (row[:, None] * (d // 2) + half)[:, None]] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    flat[base + (8 * d + vb[row])[:, None]] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    flat[base + (16 * d + row[:, None] * (d // 16) + grp)[:, None]] = ks
    flat[base + (17 * d + vsb[row])[:, None]] = vs
    # read the same tokens back
    out = []
    for code_at, scale_at, ld in (
            (row[:, None] * (d // 2) + half, 16 * d + row[:, None] * (d // 16) + grp, s["dk"]),
            (8 * d + vb[row], 17 * d + vsb[row], s["dv"])):
        c = flat[base + code_at[:, None]]
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
        sc = flat[base + scale_at[:, None]].view(torch.float8_e4m3fn).float() * 2.0 ** ld
        v = _code_values(c).view(total, hkv, d // 16, 16) * sc[..., None]
        out.append(v.view(total, hkv, d).bfloat16())
    return out


def _plain_decode(s):
    outs, lses = [], []
    hq, d = s["q"].shape[1:]
    hkv = s["pool"].shape[1]
    for i, n in enumerate(s["lens"]):
        ids = s["tables"][i, :-(-n // PAGE)].long()
        k, v = _page_values(s["pool"][ids], s["dk"], s["dv"])        # [nb, hkv, 16, d]
        k = k.transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        v = v.transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        q = s["q"][i].float().view(hkv, hq // hkv, d)
        x = (q[:, :, None, :] * k[:, None]).sum(-1) if n * hq * d < (1 << 22) else \
            torch.stack([(k * q[:, j, None]).sum(-1) for j in range(hq // hkv)], 1)
        x = x / math.sqrt(d)
        m = x.amax(-1, keepdim=True)
        p = (x - m).exp()
        z = p.sum(-1, keepdim=True)
        o = torch.stack([(p[:, j, :, None] * v).sum(1) for j in range(hq // hkv)], 1) / z
        outs.append(o.reshape(hq, d).bfloat16())
        lses.append((m + z.log()).reshape(hq))
    return [torch.stack(outs), torch.stack(lses)]


def _plain_fork(s):
    lens = s["len_list"]
    tables, counts, refs = s["tables"], s["counts"], s["refs"]
    par, chi = s["parents"].long(), s["children"].long()
    dev = _dev()
    cap = tables.shape[1]
    # fork: full pages shared, a partial last page copied into the lowest free ones
    full = torch.tensor([n // PAGE for n in lens], device=dev)
    tail = torch.tensor([i for i, n in enumerate(lens) if n % PAGE], dtype=torch.long, device=dev)
    rows = tables[par]
    live = torch.arange(cap, device=dev)[None] < full[:, None]
    tables[chi] = torch.where(live, rows, tables[chi])
    refs.scatter_add_(0, torch.where(live, rows, 0).long().view(-1), live.int().view(-1))
    if len(tail):
        free = torch.argsort((refs > 0).int(), stable=True)[:len(tail)]
        src = rows[tail, full[tail]].long()
        for p in s["pools"]:
            p[free] = p[src]
        tables[chi[tail], full[tail]] = free.int()
        refs[free] = 1
    counts[chi] = counts[par]
    # extend every child by one token: a new page where its last one is full
    grow = torch.tensor([i for i, n in enumerate(lens) if n % PAGE == 0], dtype=torch.long,
                        device=dev)
    if len(grow):
        free = torch.argsort((refs > 0).int(), stable=True)[:len(grow)]
        tables[chi[grow], full[grow]] = free.int()
        refs[free] = 1
    counts += s["add"]
    # free the children
    live = torch.arange(cap, device=dev)[None] < full[:, None] + 1
    rows = torch.where(live, tables[chi], 0).long()
    refs.scatter_add_(0, rows.view(-1), -live.int().view(-1))
    counts[chi] = 0
    return [tables, counts, refs] + s["pools"]


def _plain_compact(s):
    refs = s["refs"]
    used = refs > 0
    n = used.sum()
    ids = torch.arange(refs.numel(), device=_dev())
    src = ids[used & (ids >= n)]
    dst = ids[~used & (ids < n)]
    new = ids.clone()
    new[src] = dst
    for p in s["pools"]:
        p[dst] = p[src]
    s["refs_out"].copy_(refs)
    s["refs_out"][dst] = refs[src]
    s["refs_out"][src] = 0
    live = torch.arange(s["cap"], device=_dev())[None] < -(-s["counts"] // PAGE)[:, None]
    s["tables_out"].copy_(torch.where(live, new[s["tables"].long()].int(), s["tables_out"]))
    return [n.int().view(1), s["refs_out"], s["tables_out"]] + s["pools"]


# ------------------------------------------------------------------ the framework's operators

def _own_rope(s):
    return list(_vfa().qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], s["qw"], s["kw"],
                                    eps=s["eps"], interleaved=s["inter"]))


def _own_rope_bwd(s):
    r = _vfa().qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["pos"], s["table"], s["qw"],
                                s["kw"], eps=s["eps"], interleaved=s["inter"], workspace=s["ws"])
    return [x for x in r if x is not None]


def _own_store(s):
    vfa = _vfa()
    dk, dv = 2.0 ** s["dk"], 2.0 ** s["dv"]
    vfa.kv4_write(s["k"], s["v"], s["pool"], s["tables"], s["cu"], s["start"], dk, dv)
    return list(vfa.kv4_gather(s["pool"], s["tables"], s["cu"], s["start"], s["k"].shape[0], dk,
                               dv))


def _own_decode(s):
    return list(_vfa().kv4_decode(s["q"], s["pool"], s["tables"], s["counts"], 2.0 ** s["dk"],
                                  2.0 ** s["dv"], workspace=s["ws"]))


def _own_fork(s):
    vfa = _vfa()
    vfa.pages_fork(s["refs"], s["tables"], s["counts"], s["parents"], s["children"], s["pools"],
                   PAGE, s["ws"])
    vfa.pages_extend(s["refs"], s["tables"], s["counts"], s["add"], PAGE, s["ws"])
    vfa.pages_free(s["refs"], s["tables"], s["counts"], s["children"], PAGE)
    return [s["tables"], s["counts"], s["refs"]] + s["pools"]


def _own_compact(s):
    n = _vfa().pages_compact(s["refs"], s["tables"], s["counts"], s["pools"], PAGE, s["ws"],
                             refcounts_out=s["refs_out"], tables_out=s["tables_out"])
    return [n, s["refs_out"], s["tables_out"]] + s["pools"]


def run(state):
    op = state["op"]
    if op == "rope" and state["bwd"]:
        op = "rope_bwd"
    plain = {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "store": _plain_store,
             "decode": _plain_decode, "fork": _plain_fork, "compact": _plain_compact}
    ours = {"rope": _own_rope, "rope_bwd": _own_rope_bwd, "store": _own_store,
            "decode": _own_decode, "fork": _own_fork, "compact": _own_compact}
    return (ours if own else plain)[op](state)


# ------------------------------------------------------------------ 64-bit definitions

def _exact_rope(case, s):
    """Forward by complex products; backward by differentiating it."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=_dev()),
                       s["freq"] * s["pos"].double()[s["ax"]].T)[:, None, :]
    half = turn.shape[-1]

    def one(x, w):
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
        r = x[..., :2 * half]
        if case["inter"]:
            z = torch.view_as_complex(r.reshape(*r.shape[:-1], half, 2).contiguous()) * turn
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        return torch.cat((y, x[..., 2 * half:]), -1)

    outs, dws = [], []
    for x, w, dy in ((s["q"], s["qw"], s.get("dyq")), (s["k"], s["kw"], s.get("dyk"))):
        x = x.double()
        w = None if w is None else w.double()
        if not case["bwd"]:
            outs.append(one(x, w))
            continue
        x.requires_grad_(True)
        if w is not None:
            w.requires_grad_(True)
        y = one(x, w)
        grads = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
        outs.append(grads[0])
        dws += list(grads[1:])
    return outs + dws


def _e4m3_table():
    """All finite non-negative E4M3 values by their code 0 .. 126."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64, device=_dev())


def _nearest(x, table):
    """Index of the nearest entry of an ascending table; a tie goes to the even index."""
    hi = torch.searchsorted(table, x).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_store(s):
    e4m3 = _e4m3_table()
    e2m1 = torch.tensor(_E2M1, dtype=torch.float64, device=_dev())
    out = []
    for x, ld in ((s["k"], s["dk"]), (s["v"], s["dv"])):
        r = torch.empty(x.shape, dtype=torch.float64, device=_dev())
        for t0 in range(0, x.shape[0], 8192):
            part = x[t0:t0 + 8192].double()
            g = part.reshape(*part.shape[:-1], -1, 16) / 2.0 ** ld
            # the scale nearest to max / 6, compared at six times its size: no quotient rounds
            sc = e4m3[_nearest(g.abs().amax(-1, keepdim=True), 6.0 * e4m3)]
            y = torch.empty_like(g)
            safe = torch.where(sc > 0, sc, torch.ones_like(sc))
            # |g| against scale * midpoints: exact products of few bits
            idx = torch.zeros_like(g, dtype=torch.long)
            for i in range(7):
                mid = safe * ((e2m1[i] + e2m1[i + 1]) / 2)
                idx += ((g.abs() > mid) | ((g.abs() == mid) & (i % 2 == 1))).long()
            y = torch.sign(g) * e2m1[idx] * sc * 2.0 ** ld
            r[t0:t0 + 8192] = y.reshape(part.shape)
        out.append(r)
    return out


def _exact_decode(s):
    hq, d = s["q"].shape[1:]
    hkv = s["pool"].shape[1]
    group = hq // hkv
    e4m3 = torch.cat((_e4m3_table(), torch.zeros(1, dtype=torch.float64, device=_dev())))
    e2m1 = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float64, device=_dev())
    odd = (torch.arange(d, device=_dev()) % 2 * 4)
    t = torch.arange(PAGE, device=_dev())
    i = torch.arange(d, device=_dev())
    k_at = t[:, None] * (d // 2) + i // 2
    ks_at = 16 * d + t[:, None] * (d // 16) + i // 16
    v_at = 8 * d + _v_byte(d)
    vs_at = 17 * d + _v_scale_byte(d)[:, i // 16]
    outs, lses = [], []
    for b, n in enumerate(s["lens"]):
        pages = s["pool"][s["tables"][b, :-(-n // PAGE)].long()]
        o = torch.empty(hq, d, dtype=torch.float64, device=_dev())
        lse = torch.empty(hq, dtype=torch.float64, device=_dev())
        for h in range(hkv):
            raw = pages[:, h]
            k = (e2m1[((raw[:, k_at] >> odd) & 15).long()] * e4m3[raw[:, ks_at].long()])
            v = (e2m1[((raw[:, v_at] >> odd) & 15).long()] * e4m3[raw[:, vs_at].long()])
            k = k.reshape(-1, d)[:n] * 2.0 ** s["dk"]
            v = v.reshape(-1, d)[:n] * 2.0 ** s["dv"]
            x = s["q"][b, h * group:(h + 1) * group].double() @ k.T / math.sqrt(d)
            lse[h * group:(h + 1) * group] = torch.logsumexp(x, -1)
            o[h * group:(h + 1) * group] = torch.softmax(x, -1) @ v
        outs.append(o)
        lses.append(lse)
    return [torch.stack(outs), torch.stack(lses)]


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                  # whole numbers and copied pages
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "store":
        return _exact_store(s)
    return _exact_decode(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        words = case["axes"] * case["tokens"] * 4
        return {"bytes": n * (6 if case["bwd"] else 4) + words, "flops": n * (18 if case["bwd"] else 9)}
    lens = _lengths(case)
    if op == "store":
        n = sum(lens) * case["hkv"] * case["d"] * 2
        return {"bytes": int(n * (2 + 0.5625 + 0.5625 + 2)), "flops": n * 6}
    if op == "decode":
        n = sum(lens)
        return {"bytes": int(n * case["hkv"] * case["d"] * 1.125) + case["seqs"] * case["hq"] *
                case["d"] * 4, "flops": 4 * n * case["hq"] * case["d"]}
    page = PAGE * case["hkv"] * case["d"] * 2
    pools = 2 * case["layers"]
    if op == "fork":
        per = [lens[i % len(lens)] for i in range(case["forks"])]
        copies = sum(1 for n in per if n % PAGE)
        entries = sum(-(-n // PAGE) for n in per)
        return {"bytes": copies * pools * page * 2 + entries * 16, "flops": entries}
    used = sum(-(-m // PAGE) for m in lens)
    blocks = max(used, used * 100 // case["fill"])
    moves = used * (blocks - used) // blocks         # used pages at or above `used`, expected
    return {"bytes": moves * pools * page * 2 + used * 8 + blocks * 8, "flops": blocks}
