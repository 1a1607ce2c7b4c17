"""The operators of a bounded K/V cache, as cases that can be run and timed.

Four operators: varlen attention with a sliding window and sinks (first tokens
that stay visible), forward and backward; ``paged_decode`` (one new token per
sequence over a paged bf16 cache, with window and sinks, and with the weight
that every cached token got); ``varlen_key_weights`` (the accumulated attention
weight of a prompt's keys); and ``cache_evict`` with ``pages_truncate`` (tokens
of little weight leave the cache, and their pages go back).  With ``own`` false,
``run`` computes a case in elementary torch operations; with ``own`` true it
calls the framework's operators.

Key j is visible to query i of a sequence (both local positions) if
  j <= i + off  and  (j >= i + off - window  or  j < sinks),
off = 0 (causal 1) or Lk - Lq (causal 2); a negative window hides nothing.
"""
import math
import random

import torch

own = False

PAGE = 16                      # tokens per page
BLOCK = 128                    # query rows that the plain form takes together
FLT_MAX = torch.finfo(torch.float32).max


def _dev():
    return torch.device("cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _vfa():
    from variable_length_flashattention_gb300 import vfa
    return vfa


def _lengths(case, lo="lo", hi="hi", salt=0):
    """The case's sequence lengths: log-uniform in [lo, hi], one of them hi."""
    r = random.Random(case["lens"] + salt)
    a, b = case[lo], case[hi]
    out = [b] + [int(round(math.exp(r.uniform(math.log(a), math.log(b)))))
                 for _ in range(case["seqs"] - 1)]
    r.shuffle(out)
    return out


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short prompts: latency
        {"name": "window_short", "op": "window", "train": False, "seqs": 4, "lo": 1, "hi": 129,
         "more": 0, "lens": 1, "hq": 8, "hkv": 2, "d": 64, "causal": 1, "window": 32, "sinks": 2},
        # long-tailed prompts of a model with grouped heads
        {"name": "window_prompt", "op": "window", "train": False, "seqs": 24, "lo": 16, "hi": 8192,
         "more": 0, "lens": 2, "hq": 32, "hkv": 8, "d": 128, "causal": 1, "window": 1024, "sinks": 4},
        # prompts that continue cached contexts, odd sizes all over
        {"name": "window_continue", "op": "window", "train": False, "seqs": 31, "lo": 3, "hi": 511,
         "more": 4095, "lens": 3, "hq": 8, "hkv": 2, "d": 256, "causal": 2, "window": 500,
         "sinks": 70},
        # a training step on packed sequences: forward and backward
        {"name": "window_train", "op": "window", "train": True, "seqs": 16, "lo": 64, "hi": 2048,
         "more": 0, "lens": 4, "hq": 16, "hkv": 16, "d": 128, "causal": 1, "window": 255, "sinks": 4},
        # a training step on a few long sequences, many query heads on few kv heads
        {"name": "window_train_long", "op": "window", "train": True, "seqs": 4, "lo": 4096,
         "hi": 16381, "more": 0, "lens": 5, "hq": 16, "hkv": 2, "d": 64, "causal": 1, "window": 1024,
         "sinks": 16},
        # one step of a few short chats: latency
        {"name": "decode_short", "op": "decode", "seqs": 3, "lo": 150, "hi": 700, "lens": 6,
         "hq": 32, "hkv": 8, "d": 128, "window": 256, "sinks": 4, "weights": False},
        # a serving batch with long contexts of which the window is read
        {"name": "decode_window", "op": "decode", "seqs": 64, "lo": 1000, "hi": 65536, "lens": 7,
         "hq": 32, "hkv": 8, "d": 128, "window": 4095, "sinks": 4, "weights": False},
        # a serving batch that keeps count of what its cached tokens are worth
        {"name": "decode_weights", "op": "decode", "seqs": 32, "lo": 16, "hi": 16384, "lens": 8,
         "hq": 32, "hkv": 8, "d": 128, "window": -1, "sinks": 0, "weights": True},
        # key weights of packed short prompts
        {"name": "weights_short", "op": "weights", "seqs": 16, "lo": 8, "hi": 1000, "more": 0,
         "lens": 9, "hq": 8, "hkv": 8, "d": 64, "causal": 1, "window": -1, "sinks": 0},
        # key weights of long-tailed prompts
        {"name": "weights_prompt", "op": "weights", "seqs": 24, "lo": 16, "hi": 8192, "more": 0,
         "lens": 10, "hq": 32, "hkv": 8, "d": 128, "causal": 1, "window": -1, "sinks": 0},
        # a batch at its budget after some steps: a few tokens of every sequence leave
        {"name": "evict_step", "op": "evict", "seqs": 64, "lo": 1025, "hi": 1088, "lens": 11,
         "budget": 1024, "recent": 256, "sinks": 4, "seen": 500, "hkv": 8, "d": 128},
        # long prompts cut down to their budget
        {"name": "evict_prompt", "op": "evict", "seqs": 8, "lo": 4000, "hi": 32768, "lens": 12,
         "budget": 4096, "recent": 512, "sinks": 4, "seen": 0, "hkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "decode", "decode", "weights", "evict", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7])
    seed = rng.randrange(1 << 30)
    window, sinks = _log_int(rng, 1, 2000), rng.choice([0, 1, 3, 4, 16, 64, 100, 129, 200])
    if op in ("window", "weights"):
        seqs = rng.randint(1, 24)
        # tokens * heads * head_dim * keys seen stays below the largest listed cases'
        most = 32768 * 16 * 64 * 1024 // (hq * d)
        if op == "window":
            hi = _log_int(rng, 16, min(16384, max(16, most // (seqs * (window + sinks + BLOCK)))))
        else:
            hi = _log_int(rng, 16, min(8192, max(16, int(math.sqrt(most // seqs)))))
        causal = rng.choice([1, 2])
        case = {"op": op, "seqs": seqs, "lo": 1, "hi": hi,
                "more": _log_int(rng, 1, 2000) if causal == 2 else 0, "lens": seed, "hq": hq,
                "hkv": hkv, "d": d, "causal": causal, "window": window, "sinks": sinks}
        if op == "window":
            case["train"] = rng.random() < 0.5
        elif rng.random() < 0.7:
            case["window"], case["sinks"] = -1, 0
        return case
    if op == "decode":
        seqs = _log_int(rng, 1, 128)
        most = 64 * 4096 * 8 * 128 // (hkv * d * seqs)
        if rng.random() < 0.5:
            window, sinks = -1, 0
            hi = _log_int(rng, 1, min(65536, most))
        else:
            window = min(window, most)
            hi = _log_int(rng, 1, min(65536, 4 * most))
        return {"op": op, "seqs": seqs, "lo": 1, "hi": hi, "lens": seed,
                "hq": hkv * rng.choice([1, 2, 4, 5, 8, 12, 16]), "hkv": hkv, "d": d,
                "window": window, "sinks": sinks, "weights": rng.random() < 0.5}
    seqs = rng.randint(1, 64)
    hi = _log_int(rng, 20, min(32768, 4 * 32768 * 8 * 128 // (seqs * hkv * d)))
    budget = rng.randint(1, hi)
    return {"op": op, "seqs": seqs, "lo": max(1, hi // 8), "hi": hi, "lens": seed, "budget": budget,
            "recent": rng.randint(0, budget), "sinks": rng.choice([0, 1, 4, 17]),
            "seen": rng.choice([0, rng.randint(1, 500)]), "hkv": hkv, "d": d}


# ------------------------------------------------------------------ inputs

def _key_lengths(case, lq):
    """Keys of each sequence: its queries and the context that they continue."""
    if case["causal"] == 1:
        return lq
    r = random.Random(case["lens"] + 1)
    return [n + r.randint(0, case["more"]) for n in lq]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=_dev())


def _prepare_varlen(case, seed):
    g = _gen(seed)
    lq = _lengths(case)
    lk = _key_lengths(case, lq)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def normal(n, h):
        return torch.randn(n, h, d, generator=g, device=_dev()).bfloat16()

    s = {"q": normal(sum(lq), hq), "k": normal(sum(lk), hkv), "v": normal(sum(lk), hkv),
         "cu_q": _cu(lq), "cu_k": _cu(lk), "lq": lq, "lk": lk, "max_q": max(lq),
         "causal": case["causal"], "window": case["window"], "sinks": case["sinks"],
         "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "window":
        s["train"] = case["train"]
        if s["train"]:
            s["dout"] = normal(sum(lq), hq)
        if own:
            vfa = _vfa()
            s["ws"] = vfa.alloc_workspace(len(lq), sum(lq), sum(lk), hq, d, device=_dev())
            if s["train"]:
                s["bws"] = vfa.alloc_bwd_workspace(len(lq), sum(lq), hq, d, device=_dev(),
                                                   sink_tokens=case["sinks"])
        return s
    # what the forward pass of the prompt left, and the weights of earlier chunks
    s["lse"] = torch.cat([_sequence_lse(s, b) for b in range(len(lq))])
    s["weights"] = torch.rand(len(lq), hkv, max(lk) + 13, generator=g, device=_dev())
    s["weights_out"] = torch.zeros_like(s["weights"])
    if own:
        s["ws"] = _vfa().alloc_key_weights_workspace(len(lq), sum(lq), sum(lk), max(lq), hq,
                                                     device=_dev())
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


def _prepare_decode(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    blocks = sum(-(-n // PAGE) for n in lens)
    cap = max(-(-n // PAGE) for n in lens)

    def pool():
        return torch.randn(blocks, PAGE, hkv, d, generator=g, device=_dev(), dtype=torch.bfloat16)

    s = {"q": torch.randn(len(lens), hq, d, generator=g, device=_dev()).bfloat16(),
         "k_pool": pool(), "v_pool": pool(), "tables": _tables(lens, blocks, cap, g),
         "counts": torch.tensor(lens, dtype=torch.int32, device=_dev()), "longest": max(lens),
         "window": case["window"], "sinks": case["sinks"], "weights": None, "weights_out": None,
         "scale": 1.0 / math.sqrt(d)}
    if case["weights"]:
        s["weights"] = torch.rand(len(lens), hkv, cap * PAGE, generator=g, device=_dev())
        s["weights_out"] = torch.zeros_like(s["weights"])
    if own:
        s["ws"] = _vfa().alloc_paged_decode_workspace(len(lens), hq, hkv, d,
                                                      capacity=cap if case["weights"] else 0,
                                                      device=_dev())
    return s


def _prepare_evict(case, seed):
    g = _gen(seed)
    lens = _lengths(case)
    hkv, d, n = case["hkv"], case["d"], len(lens)
    blocks = sum(-(-x // PAGE) for x in lens) + 5
    cap = max(-(-x // PAGE) for x in lens)

    def pool():
        return torch.randn(blocks, PAGE, hkv, d, generator=g, device=_dev(), dtype=torch.bfloat16)

    tables = _tables(lens, blocks, cap, g)
    refs = torch.zeros(blocks, dtype=torch.int32, device=_dev())
    for i, x in enumerate(lens):
        refs[tables[i, :-(-x // PAGE)].long()] = 1
    # of sequences that were cut before, the first tokens have their positions written down
    known = min(min(lens), case["budget"]) if case["seen"] else 0
    positions = torch.zeros(n, hkv, cap * PAGE, dtype=torch.int32, device=_dev())
    if known:
        score = torch.rand(n, hkv, known + case["seen"], generator=g, device=_dev())
        positions[:, :, :known] = score.argsort(-1)[:, :, :known].int()
    history = torch.tensor([[known, case["seen"] if known else 0]] * n, dtype=torch.int32,
                           device=_dev())
    s = {"k_pool": pool(), "v_pool": pool(), "tables": tables, "refs": refs,
         "counts": torch.tensor(lens, dtype=torch.int32, device=_dev()),
         "budgets": torch.full((n,), case["budget"], dtype=torch.int32, device=_dev()),
         "weights": torch.randn(n, hkv, cap * PAGE, generator=g, device=_dev()).exp(),
         "positions": positions, "history": history, "sinks": case["sinks"],
         "recent": case["recent"], "longest": max(lens)}
    s["weights_out"] = torch.zeros_like(s["weights"])
    for name in ("positions", "history", "refs", "counts"):
        s[name + "_out"] = torch.zeros_like(s[name])
    s["kept"] = torch.zeros_like(s["counts"])
    if own:
        s["ws"] = _vfa().alloc_evict_workspace(n, hkv, cap, device=_dev())
    return s


def prepare(case, seed):
    s = {"window": _prepare_varlen, "weights": _prepare_varlen, "decode": _prepare_decode,
         "evict": _prepare_evict}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------ plain forms

def _blocks(s):
    """The queries in blocks of BLOCK rows, the keys that a block's rows may see, and the mask.

    (query rows [n, B], key rows [n, KK], mask [n, B, KK], block and row of every token)."""
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q.diff(), cu_k.diff()
    per = (lq + BLOCK - 1) // BLOCK
    n = sum(-(-x // BLOCK) for x in s["lq"])
    start = per.cumsum(0) - per
    seq = torch.repeat_interleave(torch.arange(len(per), device=_dev()), per, output_size=n)
    row = ((torch.arange(n, device=_dev()) - start[seq]) * BLOCK)[:, None] + \
        torch.arange(BLOCK, device=_dev())
    off = (lk - lq if s["causal"] == 2 else torch.zeros_like(lq))[seq][:, None]
    window = min(s["window"], max(s["lk"]) + max(s["lq"]))
    first = row[:, :1] + off - window
    near = first + torch.arange(window + BLOCK, device=_dev())          # the window's keys
    sink = torch.arange(s["sinks"], device=_dev()).expand(n, -1)
    edge = (row + off - window)[:, :, None]                             # first key of a row's window
    own_row = (row < lq[seq][:, None])[:, :, None]
    len_k = lk[seq][:, None, None]
    see_near = (near[:, None] >= edge.clamp(min=0)) & (near[:, None] <= (row + off)[:, :, None]) & \
        (near[:, None] < len_k) & own_row
    see_sink = (sink[:, None] < edge) & (sink[:, None] < len_k) & own_row
    key = torch.cat((sink, near), 1)
    tok = torch.arange(s["q"].shape[0], device=_dev())
    of = torch.searchsorted(cu_q, tok, right=True) - 1
    local = tok - cu_q[of]
    return ((cu_q[seq][:, None] + row).clamp(max=max(s["q"].shape[0] - 1, 0)),
            (cu_k[seq][:, None] + key).clamp(0, max(s["k"].shape[0] - 1, 0)),
            torch.cat((see_sink, see_near), 2), start[of] + local // BLOCK, local % BLOCK)


def _plain_window(s):
    q, k, v, scale = s["q"], s["k"], s["v"], s["scale"]
    t, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    rows, keys, mask, blk, at = _blocks(s)
    n, b = rows.shape

    def heads(x):                                        # [n, B, Hq, D] -> [n, Hkv, G * B, D]
        return x.float().view(n, b, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * b, d)

    def tokens(x):                                       # and back, to the packed tokens
        return x.view(n, hkv, g, b, -1)[blk, :, :, at].reshape(t, hq, -1)

    qb = heads(q[rows])
    kb, vb = (x[keys].float().permute(0, 2, 1, 3) for x in (k, v))
    x = (qb @ kb.transpose(-1, -2)).mul_(scale).view(n, hkv, g, b, -1)
    x = x.masked_fill_(~mask[:, None, None], -math.inf).view(n, hkv, g * b, -1)
    m = x.amax(-1, keepdim=True)
    p = (x - m.masked_fill(m == -math.inf, 0.0)).exp()
    z = p.sum(-1, keepdim=True)
    lse = torch.where(z > 0, m + z.log(), torch.full_like(m, -FLT_MAX))
    p = p / z.masked_fill(z == 0, 1.0)
    o = p @ vb
    res = [tokens(o).bfloat16(), tokens(lse)[..., 0]]
    if not s["train"]:
        return res
    do = heads(s["dout"][rows])
    dp = do @ vb.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = (ds @ kb) * scale
    res.append(tokens(dq).bfloat16())
    for part, f, like in ((ds.transpose(-1, -2) @ qb, scale, k), (p.transpose(-1, -2) @ do, 1.0, v)):
        acc = torch.zeros(like.shape, device=_dev())
        acc.index_add_(0, keys.reshape(-1), part.permute(0, 2, 1, 3).reshape(-1, hkv, d))
        res.append((acc * f).bfloat16())
    return res


def _plain_decode(s):
    q, tables, n = s["q"].float(), s["tables"].long(), s["counts"].long()[:, None]
    seqs, hq, d = q.shape
    hkv = s["k_pool"].shape[2]
    if s["window"] < 0 or s["window"] + s["sinks"] >= s["longest"]:
        pos = torch.arange(s["longest"], device=_dev()).expand(seqs, -1)
        live = pos < n
        if s["window"] >= 0:
            live = live & ((pos >= n - 1 - s["window"]) | (pos < s["sinks"]))
    else:
        sink = torch.arange(s["sinks"], device=_dev()).expand(seqs, -1)
        near = n - 1 - s["window"] + torch.arange(s["window"] + 1, device=_dev())
        live = torch.cat(((sink < n - 1 - s["window"]) & (sink < n), near >= 0), 1)
        pos = torch.cat((sink, near), 1).clamp(min=0)
    page = tables.gather(1, torch.where(live, pos, 0) // PAGE)
    k, v = (x[page, pos % PAGE].float().permute(0, 2, 1, 3) for x in (s["k_pool"], s["v_pool"]))
    x = (q.view(seqs, hkv, -1, d) @ k.transpose(-1, -2)).mul_(s["scale"])
    x = x.masked_fill_(~live[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    z = p.sum(-1, keepdim=True)
    p = p / z
    res = [(p @ v).reshape(seqs, hq, d).bfloat16(), (m + z.log()).reshape(seqs, hq)]
    if s["weights"] is not None:
        # the weights at their slots, those of no slot behind the last one
        size = s["weights"].shape[2]
        at = torch.where(live, pos, size)[:, None].expand(-1, hkv, -1)
        got = torch.zeros(seqs, hkv, size + 1, device=_dev()).scatter_(2, at, p.sum(2))[:, :, :size]
        seen = torch.zeros(seqs, 1, size + 1, dtype=torch.bool, device=_dev())
        seen = seen.scatter_(2, at[:, :1], True)[:, :, :size]
        # slots that are not seen keep what the output held
        out = s["weights_out"]
        out.copy_(torch.where(seen, s["weights"] + got, out))
        res.append(out)
    return res


def _seen(s, b):
    """The mask [Lq, Lk] of sequence b."""
    lq, lk = s["lq"][b], s["lk"][b]
    i = torch.arange(lq, device=_dev())[:, None] + (lk - lq if s["causal"] == 2 else 0)
    j = torch.arange(lk, device=_dev())
    m = j <= i
    if s["window"] >= 0:
        m = m & ((j >= i - s["window"]) | (j < s["sinks"]))
    return m


def _sequence_logits(s, b):
    """Logits [Hkv, G, Lq, Lk] of sequence b, -inf where a key is not seen."""
    q0, k0 = sum(s["lq"][:b]), sum(s["lk"][:b])
    hq, d = s["q"].shape[1:]
    hkv = s["k"].shape[1]
    q = s["q"][q0:q0 + s["lq"][b]].float().view(-1, hkv, hq // hkv, d).permute(1, 2, 0, 3)
    k = s["k"][k0:k0 + s["lk"][b]].float().permute(1, 2, 0)
    x = (q.reshape(hkv, -1, d) @ k).mul_(s["scale"]).view(hkv, hq // hkv, s["lq"][b], -1)
    return x.masked_fill_(~_seen(s, b), -math.inf)


def _sequence_lse(s, b):
    """The rows' log-sum-exp [Lq, Hq], -FLT_MAX where nothing is seen."""
    x = _sequence_logits(s, b)
    m = x.amax(-1, keepdim=True).clamp(min=-FLT_MAX)
    lse = (m + (x - m).exp_().sum(-1, keepdim=True).log()).clamp(min=-FLT_MAX)
    return lse[..., 0].permute(2, 0, 1).reshape(s["lq"][b], -1)


def _plain_weights(s):
    hkv = s["k"].shape[1]
    out = s["weights_out"]
    q0 = 0
    for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
        x = _sequence_logits(s, b)
        lse = s["lse"][q0:q0 + lq].view(lq, hkv, -1).permute(1, 2, 0)[..., None]
        out[b, :, :lk] = s["weights"][b, :, :lk] + (x - lse).exp_().sum((1, 2))
        q0 += lq
    return [out]


def _plain_evict(s):
    n, hkv = s["counts"].long()[:, None, None], s["k_pool"].shape[2]
    w = s["weights"][:, :, :s["longest"]]
    slot = torch.arange(s["longest"], device=_dev())
    known, gone = (s["history"][:, i].long()[:, None, None] for i in (0, 1))
    pos = torch.where(slot < known, s["positions"][:, :, :s["longest"]].long(), slot + gone)
    budget = s["budgets"].long()[:, None, None]
    b = torch.where(budget < 0, n, torch.minimum(budget, n))
    sinks = b.clamp(max=s["sinks"])
    recent = (b - sinks).clamp(max=s["recent"])
    live = slot < n
    kind = live.int() + ((pos < sinks) | (pos >= n + gone - recent)) * live
    # by kind, then by weight, then by slot: two stable sorts
    order = w.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(2, kind.gather(2, order).sort(dim=-1, descending=True, stable=True).indices)
    keep = torch.zeros_like(live.expand(-1, hkv, -1)).scatter_(2, order, (slot < b).expand(-1, hkv, -1))
    # the kept tokens past the budget go to the free slots below it, both in ascending order
    hole = ~keep & (slot < b)
    movers = (~(keep & (slot >= b))).int().argsort(dim=-1, stable=True)
    src = torch.where(hole, movers.gather(2, (hole.cumsum(-1) - 1).clamp(min=0)), slot)
    stay = slot < b
    for out, x in ((s["weights_out"], w), (s["positions_out"], pos.int())):
        o = out[:, :, :s["longest"]]
        o.copy_(torch.where(stay, x.gather(2, src), o))
    zero = s["weights_out"][:, :, :s["longest"]]
    zero.masked_fill_(live & ~stay, 0.0)
    sq, h, dst = hole.nonzero(as_tuple=True)
    frm = src[sq, h, dst]
    tables = s["tables"].long()
    pd, ps = tables[sq, dst // PAGE], tables[sq, frm // PAGE]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[pd, dst % PAGE, h] = pool[ps, frm % PAGE, h]
    kept, count = b[:, 0, 0], n[:, 0, 0]
    s["kept"].copy_(kept)
    s["history_out"].copy_(torch.stack((kept, gone[:, 0, 0] + count - kept), 1))
    # the pages behind the kept tokens go back
    page = torch.arange(tables.shape[1], device=_dev())
    up = ((page >= ((kept + PAGE - 1) // PAGE)[:, None]) & (page < ((count + PAGE - 1) // PAGE)[:, None]))
    s["refs_out"].copy_(s["refs"])
    s["refs_out"].scatter_add_(0, torch.where(up, tables, 0).view(-1), -up.int().view(-1))
    s["counts_out"].copy_(kept)
    return [s[x] for x in ("k_pool", "v_pool", "weights_out", "positions_out", "history_out", "kept",
                           "refs_out", "counts_out")]


# ------------------------------------------------------------------ the framework's operators

def _own_window(s):
    vfa = _vfa()
    out, lse = vfa.varlen_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["scale"],
                              s["causal"], workspace=s["ws"], window_left=s["window"],
                              sink_tokens=s["sinks"])
    if not s["train"]:
        return [out, lse]
    dq, dk, dv, _ = vfa.varlen_bwd(s["q"], s["k"], s["v"], out, s["dout"], lse, s["cu_q"], s["cu_k"],
                                   s["scale"], s["causal"], window_left=s["window"],
                                   workspace=s["bws"], sink_tokens=s["sinks"])
    return [out, lse, dq, dk, dv]


def _own_decode(s):
    out, lse = _vfa().paged_decode(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["counts"],
                                   window_left=s["window"], sink_tokens=s["sinks"],
                                   softmax_scale=s["scale"], key_weights=s["weights"],
                                   key_weights_out=s["weights_out"], workspace=s["ws"])
    return [out, lse] if s["weights"] is None else [out, lse, s["weights_out"]]


def _own_weights(s):
    return [_vfa().varlen_key_weights(s["q"], s["k"], s["lse"], s["cu_q"], s["cu_k"], s["max_q"],
                                      s["scale"], s["causal"], s["weights"],
                                      window_left=s["window"], sink_tokens=s["sinks"],
                                      key_weights_out=s["weights_out"], workspace=s["ws"])]


def _own_evict(s):
    vfa = _vfa()
    vfa.cache_evict(s["k_pool"], s["v_pool"], s["refs"], s["tables"], s["counts"], s["budgets"],
                    s["weights"], s["positions"], s["history"], sink_tokens=s["sinks"],
                    recent_tokens=s["recent"], key_weights_out=s["weights_out"],
                    positions_out=s["positions_out"], history_out=s["history_out"], kept=s["kept"],
                    workspace=s["ws"])
    vfa.pages_truncate(s["refs"], s["tables"], s["counts"], s["kept"], PAGE,
                       refcounts_out=s["refs_out"], token_counts_out=s["counts_out"])
    return [s[x] for x in ("k_pool", "v_pool", "weights_out", "positions_out", "history_out", "kept",
                           "refs_out", "counts_out")]


def run(state):
    plain = {"window": _plain_window, "decode": _plain_decode, "weights": _plain_weights,
             "evict": _plain_evict}
    ours = {"window": _own_window, "decode": _own_decode, "weights": _own_weights,
            "evict": _own_evict}
    return (ours if own else plain)[state["op"]](state)


# ------------------------------------------------------------------ 64-bit definitions

def _exact_varlen(case, s):
    """Sequence by sequence and kv head by kv head on whole matrices; the gradients by
    differentiating the forward pass."""
    train = case["op"] == "window" and case["train"]
    hq, d = s["q"].shape[1:]
    hkv = s["k"].shape[1]
    g = hq // hkv
    outs = [torch.zeros(s["q"].shape, dtype=torch.float64, device=_dev()),
            torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=_dev())]
    if train:
        outs += [torch.zeros(s[x].shape, dtype=torch.float64, device=_dev()) for x in "qkv"]
    if case["op"] == "weights":
        w = s["weights_out"].double()
    q0 = k0 = 0
    for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
        shift = lk - lq if case["causal"] == 2 else 0
        dist = torch.arange(lq, device=_dev())[:, None] + shift - torch.arange(lk, device=_dev())
        hidden = dist < 0
        if case["window"] >= 0:
            hidden |= (dist > case["window"]) & (torch.arange(lk, device=_dev()) >= case["sinks"])
        empty = hidden.all(1)
        for h in range(hkv):
            sq, sk = slice(q0, q0 + lq), slice(k0, k0 + lk)
            hs = slice(h * g, (h + 1) * g)
            q, k, v = s["q"][sq, hs].double(), s["k"][sk, h].double(), s["v"][sk, h].double()
            x = torch.einsum("ihd,jd->hij", q, k) / math.sqrt(d)
            if case["op"] == "weights":
                p = torch.exp(x - s["lse"][sq, hs].double().T[..., None]).masked_fill(hidden, 0.0)
                w[b, h, :lk] = s["weights"][b, h, :lk].double() + p.sum((0, 1))
                continue
            x.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(x, -1)
            outs[1][sq, hs] = torch.where(empty[:, None], -FLT_MAX, lse.T)
            p = torch.exp(x - lse.masked_fill(empty, 0.0)[..., None])
            del x
            outs[0][sq, hs] = torch.einsum("hij,jd->ihd", p, v)
            if train:
                do = s["dout"][sq, hs].double()
                outs[4][sk, h] = torch.einsum("hij,ihd->jd", p, do)
                dp = torch.einsum("ihd,jd->hij", do, v)
                dp -= torch.einsum("ihd,ihd->hi", do, outs[0][sq, hs])[..., None]
                dp *= p
                outs[2][sq, hs] = torch.einsum("hij,jd->ihd", dp, k) / math.sqrt(d)
                outs[3][sk, h] = torch.einsum("hij,ihd->jd", dp, q) / math.sqrt(d)
        q0 += lq
        k0 += lk
    return [w] if case["op"] == "weights" else outs


def _exact_decode(case, s):
    hq, d = s["q"].shape[1:]
    hkv = s["k_pool"].shape[2]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=_dev())
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=_dev())
    w = s["weights_out"].double() if case["weights"] else None
    for b, n in enumerate(_lengths(case)):
        ids = s["tables"][b, :-(-n // PAGE)].long()
        j = torch.arange(n, device=_dev())
        if case["window"] >= 0:
            j = j[(j >= n - 1 - case["window"]) | (j < case["sinks"])]
        for h in range(hkv):
            k, v = (x[ids, :, h].reshape(-1, d)[j].double() for x in (s["k_pool"], s["v_pool"]))
            x = s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(d)
            p = torch.softmax(x, -1)
            out[b, h * g:(h + 1) * g] = p @ v
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
            if w is not None:
                w[b, h, j] = s["weights"][b, h, j].double() + p.sum(0)
    return [out, lse] if w is None else [out, lse, w]


def exact(case, seed):
    if case["op"] == "evict":
        return None                                  # whole numbers and moved values
    s = prepare(case, seed)
    return _exact_decode(case, s) if case["op"] == "decode" else _exact_varlen(case, s)


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(case, lq, lk):
    """Visible (query, key) pairs of one query head in all sequences."""
    total = 0
    for a, b in zip(lq, lk):
        shift = b - a if case["causal"] == 2 else 0
        for i in range(shift, shift + a):
            seen = min(i + 1, b)
            if case["window"] >= 0:
                first = max(0, i - case["window"])
                seen = max(0, seen - first) + min(case["sinks"], first, b)
            total += seen
    return total


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    lens = _lengths(case)
    if op in ("window", "weights"):
        lk = _key_lengths(case, lens)
        hq, pairs = case["hq"], _pairs(case, lens, lk)
        q, k = sum(lens) * hq * d * 2, sum(lk) * hkv * d * 2
        if op == "weights":
            return {"bytes": q + k + sum(lens) * hq * 4 + sum(lk) * hkv * 8,
                    "flops": 2 * pairs * hq * d}
        if case["train"]:
            return {"bytes": 5 * q + 4 * k + sum(lens) * hq * 4, "flops": 14 * pairs * hq * d}
        return {"bytes": 2 * q + 2 * k + sum(lens) * hq * 4, "flops": 4 * pairs * hq * d}
    if op == "decode":
        n = sum(x if case["window"] < 0 else
                min(x, case["window"] + 1) + min(case["sinks"], max(0, x - case["window"] - 1))
                for x in lens)
        return {"bytes": n * hkv * (4 * d + (8 if case["weights"] else 0)) +
                case["seqs"] * case["hq"] * d * 4, "flops": 4 * n * case["hq"] * d}
    # eviction: weights and positions in and out; the kept tokens past the budget move
    moved = 0.0
    for n in lens:
        b = min(n, case["budget"])
        sinks = min(case["sinks"], b)
        recent = min(case["recent"], b - sinks)
        rest = n - sinks - recent                    # candidates, in no order of weight
        past = max(0, n - recent - max(b, sinks))
        moved += (recent if n - recent >= b else n - b) + \
            (b - sinks - recent) * past / max(rest, 1)
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": int(moved * hkv * 8 * d + hkv * (sum(lens) * 8 + kept * 4)),
            "flops": hkv * sum(lens)}
