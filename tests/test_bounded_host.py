"""Host-side refusals of the bounded cache's operators (no GPU): bad arguments come back with a
status before any device work.  No call here launches a kernel."""
import ctypes

import pytest

FAKE, ODD, NUL = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100002), None
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def vfa():
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


def _calls(vfa, fn, good, cases):
    """Each case changes one argument of a call that is good: (index, value, status, word)."""
    L = vfa.lib()
    for at, value, status, word in cases:
        args = list(good)
        args[at] = value
        assert getattr(L, fn)(*args) == status, (fn, at, value)
        assert word in L.vfa_last_error(), (at, value, L.vfa_last_error())


def test_forward_and_backward_with_sinks(vfa):
    bad, uns = vfa.VFA_ERR_INVALID_ARG, vfa.VFA_ERR_UNSUPPORTED
    good = [FAKE] * 5 + [4, 4, 4, 1, 2, 2, 128, 0.1, 1, 8, 4, FAKE, FAKE, FAKE, 1 << 30, NUL]
    _calls(vfa, "vfa_varlen_fwd_sinks", good, [
        (0, NUL, bad, b"null"), (15, -1, bad, b"sink_tokens"), (13, 0, bad, b"window"), (13, 3, bad, b"causal"),
        (11, 96, uns, b"head_dim"), (10, 3, bad, b"num_kv_heads"), (19, 16, bad, b"workspace"),
        (0, ODD, bad, b"aligned"), (12, NAN, bad, b"softmax_scale")])
    good = [FAKE] * 8 + [4, 4, 1, 2, 2, 128, 0.1, 1, 8, 4, FAKE, FAKE, FAKE, FAKE, 1 << 30, NUL]
    _calls(vfa, "vfa_varlen_bwd_sinks", good, [
        (0, NUL, bad, b"null"), (17, -1, bad, b"sink_tokens"), (15, 0, bad, b"window"),
        (13, 96, uns, b"head_dim"), (14, 0.0, bad, b"softmax_scale"), (22, 512, bad, b"workspace"),
        (4, ODD, bad, b"aligned")])
    L = vfa.lib()
    size = L.vfa_varlen_bwd_sinks_workspace_bytes
    plain = L.vfa_varlen_bwd_workspace_bytes
    assert size(0, 4, 2, 128, 4) == size(1, 4, 2, 96, 4) == size(1, 4, 2, 128, -1) == 0
    for d in (64, 128, 256):
        assert plain(3, 1000, 4, d) < size(3, 1000, 4, d, 1) <= size(3, 1000, 4, d, 500)
        assert size(3, 1 << 20, 4, d, 0x7fffffff) - plain(3, 1 << 20, 4, d) <= 40 << 20


def test_backward_workspace_covers_the_chunks(vfa):
    """As many partials as the chunks of any batch of these totals take."""
    import random
    rng = random.Random(1)
    for _ in range(300):
        d = rng.choice([64, 128, 256])
        step, split = {64: 96, 128: 64, 256: 32}[d], 2 if d == 256 else 1
        hkv, group = rng.choice([1, 2, 8]), rng.choice([1, 4, 7])
        lq = [rng.choice([0, 1, 50, 1000, 9000, 40000]) for _ in range(rng.randint(1, 6))]
        lk = [rng.choice([0, 1, 100, 5000]) for _ in lq]
        sinks = rng.choice([1, 4, 128, 129, 1000, 0x7fffffff])
        tiles = [-(-min(sinks, n) // 128) for n in lk]
        steps = [-(-n // step) * group for n in lq]
        total = sum(a * b for a, b in zip(tiles, steps)) * hkv * split
        per = max(32, -(-total // 152))
        parts = sum(t * c for t, c in zip(tiles, (-(-s // per) for s in steps)) if c > 1) * hkv * split
        have = vfa.lib().vfa_varlen_bwd_sinks_workspace_bytes(len(lq), sum(lq), hkv * group, d, sinks) - \
            vfa.lib().vfa_varlen_bwd_workspace_bytes(len(lq), sum(lq), hkv * group, d)
        assert parts * 2 * 128 * min(d, 128) * 4 + 12 * (len(lq) + 1) <= have


def test_paged_decode(vfa):
    bad, uns = vfa.VFA_ERR_INVALID_ARG, vfa.VFA_ERR_UNSUPPORTED
    good = [FAKE, FAKE, FAKE, 10, FAKE, 4, FAKE, 2, 8, 2, 128, 16, 4, 0.1, FAKE, FAKE, FAKE, FAKE, NUL,
            FAKE, 1 << 30, NUL]
    _calls(vfa, "vfa_paged_decode", good, [
        (0, NUL, bad, b"null"), (1, NUL, bad, b"null"), (6, NUL, bad, b"null"), (17, NUL, bad, b"null"),
        (7, 0, bad, b"size"), (10, 96, uns, b"head_dim"), (9, 3, bad, b"num_kv_heads"),
        (3, 1 << 27, uns, b"num_blocks"), (5, -1, bad, b"size"), (5, 1 << 28, uns, b"capacity"),
        (12, -1, bad, b"sink_tokens"), (13, NAN, bad, b"softmax_scale"), (13, INF, bad, b"softmax_scale"),
        (1, ODD, bad, b"aligned"), (14, ODD, bad, b"aligned"), (16, ctypes.c_void_p(0x100001), bad, b"aligned"),
        (19, NUL, bad, b"workspace"), (19, ctypes.c_void_p(0x100010), bad, b"workspace"),
        (20, 1000, bad, b"workspace"), (7, 1 << 29, uns, b"large")])
    size = vfa.lib().vfa_paged_decode_workspace_bytes
    assert size(0, 8, 2, 128, 0) == size(1, 8, 3, 128, 0) == size(1, 8, 2, 96, 0) == size(1, 8, 2, 128, -1) == 0
    assert size(4, 8, 2, 128, 3) - size(4, 8, 2, 128, 0) >= 4 * 8 * (8 + 3 * 16 * 4)


def _key_weight_partials(lq, lk, total_q, total_k, most_q, heads, kv_heads, step):
    """Bytes of the partial sums of a batch, by the rule of its chunks' length."""
    pairs = total_k // 256 + 1
    chunks = max(128, 16 * 608 // pairs)
    steps = -(-min(total_q, most_q) // 64) * heads
    per = max(16 if heads * pairs < 608 else 128, -(-steps // chunks))
    longest = max(-(-(-(-n // step) * (heads // kv_heads)) // per) for n in lq)
    return 2 * longest * kv_heads * total_k * 4


def test_key_weights_workspace_serves_smaller_calls(vfa):
    """It covers the partial sums of every batch of its sizes and of smaller ones with as many heads, and
    does not grow with the square of a prompt."""
    import random
    rng = random.Random(2)
    size = vfa.lib().vfa_varlen_key_weights_workspace_bytes
    assert size(1, 8192, 8192, 8192, 32) >= size(1, 4607, 4607, 4607, 32)
    assert size(1, 4864, 4864, 4864, 32) >= size(1, 4863, 4863, 4863, 32)
    for n in (1 << 17, 1 << 20):
        assert size(1, n, n, n, 32) <= n * 8 * (128 + 32) + 4096        # 168 MB at 131072 tokens
    assert size(2, 100, 50, 1 << 30, 4) == size(2, 100, 50, 100, 4)     # no query length is above all of them
    for _ in range(3000):
        heads = rng.choice([1, 2, 7, 8, 32, 64, 700])
        kv_heads = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
        n = rng.randint(1, 5)
        lens = lambda: [int(2 ** rng.uniform(0, 20)) * rng.randint(0, 1) for _ in range(n)]
        lq, lk = lens(), lens()
        tq, tk, most = sum(lq), sum(lk), max(lq)
        have = size(n, tq, tk, most, heads)
        assert have - 8 * (n + 1) >= max(_key_weight_partials(lq, lk, tq, tk, most, heads, kv_heads, step)
                                         for step in (64, 128))
        bigger = [x + rng.choice([0, 1, 255, 5000, 1 << 18]) for x in (n, tq, tk, most)]
        assert size(*bigger, heads) >= have


def test_paged_decode_workspace_without_room_for_logits(vfa):
    """A workspace made without key weights, however many sequences it is for, is too small with them."""
    size = vfa.lib().vfa_paged_decode_workspace_bytes
    for d in (64, 128, 256):
        none = size(4096, 32, 8, d, 0)
        assert none < size(1, 32, 8, d, 1)
        good = [FAKE, FAKE, FAKE, 10, FAKE, 1, FAKE, 1, 32, 8, d, -1, 0, 0.1, FAKE, FAKE, FAKE, FAKE, NUL,
                FAKE, none, NUL]
        _calls(vfa, "vfa_paged_decode", good, [(20, none, vfa.VFA_ERR_INVALID_ARG, b"workspace too small")])


def test_key_weights(vfa):
    bad, uns = vfa.VFA_ERR_INVALID_ARG, vfa.VFA_ERR_UNSUPPORTED
    good = [FAKE] * 5 + [4, 4, 4, 1, 2, 2, 128, 0.1, 1, 8, 4, FAKE, FAKE, 10, FAKE, 1 << 30, NUL]
    _calls(vfa, "vfa_varlen_key_weights", good, [
        (0, NUL, bad, b"null"), (2, NUL, bad, b"null"), (17, NUL, bad, b"null"), (8, 0, bad, b"size"),
        (18, -1, bad, b"size"), (10, 3, bad, b"num_kv_heads"), (11, 96, uns, b"head_dim"),
        (12, -1.0, bad, b"softmax_scale"), (12, NAN, bad, b"softmax_scale"), (13, 3, bad, b"causal"),
        (13, 0, bad, b"window"), (15, -1, bad, b"sink_tokens"), (0, ODD, bad, b"aligned"),
        (19, NUL, bad, b"workspace"), (20, 100, bad, b"workspace"), (6, 0x7fffffff, uns, b"large")])
    assert vfa.lib().vfa_varlen_key_weights_workspace_bytes(0, 1, 1, 1, 1) == 0


def test_evict_and_truncate(vfa):
    bad, uns = vfa.VFA_ERR_INVALID_ARG, vfa.VFA_ERR_UNSUPPORTED
    good = [FAKE, FAKE, FAKE, 10, FAKE, 4, FAKE, FAKE, 2, 2, 128, FAKE, FAKE, FAKE, 1, 1, FAKE, FAKE, FAKE,
            FAKE, FAKE, 1 << 30, NUL, NUL]
    _calls(vfa, "vfa_cache_evict", good, [(i, NUL, bad, b"null") for i in (0, 1, 2, 4, 6, 7, 11, 12, 13, 16, 17,
                                                                           18, 19)] + [
        (14, -1, bad, b"sink_tokens"), (15, -1, bad, b"recent_tokens"), (10, 96, uns, b"head_dim"),
        (8, 0, bad, b"size"), (0, ODD, bad, b"aligned"), (11, ctypes.c_void_p(0x100001), bad, b"aligned"),
        (20, NUL, bad, b"workspace"), (21, 8, bad, b"workspace"), (5, 1 << 28, uns, b"capacity")])
    assert vfa.lib().vfa_cache_evict_workspace_bytes(0, 1, 1) == 0
    good = [FAKE, 10, FAKE, 4, FAKE, 2, FAKE, 16, FAKE, FAKE, FAKE, 64, NUL, NUL]
    _calls(vfa, "vfa_pages_truncate", good, [
        (0, NUL, bad, b"null"), (6, NUL, bad, b"null"), (8, NUL, bad, b"null"), (9, NUL, bad, b"null"),
        (7, 0, bad, b"size"), (1, 1 << 27, uns, b"num_blocks"), (10, NUL, bad, b"workspace"),
        (11, 15, bad, b"workspace"), (6, ODD, bad, b"aligned")])


def test_binding_refuses(vfa):
    import torch
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        vfa.paged_decode(x, pool, pool, i.view(4, 1), i)
    with pytest.raises(ValueError):
        vfa.varlen_key_weights(x, x, x[..., 0].float(), i[:2], i[:2], 4, 0.1, 1, torch.zeros(1, 1, 4))
    with pytest.raises(ValueError):
        vfa.cache_evict(pool, pool, i, i.view(4, 1), i, i, torch.zeros(4, 1, 16), i, i)
    with pytest.raises(ValueError):
        vfa.pages_truncate(i, i.view(4, 1), i, i, 16)
    with pytest.raises(ValueError):
        vfa.alloc_evict_workspace(1, 1, 1 << 31, device="cpu")
    with pytest.raises(vfa.VfaError):
        vfa.alloc_paged_decode_workspace(1, 3, 2, 64, device="cpu")


def test_rows_of_more_pages_than_a_pool(vfa):
    """A row's slots, and what a thread adds to a slot's number, stay within 32 bits."""
    most, uns = 1 << 26, vfa.VFA_ERR_UNSUPPORTED
    good = [FAKE, FAKE, FAKE, 10, FAKE, 4, FAKE, 2, 8, 2, 128, 16, 4, 0.1, FAKE, FAKE, FAKE, FAKE, NUL,
            FAKE, 1 << 30, NUL]
    _calls(vfa, "vfa_paged_decode", good, [(5, most + 1, uns, b"capacity")])
    good = [FAKE, FAKE, FAKE, 10, FAKE, 4, FAKE, FAKE, 2, 2, 128, FAKE, FAKE, FAKE, 1, 1, FAKE, FAKE, FAKE,
            FAKE, FAKE, 1 << 30, NUL, NUL]
    _calls(vfa, "vfa_cache_evict", good, [(5, most + 1, uns, b"capacity")])
    L = vfa.lib()
    assert L.vfa_paged_decode_workspace_bytes(1, 2, 2, 64, most) > L.vfa_paged_decode_workspace_bytes(1, 2, 2, 64, 0)
    assert L.vfa_paged_decode_workspace_bytes(1, 2, 2, 64, most + 1) == 0
    assert L.vfa_cache_evict_workspace_bytes(1, 2, most) > 0 == L.vfa_cache_evict_workspace_bytes(1, 2, most + 1)
