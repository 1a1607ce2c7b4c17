"""The operators around attention run together, as a server and a trainer run them."""
import math

import numpy as np
import pytest
import torch

import oracle.serving as O
from test_gpu_kv4 import _bounds, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vfa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


class Server:
    """Two layers of 4-bit pools over one page state."""
    D, Hq, Hkv, BS = 64, 8, 2, 16
    DK, DV = 0.25, 0.5

    def __init__(self, vfa, blocks=40, rows=6, cap=8, layers=2, seed=0):
        self.vfa, self.rows, self.layers = vfa, rows, layers
        self.g = torch.Generator().manual_seed(seed)
        self.refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
        self.tables = torch.full((rows, cap), -1, dtype=torch.int32, device="cuda")
        self.counts = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.pools = [vfa.alloc_kv4_pool(blocks, self.Hkv, self.D) for _ in range(layers)]
        self.ws = vfa.alloc_pages_workspace(blocks, rows, rows)
        self.dec_ws = vfa.alloc_kv4_decode_workspace(rows, self.Hq, self.Hkv, self.D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = [1000.0 ** (-i / 32) for i in range(32)]
        self.table = vfa.rope_table(f)
        self.w = [(1 + 0.1 * torch.randn(self.D, generator=self.g)).cuda() for _ in range(2)]
        # what each row holds per layer, from the same quantiser in 64 bits
        self.text = [[[] for _ in range(rows)] for _ in range(layers)]

    def step(self, add):
        """Tokens for every row (add[s] of them), through every layer; returns per layer the
        queries, keys and values of the new tokens and where they start."""
        vfa = self.vfa
        start = self.counts.clone()
        vfa.pages_extend(self.refs, self.tables, self.counts, _i32(add), self.BS, self.ws,
                         status=self.status)
        cu = np.concatenate(([0], np.cumsum(add)))
        total = int(cu[-1])
        pos = torch.cat([torch.arange(n) + int(start[s]) for s, n in enumerate(add)]).int().cuda()
        out = []
        for layer in range(self.layers):
            width = (self.Hq + 2 * self.Hkv) * self.D
            qkv = torch.randn(total, width, generator=self.g).bfloat16().cuda()
            cut = self.Hq * self.D
            q = qkv[:, :cut].view(total, self.Hq, self.D)
            k = qkv[:, cut:cut + self.Hkv * self.D].view(total, self.Hkv, self.D)
            v = qkv[:, cut + self.Hkv * self.D:].view(total, self.Hkv, self.D)
            q, k = vfa.qk_norm_rope(q, k, pos, self.table, self.w[0], self.w[1])
            vfa.kv4_write(k, v, self.pools[layer], self.tables, _i32(cu), start, self.DK, self.DV,
                          status=self.status)
            kq = O.dequantise(*O.quantise(k.double().cpu().numpy(), self.DK), self.DK)
            vq = O.dequantise(*O.quantise(v.double().cpu().numpy(), self.DV), self.DV)
            for s in range(self.rows):
                self.text[layer][s] += [(kq[t], vq[t]) for t in range(cu[s], cu[s + 1])]
            out.append((q, cu, start))
        return out

    def decode(self, layer, q):
        return self.vfa.kv4_decode(q, self.pools[layer], self.tables, self.counts, self.DK, self.DV,
                                   workspace=self.dec_ws, status=self.status)

    def reference(self, layer, q):
        """O.kv4_decode's tuple, from the rows' texts laid out as pages of a plain pool."""
        n = np.array([len(t) for t in self.text[layer]])
        cap = max(1, -(-n.max() // 16))
        pool = np.zeros((self.rows * cap, self.Hkv, 18 * self.D), np.uint8)
        tables = np.arange(self.rows * cap).reshape(self.rows, cap)
        for s, text in enumerate(self.text[layer]):
            for i, (k, v) in enumerate(text):
                O.write_token(pool, tables[s, i // 16], i % 16, k, v, self.DK, self.DV)
        return O.kv4_decode(q.double().cpu().numpy(), pool, tables, n, self.DK, self.DV), n

    def check(self, layer, q, got):
        ref, n = self.reference(layer, q)
        bo, bl = _bounds(ref, n)
        out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
        assert (np.abs(out - ref[0]) <= bo).all()
        assert (np.abs(lse - ref[1]) <= bl).all()
        assert self.vfa.read_status(self.status) == 0


def test_prompt_fork_decode_free_compact(vfa):
    sv = Server(vfa)
    prompt = sv.step([37, 16, 0, 0, 50, 0])
    # the prompts attend to themselves: cached keys and values, read back, through varlen_fwd
    for layer, (q, cu, start) in enumerate(prompt):
        k, v = vfa.kv4_gather(sv.pools[layer], sv.tables, _i32(cu), start, int(cu[-1]), sv.DK, sv.DV,
                              status=sv.status)
        out, lse = vfa.varlen_fwd(q, k, v, _i32(cu), _i32(cu), 50, 0.125, 2)
        qn, kn, vn = (t.double().cpu().numpy() for t in (q, k, v))
        for s in range(6):
            for i in range(cu[s], cu[s + 1]):
                for h in range(sv.Hq):
                    x = kn[cu[s]:i + 1, h // 4] @ qn[i, h] * 0.125
                    p = np.exp(x - x.max())
                    ref = p @ vn[cu[s]:i + 1, h // 4] / p.sum()
                    # varlen_fwd's own bound
                    assert (np.abs(out[i, h].double().cpu().numpy() - ref) <= 1e-2 + 1e-2 * np.abs(ref)).all()
        ref = O.dequantise(*O.quantise(k.double().cpu().numpy(), sv.DK), sv.DK)
        assert np.array_equal(kn, ref)                     # cached values are fixed points
    # two samples of row 0, one of row 1
    vfa.pages_fork(sv.refs, sv.tables, sv.counts, _i32([0, 0, 1]), _i32([2, 3, 5]), sv.pools, sv.BS,
                   sv.ws, status=sv.status)
    for layer in range(2):
        for c, p in ((2, 0), (3, 0), (5, 1)):
            sv.text[layer][c] = list(sv.text[layer][p])
    # every row takes tokens of its own
    for add in ([1] * 6, [1] * 6, [3, 1, 1, 17, 1, 2]):
        new = sv.step(add)
        for layer, (q, cu, _) in enumerate(new):
            last = q[torch.as_tensor(cu[1:] - 1).cuda()].contiguous()
            sv.check(layer, last, sv.decode(layer, last))
    # rows 0 and 4 end; the pool is packed; the others read the same as before, bit for bit
    q = torch.randn(6, sv.Hq, sv.D, generator=sv.g).bfloat16().cuda()
    before = [sv.decode(layer, q) for layer in range(2)]
    vfa.pages_free(sv.refs, sv.tables, sv.counts, _i32([0, 4]), sv.BS, status=sv.status)
    used = vfa.pages_compact(sv.refs, sv.tables, sv.counts, sv.pools, sv.BS, sv.ws, status=sv.status)
    assert used.item() == int((sv.refs > 0).sum())
    assert (sv.refs[:used.item()] > 0).all()
    for layer in range(2):
        sv.text[layer][0], sv.text[layer][4] = [], []
        after = sv.decode(layer, q)
        keep = torch.tensor([1, 2, 3, 5]).cuda()
        ref, n = sv.reference(layer, q)
        bo, _ = _bounds(ref, n)
        assert (np.abs(after[0].double().cpu().numpy() - ref[0]) <= bo).all()
        for a, b in zip(before[layer], after):
            # (the runs of work differ, the pages' values do not)
            assert torch.allclose(a[keep].float(), b[keep].float(), rtol=2 ** -7, atol=1e-6)
        assert (after[0][torch.tensor([0, 4]).cuda()] == 0).all()


def test_captured_step_serves_every_token(vfa):
    """extend -> norm + rotation -> write -> decode captured once and replayed for 40 tokens (over
    page borders), bit for bit the eager calls; a row joins in between by a fork outside the graph."""
    rows, Hq, Hkv, D, BS = 5, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(60, rows, (Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
    table = vfa.rope_table([500.0 ** (-i / 64) for i in range(64)])
    w = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")

    def state():
        refs = torch.zeros(64, dtype=torch.int32, device="cuda")
        return dict(refs=refs, tables=torch.full((rows, 8), -1, dtype=torch.int32, device="cuda"),
                    counts=_i32([0] * rows), start=_i32([0] * rows), add=_i32([1, 1, 0, 1, 1]),
                    cu=_i32([0, 1, 2, 2, 3, 4]), pool=vfa.alloc_kv4_pool(64, Hkv, D),
                    x=torch.zeros(rows, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda"),
                    ws=vfa.alloc_pages_workspace(64, rows, 1), status=_i32([0]),
                    dws=vfa.alloc_kv4_decode_workspace(rows, Hq, Hkv, D),
                    out=torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(rows, Hq, device="cuda"))

    def step(t):
        """One token for the rows that take one; packed row i is the i-th of them."""
        t["start"].copy_(t["counts"])
        vfa.pages_extend(t["refs"], t["tables"], t["counts"], t["add"], BS, t["ws"],
                         status=t["status"])
        pick = torch.where(t["add"] > 0, 0, rows)           # the rows that take a token, first
        order = torch.argsort(pick + torch.arange(rows, device="cuda"))
        q, k, v = t["x"].split((Hq * D, Hkv * D, Hkv * D), 1)
        q, k = vfa.qk_norm_rope(q.view(rows, Hq, D), k.view(rows, Hkv, D),
                                t["start"][order].contiguous(), table, w[0], w[1])
        vfa.kv4_write(k, v.view(rows, Hkv, D), t["pool"], t["tables"], t["cu"], t["start"], 0.5, 0.25,
                      status=t["status"])
        qs = torch.empty_like(q)
        qs[order] = q
        vfa.kv4_decode(qs, t["pool"], t["tables"], t["counts"], 0.5, 0.25, out=t["out"], lse=t["lse"],
                       workspace=t["dws"], status=t["status"])

    eager, held = state(), state()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(state())                                       # (libraries and allocations are warm)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(held)
        torch.cuda.synchronize()
        for i in range(40):
            if i == 21:                                     # row 2 becomes a sample of row 1
                for t in (eager, held):
                    vfa.pages_fork(t["refs"], t["tables"], t["counts"], _i32([1]), _i32([2]),
                                   [t["pool"]], BS, t["ws"], status=t["status"])
                    t["add"].fill_(1)
                    t["cu"].copy_(torch.arange(rows + 1, device="cuda"))
            for t in (eager, held):
                t["x"].copy_(qkv[i])
            step(eager)
            graph.replay()
            assert torch.equal(eager["out"], held["out"]) and torch.equal(eager["lse"], held["lse"]), i
        side.synchronize()
    for name in ("refs", "tables", "counts", "pool", "status"):
        assert torch.equal(eager[name], held[name]), name
    assert held["status"].item() == 0
    assert held["counts"].tolist() == [40, 40, 40, 40, 40]
    assert (held["out"].float().abs().amax((1, 2)) > 0).all()


def test_bf16_pools_moved_right_before_a_decode_step(vfa):
    """decode_step reads its pools before it waits for the kernel ahead of it; the page
    operations must have finished by then, without a synchronisation between."""
    g = torch.Generator(device="cuda").manual_seed(0)
    blocks, rows, cap, Hkv, D = 6000, 8, 260, 8, 128
    kp, vp = (torch.randn(blocks, 16, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
              for _ in range(2))
    perm = torch.randperm(blocks, generator=g, device="cuda").int()[:rows * 256]
    tables = torch.zeros(rows, cap, dtype=torch.int32, device="cuda")
    tables[:, :256] = perm.view(rows, 256)
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[perm.long()] = 1
    counts = torch.full((rows,), 4096, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, 32, D, generator=g, device="cuda").bfloat16()
    ws = vfa.alloc_pages_workspace(blocks, rows, rows)
    nb = torch.full((rows,), 256, dtype=torch.int32, device="cuda")

    def decode():
        m, l = (torch.empty(rows, 32, device="cuda") for _ in range(2))
        o = torch.empty(rows, 32, D, device="cuda")
        vfa.decode_init(m, l, o)
        return m, l, o

    def step(st):
        vfa.decode_step(q, kp, vp, tables, nb, *st)
        return vfa.decode_finalize(st[1], st[2])

    want = step(decode())
    st = decode()
    torch.cuda.synchronize()
    vfa.pages_compact(refs, tables, counts, [kp, vp], 16, ws)
    got = step(st)
    # the pages' places differ, their values and order do not
    assert torch.equal(want, got)


def test_side_stream_with_its_own_allocations(vfa):
    """stream=: the results allocated inside belong to that stream and are right there."""
    s = torch.cuda.Stream()
    x = torch.randn(4000, 10, 128, device="cuda").bfloat16()
    q, k = x[:, :8], x[:, 8:]
    pos = torch.arange(4000, device="cuda", dtype=torch.int32)
    table = vfa.rope_table([10.0 ** (-i / 8) for i in range(64)])
    w = torch.ones(128, device="cuda")
    want = vfa.qk_norm_rope(q, k, pos, table, w, w)
    wantb = vfa.qk_norm_rope_bwd(q, k, want[0], want[1], pos, table, w, w)
    torch.cuda.synchronize()
    got = vfa.qk_norm_rope(q, k, pos, table, w, w, stream=s)
    gotb = vfa.qk_norm_rope_bwd(q, k, got[0], got[1], pos, table, w, w, stream=s)
    s.synchronize()
    for a, b in zip((*want, *wantb), (*got, *gotb)):
        assert torch.equal(a, b)


def test_training_step_gradients(vfa):
    """norm + rotation -> varlen_fwd -> varlen_bwd -> backward of norm + rotation.

    The last stage is held to the 64-bit formula on the gradients that reach it (its tolerance
    is derived in test_gpu_rope.py), and the whole chain to 64-bit autograd: along it q, k, out,
    P, dS and the gradients are rounded to bf16, seven roundings of at most 2^-8 relative to
    each value, and a direction of the loss averages them; 16 * 2^-8 of the gradient's norm
    leaves a factor of two for their propagation through the softmax."""
    g = torch.Generator().manual_seed(0)
    D, Hq, Hkv = 64, 4, 2
    lens = [33, 1, 100]
    T = sum(lens)
    cu = np.concatenate(([0], np.cumsum(lens)))
    x = [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv)]
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)]
    dout = torch.randn(T, Hq, D, generator=g).bfloat16()
    pos = torch.cat([torch.arange(n) for n in lens]).int()
    f = [100.0 ** (-i / 16) for i in range(16)]
    dq_, dk_, dv_ = (t.cuda() for t in x)
    wd = [t.cuda() for t in w]
    table = vfa.rope_table(f)
    q, k = vfa.qk_norm_rope(dq_, dk_, pos.cuda(), table, wd[0], wd[1])
    out, lse = vfa.varlen_fwd(q, k, dv_, _i32(cu), _i32(cu), max(lens), 0.125, 1)
    gq, gk, gv, _ = vfa.varlen_bwd(q, k, dv_, out, dout.cuda(), lse, _i32(cu), _i32(cu), 0.125, 1)
    got = vfa.qk_norm_rope_bwd(dq_, dk_, gq, gk, pos.cuda(), table, wd[0], wd[1])

    # 64-bit autograd of the whole chain
    leaves = [t.double().requires_grad_(True) for t in (*x, *w)]
    ang = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64)

    def turn(y):
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        a, b = y[..., :16], y[..., 16:32]
        return torch.cat((a * c - b * s, b * c + a * s, y[..., 32:]), -1)

    nr = lambda y, wt: turn(y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * wt)
    q64, k64, v64 = nr(leaves[0], leaves[3]), nr(leaves[1], leaves[4]), leaves[2]
    loss = 0
    for a, b in zip(cu[:-1], cu[1:]):
        s = torch.einsum("ihd,jhd->hij", q64[a:b], k64[a:b].repeat_interleave(2, 1)) * 0.125
        s = s.masked_fill(~torch.ones(b - a, b - a, dtype=torch.bool).tril(), -math.inf)
        o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v64[a:b].repeat_interleave(2, 1))
        loss = loss + (o * dout[a:b].double()).sum()
    want = torch.autograd.grad(loss, leaves)
    for name, a, b in zip(("dq", "dk", "dv", "dwq", "dwk"),
                          (got[0], got[1], gv, got[2], got[3]), want):
        err = (a.double().cpu() - b).norm() / b.norm()
        assert err <= 16 * 2.0 ** -8, (name, float(err))


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_taken_on_while_some_are_still_written(vfa, D):
    """varlen_bwd and the rotation's backward with nothing between them.  One tile of keys and 64
    query heads on one kv head: the kernel of dk and dv is one CTA's long loop, that of dq is done
    far earlier.  The rotation's backward must see the finished dk: bit for bit the gradients
    from finished tensors."""
    g = torch.Generator(device="cuda").manual_seed(D)
    Lq, Lk, H = 4096, 128, 64
    q, dout = (torch.randn(Lq, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(Lk, 1, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    cuq, cuk = _i32([0, Lq]), _i32([0, Lk])
    out, lse = vfa.varlen_fwd(q, k, v, cuq, cuk, Lq, D ** -0.5, 0)
    table = vfa.rope_table([100.0 ** (-i / 16) for i in range(16)])
    pos = torch.arange(Lk, dtype=torch.int32, device="cuda")
    w = torch.ones(D, device="cuda")
    few = torch.randn(Lk, 1, D, generator=g, device="cuda").bfloat16()
    # every buffer exists before the two calls: an allocation's own kernel would come between
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, float("nan")), torch.empty_like(v)
    ws = vfa.alloc_bwd_workspace(1, Lq, H, D)
    rws = vfa.alloc_qk_norm_rope_bwd_workspace(D)
    outs = [torch.empty_like(few), torch.empty_like(few), torch.empty_like(w), torch.empty_like(w)]

    def rope():
        return vfa.qk_norm_rope_bwd(few, k, few, dk, pos, table, w, w, dq=outs[0], dk=outs[1],
                                    dq_weight=outs[2], dk_weight=outs[3], workspace=rws)

    torch.cuda.synchronize()
    vfa.varlen_bwd(q, k, v, out, dout, lse, cuq, cuk, D ** -0.5, 0, dq=dq, dk=dk, dv=dv, workspace=ws)
    rope()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    assert torch.isfinite(dk.float()).all()
    for a, b in zip(got, rope()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("splits", [1, 4])
def test_pages_overwritten_behind_a_decode_step_without_tokens(vfa, splits):
    """A long decode step, one whose tiles are all empty, and a copy over the first one's pages,
    with nothing between them: the copy must not start while the first step still reads."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, per, Hkv, D = 4, 1000, 8, 128
    blocks = 2 * rows * per
    kp, vp = (torch.randn(blocks, 16, Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
              for _ in range(2))
    kp[::2] = float("nan")                                 # no row lists the even pages
    tables = torch.arange(1, blocks, 2, dtype=torch.int32, device="cuda").view(rows, per)
    dst = tables.flip(1).reshape(-1).contiguous()          # the pages read last are copied first
    src = dst - 1
    q = torch.randn(rows, 32, D, generator=g, device="cuda").bfloat16()
    full, none = (torch.full((rows,), n, dtype=torch.int32, device="cuda") for n in (per, 0))
    ws = vfa.alloc_decode_split_workspace(rows, 32, Hkv, D, splits) if splits > 1 else None

    def state():
        m, l = (torch.empty(rows, 32, device="cuda") for _ in range(2))
        o = torch.empty(rows, 32, D, device="cuda")
        vfa.decode_init(m, l, o)
        return m, l, o

    def step(n, st):
        if splits > 1:
            vfa.decode_step_split(q, kp, vp, tables, n, *st, splits, ws)
        else:
            vfa.decode_step(q, kp, vp, tables, n, *st)

    want = state()
    step(full, want)
    got = state()
    torch.cuda.synchronize()
    step(full, got)
    step(none, got)
    vfa.pages_copy([kp, vp], src, dst)
    torch.cuda.synchronize()
    assert torch.isnan(kp).all()
    for a, b in zip(want, got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
