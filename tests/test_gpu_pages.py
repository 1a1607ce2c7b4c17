"""GPU page operations against the plain ones: whole numbers and page bytes, all equal."""
import numpy as np
import pytest
import torch

import oracle.serving as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vfa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from variable_length_flashattention_gb300 import build, vfa as binding
    build.build()
    return binding


class State:
    """One page state on the host (the definition) and on the device."""

    def __init__(self, vfa, blocks, S, cap, bs, page_shapes=((8, 64), (3, 16)), forks=64, seed=0):
        self.vfa, self.bs = vfa, bs
        rng = np.random.default_rng(seed)
        self.refs = np.zeros(blocks, np.int32)
        self.tables = np.full((S, cap), -7, np.int32)
        self.counts = np.zeros(S, np.int32)
        self.pools = [rng.integers(0, 256, (blocks, *s), dtype=np.uint8) for s in page_shapes]
        self.d_refs, self.d_tables, self.d_counts = (torch.from_numpy(x.copy()).cuda() for x in
                                                     (self.refs, self.tables, self.counts))
        self.d_pools = [torch.from_numpy(p.copy()).cuda() for p in self.pools]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = vfa.alloc_pages_workspace(blocks, S, forks)
        self.ws.fill_(0xa5)                            # needs no initial value

    def i32(self, x):
        return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()

    def extend(self, add):
        ok = O.extend(self.refs, self.tables, self.counts, np.asarray(add, np.int32), self.bs)
        self.vfa.pages_extend(self.d_refs, self.d_tables, self.d_counts, self.i32(add), self.bs,
                              self.ws, status=self.status)
        self.check(0 if ok else self.vfa.VFA_ERR_NO_PAGES)

    def fork(self, parents, children):
        ok = O.fork(self.refs, self.tables, self.counts, parents, children, self.pools, self.bs)
        self.vfa.pages_fork(self.d_refs, self.d_tables, self.d_counts, self.i32(parents),
                            self.i32(children), self.d_pools, self.bs, self.ws,
                            status=self.status)
        self.check(0 if ok else self.vfa.VFA_ERR_NO_PAGES)

    def free(self, seqs):
        O.free(self.refs, self.tables, self.counts, seqs, self.bs)
        self.vfa.pages_free(self.d_refs, self.d_tables, self.d_counts, self.i32(seqs), self.bs,
                            status=self.status)
        self.check(0)

    def compact(self):
        n = O.compact(self.refs, self.tables, self.counts, self.pools, self.bs)
        got = self.vfa.pages_compact(self.d_refs, self.d_tables, self.d_counts, self.d_pools,
                                     self.bs, self.ws, status=self.status)
        assert got.item() == n
        self.check(0)

    def check(self, status):
        assert self.vfa.read_status(self.status) == status
        self.status.zero_()
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_counts.cpu().numpy(), self.counts)
        for d, p in zip(self.d_pools, self.pools):
            assert np.array_equal(d.cpu().numpy(), p)


@pytest.mark.parametrize("blocks,S,cap,bs,seed", [
    (1, 1, 1, 1, 0), (40, 6, 9, 4, 1), (4096, 33, 60, 16, 2), (4097, 70, 40, 16, 3),
    (9001, 1500, 3, 16, 4), (300, 5, 50, 7, 5)])
def test_random_histories(vfa, blocks, S, cap, bs, seed):
    st = State(vfa, blocks, S, cap, bs, seed=seed)
    rng = np.random.default_rng(seed)
    for step in range(8):
        room = cap * bs - st.counts
        add = np.minimum(room, rng.integers(0, 2 * bs + 1, S)) * (rng.random(S) < 0.7)
        if step % 2:
            add = np.minimum(add, 1)
        st.extend(add)
        empty = np.flatnonzero(st.counts == 0)[:64]
        live = np.flatnonzero(st.counts > 0)
        if len(empty) and len(live):
            n = rng.integers(1, len(empty) + 1)
            parents = rng.choice(live, n)
            parents[rng.random(n) < 0.1] = -1
            st.fork(parents, rng.permutation(empty)[:n])
        gone = np.flatnonzero(rng.random(S) < 0.4)
        st.free(np.concatenate((gone, gone[:1], [-1])))      # one row twice, one padding entry
        if step % 3 == 2:
            st.compact()
        used = (st.refs > 0).sum()
        assert used <= blocks


def test_fork_of_a_row_that_ends_on_a_page_and_of_an_empty_one(vfa):
    st = State(vfa, 64, 8, 6, 4)
    st.extend([8, 0, 5, 0, 0, 0, 0, 0])
    st.fork([0, 1, 2, 2], [3, 4, 5, 6])
    st.extend([1, 1, 1, 1, 1, 1, 1, 0])
    st.free([0, 2])
    st.compact()


def test_pages_run_out(vfa):
    st = State(vfa, 10, 4, 10, 4)
    st.extend([20, 12, 0, 0])             # 8 pages
    st.extend([12, 0, 0, 0])              # 3 more: refused, nothing changes
    st.extend([8, 0, 0, 0])               # exactly all
    st.free([1])
    st.extend([0, 12, 0, 0])
    st.free([0])
    st.extend([26, 0, 0, 0])              # 7 pages, the last one partly filled: none left
    st.fork([0], [2])                     # no page for the copy: refused


def test_large_requests(vfa):
    """Thousands of pages in one call, over several chunks of the pool."""
    st = State(vfa, 30000, 9, 6000, 16, page_shapes=((1, 16),))
    st.extend([16 * 5000 + 3, 0, 16 * 6000, 1, 0, 16 * 4000 - 1, 0, 0, 0])
    st.free([2])
    st.extend([0, 16 * 5999 + 1, 0, 5, 0, 33, 0, 0, 0])
    st.fork([0, 1, 1, 5], [2, 4, 6, 7])
    st.free([0, 1])
    st.compact()


def test_refusals_change_nothing(vfa):
    st = State(vfa, 30, 6, 5, 4)
    st.extend([9, 4, 0, 0, 0, 0])
    v = st.vfa

    def refused(call):
        call()
        st.check(v.VFA_ERR_BAD_BLOCK)

    ext = lambda add: v.pages_extend(st.d_refs, st.d_tables, st.d_counts, st.i32(add), 4, st.ws,
                                     status=st.status)
    fork = lambda p, c: v.pages_fork(st.d_refs, st.d_tables, st.d_counts, st.i32(p), st.i32(c),
                                     st.d_pools, 4, st.ws, status=st.status)
    refused(lambda: ext([0, -1, 0, 0, 0, 0]))              # a negative addition
    refused(lambda: ext([12, 1, 0, 0, 0, 0]))              # past the row's capacity
    refused(lambda: ext([0, 2 ** 31 - 1, 0, 0, 0, 0]))
    refused(lambda: fork([0, 0], [2, 2]))                  # a child twice
    refused(lambda: fork([0], [1]))                        # a child in use
    refused(lambda: fork([0, 0], [2, 6]))                  # a child out of range
    refused(lambda: fork([6], [2]))                        # a parent out of range
    refused(lambda: v.pages_free(st.d_refs, st.d_tables, st.d_counts, st.i32([6]), 4,
                                 status=st.status))
    st.fork([0, 1], [2, 3])                                # and the state still works


def test_token_counts_stay_within_32_bits(vfa):
    st = State(vfa, 8, 2, 4, 2 ** 30)
    st.extend([2 ** 30 + 5, 0])
    v = st.vfa
    v.pages_extend(st.d_refs, st.d_tables, st.d_counts, st.i32([2 ** 30, 1]), st.bs, st.ws,
                   status=st.status)
    st.check(v.VFA_ERR_BAD_BLOCK)                          # 2^31 + 5 tokens: nothing changes
    st.extend([2 ** 30 - 6, 2 ** 30])
    st.free([0])


def test_bad_table_entries_are_recorded(vfa):
    st = State(vfa, 30, 4, 5, 4)
    st.extend([9, 4, 0, 0])
    v = st.vfa
    st.d_tables[0, 0] = 30                                 # a full page out of range
    v.pages_fork(st.d_refs, st.d_tables, st.d_counts, st.i32([0]), st.i32([2]), st.d_pools, 4,
                 st.ws, status=st.status)
    assert v.read_status(st.status) == v.VFA_ERR_BAD_BLOCK
    assert st.d_tables[2, 0].item() == 30 and st.d_counts[2].item() == 9
    assert st.d_refs[st.d_tables[0, 1].long()].item() == 2
    st.status.zero_()
    v.pages_free(st.d_refs, st.d_tables, st.d_counts, st.i32([0, 2]), 4, status=st.status)
    assert v.read_status(st.status) == v.VFA_ERR_BAD_BLOCK
    st.status.zero_()
    st.d_tables[1, 0] = 29                                 # a page nobody counts
    v.pages_compact(st.d_refs, st.d_tables, st.d_counts, st.d_pools, 4, st.ws, status=st.status)
    assert v.read_status(st.status) == v.VFA_ERR_BAD_BLOCK
    st.status.zero_()
    v.pages_free(st.d_refs, st.d_tables, st.d_counts, st.i32([1]), 4, status=st.status)
    assert v.read_status(st.status) == v.VFA_ERR_BAD_BLOCK
    assert (st.d_refs >= 0).all()
    # a last page out of range: the fork is refused as a whole
    st.status.zero_()
    st.d_counts[3] = 6
    st.d_tables[3, 1] = -3
    v.pages_fork(st.d_refs, st.d_tables, st.d_counts, st.i32([3]), st.i32([0]), st.d_pools, 4,
                 st.ws, status=st.status)
    assert v.read_status(st.status) == v.VFA_ERR_BAD_BLOCK and st.d_counts[0].item() == 0


def test_compact_into_other_tables(vfa):
    st = State(vfa, 500, 5, 40, 4, seed=9)
    st.extend([100, 70, 33, 0, 9])
    st.free([0])
    st.extend([13, 0, 0, 50, 0])
    st.free([1])
    refs, tables, pools = st.d_refs.clone(), st.d_tables.clone(), None
    r_out, t_out = torch.full_like(st.d_refs, 77), torch.full_like(st.d_tables, 77)
    n = st.vfa.pages_compact(st.d_refs, st.d_tables, st.d_counts, st.d_pools, 4, st.ws,
                             refcounts_out=r_out, tables_out=t_out, status=st.status)
    assert torch.equal(refs, st.d_refs) and torch.equal(tables, st.d_tables)
    want = O.compact(st.refs, st.tables, st.counts, st.pools, 4)
    assert n.item() == want and np.array_equal(r_out.cpu().numpy(), st.refs)
    live = np.arange(40)[None] < -(-st.counts // 4)[:, None]
    assert np.array_equal(t_out.cpu().numpy(), np.where(live, st.tables, 77))
    for d, p in zip(st.d_pools, st.pools):
        assert np.array_equal(d.cpu().numpy(), p)


def test_copy_past_32_bits(vfa):
    """Pages beyond 4 GiB of a pool, copied and compacted."""
    page = 1 << 20
    pool = torch.zeros((1 << 32) // page + 9, page, dtype=torch.uint8, device="cuda")
    last = pool.shape[0] - 1
    x = torch.randint(0, 256, (2, page), dtype=torch.uint8, device="cuda")
    pool[last], pool[last - 2] = x[0], x[1]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    vfa.pages_copy([pool], i32([last, last - 2]), i32([last - 1, 5]))
    assert torch.equal(pool[last - 1], x[0]) and torch.equal(pool[5], x[1])
    refs = torch.zeros(last + 1, dtype=torch.int32, device="cuda")
    refs[[last - 2, last]] = 1
    tables = i32([[last, last - 2]])
    used = vfa.pages_compact(refs, tables, i32([32]), [pool], 16, vfa.alloc_pages_workspace(last + 1, 1))
    assert used.item() == 2 and tables.tolist() == [[1, 0]]
    assert torch.equal(pool[1], x[0]) and torch.equal(pool[0], x[1])


@pytest.mark.parametrize("shape", [(16,), (48,), (4096,), (5, 16), (2304,), (16, 8, 64)])
def test_copy(vfa, shape):
    rng = np.random.default_rng(1)
    pools = [rng.integers(0, 256, (50, *shape), dtype=np.uint8) for _ in range(3)]
    dev = [torch.from_numpy(p.copy()).cuda() for p in pools]
    src, dst = [4, 4, -1, 9, 49], [0, 1, 2, 48, 3]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    vfa.pages_copy(dev, i32(src), i32(dst), status=status)
    for p, d in zip(pools, dev):
        for a, b in zip(src, dst):
            if a >= 0:
                p[b] = p[a]
        assert np.array_equal(d.cpu().numpy(), p)
    assert vfa.read_status(status) == 0
    vfa.pages_copy(dev, i32([50, 3, 5]), i32([0, 50, 6]), status=status)
    assert vfa.read_status(status) == vfa.VFA_ERR_BAD_BLOCK
    for p, d in zip(pools, dev):
        p[6] = p[5]
        assert np.array_equal(d.cpu().numpy(), p)


def test_captured_cycle(vfa):
    """Fork, extend and free in one graph, replayed: the state after each replay is the same."""
    st = State(vfa, 200, 12, 10, 4, seed=2)
    st.extend([13, 8, 30] + [0] * 9)
    parents, children = st.i32([0, 1, 2, 0]), st.i32([4, 5, 6, 7])
    add = st.i32([0] * 4 + [1, 1, 1, 1] + [0] * 4)
    v = st.vfa

    def cycle():
        v.pages_fork(st.d_refs, st.d_tables, st.d_counts, parents, children, st.d_pools, 4, st.ws)
        v.pages_extend(st.d_refs, st.d_tables, st.d_counts, add, 4, st.ws)
        v.pages_free(st.d_refs, st.d_tables, st.d_counts, children, 4)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cycle()
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    O.fork(st.refs, st.tables, st.counts, [0, 1, 2, 0], [4, 5, 6, 7], st.pools, 4)
    O.extend(st.refs, st.tables, st.counts, np.array([0] * 4 + [1] * 4 + [0] * 4, np.int32), 4)
    O.free(st.refs, st.tables, st.counts, [4, 5, 6, 7], 4)
    st.check(0)


@pytest.mark.parametrize("blocks", [6, 32768, 32769, 70000])
def test_fork_of_rows_that_list_free_pages(vfa, blocks):
    """A full page that is not in use when the call is made is listed in the child, not counted
    and recorded, also where the same call hands that page out as another child's own copy."""
    st = State(vfa, blocks, 8, 6, 4, page_shapes=((2, 16),), seed=blocks)
    last = blocks - 1
    # rows 0 and 1 end in a partly filled page (1, last); page 0 and 3 are free and listed
    st.refs[[1, 2, last]] = 1
    st.tables[0, :2], st.tables[1, :3] = (0, 1), (3, 2, last)
    st.counts[:2] = 6, 10
    st.d_refs.copy_(torch.from_numpy(st.refs))
    st.d_tables.copy_(torch.from_numpy(st.tables))
    st.d_counts.copy_(torch.from_numpy(st.counts))
    st.vfa.pages_fork(st.d_refs, st.d_tables, st.d_counts, st.i32([0, 1]), st.i32([2, 4]),
                      st.d_pools, 4, st.ws, status=st.status)
    # the lowest free pages in the order of the entries: 0 and 3, the ones listed above
    st.tables[2, :2], st.tables[4, :3] = (0, 0), (3, 2, 3)
    st.counts[[2, 4]] = 6, 10
    st.refs[[0, 2, 3]] = 1, 2, 1
    st.pools[0][0], st.pools[0][3] = st.pools[0][1], st.pools[0][last]
    st.check(st.vfa.VFA_ERR_BAD_BLOCK)


@pytest.mark.parametrize("blocks,S,seed", [(32768, 24, 6), (32769, 24, 7), (36864, 5, 8),
                                           (36865, 40, 9), (70000, 24, 10)])
def test_histories_of_large_pools(vfa, blocks, S, seed):
    """Pools around and above the largest that one CTA plans (32768 pages): thousands of pages
    given, shared, taken back and moved over many chunks, some requests without enough pages."""
    bs = 3
    cap = 3 * blocks // S
    st = State(vfa, blocks, S, cap, bs, page_shapes=((1, 16), (2, 16)), forks=S, seed=seed)
    rng = np.random.default_rng(seed)
    refused = moved = 0
    for step in range(9):
        free = int((st.refs <= 0).sum())
        want = rng.random(S) ** 3 * (rng.random(S) < 0.7)
        # half of the free pages, or (every third step) more than there are
        want = want / max(want.sum(), 1e-9) * free * bs * (1.4 if step % 3 == 1 else 0.5)
        add = np.minimum(want.astype(np.int64) + (rng.random(S) < 0.3), cap * bs - st.counts)
        before = st.counts.copy()
        st.extend(add)
        refused += bool(add.any() and np.array_equal(before, st.counts))
        empty, live = np.flatnonzero(st.counts == 0), np.flatnonzero(st.counts > 0)
        if len(empty) and len(live):
            n = rng.integers(1, len(empty) + 1)
            parents = rng.choice(live, n)
            parents[rng.random(n) < 0.1] = -1
            pools = st.pools, st.d_pools
            if step % 4 == 2:                              # the pages alone, no pool
                st.pools, st.d_pools = [], []
            st.fork(parents, rng.permutation(empty)[:n])
            st.pools, st.d_pools = pools
        gone = np.flatnonzero(rng.random(S) < 0.4)
        st.free(np.concatenate((gone, gone[:1], [-1])))
        if step % 3 == 2:
            used = int((st.refs > 0).sum())
            moved += int((st.refs[used:] > 0).sum())
            st.compact()
    assert refused >= 1 and moved > 1000


def test_refusals_of_a_large_pool_change_nothing(vfa):
    st = State(vfa, 40000, 6, 39000, 4, page_shapes=((1, 16),))
    st.extend([4 * 38997 + 1, 4, 0, 0, 0, 0])
    v = st.vfa

    def refused(call, code):
        call()
        st.check(code)

    ext = lambda add: v.pages_extend(st.d_refs, st.d_tables, st.d_counts, st.i32(add), 4, st.ws,
                                     status=st.status)
    fork = lambda p, c: v.pages_fork(st.d_refs, st.d_tables, st.d_counts, st.i32(p), st.i32(c),
                                     st.d_pools, 4, st.ws, status=st.status)
    refused(lambda: ext([0, -1, 0, 0, 0, 0]), v.VFA_ERR_BAD_BLOCK)
    refused(lambda: ext([16, 0, 0, 0, 0, 0]), v.VFA_ERR_BAD_BLOCK)       # past the row's capacity
    refused(lambda: ext([0, 4 * 1002, 0, 0, 0, 0]), v.VFA_ERR_NO_PAGES)
    refused(lambda: fork([0, 0], [2, 2]), v.VFA_ERR_BAD_BLOCK)
    refused(lambda: fork([0], [1]), v.VFA_ERR_BAD_BLOCK)
    refused(lambda: fork([0, 6], [2, 3]), v.VFA_ERR_BAD_BLOCK)
    st.extend([0, 4 * 1001, 0, 0, 0, 0])                   # exactly the rest
    refused(lambda: fork([0], [2]), v.VFA_ERR_NO_PAGES)    # no page for the copy
    st.free([0])
    st.fork([1, 1], [2, 5])
    st.compact()


@pytest.mark.parametrize("blocks", [20000, 40000])
def test_more_rows_than_one_cta_keeps(vfa, blocks):
    """5000 rows: the rows' places are kept in the workspace (a CTA's shared memory holds 4096)."""
    test_random_histories(vfa, blocks, 5000, 3, 16, blocks)


def test_captured_cycle_of_a_large_pool(vfa):
    """Fork, extend and free in one graph, replayed over several chunks."""
    st = State(vfa, 50000, 12, 9000, 4, page_shapes=((1, 16),), seed=2)
    st.extend([4 * 8000 + 1, 4 * 3000, 30] + [0] * 9)
    st.free([1])
    st.extend([0, 4 * 4000 + 3] + [0] * 10)
    parents, children = st.i32([0, 1, 2, 0]), st.i32([4, 5, 6, 7])
    add = st.i32([0] * 4 + [5, 1, 4000, 1] + [0] * 4)
    v = st.vfa

    def cycle():
        v.pages_fork(st.d_refs, st.d_tables, st.d_counts, parents, children, st.d_pools, 4, st.ws)
        v.pages_extend(st.d_refs, st.d_tables, st.d_counts, add, 4, st.ws)
        v.pages_free(st.d_refs, st.d_tables, st.d_counts, children, 4)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            cycle()
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        O.fork(st.refs, st.tables, st.counts, [0, 1, 2, 0], [4, 5, 6, 7], st.pools, 4)
        O.extend(st.refs, st.tables, st.counts,
                 np.array([0] * 4 + [5, 1, 4000, 1] + [0] * 4, np.int32), 4)
        O.free(st.refs, st.tables, st.counts, [4, 5, 6, 7], 4)
    st.check(0)
