// key_weights.cu -- the accumulated attention weight of packed keys:
//   weights[b, hk, j] += sum over the query heads of kv head hk and the queries i
//                        that see key j of exp(scale q_i.k_j - lse_i).
//
// The column sums of the attention matrix.  With keys as the rows of the score
// tile a column sum is a row sum, which one thread adds up in registers:
//   * a unit is (kv head, pair of 128-key tiles, chunk of steps); a step is a block
//     of queries of one query head.  The pair of K tiles stays in shared memory,
//     the blocks stream past through a TMA ring, each read once for 256 keys;
//   * the tensor core forms S^T = K Q^T of each tile into one of two TMEM buffers of
//     its own; a warpgroup takes half of the columns of one tile, one key row per
//     thread, and adds 2^(s scale log2e - lse log2e) over the row's visible columns,
//     four chains of two side by side, block after block: the order of a sum is
//     fixed.  -lse log2e of a step's queries comes from a warp of its own through
//     a ring;
//   * a unit's sums go to the workspace, and a second kernel adds them over the
//     chunks and halves, in order, to the weights.
// One CTA per SM takes units from an atomic counter.
//
// Bound.  38577 tokens of 32 + 8 heads of 128 take 0.8 ms, 1.0 PFLOP/s (52% of the
// measured peak).  The products alone, with every handshake, take 0.55, the
// exponentials (32 a cycle and SM) 0.38; the rest is their overlap, which four warps per
// scheduler do not complete.  Steps on the way: one tile per unit 1.26 ms; eight
// warps and a tile's masked steps in the common code 0.94, in code of their own
// 0.82.  K as an operand in TMEM was the same (0.83).
#include <algorithm>
#include <cfloat>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace vfa {

namespace {

constexpr int kTiles = 2;          // key tiles of a unit
constexpr int kMathWarps = 16;     // a warpgroup per tile and half of the columns
constexpr int kStatWarp = 2, kFirstMathWarp = 4;
constexpr int kThreads = (kFirstMathWarp + kMathWarps) * 32;
// 640 threads launch with 96 registers each: 128 * 64 + 512 * 104 = 640 * 96
constexpr int kLoadRegs = 64;
constexpr int kMathRegs = 104;
constexpr int kFewUnits = 608;     // four for every SM
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct KwCfg {
    static constexpr int DB = D / 64;
    static constexpr int STEP = key_weights_rows(D);
    static constexpr int NCH = STEP / 32, NH = NCH / 2;     // 32-column chunks; of a warpgroup's half
    static constexpr int NSTAT = 4;                         // stages of the queries' -lse log2(e)
    static constexpr uint32_t TILE = kOwn * D * 2;          // a tile of K
    static constexpr uint32_t BLOCK = STEP * D * 2;         // a block of Q
    static constexpr int NSTAGE = D == 64 ? 8 : (D == 128 ? 4 : 2);
    static constexpr int NUM_BARS = 2 * NSTAGE + 4 * kTiles + 4 + 2 + 1 + 2 * NSTAT;
    static constexpr uint32_t STAT = STEP * sizeof(float);
    static constexpr size_t SMEM = 1024 + kTiles * TILE + NSTAGE * BLOCK + NSTAT * STAT + NUM_BARS * 8;
    static constexpr uint32_t IDESC = idesc_bf16_f32(kOwn, STEP, false, false);
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(kTiles * 2 * STEP <= 512, "TMEM budget");
};

// The blocks of `step` queries that see key tile t of a sequence: [first, end).
struct Blocks {
    int first, end;
    __device__ __forceinline__ bool has(int b) const { return b >= first && b < end; }
};

__device__ __forceinline__ Blocks blocks_of(const KeyWeightArgs &a, int lq, int lk, int t, int step)
{
    const long long off = a.causal == 2 ? lk - lq : 0;
    const long long j_lo = static_cast<long long>(t) * kOwn, j_hi = min(static_cast<long long>(lk), j_lo + kOwn);
    const long long lo = a.causal ? max(0ll, j_lo - off) : 0;
    long long hi = lq - 1;
    if (a.window_left >= 0 && j_lo >= a.sink_tokens)
        hi = min(hi, j_hi - 1 - off + a.window_left);
    Blocks b;
    b.first = lo <= hi && j_lo < lk ? static_cast<int>(lo / step) : 0;
    b.end = lo <= hi && j_lo < lk ? static_cast<int>(hi / step) + 1 : 0;
    return b;
}

// The blocks that see a tile of the pair t, t + 1: what lies between the two is
// among them (no block sees neither).
__device__ __forceinline__ Blocks pair_blocks(const Blocks &x, const Blocks &y)
{
    if (x.end <= x.first)
        return y;
    if (y.end <= y.first)
        return x;
    Blocks b;
    b.first = min(x.first, y.first);
    b.end = max(x.end, y.end);
    return b;
}

__global__ void __launch_bounds__(kPrepThreads) kw_prep_kernel(const KeyWeightArgs a)
{
    grid_wait();
    grid_release();
    __shared__ int warp_sums[32];
    __shared__ int s_bad;
    const int B = a.batch;
    if (threadIdx.x == 0)
        s_bad = a.cu_q[0] != 0 || a.cu_k[0] != 0 || a.cu_q[B] != a.total_q || a.cu_k[B] != a.total_k;
    __syncthreads();
    auto pairs_of = [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b], lk = a.cu_k[b + 1] - a.cu_k[b];
        // (compared, too: a difference of 32 bits may wrap)
        if (a.cu_q[b + 1] < a.cu_q[b] || a.cu_k[b + 1] < a.cu_k[b] || lq > a.max_seqlen_q ||
            lk > a.weight_stride) {
            s_bad = 1;
            return 0;
        }
        return lk / (kTiles * kOwn) + (lk % (kTiles * kOwn) != 0);
    };
    block_prefix(B, a.pair_start, warp_sums, pairs_of);
    block_prefix(B, a.unit_start, warp_sums, [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b];
        const long long steps = lq > 0 ? (static_cast<long long>(lq) + a.step - 1) / a.step *
                                             (a.num_heads / a.num_kv_heads)
                                       : 0;
        return pairs_of(b) * static_cast<int>((steps + a.chunk_steps - 1) / a.chunk_steps);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
        a.status[1] = 0;                         // the main kernel's unit counter
        *a.status = s_bad ? VFA_ERR_BAD_SEQLENS : VFA_OK;
    }
}

struct KwUnit {
    int t, kh, chunk;            // first key tile of the pair, kv head, chunk
    int q0, lq, k0, lk;
    Blocks tile[kTiles], both;   // blocks that see each tile, and either
    int s0, n;                   // steps [s0, s0 + n) of group x (both.end - both.first)
    int valid;                   // 0: no more units
};

// Sums of this thread's key row over 32 columns: p = 2^(s scale_log2 + nl), nl of every
// column from shared memory, all of them asked for before the first is used.  MASK: where
// a column's bit of `see` is 0 p is 0, whatever the query's score and lse are.
template <bool MASK>
__device__ __forceinline__ void add_weights(const uint32_t (&sr)[32], float scale_log2, uint32_t stat,
                                            float2 (&acc)[4], uint32_t see = 0xffffffffu)
{
    uint4 nl[4];
    const float2 c2 = make_float2(scale_log2, scale_log2);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        if (e % 16 == 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                nl[u] = ld_shared_v4(stat + e * 4 + u * 16);
        }
        const uint4 q = nl[e / 4 % 4];
        const float2 t = __ffma2_rn(
            make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2,
            make_float2(__uint_as_float(e & 2 ? q.z : q.x), __uint_as_float(e & 2 ? q.w : q.y)));
        float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        if (MASK) {
            p.x = see >> e & 1u ? p.x : 0.f;
            p.y = see >> (e + 1) & 1u ? p.y : 0.f;
        }
        acc[e / 2 % 4] = __fadd2_rn(acc[e / 2 % 4], p);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kw_main_kernel(const __grid_constant__ KeyWeightArgs a)
{
    using C = KwCfg<D>;
    constexpr int DB = C::DB, NSTAGE = C::NSTAGE, STEP = C::STEP, NCH = C::NCH, NH = C::NH, NSTAT = C::NSTAT;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort;
    __shared__ KwUnit s_unit[2];

    grid_wait();
    if (*a.status != VFA_OK)
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int H = a.num_heads, group = H / a.num_kv_heads;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sK = (raw + 1023u) & ~1023u;
    const uint32_t sRing = sK + kTiles * C::TILE;
    const uint32_t sStat = sRing + NSTAGE * C::BLOCK;
    const uint32_t bars = sStat + NSTAT * C::STAT;
    auto ring_full = [&](int i) { return bars + 8u * i; };
    auto ring_empty = [&](int i) { return bars + 8u * (NSTAGE + i); };
    constexpr uint32_t E = 2 * NSTAGE;
    // score buffers: two per tile
    auto s_full = [&](int x, int i) { return bars + 8u * (E + 2 * x + i); };
    auto s_free = [&](int x, int i) { return bars + 8u * (E + 2 * kTiles + 2 * x + i); };
    auto unit_full = [&](int x) { return bars + 8u * (E + 4 * kTiles + x); };
    auto unit_empty = [&](int x) { return bars + 8u * (E + 4 * kTiles + 2 + x); };
    const uint32_t own_full = bars + 8u * (E + 4 * kTiles + 4);
    const uint32_t own_empty = bars + 8u * (E + 4 * kTiles + 5);
    const uint32_t drain_bar = bars + 8u * (E + 4 * kTiles + 6);
    auto stat_full = [&](int i) { return bars + 8u * (E + 4 * kTiles + 7 + i); };
    auto stat_empty = [&](int i) { return bars + 8u * (E + 4 * kTiles + 7 + NSTAT + i); };
    volatile int *abort = &s_abort;

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(ring_full(i), 1);
            mbar_init(ring_empty(i), 1);
        }
        for (int x = 0; x < kTiles; ++x)
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full(x, i), 1);
                mbar_init(s_free(x, i), 256);       // tile x's warpgroups
            }
        for (int x = 0; x < 2; ++x) {
            mbar_init(unit_full(x), 1);
            mbar_init(unit_empty(x), 2 + kMathWarps);
        }
        mbar_init(own_full, 1);
        mbar_init(own_empty, 1);
        for (int i = 0; i < NSTAT; ++i) {
            mbar_init(stat_full(i), 1);
            mbar_init(stat_empty(i), kMathWarps);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem_base;

    auto take_unit = [&](uint32_t n, KwUnit &w) -> bool {
        if (!mbar_wait_warp(unit_full(n & 1), (n >> 1) & 1u, abort))
            return false;
        w = s_unit[n & 1];
        return w.valid;
    };

    if (warp < kFirstMathWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (warp == 0) {
        // ------------------------------------------------------------ units, K and Q
        if (lane == 0) {
            tma_prefetch_map(&a.tm_q);
            tma_prefetch_map(&a.tm_k);
            const int units = a.unit_start[a.batch];
            uint32_t g = 0, owns = 0;
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                if (!mbar_wait(unit_empty(n & 1), ((n >> 1) & 1u) ^ 1u, abort))
                    break;
                KwUnit w;
                for (;;) {
                    // the next unit with a step
                    const int u = atomicAdd(a.status + 1, 1);
                    w.valid = u < units * static_cast<long long>(a.num_kv_heads);
                    if (!w.valid)
                        break;
                    w.kh = u / units;
                    const int b = owner_of(a.unit_start, a.batch, u % units);
                    w.q0 = a.cu_q[b];
                    w.lq = a.cu_q[b + 1] - w.q0;
                    w.k0 = a.cu_k[b];
                    w.lk = a.cu_k[b + 1] - w.k0;
                    const int pairs = a.pair_start[b + 1] - a.pair_start[b];
                    const int x = u % units - a.unit_start[b];
                    w.t = x % pairs * kTiles;
                    w.chunk = x / pairs;
                    for (int i = 0; i < kTiles; ++i)
                        w.tile[i] = blocks_of(a, w.lq, w.lk, w.t + i, STEP);
                    w.both = pair_blocks(w.tile[0], w.tile[1]);
                    w.s0 = w.chunk * a.chunk_steps;
                    w.n = min(a.chunk_steps, (w.both.end - w.both.first) * group - w.s0);
                    if (w.n > 0)
                        break;
                }
                s_unit[n & 1] = w;
                mbar_arrive(unit_full(n & 1));
                if (!w.valid)
                    break;
                if (!mbar_wait(own_empty, (owns & 1u) ^ 1u, abort))
                    break;
                mbar_arrive_expect_tx(own_full, kTiles * C::TILE);
                for (int i = 0; i < kTiles; ++i)
                    load_rows<DB, kOwn>(sK + i * C::TILE, &a.tm_k, own_full, w.kh,
                                        w.k0 + (w.t + i) * kOwn, kOwn);
                ++owns;
                const int per = w.both.end - w.both.first;
                int head = w.s0 / per, blk = w.both.first + w.s0 % per;
                for (int s = 0; s < w.n; ++s, ++g) {
                    const int st = g % NSTAGE;
                    if (!mbar_wait(ring_empty(st), ((g / NSTAGE) & 1u) ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(ring_full(st), C::BLOCK);
                    load_rows<DB, STEP>(sRing + st * C::BLOCK, &a.tm_q, ring_full(st), w.kh * group + head,
                                        w.q0 + blk * STEP, STEP);
                    if (++blk == w.both.end) {
                        blk = w.both.first;
                        ++head;
                    }
                }
            }
            if (*abort) {
                // the last fills may be in flight
                if (owns > 0)
                    mbar_wait_drain(own_full, (owns - 1) & 1u);
                for (int st = 0; st < NSTAGE; ++st) {
                    const uint32_t fills = g / NSTAGE + (static_cast<uint32_t>(st) < g % NSTAGE ? 1u : 0u);
                    if (fills > 0)
                        mbar_wait_drain(ring_full(st), (fills - 1) & 1u);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        uint32_t g = 0, owns = 0, used[kTiles] = {0, 0};        // buffers of each tile so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            KwUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            if (!mbar_wait_warp(own_full, owns & 1u, abort)) {
                ok = false;
                break;
            }
            ++owns;
            int blk = w.both.first + w.s0 % (w.both.end - w.both.first);
            for (int s = 0; s < w.n && ok; ++s, ++g) {
                const int st = g % NSTAGE;
                if (!mbar_wait_warp(ring_full(st), (g / NSTAGE) & 1u, abort)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int x = 0; x < kTiles; ++x) {
                    if (!w.tile[x].has(blk))
                        continue;
                    const int i = used[x] & 1;
                    if (!mbar_wait_warp(s_free(x, i), ((used[x] >> 1) & 1u) ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_scores<D, STEP>(tmem + (2 * x + i) * STEP, sK + x * C::TILE, sRing + st * C::BLOCK,
                                          C::IDESC);
                    mma_commit_w(s_full(x, i));
                    ++used[x];
                }
                mma_commit_w(ring_empty(st));
                if (s == w.n - 1)
                    mma_commit_w(own_empty);
                blk = blk + 1 == w.both.end ? w.both.first : blk + 1;
            }
        }
        if (!ok || *abort) {
            mma_commit_w(drain_bar);
            mbar_wait_drain(drain_bar, 0);
        }
    } else if (warp == kStatWarp) {
        // ------------------------------------------------------------ -lse log2(e) of the queries
        uint32_t g = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            KwUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            const int per = w.both.end - w.both.first;
            int head = w.s0 / per, blk = w.both.first + w.s0 % per;
            // NCH per lane, loaded a step ahead
            float nl[NCH];
            auto load = [&]() {
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int i = blk * STEP + 32 * c + lane;
                    nl[c] = i < w.lq ? -__ldg(a.lse + static_cast<size_t>(w.q0 + i) * H + w.kh * group + head) *
                                           kLog2e
                                     : 0.f;
                }
            };
            load();
            for (int s = 0; s < w.n; ++s, ++g) {
                const int st = g % NSTAT;
                if (!mbar_wait_warp(stat_empty(st), ((g / NSTAT) & 1u) ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                float *dst = reinterpret_cast<float *>(smem_raw + (sStat + st * C::STAT - raw));
#pragma unroll
                for (int c = 0; c < NCH; ++c)       // a query that sees nothing (lse = -FLT_MAX) is hidden
                    dst[32 * c + lane] = nl[c] > FLT_MAX ? 0.f : nl[c];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(stat_full(st));
                if (++blk == w.both.end) {
                    blk = w.both.first;
                    ++head;
                }
                if (s + 1 < w.n)
                    load();
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMathRegs));
        // ------------------------------------------------------------ weights
        const int quarter = warp & 3, wg = (warp - kFirstMathWarp) >> 2;
        const int x = wg & 1, half = wg >> 1;         // its tile, half of the columns
        const int r = quarter * 32 + lane;            // key row of the tile
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t g = 0, used = 0;                     // steps, buffers of the tile so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            KwUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            const long long off = a.causal == 2 ? w.lk - w.lq : 0;
            const long long olo = static_cast<long long>(w.t + x) * kOwn;
            const int own = (w.t + x) * kOwn + r;
            const int wl = own < a.sink_tokens ? -1 : a.window_left;
            const Blocks mine = x ? w.tile[1] : w.tile[0];
            float2 acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = make_float2(0.f, 0.f);
            int s = 0, blk = w.both.first + w.s0 % (w.both.end - w.both.first);
            // a step's queries are read, or its block does not see the tile
            auto pass = [&]() {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(stat_empty(g % NSTAT));
                ++g;
                ++s;
                blk = blk + 1 == w.both.end ? w.both.first : blk + 1;
            };
            while (s < w.n && ok) {
                // (a step that passes by is waited for too: its stage is not given up twice)
                ok = mbar_wait_warp(stat_full(g % NSTAT), (g / NSTAT) & 1u, abort);
                if (!ok)
                    break;
                if (!mine.has(blk)) {
                    pass();
                    continue;
                }
                const int i = used & 1;
                const uint32_t stat = sStat + g % NSTAT * C::STAT;
                const long long slo = static_cast<long long>(blk) * STEP;
                // a block every pair of which is visible needs no mask
                const bool full = olo + kOwn <= w.lk && slo + STEP <= w.lq &&
                                  (!a.causal || olo + kOwn - 1 <= slo + off) &&
                                  (a.window_left < 0 || olo >= slo + STEP - 1 + off - a.window_left ||
                                   olo + kOwn <= a.sink_tokens);
                ok = mbar_wait_warp(s_full(x, i), (used >> 1) & 1u, abort);
                if (!ok)
                    break;
                ++used;
                tc_fence_after();
                const uint32_t addr = tmem + lane_addr + (2 * x + i) * STEP;
                if (full) {
                    uint32_t ra[32], rb[32];
                    tmem_ld32(addr + 32 * half * NH, ra);
                    tmem_wait_ld_r(ra);
                    if constexpr (NH == 2) {
                        // the second chunk is on its way while the first is added up
                        tmem_ld32(addr + 32 * half * NH + 32, rb);
                        add_weights<false>(ra, a.scale_log2, stat + 128 * half * NH, acc);
                        tmem_wait_ld_r(rb);
                    }
                    tc_fence_before();
                    mbar_arrive(s_free(x, i));
                    add_weights<false>(NH == 2 ? rb : ra, a.scale_log2, stat + 128 * (half * NH + NH - 1), acc);
                } else {
                    // little code for the few masked steps
#pragma unroll 1
                    for (int c = half * NH; c < half * NH + NH; ++c) {
                        uint32_t sr[32];
                        tmem_ld32(addr + 32 * c, sr);
                        tmem_wait_ld_r(sr);
                        int lo, hi;
                        key_row_span(own, slo + 32 * c, w.lk, w.lq, a.causal, wl, off, &lo, &hi);
                        add_weights<true>(sr, a.scale_log2, stat + 128 * c, acc, below(hi) & ~below(lo));
                    }
                    tc_fence_before();
                    mbar_arrive(s_free(x, i));
                }
                pass();
            }
            if (!ok)
                break;
            const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            if (own < w.lk)
                a.part[(static_cast<size_t>(w.chunk * 2 + half) * a.num_kv_heads + w.kh) * a.total_k + w.k0 + own] =
                    sum.x + sum.y;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort && tid == 0)
        atomicCAS(a.status, VFA_OK, VFA_ERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The sums of a pair's units added to the weights, one thread per key.
__global__ void __launch_bounds__(kTiles * kOwn) kw_sum_kernel(const KeyWeightArgs a)
{
    grid_wait();
    if (*a.status != VFA_OK)
        return;
    const int kh = blockIdx.y, group = a.num_heads / a.num_kv_heads;
    for (int gp = blockIdx.x; gp < a.pair_start[a.batch]; gp += gridDim.x) {
        const int b = owner_of(a.pair_start, a.batch, gp), t = (gp - a.pair_start[b]) * kTiles;
        const int k0 = a.cu_k[b], lk = a.cu_k[b + 1] - k0, lq = a.cu_q[b + 1] - a.cu_q[b];
        const int j = t * kOwn + threadIdx.x;
        const Blocks both = pair_blocks(blocks_of(a, lq, lk, t, a.step), blocks_of(a, lq, lk, t + 1, a.step));
        const int parts = 2 * (((both.end - both.first) * group + a.chunk_steps - 1) / a.chunk_steps);
        if (j >= lk)
            continue;
        const size_t at = (static_cast<size_t>(b) * a.num_kv_heads + kh) * a.weight_stride + j;
        const float *src = a.part + static_cast<size_t>(kh) * a.total_k + k0 + j;
        const float old = a.weights[at];
        float sum = 0.f;
#pragma unroll 4
        for (int c = 0; c < parts; ++c)
            sum += __ldcg(src + static_cast<size_t>(c) * a.num_kv_heads * a.total_k);
        a.weights_out[at] = old + sum;
    }
}

// Steps of a unit: 128, or 16 where that leaves SMs without a unit; more where a prompt
// would have over most_chunks() of them, since every chunk costs 8 bytes per key and kv head
// (one prompt of 131072 tokens with 32 heads: 168 MB instead of 570).
constexpr int kChunks = 128;                // of the longest prompt in all kv heads, where
constexpr int kChunkPairs = 16 * kFewUnits; // this many (pair, chunk) are no fewer

long long most_chunks(int total_k)
{
    const long long pairs = total_k / (kTiles * kOwn) + 1;
    return std::max<long long>(kChunks, kChunkPairs / pairs);
}

bool few_pairs(int total_k, int num_heads)
{
    return static_cast<long long>(num_heads) * (total_k / (kTiles * kOwn) + 1) < kFewUnits;
}

// Steps of the longest prompt in all heads, of 64 queries (the fewest a step has).
long long steps_of(int total_q, int max_seqlen_q, int num_heads)
{
    return (static_cast<long long>(std::min(total_q, max_seqlen_q)) + 63) / 64 * num_heads;
}

int chunk_steps_for(int total_q, int total_k, int max_seqlen_q, int num_heads)
{
    const long long most = most_chunks(total_k);
    const long long per = (steps_of(total_q, max_seqlen_q, num_heads) + most - 1) / most;
    return static_cast<int>(std::max<long long>(few_pairs(total_k, num_heads) ? 16 : 128, per));
}

// Partial sums for chunks of `base` steps or more: each kv head has
// steps / base or most_chunks() whole ones, and one that is not.  No less for a larger total_k.
long long partials(long long steps, int base, int total_k, int num_heads)
{
    const double whole = std::min(static_cast<double>(steps / base) * total_k,
                                  std::max(static_cast<double>(kChunks) * total_k,
                                           static_cast<double>(kChunkPairs) * kTiles * kOwn));
    return static_cast<long long>(whole) + static_cast<long long>(num_heads) * total_k;
}

template <int D>
cudaError_t launch_d(const KeyWeightArgs &a, int sm_count, cudaStream_t s)
{
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_done[dev]) {
        if ((e = cudaFuncSetAttribute(kw_main_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(KwCfg<D>::SMEM))) != cudaSuccess)
            return e;
        if (dev < 64)
            attr_done[dev] = 1;
    }
    if ((e = launch_dependent(kw_prep_kernel, dim3(1), kPrepThreads, 0, s, a)) != cudaSuccess ||
        (e = launch_dependent(kw_main_kernel<D>, dim3(sm_count), kThreads, KwCfg<D>::SMEM, s, a)) !=
            cudaSuccess)
        return e;
    const long long pairs = static_cast<long long>(a.total_k) / (kTiles * kOwn) + a.batch;
    return launch_dependent(kw_sum_kernel,
                            dim3(static_cast<unsigned>(std::min<long long>(pairs, 65535)), a.num_kv_heads),
                            kTiles * kOwn, 0, s, a);
}

size_t list_bytes(int batch)
{
    return (256 + 2 * (static_cast<size_t>(batch) + 1) * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

}  // namespace

size_t key_weights_workspace_bytes(int batch, int total_q, int total_k, int max_seqlen_q, int num_heads)
{
    // room for long chunks, and for short ones of as many keys as have them: a
    // workspace serves smaller calls too
    const long long steps = steps_of(total_q, max_seqlen_q, num_heads);
    const long long short_pairs = (kFewUnits - 1) / num_heads;         // few_pairs() up to here
    const int short_k = static_cast<int>(std::min<long long>(total_k, short_pairs * kTiles * kOwn - 1));
    long long most = partials(steps, 128, total_k, num_heads);
    if (short_k > 0)
        most = std::max(most, partials(steps, 16, short_k, num_heads));
    return list_bytes(batch) + 2 * static_cast<size_t>(most) * sizeof(float);
}

cudaError_t launch_key_weights(int head_dim, KeyWeightArgs &a, void *workspace, int sm_count,
                               cudaStream_t stream)
{
    uint8_t *p = static_cast<uint8_t *>(workspace);
    a.status = reinterpret_cast<int32_t *>(p);
    a.pair_start = reinterpret_cast<int32_t *>(p + 256);
    a.unit_start = a.pair_start + a.batch + 1;
    a.part = reinterpret_cast<float *>(p + list_bytes(a.batch));
    a.chunk_steps = chunk_steps_for(a.total_q, a.total_k, a.max_seqlen_q, a.num_heads);
    a.step = key_weights_rows(head_dim);
    switch (head_dim) {
    case 64: return launch_d<64>(a, sm_count, stream);
    case 128: return launch_d<128>(a, sm_count, stream);
    case 256: return launch_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
