// key_weights.cu -- the accumulated attention weight of packed keys:
//   weights[b, hk, j] += sum over the query heads of kv head hk and the queries i
//                        that see key j of exp(scale q_i.k_j - lse_i).
//
// The column sums of the attention matrix.  With keys as the rows of the score
// tile a column sum is a row sum, which one thread adds up in registers:
//   * a unit is (query head, 128-key tile, chunk of its query blocks): K stays in
//     shared memory, blocks of 128 queries stream past it through a TMA ring;
//   * the tensor core forms S^T = K Q^T (128 x 128) into one of four TMEM
//     buffers; two warpgroups take a unit's blocks in turn (the first one block 0
//     of every unit: the order of a sum does not depend on the CTA's other units),
//     one key row per thread, and add 2^(s scale log2e - lse log2e) over the row's visible columns, four
//     chains of two side by side;
//   * the sums of a unit's two warpgroups go to the workspace, and a second kernel
//     adds them over chunks and query heads, in a fixed order, to the weights.
// One CTA per SM takes units from an atomic counter; consecutive units overlap
// (the next unit's K loads and its first scores run while the current one ends).
//
// Bound: the tensor core (2 D flops per visible pair and query head against one
// exponential and 2.3 instructions of a thread).
#include <algorithm>
#include <cfloat>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace vfa {

namespace {

constexpr int kStep = 128;         // queries of a block
constexpr int kBufs = 4;           // score buffers in TMEM
constexpr int kMathWarps = 8;      // two warpgroups
constexpr int kFirstMathWarp = 4;
constexpr int kThreads = (kFirstMathWarp + kMathWarps) * 32;
constexpr int kFewUnits = 608;      // four for every SM
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct KwCfg {
    static constexpr int DB = D / 64;
    static constexpr uint32_t TILE = kOwn * D * 2;          // a tile of K or a block of Q
    static constexpr int KBUF = D == 256 ? 1 : 2;
    static constexpr int NSTAGE = D == 64 ? 6 : (D == 128 ? 4 : 2);
    static constexpr int NUM_BARS = 2 * NSTAGE + 2 * kBufs + 4 + 2 * KBUF + 1;
    static constexpr uint32_t STAT = kStep * sizeof(float); // per math warp: -lse log2(e)
    static constexpr size_t SMEM = 1024 + (KBUF + NSTAGE) * TILE + kMathWarps * STAT + NUM_BARS * 8;
    static constexpr uint32_t IDESC = idesc_bf16_f32(kOwn, kStep, false, false);
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(kBufs * kStep <= 512, "TMEM budget");
};

// The query blocks that see key tile t: [first, first + n).
struct Blocks {
    int first, n;
};

__device__ __forceinline__ Blocks blocks_of(const KeyWeightArgs &a, int lq, int lk, int t)
{
    const long long off = a.causal == 2 ? lk - lq : 0;
    const long long j_lo = static_cast<long long>(t) * kOwn, j_hi = min(static_cast<long long>(lk), j_lo + kOwn);
    const long long lo = a.causal ? max(0ll, j_lo - off) : 0;
    long long hi = lq - 1;
    if (a.window_left >= 0 && j_lo >= a.sink_tokens)
        hi = min(hi, j_hi - 1 - off + a.window_left);
    Blocks b;
    b.first = lo <= hi ? static_cast<int>(lo / kStep) : 0;
    b.n = lo <= hi ? static_cast<int>(hi / kStep) + 1 - b.first : 0;
    return b;
}

__global__ void __launch_bounds__(kPrepThreads) kw_prep_kernel(const KeyWeightArgs a)
{
    grid_wait();
    __shared__ int warp_sums[32];
    __shared__ int s_bad;
    const int B = a.batch;
    if (threadIdx.x == 0)
        s_bad = a.cu_q[0] != 0 || a.cu_k[0] != 0 || a.cu_q[B] != a.total_q || a.cu_k[B] != a.total_k;
    __syncthreads();
    auto tiles_of = [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b], lk = a.cu_k[b + 1] - a.cu_k[b];
        if (lq < 0 || lk < 0 || lq > a.max_seqlen_q || lk > a.weight_stride) {
            s_bad = 1;
            return 0;
        }
        return lk / kOwn + (lk % kOwn != 0);
    };
    block_prefix(B, a.tile_start, warp_sums, tiles_of);
    block_prefix(B, a.unit_start, warp_sums, [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b];
        const int blocks = lq > 0 ? lq / kStep + (lq % kStep != 0) : 0;
        return tiles_of(b) * ((blocks + a.chunk_steps - 1) / a.chunk_steps);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
        a.status[1] = 0;                         // the main kernel's unit counter
        *a.status = s_bad ? VFA_ERR_BAD_SEQLENS : VFA_OK;
    }
}

struct KwUnit {
    int t, head, chunk;          // key tile in its sequence, query head, chunk
    int q0, lq, k0, lk;
    int first, n;                // query blocks [first, first + n)
    int valid;                   // 0: no more units
};

// Sums of this thread's key row over one block's columns: p = 2^(s scale_log2 + nl),
// nl of every column from shared memory.
template <bool MASK>
__device__ __forceinline__ void add_weights(const uint32_t (&sr)[32], float scale_log2, uint32_t stat,
                                            int lo, int hi, float2 (&acc)[4])
{
    const float2 c2 = make_float2(scale_log2, scale_log2);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const uint4 nl = ld_shared_v4(stat + e * 4);
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
            const float2 t = __ffma2_rn(
                make_float2(__uint_as_float(sr[e + u]), __uint_as_float(sr[e + u + 1])), c2,
                make_float2(__uint_as_float(u ? nl.z : nl.x), __uint_as_float(u ? nl.w : nl.y)));
            float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            if (MASK) {
                p.x = (e + u >= lo && e + u < hi) ? p.x : 0.f;
                p.y = (e + u + 1 >= lo && e + u + 1 < hi) ? p.y : 0.f;
            }
            acc[(e + u) / 2 % 4] = __fadd2_rn(acc[(e + u) / 2 % 4], p);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kw_main_kernel(const __grid_constant__ KeyWeightArgs a)
{
    using C = KwCfg<D>;
    constexpr int DB = C::DB, NSTAGE = C::NSTAGE, KBUF = C::KBUF;
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
    const uint32_t sRing = sK + KBUF * C::TILE;
    const uint32_t sStat = sRing + NSTAGE * C::TILE;
    const uint32_t bars = sStat + kMathWarps * C::STAT;
    auto ring_full = [&](int i) { return bars + 8u * i; };
    auto ring_empty = [&](int i) { return bars + 8u * (NSTAGE + i); };
    constexpr uint32_t E = 2 * NSTAGE;
    auto s_full = [&](int x) { return bars + 8u * (E + x); };
    auto s_free = [&](int x) { return bars + 8u * (E + kBufs + x); };
    auto unit_full = [&](int x) { return bars + 8u * (E + 2 * kBufs + x); };
    auto unit_empty = [&](int x) { return bars + 8u * (E + 2 * kBufs + 2 + x); };
    auto own_full = [&](int x) { return bars + 8u * (E + 2 * kBufs + 4 + x); };
    auto own_empty = [&](int x) { return bars + 8u * (E + 2 * kBufs + 4 + KBUF + x); };
    const uint32_t drain_bar = bars + 8u * (E + 2 * kBufs + 4 + 2 * KBUF);
    volatile int *abort = &s_abort;

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(ring_full(i), 1);
            mbar_init(ring_empty(i), 1);
        }
        for (int x = 0; x < kBufs; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(s_free(x), 128);              // the warpgroup that read it
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(unit_full(x), 1);
            mbar_init(unit_empty(x), 1 + kMathWarps);
        }
        for (int x = 0; x < KBUF; ++x) {
            mbar_init(own_full(x), 1);
            mbar_init(own_empty(x), 1);
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
                    // the next unit with a block to look at
                    const int u = atomicAdd(a.status + 1, 1);
                    w.valid = u < units * static_cast<long long>(H);
                    if (!w.valid)
                        break;
                    w.head = u / units;
                    const int b = owner_of(a.unit_start, a.batch, u % units);
                    w.q0 = a.cu_q[b];
                    w.lq = a.cu_q[b + 1] - w.q0;
                    w.k0 = a.cu_k[b];
                    w.lk = a.cu_k[b + 1] - w.k0;
                    const int tiles = a.tile_start[b + 1] - a.tile_start[b];
                    const int x = u % units - a.unit_start[b];
                    w.t = x % tiles;
                    w.chunk = x / tiles;
                    const Blocks bl = blocks_of(a, w.lq, w.lk, w.t);
                    const int skip = w.chunk * a.chunk_steps;
                    w.first = bl.first + skip;
                    w.n = min(a.chunk_steps, bl.n - skip);
                    if (w.n > 0)
                        break;
                }
                s_unit[n & 1] = w;
                mbar_arrive(unit_full(n & 1));
                if (!w.valid)
                    break;
                const int slot = owns % KBUF;
                if (!mbar_wait(own_empty(slot), ((owns / KBUF) & 1u) ^ 1u, abort))
                    break;
                mbar_arrive_expect_tx(own_full(slot), C::TILE);
                load_rows<DB, kOwn>(sK + slot * C::TILE, &a.tm_k, own_full(slot), w.head / group,
                                    w.k0 + w.t * kOwn, kOwn);
                ++owns;
                for (int s = 0; s < w.n; ++s, ++g) {
                    const int st = g % NSTAGE;
                    if (!mbar_wait(ring_empty(st), ((g / NSTAGE) & 1u) ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(ring_full(st), C::TILE);
                    load_rows<DB, kStep>(sRing + st * C::TILE, &a.tm_q, ring_full(st), w.head,
                                         w.q0 + (w.first + s) * kStep, kStep);
                }
            }
            if (*abort) {
                // the last fills may be in flight
                for (int x = 0; x < KBUF; ++x) {
                    const uint32_t fills = owns / KBUF + (static_cast<uint32_t>(x) < owns % KBUF ? 1u : 0u);
                    if (fills > 0)
                        mbar_wait_drain(own_full(x), (fills - 1) & 1u);
                }
                for (int st = 0; st < NSTAGE; ++st) {
                    const uint32_t fills = g / NSTAGE + (static_cast<uint32_t>(st) < g % NSTAGE ? 1u : 0u);
                    if (fills > 0)
                        mbar_wait_drain(ring_full(st), (fills - 1) & 1u);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // step s of a unit goes to buffer (buf + s) % 4, buf even; phase: one bit per buffer
        uint32_t g = 0, owns = 0, buf = 0, phase = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            KwUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            const int slot = owns % KBUF;
            if (!mbar_wait_warp(own_full(slot), (owns / KBUF) & 1u, abort)) {
                ok = false;
                break;
            }
            for (int s = 0; s < w.n; ++s, ++g) {
                const int st = g % NSTAGE, x = (buf + s) % kBufs;
                if (!mbar_wait_warp(ring_full(st), (g / NSTAGE) & 1u, abort) ||
                    !mbar_wait_warp(s_free(x), ((phase >> x) & 1u) ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                phase ^= 1u << x;
                tc_fence_after();
                issue_scores<D, kStep>(tmem + x * kStep, sK + slot * C::TILE, sRing + st * C::TILE,
                                       C::IDESC);
                mma_commit_w(s_full(x));
                mma_commit_w(ring_empty(st));
                if (s == w.n - 1)
                    mma_commit_w(own_empty(slot));
            }
            ++owns;
            buf += (w.n + 1) & ~1;
        }
        if (!ok || *abort) {
            mma_commit_w(drain_bar);
            mbar_wait_drain(drain_bar, 0);
        }
    } else if (warp >= kFirstMathWarp) {
        // ------------------------------------------------------------ weights
        const int quarter = warp & 3, half = (warp - kFirstMathWarp) >> 2;
        const int r = quarter * 32 + lane;            // key row of the tile
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t wstat = sStat + (warp - kFirstMathWarp) * C::STAT;
        float *stat = reinterpret_cast<float *>(smem_raw + (wstat - raw));
        uint32_t buf = 0, phase = 0;
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
            const long long olo = static_cast<long long>(w.t) * kOwn;
            const int own = w.t * kOwn + r;
            const int wl = own < a.sink_tokens ? -1 : a.window_left;
            // -lse log2(e) of a block's queries, 4 per lane, loaded a turn ahead
            float nl[4] = {0.f, 0.f, 0.f, 0.f};
            auto load_stats = [&](int s) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = (w.first + s) * kStep + 32 * c + lane;
                    nl[c] = s < w.n && i < w.lq
                                ? -__ldg(a.lse + static_cast<size_t>(w.q0 + i) * H + w.head) * kLog2e
                                : 0.f;
                }
            };
            float2 acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = make_float2(0.f, 0.f);
            load_stats(half);
            for (int s = half; s < w.n; s += 2) {
                const int x = (buf + s) % kBufs;
                __syncwarp();                       // the last block's stats are read
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    stat[32 * c + lane] = nl[c];
                __syncwarp();
                load_stats(s + 2);
                const long long slo = static_cast<long long>(w.first + s) * kStep;
                // a block every pair of which is visible needs no mask
                const bool full = olo + kOwn <= w.lk && slo + kStep <= w.lq &&
                                  (!a.causal || olo + kOwn - 1 <= slo + off) &&
                                  (a.window_left < 0 || olo >= slo + kStep - 1 + off - a.window_left ||
                                   olo + kOwn <= a.sink_tokens);
                ok = mbar_wait_warp(s_full(x), (phase >> x) & 1u, abort);
                if (!ok)
                    break;
                phase ^= 1u << x;
                tc_fence_after();
                const uint32_t addr = tmem + lane_addr + x * kStep;
                uint32_t sr[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(addr + 32 * c, sr[c]);
                tmem_wait_ld_r(sr[0]);
                tmem_bind_r(sr[1]);
                tmem_bind_r(sr[2]);
                tmem_bind_r(sr[3]);
                tc_fence_before();
                mbar_arrive(s_free(x));
                if (full) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        add_weights<false>(sr[c], a.scale_log2, wstat + 128 * c, 0, 32, acc);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        int lo, hi;
                        key_row_span(own, slo + 32 * c, w.lk, w.lq, a.causal, wl, off, &lo, &hi);
                        add_weights<true>(sr[c], a.scale_log2, wstat + 128 * c, lo, hi, acc);
                    }
                }
            }
            if (!ok)
                break;
            const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
            if (own < w.lk)
                a.part[(static_cast<size_t>(w.chunk * 2 + half) * H + w.head) * a.total_k + w.k0 + own] =
                    sum.x + sum.y;
            buf += (w.n + 1) & ~1;
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

// The sums of a key tile's units added to the weights, one thread per key.
__global__ void __launch_bounds__(kOwn) kw_sum_kernel(const KeyWeightArgs a)
{
    grid_wait();
    if (*a.status != VFA_OK)
        return;
    const int kh = blockIdx.y, group = a.num_heads / a.num_kv_heads;
    for (int gt = blockIdx.x; gt < a.tile_start[a.batch]; gt += gridDim.x) {
        const int b = owner_of(a.tile_start, a.batch, gt), t = gt - a.tile_start[b];
        const int k0 = a.cu_k[b], lk = a.cu_k[b + 1] - k0, lq = a.cu_q[b + 1] - a.cu_q[b];
        const int j = t * kOwn + threadIdx.x;
        const int parts = 2 * ((blocks_of(a, lq, lk, t).n + a.chunk_steps - 1) / a.chunk_steps);
        if (j >= lk)
            continue;
        float sum = 0.f;
        for (int p = 0; p < parts; ++p) {
            const float *src = a.part + (static_cast<size_t>(p) * a.num_heads + kh * group) * a.total_k + k0 + j;
#pragma unroll 4
            for (int h = 0; h < group; ++h)
                sum += __ldcg(src + static_cast<size_t>(h) * a.total_k);
        }
        const size_t at = (static_cast<size_t>(b) * a.num_kv_heads + kh) * a.weight_stride + j;
        a.weights_out[at] = a.weights[at] + sum;
    }
}

// Blocks of a chunk: long ones, but where that leaves SMs without a unit.
int chunk_steps_for(int total_k, int num_heads)
{
    return static_cast<long long>(num_heads) * (total_k / kOwn + 1) < kFewUnits ? 8 : 64;
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
    const long long tiles = static_cast<long long>(a.total_k) / kOwn + a.batch;
    return launch_dependent(kw_sum_kernel,
                            dim3(static_cast<unsigned>(std::min<long long>(tiles, 65535)), a.num_kv_heads),
                            kOwn, 0, s, a);
}

size_t list_bytes(int batch)
{
    return (256 + 2 * (static_cast<size_t>(batch) + 1) * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

// chunks of the longest sequence, with the fewest blocks a chunk may have
long long most_chunks(int max_seqlen_q, int steps)
{
    return ((static_cast<long long>(max_seqlen_q) + kStep - 1) / kStep + steps - 1) / steps;
}

}  // namespace

size_t key_weights_workspace_bytes(int batch, int total_k, int max_seqlen_q, int num_heads)
{
    const long long parts =
        2 * most_chunks(max_seqlen_q, chunk_steps_for(total_k, num_heads));
    return list_bytes(batch) + static_cast<size_t>(parts) * num_heads * total_k * sizeof(float);
}

cudaError_t launch_key_weights(int head_dim, KeyWeightArgs &a, void *workspace, int sm_count,
                               cudaStream_t stream)
{
    uint8_t *p = static_cast<uint8_t *>(workspace);
    a.status = reinterpret_cast<int32_t *>(p);
    a.tile_start = reinterpret_cast<int32_t *>(p + 256);
    a.unit_start = a.tile_start + a.batch + 1;
    a.part = reinterpret_cast<float *>(p + list_bytes(a.batch));
    a.chunk_steps = chunk_steps_for(a.total_k, a.num_heads);
    switch (head_dim) {
    case 64: return launch_d<64>(a, sm_count, stream);
    case 128: return launch_d<128>(a, sm_count, stream);
    case 256: return launch_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
