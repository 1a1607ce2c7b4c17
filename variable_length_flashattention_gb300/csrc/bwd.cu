// bwd.cu -- variable-length attention backward on sm_103a (head_dim 64, 128,
// 256).
//
// Gradients of the forward (scaled scores, causal / bottom-right / sliding-
// window masks on local positions, softmax over the visible keys) for an
// upstream gradient dO, given the forward's out and natural-log lse.  With
// P = exp(scale * q.k - lse), dP = dO V^T, Delta = rowsum(dO * out) and
// dS = P * (dP - Delta):
//   dV = P^T dO,   dK = scale * dS^T Q,   dQ = scale * dS K.
//
// Four kernels, none of them with atomics, so every gradient is
// deterministic:
//   * bwd_prep: one CTA validates cu_seqlens and writes each sequence's first
//     global key tile and first global q tile (prefix sums of
//     ceil(L / 128));
//   * bwd_delta: Delta[t, h] = sum_d dO * out, one warp per (token, head);
//   * the dK/dV kernel (bwd_main_kernel<D, false>): for each 128-key tile and
//     kv head -- at head_dim 256 each column half of dK and dV -- K and V
//     stay in shared memory; the query rows that see a key of the tile stream
//     past in steps of STEP rows (64; 32 at head_dim 256), every query head of
//     the group, Q and dO through a TMA ring.  Per step the tensor core forms
//     S^T = K Q^T and dP^T = V dO^T into one of two TMEM buffers; eight warps
//     turn them into P^T and dS^T (bf16, written back over the columns they
//     read), and the tensor core accumulates dV += P^T dO and dK += dS^T Q in
//     TMEM with both A operands read from TMEM.  With two buffers the next
//     step's S^T / dP^T run on the tensor core while this step's are being
//     exponentiated;
//   * the dQ kernel (bwd_main_kernel<D, true>): for each 128-query tile and
//     head, the same with the roles swapped: Q, dO stay, K and V stream past
//     in blocks of STEP keys (96; 32 at head_dim 256, through their own TMA
//     maps with boxes of that height); S = Q K^T, dP = dO V^T into two TMEM
//     buffers, dS (bf16, over dP) and dQ += dS K in TMEM.  dQ leaves as bf16
//     once, so no fp32 sum and no second pass exist.  It is launched with
//     programmatic dependent launch and starts on the SMs the dK/dV kernel's
//     CTAs leave (it reads nothing that kernel writes).
// Both are persistent: one CTA per SM takes (tile, head) units from an atomic
// counter, and consecutive units overlap (the next unit's own tiles load and
// its first score products run while the current one finishes).  dK, dV and
// dQ leave through a per-warp shared-memory stage.
// Sinks (keys j < sink_tokens that a window leaves visible; the instantiations
// with SINK).  A query tile's sink blocks are streamed ahead of its window's.
// A key tile that holds sinks sees every later query of its sequence, where
// the others see a window: its steps are cut into chunks that are units of
// their own, about kSinkUnits in all, whose dV and dK go to the workspace in
// fp32; bwd_sinks_kernel adds them in the order of the chunks.
// The math warps evaluate masks only on steps that need them, as one
// interval of visible columns per thread.  Every wait is bounded; on expiry
// the CTA records VFA_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and
// exits.
#include <algorithm>
#include <cfloat>
#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace vfa {

namespace {

constexpr int kMathWarps = 8;      // four TMEM lane quarters x two column halves
constexpr int kFirstMathWarp = 4;
constexpr int kMathThreads = kMathWarps * 32;
constexpr int kThreads = (kFirstMathWarp + kMathWarps) * 32;   // + TMA, MMA, two idle warps
constexpr uint32_t kEpiStage = 32 * 64;    // per math warp: 32 rows x 32 bf16 columns of output
constexpr float kLog2e = 1.4426950408889634f;

// Shapes per head_dim and kernel (DQ: the dQ kernel).  STEP rows (queries,
// resp. keys) stream past per step, as many as TMEM holds two buffers of:
// 96 keys past a query tile (dQ + 2 x (2 x 96) columns at head_dim 128), 64
// queries past a key tile at head_dim 128 (dK, dV and 2 x (2 x 64)) and 96
// at head_dim 64; N = 96 score products run at 56.9 cycles against 48.9 at
// N = 64 for 1.5x the work.  32 either way at head_dim 256, so that the own
// tiles and a two-stage ring fit shared memory.  The dK/dV kernel splits dK and dV into DSPLIT column
// halves, one CTA each (at head_dim 256 the two accumulators would fill TMEM
// alone).
template <int D, bool DQ>
struct BwdCfg {
    static constexpr int DB = D / 64;                       // 128-byte column blocks per row
    static constexpr int STEP = DQ ? bwd_dq_step_rows(D) : bwd_kv_step_rows(D);   // TMA box height
    static constexpr int OWN_BOX = bwd_step_rows(D);        // box height of the own-tile maps
    static constexpr int NCH = STEP / 32;                   // 32-column chunks per step
    static constexpr int DSPLIT = D == 256 ? 2 : 1;
    static constexpr int DKV = D / DSPLIT;                  // dK / dV columns per CTA
    static constexpr uint32_t OWN_BYTES = kOwn * D * 2;     // a 128-row tile
    static constexpr uint32_t STEP_BYTES = STEP * D * 2;    // a STEP-row tile
    // streamed-tile ring stages (three 96-key stages at head_dim 128 fill
    // shared memory)
    static constexpr int NSTAGE = D == 256 ? 2 : (DQ && STEP == 96 && D == 128 ? 3 : 4);
    static constexpr uint32_t STAGE_BYTES = 2 * STEP_BYTES; // (Q, dO) or (K, V)
    // per math warp: -lse log2(e) and -Delta of a step's query columns (the
    // dK/dV kernel only; the dQ kernel keeps its rows' in registers)
    static constexpr uint32_t STAT_BYTES = DQ ? 0 : 256 * NCH;
    // TMEM.  dK/dV kernel: dV, dK (DKV columns each), then two buffers of S^T
    // (STEP columns) + dP^T (STEP).  dQ kernel: dQ (D), then the two buffers.
    static constexpr uint32_t COL_DV = 0, COL_DK = DKV, KV_BUF = 2 * DKV;
    static constexpr uint32_t COL_DQ = 0, Q_BUF = D;
    static constexpr uint32_t BUF_STRIDE = 2 * STEP;
    static constexpr uint32_t TMEM_COLS = 512;
    // ring full / empty per stage; s_full, p_full, unit_full, unit_empty per
    // buffer; own_full, own_empty, acc_done, epi_done, drain
    static constexpr int NUM_BARS = 2 * NSTAGE + 8 + 5;
    static constexpr size_t SMEM = 1024 + 2 * OWN_BYTES + NSTAGE * STAGE_BYTES +
                                   kMathWarps * (STAT_BYTES + kEpiStage) + NUM_BARS * 8 + 64;
    // S^T / dP^T (keys x STEP queries) and S / dP (queries x STEP keys): both K-major
    static constexpr uint32_t IDESC_T = idesc_bf16_f32(kOwn, STEP, false, false);
    // dV, dK (DKV columns) and dQ (D columns): A from TMEM, B (dO, Q or K rows) MN-major
    static constexpr uint32_t IDESC_KV = idesc_bf16_f32(kOwn, DKV, false, true);
    static constexpr uint32_t IDESC_DQ = idesc_bf16_f32(kOwn, D, false, true);
    static_assert((DQ ? Q_BUF : KV_BUF) + 2 * BUF_STRIDE <= TMEM_COLS, "TMEM budget");
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(STEP % 32 == 0 && STEP <= 256 && kOwn % OWN_BOX == 0, "step shape");
};

// ------------------------------------------------------------ prep

// Key tiles of a sequence of lk keys that hold sinks.
__device__ __forceinline__ int sink_tiles(const BwdArgs &a, int lk)
{
    return (min(a.sink_tokens, lk) + kOwn - 1) / kOwn;
}

// STEP: queries of a step of the dK/dV kernel; SPLIT: its units per key tile.
template <int STEP, int SPLIT, bool SINK>
__global__ void __launch_bounds__(kPrepThreads) bwd_prep_kernel(const BwdArgs a)
{
    grid_release();             // the Delta kernel reads nothing of this one's
    __shared__ int warp_sums[32];
    __shared__ int s_bad;
    __shared__ unsigned long long s_steps;
    const int B = a.batch;
    if (threadIdx.x == 0)
        s_steps = 0;
    if (threadIdx.x == 0)
        s_bad = (a.cu_q[0] != 0 || a.cu_k[0] != 0 || a.cu_q[B] != a.total_q ||
                 a.cu_k[B] != a.total_k);
    __syncthreads();
    block_prefix(B, a.ktile_start, warp_sums, [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b], lk = a.cu_k[b + 1] - a.cu_k[b];
        if (lq < 0 || lk < 0) {
            s_bad = 1;
            return 0;
        }
        return (lk + kOwn - 1) / kOwn;
    });
    block_prefix(B, a.qtile_start, warp_sums, [&](int b) {
        const int lq = a.cu_q[b + 1] - a.cu_q[b];
        return lq > 0 ? (lq + kOwn - 1) / kOwn : 0;
    });
    __syncthreads();
    if (SINK && !s_bad) {
        // steps of a sequence's first sink tile (the others have as many or fewer)
        auto steps_of = [&](int b) {
            const int lq = a.cu_q[b + 1] - a.cu_q[b];
            return static_cast<long long>((lq + STEP - 1) / STEP) * (a.num_heads / a.num_kv_heads);
        };
        auto tiles_of = [&](int b) { return sink_tiles(a, a.cu_k[b + 1] - a.cu_k[b]); };
        unsigned long long mine = 0;
        for (int b = threadIdx.x; b < B; b += kPrepThreads)
            mine += steps_of(b) * tiles_of(b);
        if (mine)
            atomicAdd(&s_steps, mine);
        __syncthreads();
        const unsigned long long all = s_steps * a.num_kv_heads * SPLIT;
        const long long per =
            max(static_cast<long long>(kSinkMinSteps),
                static_cast<long long>((all + kSinkUnits - 1) / kSinkUnits));
        auto chunks_of = [&](int b) { return max(1, static_cast<int>((steps_of(b) + per - 1) / per)); };
        for (int b = threadIdx.x; b < B; b += kPrepThreads)
            a.sink_chunks[b] = chunks_of(b);
        if (threadIdx.x == 0)
            a.sink_chunks[B] = static_cast<int>(min(per, 0x7fffffffll));
        block_prefix(B, a.sink_start, warp_sums, [&](int b) { return tiles_of(b) * chunks_of(b); });
        block_prefix(B, a.part_start, warp_sums, [&](int b) {
            return chunks_of(b) > 1 ? tiles_of(b) * chunks_of(b) : 0;
        });
        block_prefix(B, a.cut_start, warp_sums, [&](int b) { return chunks_of(b) > 1 ? tiles_of(b) : 0; });
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.status[1] = 0;                 // unit counters of the two main kernels
        a.status[2] = 0;
        *a.status = s_bad ? VFA_ERR_BAD_SEQLENS : VFA_OK;
    }
}

// ------------------------------------------------------------ Delta
//
// Runs beside the prep kernel, one CTA's chain of prefix sums, and waits for it
// before it ends: the dK/dV kernel behind it waits for this one alone.

template <int D>
__global__ void bwd_delta_kernel(const BwdArgs a)
{
    grid_release();
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(a.total_q) * a.num_heads;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    const __nv_bfloat16 *o = static_cast<const __nv_bfloat16 *>(a.out);
    const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(a.dout);
    for (long long r = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         r < rows; r += warps) {
        float s = 0.f;
#pragma unroll
        for (int d = lane * 2; d < D; d += 64) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(o + r * D + d);
            const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162 *>(g + r * D + d);
            s += __bfloat162float(x.x) * __bfloat162float(y.x) +
                 __bfloat162float(x.y) * __bfloat162float(y.y);
        }
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o2);
        if (lane == 0)
            a.delta[r] = s;
    }
    grid_wait();
}

// The same for the instantiations with sinks: D / 8 lanes per row with 16-byte loads, two
// rows of a lane in flight (49879 tokens of 16 heads of 64: 37 us, 59 with a warp per
// row; the order of a sum, and with it the last bits, differs from the other's).
template <int D>
__global__ void __launch_bounds__(256) bwd_delta_wide_kernel(const BwdArgs a)
{
    grid_release();
    constexpr int LANES = D / 8, TURNS = 2;
    const long long rows = static_cast<long long>(a.total_q) * a.num_heads;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x / LANES;
    const int l = threadIdx.x % LANES;
    const uint4 *o = static_cast<const uint4 *>(a.out), *g = static_cast<const uint4 *>(a.dout);
    // whole warps go round together: the last turns' lanes past the end take part in the sums
    const long long first = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / LANES;
    const long long warp_first = (static_cast<long long>(blockIdx.x) * blockDim.x + (threadIdx.x & ~31)) / LANES;
    for (long long r = first, w = warp_first; w < rows; r += step * TURNS, w += step * TURNS) {
        uint4 x[TURNS], y[TURNS];
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const long long row = r + t * step;
            x[t] = y[t] = make_uint4(0, 0, 0, 0);
            if (row < rows) {
                x[t] = __ldcs(o + row * LANES + l);
                y[t] = __ldg(g + row * LANES + l);
            }
        }
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const uint32_t xs[4] = {x[t].x, x[t].y, x[t].z, x[t].w}, ys[4] = {y[t].x, y[t].y, y[t].z, y[t].w};
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s += __uint_as_float(xs[e] << 16) * __uint_as_float(ys[e] << 16) +
                     __uint_as_float(xs[e] & 0xffff0000u) * __uint_as_float(ys[e] & 0xffff0000u);
#pragma unroll
            for (int k = LANES / 2; k > 0; k >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, k);
            if (l == 0 && r + t * step < rows)
                a.delta[r + t * step] = s;
        }
    }
    grid_wait();
}

// ------------------------------------------------------------ shared pieces

// Query i's visible keys among j_base, j_base + 1, ... (the dQ kernel's
// columns): j < Lk, and j <= i + off (causal), j >= i + off - window_left.
__device__ __forceinline__ void query_row_span(long long i, long long j_base, int lk, int lq,
                                               int causal, int wl, long long off, int *lo,
                                               int *hi)
{
    long long l = (causal && wl >= 0) ? i + off - wl - j_base : 0;
    long long h = lk - j_base;
    if (causal)
        h = min(h, i + off - j_base + 1);
    if (i >= lq)
        h = l;
    *lo = clamp_col(l);
    *hi = clamp_col(h);
}

// -lse log2(e); of a row without visible keys (lse = -FLT_MAX, or -inf from elsewhere), whose
// scores are all hidden, 0
__device__ __forceinline__ float neg_lse(float lse)
{
    return lse <= -FLT_MAX ? 0.f : -lse * kLog2e;
}

// P^T and dS^T of this thread's key row over its NC query columns: p =
// 2^(s scale_log2 + nl)
// and ds = p (dp + nd), with nl = -lse log2(e) and nd = -Delta of each column
// read from shared memory (NC floats each at wstat, wstat + 128).
template <int NC>
__device__ __forceinline__ void key_row_grads(const uint32_t (&sr)[NC], const uint32_t (&dr)[NC],
                                              float scale_log2, uint32_t wstat,
                                              uint32_t (&pk)[NC / 2], uint32_t (&dk2)[NC / 2])
{
    const float2 c2 = make_float2(scale_log2, scale_log2);
#pragma unroll
    for (int e = 0; e < NC; e += 4) {
        const uint4 nl4 = ld_shared_v4(wstat + e * 4);
        const uint4 nd4 = ld_shared_v4(wstat + 128 + e * 4);
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
            const uint32_t nla = u ? nl4.z : nl4.x, nlb = u ? nl4.w : nl4.y;
            const uint32_t nda = u ? nd4.z : nd4.x, ndb = u ? nd4.w : nd4.y;
            const float2 t = __ffma2_rn(make_float2(__uint_as_float(sr[e + u]),
                                                    __uint_as_float(sr[e + u + 1])),
                                        c2, make_float2(__uint_as_float(nla),
                                                        __uint_as_float(nlb)));
            const float p0 = ex2_approx(t.x), p1 = ex2_approx(t.y);
            const float2 g = __fadd2_rn(make_float2(__uint_as_float(dr[e + u]),
                                                    __uint_as_float(dr[e + u + 1])),
                                        make_float2(__uint_as_float(nda), __uint_as_float(ndb)));
            const float2 ds = __fmul2_rn(make_float2(p0, p1), g);
            pk[(e + u) >> 1] = pack_bf16x2(p0, p1);
            dk2[(e + u) >> 1] = pack_bf16x2(ds.x, ds.y);
        }
    }
}

// dS of this thread's query row over its NC key columns: p = 2^(s
// scale_log2 + nl), ds = p (dp + nd) with the
// row's nl = -lse log2(e) and nd = -Delta.
template <int NC>
__device__ __forceinline__ void query_row_grads(const uint32_t (&sr)[NC], const uint32_t (&dr)[NC],
                                                float scale_log2, float nl, float nd,
                                                uint32_t (&dk2)[NC / 2])
{
    const float2 c2 = make_float2(scale_log2, scale_log2);
    const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
#pragma unroll
    for (int e = 0; e < NC; e += 2) {
        const float2 t = __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])),
                                    c2, nl2);
        const float p0 = ex2_approx(t.x), p1 = ex2_approx(t.y);
        const float2 g = __fadd2_rn(make_float2(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])),
                                    nd2);
        const float2 ds = __fmul2_rn(make_float2(p0, p1), g);
        dk2[e >> 1] = pack_bf16x2(ds.x, ds.y);
    }
}

// D += A B over K = STEP streamed rows: A (128 x STEP, bf16 pairs) in TMEM at
// a_tmem, written by the math warps in chunks of 32 columns (chunk c's 32
// values packed into the first 16 of its own 32 columns); B the STEP-row tile
// in shared memory from column block b_buf on, MN-major.
template <int STEP>
__device__ __forceinline__ void issue_accumulate(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_buf,
                                                 uint32_t idesc, bool first)
{
    const uint64_t b0 = sdesc_sw128(b_buf, STEP * 128, 1024);
#pragma unroll
    for (int kk = 0; kk < STEP / 16; ++kk) {
        const uint32_t a = a_tmem + 32 * (kk >> 1) + 8 * (kk & 1);
        const uint64_t bo = (kk * 16 * 128) >> 4;
        if (kk == 0 && first)
            mma_ts_w<0>(d_tmem, a, b0 + bo, idesc);
        else
            mma_ts_w<1>(d_tmem, a, b0 + bo, idesc);
    }
}

// NC consecutive TMEM columns of this warp's lanes into r (warp-collective),
// and NC / 2 packed columns back.
template <int NC>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[NC])
{
    if constexpr (NC == 32)
        tmem_ld32(taddr, r);
    else
        tmem_ld16(taddr, r);
}

template <int NC>
__device__ __forceinline__ void wait_cols(uint32_t (&r)[NC], uint32_t (&q)[NC])
{
    if constexpr (NC == 32) {
        tmem_wait_ld_r(r);
        tmem_bind_r(q);
    } else {
        tmem_wait_ld_r16(r);
        asm volatile(""
                     : "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]), "+r"(q[4]), "+r"(q[5]),
                       "+r"(q[6]), "+r"(q[7]), "+r"(q[8]), "+r"(q[9]), "+r"(q[10]), "+r"(q[11]),
                       "+r"(q[12]), "+r"(q[13]), "+r"(q[14]), "+r"(q[15])
                     :
                     : "memory");
    }
}

template <int NP>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[NP])
{
    if constexpr (NP == 16) {
        tmem_st16(taddr, r);
    } else {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], "
                     "{%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                     "r"(r[6]), "r"(r[7])
                     : "memory");
    }
}

// 32 accumulator columns of this warp's 32 rows (fp32 in TMEM at taddr; the
// thread's lane is its row) * f -> bf16 at dst0 (the warp's first row, the
// chunk's first column; rows row_stride elements apart).  The values pass
// through the warp's 2 KB stage (row segments swizzled by row, so the writes
// are conflict-free) so that every global store instruction writes eight
// whole 64-byte row segments; rows n_valid and later are not written.
__device__ __forceinline__ void store_tile32(uint32_t taddr, float f, uint32_t stage, int lane,
                                             __nv_bfloat16 *dst0, size_t row_stride, int n_valid)
{
    uint32_t rr[32];
    tmem_ld32(taddr, rr);
    tmem_wait_ld_r(rr);
    const uint32_t row = stage + lane * 64;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        st_shared_v4(row + ((c ^ ((lane >> 1) & 3)) << 4),
                     pack_bf16x2(__uint_as_float(rr[8 * c + 0]) * f, __uint_as_float(rr[8 * c + 1]) * f),
                     pack_bf16x2(__uint_as_float(rr[8 * c + 2]) * f, __uint_as_float(rr[8 * c + 3]) * f),
                     pack_bf16x2(__uint_as_float(rr[8 * c + 4]) * f, __uint_as_float(rr[8 * c + 5]) * f),
                     pack_bf16x2(__uint_as_float(rr[8 * c + 6]) * f, __uint_as_float(rr[8 * c + 7]) * f));
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int rw = 8 * k + (lane >> 2), ch = lane & 3;
        const uint4 v = ld_shared_v4(stage + rw * 64 + ((ch ^ ((rw >> 1) & 3)) << 4));
        if (rw < n_valid)
            *reinterpret_cast<uint4 *>(dst0 + rw * row_stride + ch * 8) = v;
    }
    __syncwarp();
}

// 32 accumulator columns of the thread's row, as they are.
__device__ __forceinline__ void store_part32(uint32_t taddr, float *dst)
{
    uint32_t rr[32];
    tmem_ld32(taddr, rr);
    tmem_wait_ld_r(rr);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        reinterpret_cast<uint4 *>(dst)[c] =
            make_uint4(rr[4 * c], rr[4 * c + 1], rr[4 * c + 2], rr[4 * c + 3]);
}

// ------------------------------------------------------------ the two main kernels

// One unit of work, decoded by the loading warp and handed to the others
// through a two-slot shared-memory ring.  dK/dV kernel: (kv head, 128-key
// tile, column half); dQ kernel: (head, 128-query tile).
struct BwdUnit {
    int b, t, head, dh;          // sequence, tile in it, (kv) head, column half
    int q0, lq, k0, lk;          // the sequence's rows and lengths
    int first, n_blk, n_steps;   // streamed blocks [first, first + n_blk); steps (x group)
    int valid;                   // 0: no more units
    // with sinks: dQ: blocks [0, n_sink) come first; dK/dV: this unit's first step of
    // its tile's, the partial it writes (-1: the gradients themselves), and whether
    // there is nothing to do (a tile whose chunks are units)
    int n_sink, step0, part, skip;
};

// Unit u of the dK/dV kernel (DQ false) or the dQ kernel (DQ true); `tiles`
// is the number of 128-row tiles of all sequences.
template <int D, bool DQ, bool SINK>
__device__ BwdUnit decode_unit(const BwdArgs &a, int u, int tiles)
{
    using C = BwdCfg<D, DQ>;
    constexpr int STEP = C::STEP;
    constexpr int SPLIT = DQ ? 1 : C::DSPLIT;
    BwdUnit w;
    const int per_head = tiles * SPLIT;
    const int n_heads = DQ ? a.num_heads : a.num_kv_heads;
    w.n_sink = w.step0 = w.skip = 0;
    w.part = -1;
    // the chunks of the sinks' tiles come first
    const int sink_units = SINK && !DQ ? a.sink_start[a.batch] * SPLIT : 0;
    const bool chunked = SINK && !DQ && u < sink_units * n_heads;
    u -= SINK && !chunked ? sink_units * n_heads : 0;
    w.valid = chunked || u < per_head * n_heads;
    if (!w.valid)
        return w;
    const int per_row = chunked ? sink_units : per_head;
    w.head = u / per_row;
    const int r = u % per_row;
    // dQ: each head's tiles run last-first (a causal sequence's longest key
    // ranges first); dK/dV: in order (a sequence's first key tiles see the
    // most queries); a key tile's column halves are neighbours
    int gt = r / SPLIT;
    w.dh = r % SPLIT;
    if (DQ)
        gt = tiles - 1 - gt;
    const int32_t *start = DQ ? a.qtile_start : chunked ? a.sink_start : a.ktile_start;
    w.b = owner_of(start, a.batch, gt);
    w.t = gt - start[w.b];
    int chunk = 0, chunks = 1;
    if (chunked) {
        chunks = a.sink_chunks[w.b];
        if (chunks > 1)
            w.part = ((a.part_start[w.b] + w.t) * a.num_kv_heads + w.head) * SPLIT + w.dh;
        chunk = w.t % chunks;
        w.t /= chunks;
    }
    w.q0 = a.cu_q[w.b];
    w.lq = a.cu_q[w.b + 1] - w.q0;
    w.k0 = a.cu_k[w.b];
    w.lk = a.cu_k[w.b + 1] - w.k0;
    const long long off = a.causal == 2 ? w.lk - w.lq : 0;
    const int wl = a.window_left;
    long long lo, hi;
    if (!DQ) {
        // queries that see a key of this tile: i >= j - off (causal),
        // i <= j - off + window_left (window)
        const int j_lo = w.t * kOwn, j_hi = min(w.lk, j_lo + kOwn);
        lo = a.causal ? max(0ll, j_lo - off) : 0;
        hi = w.lq - 1;
        const bool holds_sinks = SINK && j_lo < a.sink_tokens;
        if (wl >= 0 && !holds_sinks)
            hi = min(hi, static_cast<long long>(j_hi) - 1 - off + wl);
        w.skip = holds_sinks && !chunked;
    } else {
        // keys some row of this tile sees: j <= i + off (causal), j >= i + off
        // - window_left (window)
        const int i_lo = w.t * kOwn, i_hi = min(w.lq, i_lo + kOwn);
        lo = (a.causal && wl >= 0) ? max(0ll, i_lo + off - wl) : 0;
        hi = w.lk - 1;
        if (a.causal)
            hi = min(hi, static_cast<long long>(i_hi) - 1 + off);
    }
    w.first = lo <= hi ? static_cast<int>(lo / STEP) : 0;
    w.n_blk = lo <= hi ? static_cast<int>(hi / STEP) + 1 - w.first : 0;
    w.n_steps = DQ ? w.n_blk : w.n_blk * (a.num_heads / a.num_kv_heads);
    if (SINK && DQ) {
        // sink blocks below the window's; all of them where the window is past the keys
        const long long seen = lo <= hi ? min(lo / STEP * STEP, static_cast<long long>(w.lk))
                                        : max(0ll, hi + 1);
        w.n_sink = static_cast<int>((min(static_cast<long long>(a.sink_tokens), seen) + STEP - 1) / STEP);
        w.n_steps += w.n_sink;
    }
    if (chunked) {
        const int per = a.sink_chunks[a.batch];
        w.step0 = static_cast<int>(min(static_cast<long long>(chunk) * per,
                                       static_cast<long long>(w.n_steps)));
        w.n_steps = chunks > 1 ? min(per, w.n_steps - w.step0) : w.n_steps;
    }
    if (w.skip)
        w.n_steps = 0;
    return w;
}

// The streamed block of the unit's step s.
template <bool DQ, bool SINK>
__device__ __forceinline__ int block_of(const BwdUnit &w, int s)
{
    if (DQ)
        return SINK ? (s < w.n_sink ? s : w.first + s - w.n_sink) : w.first + s;
    return w.first + (SINK ? s + w.step0 : s) % w.n_blk;
}

// Persistent CTAs, one per SM, take units from an atomic counter.  Warp 0
// loads (the unit's own 128-row tiles once, the streamed tiles per step),
// warp 1 issues the MMAs, warps 4-11 do the elementwise work: warp w owns
// TMEM lanes (own rows) 32 (w % 4) .. +31; warpgroup g = (w - 4) / 4 takes
// the steps held in TMEM buffer g, all STEP columns of each.
//
// dK/dV kernel (DQ false): own = K, V of a key tile; a step is a block of
// STEP queries of one query head of the group; per step
//   MMA:  S^T = K Q^T, dP^T = V dO^T -> buffer x (s_full(x));
//         then, for the previous step: dV += P^T dO, dK += dS^T Q
//   math: P^T = 2^(s scale log2e - lse log2e) (masked: 0), dS^T = P^T (dP^T -
//         Delta) -> bf16 over S^T / dP^T (p_full(x))
// dQ kernel (DQ true): own = Q, dO of a query tile; a step is a block of
// STEP keys; S = Q K^T, dP = dO V^T; dS (over dP); dQ += dS K.
//
// Across units nothing restarts: the step counter (ring stage, TMEM buffer
// and their barrier phases) runs on, the next unit's own tiles load as soon
// as the last score products of the current one have read the old ones, and
// the next unit's first scores run during the current unit's epilogue; only
// its first accumulating product waits for the epilogue (epi_done) to have
// read the accumulators.
template <int D, bool DQ, bool SINK>
__global__ void __launch_bounds__(kThreads, 1) bwd_main_kernel(const __grid_constant__ BwdArgs a)
{
    using C = BwdCfg<D, DQ>;
    constexpr int DB = C::DB, NSTAGE = C::NSTAGE, STEP = C::STEP, NCH = C::NCH;
    constexpr int NACC = DQ ? D : C::DKV;        // accumulator columns (each)
    constexpr int DH = NACC / 2;                  // accumulator columns per math thread
    constexpr uint32_t BUF = DQ ? C::Q_BUF : C::KV_BUF;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ int s_abort;
    __shared__ BwdUnit s_unit[2];

    // The dK/dV kernel waits for the Delta kernel, and with it for the prep kernel.  The
    // dQ kernel, launched next with programmatic dependent launch, reads what
    // those two wrote and nothing this kernel writes: from here on let it take each SM
    // this kernel's CTAs leave.
    if (!DQ) {
        grid_wait();
        grid_release();
    } else if (SINK) {
        grid_release();             // the sums of the sinks' chunks, always next, wait for it
    }
    // The dQ kernel waits for the dK/dV kernel before it ends: what is launched
    // behind it in the same way waits for the dQ kernel alone, and may read dK
    // and dV.
    auto wait_for_dkv = [] {
        if (DQ)
            asm volatile("griddepcontrol.wait;" ::: "memory");
    };
    if (*a.status != VFA_OK) {
        wait_for_dkv();
        return;
    }
    const int B = a.batch, H = a.num_heads, Hkv = a.num_kv_heads;
    const int tiles = DQ ? a.qtile_start[B] : a.ktile_start[B];
    int32_t *counter = a.status + (DQ ? 2 : 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3;
    const int half = warp >= kFirstMathWarp ? (warp - kFirstMathWarp) >> 2 : 0;
    const int r = quarter * 32 + lane;            // own row of math threads

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sOwn0 = base, sOwn1 = sOwn0 + C::OWN_BYTES;     // K, V  /  Q, dO
    const uint32_t sRing = sOwn1 + C::OWN_BYTES;                    // stage: Q, dO  /  K, V
    const uint32_t sStat = sRing + NSTAGE * C::STAGE_BYTES;         // per math warp: nl, -Delta
    const uint32_t sEpi = sStat + kMathWarps * C::STAT_BYTES;       // per math warp: output stage
    const uint32_t bars = sEpi + kMathWarps * kEpiStage;
    auto ring_full = [&](int st) { return bars + 8u * st; };
    auto ring_empty = [&](int st) { return bars + 8u * (NSTAGE + st); };
    auto s_full = [&](int x) { return bars + 8u * (2 * NSTAGE + x); };
    auto p_full = [&](int x) { return bars + 8u * (2 * NSTAGE + 2 + x); };
    auto unit_full = [&](int x) { return bars + 8u * (2 * NSTAGE + 4 + x); };
    auto unit_empty = [&](int x) { return bars + 8u * (2 * NSTAGE + 6 + x); };
    const uint32_t own_full = bars + 8u * (2 * NSTAGE + 8);
    const uint32_t own_empty = bars + 8u * (2 * NSTAGE + 9);
    const uint32_t acc_done = bars + 8u * (2 * NSTAGE + 10);
    const uint32_t epi_done = bars + 8u * (2 * NSTAGE + 11);
    const uint32_t drain_bar = bars + 8u * (2 * NSTAGE + 12);
    auto stage0 = [&](int st) { return sRing + st * C::STAGE_BYTES; };
    auto stage1 = [&](int st) { return sRing + st * C::STAGE_BYTES + C::STEP_BYTES; };
    volatile int *abort = &s_abort;

    if (tid == 0) {
        s_abort = 0;
        for (int st = 0; st < NSTAGE; ++st) {
            mbar_init(ring_full(st), 1);
            mbar_init(ring_empty(st), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(x), 1);
            mbar_init(p_full(x), kMathThreads / 2);    // buffer x's warpgroup
            mbar_init(unit_full(x), 1);
            mbar_init(unit_empty(x), 1 + kMathWarps);
        }
        mbar_init(own_full, 1);
        mbar_init(own_empty, 1);
        mbar_init(acc_done, 1);
        mbar_init(epi_done, kMathThreads);
        mbar_init(drain_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem_base;

    // Consumers take unit n from the ring; false at the end (or on abort).
    auto take_unit = [&](uint32_t n, BwdUnit &w) -> bool {
        if (!mbar_wait_warp(unit_full(n & 1), (n >> 1) & 1u, abort))
            return false;
        w = s_unit[n & 1];
        return w.valid;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            tma_prefetch_map(&a.tm_q);
            tma_prefetch_map(&a.tm_k);
            tma_prefetch_map(&a.tm_v);
            tma_prefetch_map(&a.tm_do);
            const CUtensorMap *own0 = DQ ? &a.tm_q : &a.tm_k, *own1 = DQ ? &a.tm_do : &a.tm_v;
            const CUtensorMap *str0 = DQ ? &a.tm_ks : &a.tm_qs, *str1 = DQ ? &a.tm_vs : &a.tm_dos;
            tma_prefetch_map(str0);
            tma_prefetch_map(str1);
            uint32_t g = 0, owns = 0;
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                if (!mbar_wait(unit_empty(n & 1), ((n >> 1) & 1u) ^ 1u, abort))
                    break;
                const BwdUnit w = decode_unit<D, DQ, SINK>(a, atomicAdd(counter, 1), tiles);
                s_unit[n & 1] = w;
                mbar_arrive(unit_full(n & 1));
                if (!w.valid)
                    break;
                if (w.n_steps == 0)
                    continue;
                // the previous unit's score products have read the own tiles
                if (!mbar_wait(own_empty, (owns & 1u) ^ 1u, abort))
                    break;
                mbar_arrive_expect_tx(own_full, 2 * C::OWN_BYTES);
                const int own_row = (DQ ? w.q0 : w.k0) + w.t * kOwn;
                load_rows<DB, C::OWN_BOX>(sOwn0, own0, own_full, w.head, own_row, kOwn);
                load_rows<DB, C::OWN_BOX>(sOwn1, own1, own_full, w.head, own_row, kOwn);
                ++owns;
                const int group = H / Hkv;
                for (int s = 0; s < w.n_steps; ++s, ++g) {
                    const int st = g % NSTAGE;
                    if (!mbar_wait(ring_empty(st), ((g / NSTAGE) & 1u) ^ 1u, abort)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(ring_full(st), C::STAGE_BYTES);
                    // dK/dV: step s = (query head of the group, query block);
                    // dQ: key block of the head's kv head
                    const int blk = block_of<DQ, SINK>(w, s);
                    const int row = (DQ ? w.k0 : w.q0) + blk * STEP;
                    const int head = DQ ? w.head / group
                                        : w.head * group + (SINK ? s + w.step0 : s) / w.n_blk;
                    load_rows<DB, STEP>(stage0(st), str0, ring_full(st), head, row, STEP);
                    load_rows<DB, STEP>(stage1(st), str1, ring_full(st), head, row, STEP);
                }
            }
            if (*abort) {
                // the last fill of each stage and of the own tiles may be in flight
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
        // All 32 lanes run this loop on warp-uniform values; one elected lane
        // issues each MMA and commit.
        uint32_t g = 0, owns = 0, units = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            BwdUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            if (w.n_steps == 0)
                continue;
            if (!mbar_wait_warp(own_full, owns & 1u, abort)) {
                ok = false;
                break;
            }
            ++owns;
            // this unit's column half of the streamed tiles' columns (dK/dV at
            // head_dim 256): DKV / 64 column blocks on
            const uint32_t col0 = DQ ? 0u : w.dh * (C::DKV / 64) * (STEP * 128);
            for (int s = 0; s <= w.n_steps && ok; ++s) {
                if (s < w.n_steps) {
                    const uint32_t gs = g + s;
                    const int st = gs % NSTAGE, x = gs & 1;
                    if (!mbar_wait_warp(ring_full(st), (gs / NSTAGE) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // buffer x was last read by step gs - 2's products, issued earlier
                    const uint32_t buf = tmem + BUF + C::BUF_STRIDE * x;
                    issue_scores<D, STEP>(buf, sOwn0, stage0(st), C::IDESC_T);
                    issue_scores<D, STEP>(buf + STEP, sOwn1, stage1(st), C::IDESC_T);
                    mma_commit_w(s_full(x));
                    if (s == w.n_steps - 1)
                        mma_commit_w(own_empty);        // own tiles free once these complete
                }
                if (s >= 1) {
                    const uint32_t gp = g + s - 1;
                    const int stp = gp % NSTAGE, xp = gp & 1;
                    if (!mbar_wait_warp(p_full(xp), (gp >> 1) & 1u, abort) ||
                        (s == 1 && !mbar_wait_warp(epi_done, (units & 1u) ^ 1u, abort))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t buf = tmem + BUF + C::BUF_STRIDE * xp;
                    if (DQ) {
                        issue_accumulate<STEP>(tmem + C::COL_DQ, buf + STEP, stage0(stp),
                                               C::IDESC_DQ, s == 1);
                    } else {
                        issue_accumulate<STEP>(tmem + C::COL_DV, buf, stage1(stp) + col0,
                                               C::IDESC_KV, s == 1);
                        issue_accumulate<STEP>(tmem + C::COL_DK, buf + STEP, stage0(stp) + col0,
                                               C::IDESC_KV, s == 1);
                    }
                    mma_commit_w(ring_empty(stp));
                }
            }
            if (!ok)
                break;
            mma_commit_w(acc_done);
            g += w.n_steps;
            ++units;
        }
        if (!ok || *abort) {
            mma_commit_w(drain_bar);
            mbar_wait_drain(drain_bar, 0);
        }
    } else if (warp >= kFirstMathWarp) {
        // ------------------------------------------------------------ elementwise, epilogue
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        // per warp and 32-column chunk: 32 nl, then 32 -Delta
        const uint32_t wstat = sStat + (warp - kFirstMathWarp) * C::STAT_BYTES;
        float *stat = reinterpret_cast<float *>(smem_raw + (wstat - raw));
        const float scale_log2 = a.scale_log2;
        uint32_t g = 0, units = 0;
        bool ok = true;
        __nv_bfloat16 *dq = static_cast<__nv_bfloat16 *>(a.dq);
        __nv_bfloat16 *dk = static_cast<__nv_bfloat16 *>(a.dk);
        __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv);
        for (uint32_t n = 0; ok; ++n) {
            BwdUnit w;
            const bool more = take_unit(n, w);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(unit_empty(n & 1));
            if (!more)
                break;
            const long long off = a.causal == 2 ? w.lk - w.lq : 0;
            const int wl = a.window_left;
            const int own = w.t * kOwn + r;       // this thread's own row (key or query)
            // where this thread's accumulator columns go
            size_t row_out;
            if (DQ)
                row_out = (static_cast<size_t>(w.q0 + own) * H + w.head) * D + half * DH;
            else
                row_out = (static_cast<size_t>(w.k0 + own) * Hkv + w.head) * D + w.dh * C::DKV +
                          half * DH;
            const bool own_valid = DQ ? own < w.lq : own < w.lk;
            if (SINK && !DQ && w.skip)
                continue;
            // a chunk's partial: dV, then dK, 128 rows of DKV columns each
            float *part = nullptr;
            if (SINK && !DQ && w.part >= 0)
                part = a.part + (static_cast<size_t>(w.part) * 2 * kOwn + r) * C::DKV + half * DH;
            if (w.n_steps == 0 && part) {
#pragma unroll
                for (int d = 0; d < DH; d += 4) {
                    *reinterpret_cast<float4 *>(part + d) = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4 *>(part + kOwn * C::DKV + d) =
                        make_float4(0.f, 0.f, 0.f, 0.f);
                }
                continue;
            }
            if (w.n_steps == 0) {
                // no key / query pairs: zero gradients
                if (own_valid) {
#pragma unroll
                    for (int d = 0; d < DH; d += 8) {
                        if (DQ) {
                            *reinterpret_cast<uint4 *>(dq + row_out + d) = make_uint4(0, 0, 0, 0);
                        } else {
                            *reinterpret_cast<uint4 *>(dk + row_out + d) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(dv + row_out + d) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                continue;
            }
            // dQ: this thread's row constants
            float nl_row = 0.f, nd_row = 0.f;
            if (DQ && own_valid) {
                const size_t srow = static_cast<size_t>(w.q0 + own) * H + w.head;
                nl_row = neg_lse(a.lse[srow]);
                nd_row = -a.delta[srow];
            }
            const int group = H / Hkv;
            // The two warpgroups take the steps in turn (warpgroup x the steps
            // in TMEM buffer x), each doing all STEP columns of its rows in
            // chunks of 32, so two steps are in the works at once.
            for (int s = (half - static_cast<int>(g & 1u)) & 1; s < w.n_steps && ok; s += 2) {
                const uint32_t gs = g + s;
                const int x = gs & 1;
                const int blk = block_of<DQ, SINK>(w, s);
                const int c0 = blk * STEP;                 // the step's first streamed column
                if (!DQ) {
                    // -lse log2(e) and -Delta of the step's query columns
                    const int hq = w.head * group + (SINK ? s + w.step0 : s) / w.n_blk;
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        const int i = c0 + 32 * c + lane;
                        const size_t srow = static_cast<size_t>(w.q0 + i) * H + hq;
                        stat[64 * c + lane] = i < w.lq ? neg_lse(a.lse[srow]) : 0.f;
                        stat[64 * c + 32 + lane] = i < w.lq ? -a.delta[srow] : 0.f;
                    }
                    __syncwarp();
                }
                // a step every (own, streamed) pair of which is visible needs no mask
                const long long slo = static_cast<long long>(c0);
                const long long olo = static_cast<long long>(w.t) * kOwn;
                bool full;
                if (DQ)
                    full = slo + STEP <= w.lk && olo + kOwn <= w.lq &&
                           (!a.causal || slo + STEP - 1 <= olo + off) &&
                           (wl < 0 || slo >= olo + kOwn - 1 + off - wl ||
                            (SINK && slo + STEP <= a.sink_tokens));
                else
                    full = olo + kOwn <= w.lk && slo + STEP <= w.lq &&
                           (!a.causal || olo + kOwn - 1 <= slo + off) &&
                           (wl < 0 || olo >= slo + STEP - 1 + off - wl ||
                            (SINK && olo + kOwn <= a.sink_tokens));
                ok = mbar_wait_warp(s_full(x), (gs >> 1) & 1u, abort);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < NCH; ++c) {
                    const uint32_t st_addr = tmem + lane_addr + BUF + C::BUF_STRIDE * x + 32 * c;
                    uint32_t sr[32], dr[32];
                    ld_cols<32>(st_addr, sr);
                    ld_cols<32>(st_addr + STEP, dr);
                    wait_cols<32>(sr, dr);
                    uint32_t dk2[16];
                    const int cb = c0 + 32 * c;            // the chunk's first streamed column
                    if (DQ) {
                        if (!full) {
                            int lo, hi;
                            query_row_span(own, cb, w.lk, w.lq, a.causal, wl, off, &lo, &hi);
                            if (own >= w.lq)
                                hi = -1;                   // no row: no sinks either
                            uint32_t from = ~below(lo);
                            if (SINK)
                                from |= below(a.sink_tokens - cb);
                            hide(sr, below(hi) & from);
                        }
                        query_row_grads(sr, dr, scale_log2, nl_row, nd_row, dk2);
                    } else {
                        uint32_t pk[16];
                        const uint32_t cstat = wstat + 256 * c;
                        if (!full) {
                            int lo, hi;
                            key_row_span(own, cb, w.lk, w.lq, a.causal,
                                         SINK && own < a.sink_tokens ? -1 : wl, off, &lo, &hi);
                            hide(sr, below(hi) & ~below(lo));
                        }
                        key_row_grads(sr, dr, scale_log2, cstat, pk, dk2);
                        // P^T (bf16 pairs) over the first half of the chunk's S^T columns
                        st_cols<16>(st_addr, pk);
                    }
                    // dS (bf16 pairs) over the first half of the chunk's dP columns
                    st_cols<16>(st_addr + STEP, dk2);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full(x));
            }
            if (!ok)
                break;
            ok = mbar_wait_warp(acc_done, units & 1u, abort);
            if (!ok)
                break;
            tc_fence_after();
            {
                // this warp's 32 rows start at own row w.t * 128 + 32 * quarter
                const int wrow = w.t * kOwn + quarter * 32;
                const int n_valid = (DQ ? w.lq : w.lk) - wrow;
                const uint32_t stage = sEpi + (warp - kFirstMathWarp) * kEpiStage;
                const size_t stride = static_cast<size_t>(DQ ? H : Hkv) * D;
                const size_t base_out = row_out - static_cast<size_t>(lane) * stride;
#pragma unroll 1
                for (int cb = 0; cb < DH; cb += 32) {
                    if (SINK && !DQ && part) {
                        store_part32(tmem + lane_addr + C::COL_DV + half * DH + cb, part + cb);
                        store_part32(tmem + lane_addr + C::COL_DK + half * DH + cb,
                                     part + kOwn * C::DKV + cb);
                    } else if (DQ) {
                        store_tile32(tmem + lane_addr + C::COL_DQ + half * DH + cb, a.scale, stage,
                                     lane, dq + base_out + cb, stride, n_valid);
                    } else {
                        store_tile32(tmem + lane_addr + C::COL_DV + half * DH + cb, 1.f, stage,
                                     lane, dv + base_out + cb, stride, n_valid);
                        store_tile32(tmem + lane_addr + C::COL_DK + half * DH + cb, a.scale, stage,
                                     lane, dk + base_out + cb, stride, n_valid);
                    }
                }
            }
            // the accumulators may be overwritten by the next unit's products
            tc_fence_before();
            mbar_arrive(epi_done);
            g += w.n_steps;
            ++units;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort && tid == 0)
        atomicCAS(a.status, VFA_OK, VFA_ERR_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    wait_for_dkv();
}

// dV and dK of the sinks' tiles that were cut: the chunks' partials in order.
// A CTA takes kSinkRows rows of a tile and kv head at a time, a thread four
// columns of them.
constexpr int kSinkRows = 4, kSinkShares = kOwn / kSinkRows;

template <int D>
__global__ void __launch_bounds__(2 * kSinkRows * D / 4) bwd_sinks_kernel(const BwdArgs a)
{
    using C = BwdCfg<D, false>;
    grid_wait();
    if (*a.status != VFA_OK)
        return;
    const int sub_row = threadIdx.x / (D / 4) % kSinkRows;
    const bool is_dk = threadIdx.x >= kSinkRows * D / 4;
    const int col = threadIdx.x % (D / 4) * 4, dh = col / C::DKV;
    const long long items = static_cast<long long>(a.cut_start[a.batch]) * a.num_kv_heads * kSinkShares;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int row = static_cast<int>(it % kSinkShares) * kSinkRows + sub_row;
        const int head = static_cast<int>(it / kSinkShares % a.num_kv_heads);
        const int cut = static_cast<int>(it / kSinkShares / a.num_kv_heads);
        const int b = owner_of(a.cut_start, a.batch, cut), t = cut - a.cut_start[b];
        const int chunks = a.sink_chunks[b], k0 = a.cu_k[b], key = t * kOwn + row;
        if (key >= a.cu_k[b + 1] - k0)
            continue;
        const size_t stride = static_cast<size_t>(a.num_kv_heads) * C::DSPLIT * 2 * kOwn * C::DKV;
        const float *src =
            a.part +
            ((((static_cast<size_t>(a.part_start[b]) + t * chunks) * a.num_kv_heads + head) * C::DSPLIT + dh) *
                 2 * kOwn + (is_dk ? kOwn : 0) + row) * C::DKV + col % C::DKV;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int c = 0; c < chunks; ++c) {
            const float4 p = __ldcs(reinterpret_cast<const float4 *>(src + c * stride));
            s.x += p.x;
            s.y += p.y;
            s.z += p.z;
            s.w += p.w;
        }
        const float f = is_dk ? a.scale : 1.f;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_dk ? a.dk : a.dv) +
                             (static_cast<size_t>(k0 + key) * a.num_kv_heads + head) * D + col;
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16x2(s.x * f, s.y * f), pack_bf16x2(s.z * f, s.w * f));
    }
}

template <int D, bool SINK>
cudaError_t launch_bwd_d(const BwdArgs &a, int key_tile_bound, int q_tile_bound, int sm_count,
                         cudaStream_t s)
{
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && !attr_done[dev]) {
        if ((e = cudaFuncSetAttribute(bwd_main_kernel<D, false, SINK>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(BwdCfg<D, false>::SMEM))) != cudaSuccess ||
            (e = cudaFuncSetAttribute(bwd_main_kernel<D, true, SINK>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(BwdCfg<D, true>::SMEM))) != cudaSuccess)
            return e;
        attr_done[dev] = 1;
    }
    bwd_prep_kernel<BwdCfg<D, false>::STEP, BwdCfg<D, false>::DSPLIT, SINK>
        <<<1, kPrepThreads, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    if ((e = launch_dependent(SINK ? bwd_delta_wide_kernel<D> : bwd_delta_kernel<D>, dim3(sm_count * 8), 256, 0,
                              s, a)) != cudaSuccess)
        return e;
    // persistent grids: one CTA per SM (fewer when there are fewer units)
    const long long kv_units =
        static_cast<long long>(key_tile_bound) * BwdCfg<D, false>::DSPLIT * a.num_kv_heads;
    const long long q_units = static_cast<long long>(q_tile_bound) * a.num_heads;
    if (kv_units > 0) {
        const int grid = SINK ? sm_count : static_cast<int>(std::min<long long>(kv_units, sm_count));
        if ((e = launch_dependent(bwd_main_kernel<D, false, SINK>, dim3(grid), kThreads,
                                  BwdCfg<D, false>::SMEM, s, a)) != cudaSuccess)
            return e;
    }
    if (q_units > 0) {
        // Programmatic dependent launch: the dQ kernel's CTAs start on the SMs
        // the dK/dV kernel's CTAs leave, without waiting for the whole grid.  It
        // reads only the prep and Delta kernels' output, complete before any
        // dK/dV CTA let it start, so it waits (griddepcontrol.wait) only at its
        // end; its atomic unit counter balances CTAs that start late.
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(q_units, sm_count)));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = BwdCfg<D, true>::SMEM;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = kv_units > 0 ? 1 : 0;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, bwd_main_kernel<D, true, SINK>, a)) != cudaSuccess)
            return e;
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
    }
    if (SINK && kv_units > 0 && q_units > 0) {
        // behind the dQ kernel, which waits for the dK/dV kernel
        if ((e = launch_dependent(bwd_sinks_kernel<D>, dim3(4 * sm_count), 2 * kSinkRows * D / 4, 0, s, a)) !=
            cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// Most partials of chunks: a tile is cut where it has over `per` steps, which
// gives less than twice its steps over `per`; all tiles' steps over `per` are at
// most kSinkUnits, and `per` is at least kSinkMinSteps.
size_t sink_parts(int batch, int total_q, int num_heads, int head_dim, int sink_tokens)
{
    const long long split = head_dim == 256 ? 2 : 1;
    const long long tiles = (static_cast<long long>(sink_tokens) + kOwn - 1) / kOwn;
    const long long blocks = total_q / bwd_kv_step_rows(head_dim) + static_cast<long long>(batch);
    // a double, since the product may pass 64 bits
    const double steps = static_cast<double>(split * num_heads) * tiles * blocks;
    return 2 * static_cast<size_t>(std::min<double>(kSinkUnits, steps / kSinkMinSteps + 1));
}

}  // namespace

size_t bwd_workspace_bytes(int batch, int total_q, int num_heads, int head_dim)
{
    (void)head_dim;
    size_t n = 256;                                                   // status word
    n += (static_cast<size_t>(batch) + 1) * sizeof(int32_t);          // key tile starts
    n = (n + 255) & ~static_cast<size_t>(255);
    n += (static_cast<size_t>(batch) + 1) * sizeof(int32_t);          // q tile starts
    n = (n + 255) & ~static_cast<size_t>(255);
    n += static_cast<size_t>(total_q) * num_heads * sizeof(float);    // Delta
    return (n + 255) & ~static_cast<size_t>(255);
}

void bwd_workspace_split(void *ws, int batch, int total_q, int num_heads, BwdArgs *a)
{
    (void)total_q;
    (void)num_heads;
    uint8_t *p = static_cast<uint8_t *>(ws);
    a->status = reinterpret_cast<int32_t *>(p);
    size_t n = 256;
    a->ktile_start = reinterpret_cast<int32_t *>(p + n);
    n += (static_cast<size_t>(batch) + 1) * sizeof(int32_t);
    n = (n + 255) & ~static_cast<size_t>(255);
    a->qtile_start = reinterpret_cast<int32_t *>(p + n);
    n += (static_cast<size_t>(batch) + 1) * sizeof(int32_t);
    n = (n + 255) & ~static_cast<size_t>(255);
    a->delta = reinterpret_cast<float *>(p + n);
}

size_t bwd_sinks_workspace_bytes(int batch, int total_q, int num_heads, int head_dim,
                                 int sink_tokens)
{
    const size_t lists = (4 * (static_cast<size_t>(batch) + 1) * sizeof(int32_t) + 255) &
                         ~static_cast<size_t>(255);
    const size_t part = 2 * static_cast<size_t>(kOwn) * (head_dim == 256 ? 128 : head_dim) * sizeof(float);
    return bwd_workspace_bytes(batch, total_q, num_heads, head_dim) + lists +
           sink_parts(batch, total_q, num_heads, head_dim, sink_tokens) * part;
}

void bwd_sinks_workspace_split(void *ws, int batch, int total_q, int num_heads, BwdArgs *a)
{
    bwd_workspace_split(ws, batch, total_q, num_heads, a);
    const size_t n = static_cast<size_t>(batch) + 1;
    int32_t *p = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) +
                                             bwd_workspace_bytes(batch, total_q, num_heads, 0));
    a->sink_start = p;
    a->sink_chunks = p + n;
    a->part_start = p + 2 * n;
    a->cut_start = p + 3 * n;
    a->part = reinterpret_cast<float *>(p) + ((4 * n + 63) & ~static_cast<size_t>(63));
}

cudaError_t launch_bwd(int head_dim, const BwdArgs &a, int key_tile_bound, int q_tile_bound,
                       int sm_count, cudaStream_t stream)
{
    const bool sinks = a.window_left >= 0 && a.sink_tokens > 0;
    auto run = [&](auto with, auto without) {
        return (sinks ? with : without)(a, key_tile_bound, q_tile_bound, sm_count, stream);
    };
    switch (head_dim) {
    case 64: return run(launch_bwd_d<64, true>, launch_bwd_d<64, false>);
    case 128: return run(launch_bwd_d<128, true>, launch_bwd_d<128, false>);
    case 256: return run(launch_bwd_d<256, true>, launch_bwd_d<256, false>);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
