// tiles.cuh -- what the kernels that keep a 128-row tile and stream others past it
// share: prefix sums over sequences, the tile loads and the score products.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace vfa {

constexpr int kOwn = 128;          // rows of a CTA's own tile (keys, resp. queries)
constexpr int kPrepThreads = 1024;

// Exclusive prefix sum over blockDim.x-wide chunks of per-sequence counts;
// out[b] = sum of count(b') for b' < b, out[B] = the total.
template <typename CountFn>
__device__ void block_prefix(int B, int32_t *out, int *warp_sums, CountFn count)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int base = 0; base < B; base += kPrepThreads) {
        const int b = base + tid;
        const int nt = b < B ? count(b) : 0;
        int x = nt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            warp_sums[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int w = warp_sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o)
                    w += y;
            }
            warp_sums[lane] = w;
        }
        __syncthreads();
        const int excl = x - nt + (warp > 0 ? warp_sums[warp - 1] : 0);
        if (b < B)
            out[b] = carry + excl;
        carry += warp_sums[31];
        __syncthreads();
    }
    if (tid == 0)
        out[B] = carry;
}

// Largest b with start[b] <= gt (start is a non-decreasing prefix sum).
__device__ __forceinline__ int owner_of(const int32_t *start, int B, int gt)
{
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= gt)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The visible part of (at most 32) consecutive columns, [lo, hi) (empty when hi <= lo),
// clamped to [-1, 33] so it fits an int.
__device__ __forceinline__ int clamp_col(long long x)
{
    return static_cast<int>(x < -1 ? -1 : (x > 33 ? 33 : x));
}

// Key j's visible queries among i_base, i_base + 1, ... (the columns
// of a key tile's scores): i < Lq, and i >= j - off (causal), i <= j - off + window_left.
__device__ __forceinline__ void key_row_span(long long j, long long i_base, int lk, int lq,
                                             int causal, int wl, long long off, int *lo, int *hi)
{
    long long l = causal ? j - off - i_base : 0;
    long long h = lq - i_base;
    if (wl >= 0)
        h = min(h, j - off + wl - i_base + 1);
    if (j >= lk)
        h = l;
    *lo = clamp_col(l);
    *hi = clamp_col(h);
}

// The columns below x, one bit each.
__device__ __forceinline__ uint32_t below(int x)
{
    const int n = min(32, max(0, x));
    return n == 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Scores of hidden columns (bits of `see` that are 0) become -inf: their p is 0.  Where a
// warp sees all of a chunk nothing is done; the rest of a step is the same code
// for masked and unmasked ones, which a short range of steps would fetch anew.
__device__ __forceinline__ void hide(uint32_t (&sr)[32], uint32_t see)
{
    if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            sr[e] = see >> e & 1u ? sr[e] : __float_as_uint(-INFINITY);
    }
}

// Loads a tile of `rows` rows (a multiple of the map's box height BOX) of
// every 64-column block of row `row0`, head `head` into a 128-byte-swizzled
// buffer holding `rows` rows per column block.
template <int DB, int BOX>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                          int head, int row0, int rows)
{
    for (int db = 0; db < DB; ++db)
        for (int r = 0; r < rows; r += BOX)
            tma_load_3d(dst + db * (rows * 128) + r * 128, map, bar, db * 64, head, row0 + r);
}

// S (or S^T) = A B^T over K = D for A a 128-row operand and B a STEP-row
// operand, both K-major in 128-byte-swizzled column blocks.
template <int D, int STEP>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint32_t a_buf, uint32_t b_buf,
                                             uint32_t idesc)
{
    const uint64_t a0 = sdesc_sw128(a_buf, 16, 1024), b0 = sdesc_sw128(b_buf, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t ao = ((kk >> 2) * (kOwn * 128) + (kk & 3) * 32) >> 4;
        const uint64_t bo = ((kk >> 2) * (STEP * 128) + (kk & 3) * 32) >> 4;
        if (kk == 0)
            mma_ss_w<0>(d_tmem, a0 + ao, b0 + bo, idesc);
        else
            mma_ss_w<1>(d_tmem, a0 + ao, b0 + bo, idesc);
    }
}

}  // namespace vfa
