// rope.cu -- RMS norm of each query and key head and the rotation of its
// position in one pass, forward and backward.
//
// Per (token, head) vector x of D elements, weight w, pair (a, b) of
// dimensions with frequency i (halves: (i, i + R/2); interleaved:
// (2i, 2i + 1)) and angle phi_i = inv_freq_i * position[axis_i]:
//   r = (mean(x^2) + eps)^-1/2,  n = x r w
//   y_a = n_a cos(phi) - n_b sin(phi),  y_b = n_b cos(phi) + n_a sin(phi)
// and for the gradient, g = the rotation of dy by -phi:
//   dw = sum over tokens and heads of g x r,
//   dx = r (u - x r^2 mean(u x)),  u = g w.
//
// Angles are fixed point: the table holds inv_freq / (2 pi) in units of
// 2^-64 of a turn, and position * step modulo 2^64 is the angle's fraction of
// a turn with no rounding, so position 2^30 is as accurate as position 1 (a
// 32-bit product would have lost the angle near position 2^20).
//
// Bound: HBM.  Forward 4 bytes per element, backward 6, about 10 and 20
// flops.  A lane holds 8 dimensions of a head as two 8-byte pieces that
// contain both members of its four pairs, so D/8 lanes hold a head and the
// only exchange is the sum of the norm.  (16 dimensions per lane halve the
// load instructions but double the weights, sines and sums of dw a lane keeps:
// 150 registers and 8 warps per SM in the backward, 265 us where this takes
// 202.)  A warp takes one token (or, when there are few, a share of its
// heads) and works out the token's sines and cosines once for all its heads.
#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vfa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFwdUnroll = 4;           // head iterations whose loads are in flight together
constexpr int kBwdUnroll = 2;
constexpr int kBwdCtas = 3;             // resident per SM

__device__ __forceinline__ void unpack4(const uint2 v, float *f)
{
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ uint2 pack4(const float *f)
{
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// The 8 dimensions of lane piece p of a head: [a, a + 4) and [b, b + 4).
template <bool INTER>
__device__ __forceinline__ void lane_dims(int p, int half, int *a, int *b)
{
    if (!INTER && 4 * p < half) {
        *a = 4 * p;
        *b = half + 4 * p;
    } else {
        *a = 8 * p;                     // interleaved pairs, or dimensions past the rotated ones
        *b = 8 * p + 4;
    }
}

// x[0..3] = dims [a, a+4), x[4..7] = dims [b, b+4); pair j is (x[j], x[4+j])
// for halves and (x[2j], x[2j+1]) for interleaved pairs.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[4], const float (&s)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : 4 + j;
        const float xa = x[ia], xb = x[ib];
        x[ia] = xa * c[j] - xb * s[j];
        x[ib] = xb * c[j] + xa * s[j];
    }
}

// Cosines and sines of token t for frequencies 4p .. 4p + 3 (1 and 0 past the
// rotated ones).  The warp's lane groups (one per head it holds) work out a
// share each and exchange.
template <int D>
__device__ __forceinline__ void angles(const RopeArgs &a, int t, int lane, float (&c)[4],
                                       float (&s)[4])
{
    constexpr int LPH = D / 8, GROUPS = 32 / LPH, PER = 4 / GROUPS;
    const int p = lane % LPH, g = lane / LPH;
    float mc[PER], ms[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = 4 * p + g * PER + e;
        mc[e] = 1.f;
        ms[e] = 0.f;
        if (i < a.half) {
            const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2 *>(a.table) + i);
            // an axis outside the positions' reads the last one
            const unsigned long long ax = f.y < static_cast<unsigned long long>(a.num_axes)
                                              ? f.y
                                              : static_cast<unsigned long long>(a.num_axes - 1);
            const long long pos = __ldg(a.positions + ax * a.tokens + t);
            const unsigned long long turn = static_cast<unsigned long long>(pos) * f.x;
            const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
            sincospif(x, &ms[e], &mc[e]);       // x in [-1, 1): half turns
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int src = (j / PER) * LPH + p;
        c[j] = __shfl_sync(0xffffffffu, mc[j % PER], src);
        s[j] = __shfl_sync(0xffffffffu, ms[j % PER], src);
    }
}

template <int D>
__device__ __forceinline__ float head_sum(float v)
{
#pragma unroll
    for (int off = 1; off < D / 8; off <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ void load_weight(const float *w, int da, int db, float (&o)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o[j] = w ? __ldg(w + da + j) : 1.f;
        o[4 + j] = w ? __ldg(w + db + j) : 1.f;
    }
}

__device__ __forceinline__ uint2 load_piece(const __nv_bfloat16 *p)
{
    return __ldcs(reinterpret_cast<const uint2 *>(p));
}

__device__ __forceinline__ void store_piece(__nv_bfloat16 *p, const float *f)
{
    *reinterpret_cast<uint2 *>(p) = pack4(f);
}

// A unit of work: head iterations [i0, i1) of token t, the query heads first.
struct Unit {
    int t, i0, i1;

    __device__ __forceinline__ Unit(const RopeArgs &a, long long u, int iters)
    {
        const int per = (iters + a.segments - 1) / a.segments;
        t = static_cast<int>(u / a.segments);
        i0 = static_cast<int>(u % a.segments) * per;
        i1 = min(iters, i0 + per);
    }
};

// ------------------------------------------------------------ forward

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rope_fwd_kernel(const RopeArgs a)
{
    constexpr int LPH = D / 8, HPW = 32 / LPH, U = kFwdUnroll;
    grid_wait();
    const int lane = threadIdx.x & 31;
    const int p = lane % LPH, g = lane / LPH;
    int da, db;
    lane_dims<INTER>(p, a.half, &da, &db);
    const bool turns = 4 * p < a.half;
    const int iq = (a.heads[0] + HPW - 1) / HPW, ik = (a.heads[1] + HPW - 1) / HPW;
    const long long units = static_cast<long long>(a.tokens) * a.segments;
    const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += nwarps) {
        const Unit un(a, u, iq + ik);
        float c[4], s[4];
        bool have_angles = false;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int base = which ? iq : 0;
            const int e0 = max(un.i0 - base, 0), e1 = min(un.i1 - base, which ? ik : iq);
            const int H = a.heads[which];
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.x[which]) +
                                       un.t * a.x_stride[which];
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.y[which]) + un.t * a.y_stride[which];
            const bool norm = a.weight[which] != nullptr;
            float w[8];
            if (e0 < e1)
                load_weight(a.weight[which], da, db, w);
            for (int e = e0; e < e1; e += U) {
                uint2 ra[U], rb[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = (e + k) * HPW + g;
                    ra[k] = rb[k] = make_uint2(0, 0);
                    if (e + k < e1 && h < H) {
                        ra[k] = load_piece(src + h * D + da);
                        rb[k] = load_piece(src + h * D + db);
                    }
                }
                if (!have_angles) {                 // behind the first loads
                    angles<D>(a, un.t, lane, c, s);
                    have_angles = true;
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = (e + k) * HPW + g;
                    float x[8];
                    unpack4(ra[k], x);
                    unpack4(rb[k], x + 4);
                    if (norm) {
                        float q = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            q = fmaf(x[j], x[j], q);
                        const float r = rsqrtf(head_sum<D>(q) * (1.f / D) + a.eps);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = x[j] * r * w[j];
                    }
                    if (turns)
                        rotate<INTER>(x, c, s);
                    if (e + k < e1 && h < H) {
                        store_piece(dst + h * D + da, x);
                        store_piece(dst + h * D + db, x + 4);
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------ backward
//
// A persistent grid whose warps take fixed units, so the sums of dw run in a
// fixed order: per lane over its units, then over the warp's lane groups, the
// CTA's warps, and (second kernel) the CTAs.  No atomics.

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdCtas) rope_bwd_kernel(const RopeArgs a)
{
    constexpr int LPH = D / 8, HPW = 32 / LPH, U = kBwdUnroll;
    __shared__ float s_dw[kWarps][D];
    grid_wait();
    if (a.dweight[0] || a.dweight[1])
        grid_release();                             // the sums of dw follow
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = lane % LPH, g = lane / LPH;
    int da, db;
    lane_dims<INTER>(p, a.half, &da, &db);
    const bool turns = 4 * p < a.half;
    const int iq = (a.heads[0] + HPW - 1) / HPW, ik = (a.heads[1] + HPW - 1) / HPW;
    float dw[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        dw[0][j] = dw[1][j] = 0.f;
    const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
    const long long units = static_cast<long long>(a.tokens) * a.segments;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + warp; u < units; u += nwarps) {
        const Unit un(a, u, iq + ik);
        float c[4], s[4];
        bool have_angles = false;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int base = which ? iq : 0;
            const int e0 = max(un.i0 - base, 0), e1 = min(un.i1 - base, which ? ik : iq);
            const int H = a.heads[which];
            const bool norm = a.weight[which] != nullptr;
            const __nv_bfloat16 *px = static_cast<const __nv_bfloat16 *>(a.x[which]) +
                                      un.t * a.x_stride[which];
            const __nv_bfloat16 *pdy = static_cast<const __nv_bfloat16 *>(a.dy[which]) +
                                       un.t * a.dy_stride[which];
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.y[which]) + un.t * a.y_stride[which];
            float w[8];
            if (e0 < e1)
                load_weight(a.weight[which], da, db, w);
#pragma unroll 1
            for (int e = e0; e < e1; e += U) {
                uint2 xa[U], xb[U], ya[U], yb[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = (e + k) * HPW + g;
                    xa[k] = xb[k] = ya[k] = yb[k] = make_uint2(0, 0);
                    if (e + k < e1 && h < H) {
                        ya[k] = load_piece(pdy + h * D + da);
                        yb[k] = load_piece(pdy + h * D + db);
                        if (norm) {
                            xa[k] = load_piece(px + h * D + da);
                            xb[k] = load_piece(px + h * D + db);
                        }
                    }
                }
                if (!have_angles) {                 // behind the first loads
                    angles<D>(a, un.t, lane, c, s);
                    have_angles = true;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[j] = -s[j];
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int h = (e + k) * HPW + g;
                    float y[8];
                    unpack4(ya[k], y);
                    unpack4(yb[k], y + 4);
                    if (turns)
                        rotate<INTER>(y, c, s);
                    if (norm) {
                        float x[8];
                        unpack4(xa[k], x);
                        unpack4(xb[k], x + 4);
                        float q = 0.f, d = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            q = fmaf(x[j], x[j], q);
                            d = fmaf(y[j] * w[j], x[j], d);
                        }
                        const float r = rsqrtf(head_sum<D>(q) * (1.f / D) + a.eps);
                        const float m = head_sum<D>(d) * (1.f / D) * r * r;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            dw[which][j] = fmaf(y[j] * r, x[j], dw[which][j]);
                            y[j] = r * (y[j] * w[j] - x[j] * m);
                        }
                    }
                    if (e + k < e1 && h < H) {
                        store_piece(dst + h * D + da, y);
                        store_piece(dst + h * D + db, y + 4);
                    }
                }
            }
        }
    }
    // partial[cta][which][d]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!a.dweight[which])
            continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int off = LPH; off < 32; off <<= 1)
                dw[which][j] += __shfl_xor_sync(0xffffffffu, dw[which][j], off);
        }
        __syncthreads();                            // s_dw's readers of the queries' turn
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s_dw[warp][da + j] = dw[which][j];
                s_dw[warp][db + j] = dw[which][4 + j];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                v += s_dw[k][d];
            a.partial[(static_cast<long long>(blockIdx.x) * 2 + which) * D + d] = v;
        }
    }
}

// dw[which][d] = the sum of the CTAs' partial sums: 32 slices of the CTAs per
// column, then the slices.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const RopeArgs a, const int D)
{
    __shared__ float s[32][33];
    grid_wait();
    const int which = blockIdx.y;
    const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
    if (!a.dweight[which])
        return;
    float v = 0.f;
#pragma unroll 8
    for (int i = slice; i < a.ctas; i += 32)
        v += a.partial[(static_cast<long long>(i) * 2 + which) * D + blockIdx.x * 32 + col];
    s[slice][col] = v;
    __syncthreads();
    v = s[col][slice];                              // column `slice`, slice `col`
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    if (col == 0)
        a.dweight[which][blockIdx.x * 32 + slice] = v;
}

// One warp per token keeps a token's sines to one warp; with fewer tokens than
// warps that fill the GPU, a token's heads are spread over several.
int head_segments(const RopeArgs &a, int iters, int sm_count)
{
    const long long want = static_cast<long long>(sm_count) * 32;
    const long long seg = (want + a.tokens - 1) / a.tokens;
    return static_cast<int>(seg < 1 ? 1 : (seg > iters ? iters : seg));
}

template <int D>
cudaError_t launch_fwd_d(RopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int HPW = 32 / (D / 8);
    a.segments = head_segments(a, (a.heads[0] + HPW - 1) / HPW + (a.heads[1] + HPW - 1) / HPW,
                               sm_count);
    const long long units = static_cast<long long>(a.tokens) * a.segments;
    long long grid = (units + kWarps - 1) / kWarps;
    if (grid > (1 << 20))
        grid = 1 << 20;
    const auto kernel = a.interleaved ? rope_fwd_kernel<D, true> : rope_fwd_kernel<D, false>;
    return launch_dependent(kernel, dim3(static_cast<int>(grid)), kThreads, 0, stream, a);
}

template <int D>
cudaError_t launch_bwd_d(RopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int HPW = 32 / (D / 8);
    a.segments = head_segments(a, (a.heads[0] + HPW - 1) / HPW + (a.heads[1] + HPW - 1) / HPW,
                               sm_count);
    const long long need = (static_cast<long long>(a.tokens) * a.segments + kWarps - 1) / kWarps;
    long long grid = static_cast<long long>(sm_count) * kBwdCtas;
    grid = grid < need ? grid : need;
    grid = grid < kRopeMaxCtas ? grid : kRopeMaxCtas;
    a.ctas = static_cast<int>(grid);
    const auto kernel = a.interleaved ? rope_bwd_kernel<D, true> : rope_bwd_kernel<D, false>;
    const cudaError_t e = launch_dependent(kernel, dim3(a.ctas), kThreads, 0, stream, a);
    if (e != cudaSuccess || (!a.dweight[0] && !a.dweight[1]))
        return e;
    return launch_dependent(rope_dw_kernel, dim3(D / 32, 2), 1024, 0, stream, a, D);
}

}  // namespace

cudaError_t launch_rope_fwd(int head_dim, RopeArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.tokens == 0)
        return cudaSuccess;
    switch (head_dim) {
    case 64: return launch_fwd_d<64>(a, sm_count, stream);
    case 128: return launch_fwd_d<128>(a, sm_count, stream);
    case 256: return launch_fwd_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_rope_bwd(int head_dim, RopeArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.tokens == 0) {                    // no rows: dw is a sum over no CTAs
        if (a.dweight[0] || a.dweight[1])
            return launch_dependent(rope_dw_kernel, dim3(head_dim / 32, 2), 1024, 0, stream,
                                    a, head_dim);
        return cudaSuccess;
    }
    switch (head_dim) {
    case 64: return launch_bwd_d<64>(a, sm_count, stream);
    case 128: return launch_bwd_d<128>(a, sm_count, stream);
    case 256: return launch_bwd_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
