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
// flops.  A lane holds 16 dimensions of a head as two 16-byte pieces that
// contain both members of its eight pairs, so D/16 lanes hold a head and the
// only exchange is the sum of the norm.  A warp takes one token (or, when
// there are few, a share of its heads) and works out the token's eight
// sines and cosines per lane once for all its heads.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace vfa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;              // head iterations whose loads are in flight together

__device__ __forceinline__ void unpack8(const uint4 v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// The 16 dimensions of lane piece p of a head: [a, a + 8) and [b, b + 8).
template <bool INTER>
__device__ __forceinline__ void lane_dims(int p, int half, int *a, int *b)
{
    if (!INTER && 8 * p < half) {
        *a = 8 * p;
        *b = half + 8 * p;
    } else {
        *a = 16 * p;                    // interleaved pairs, or dimensions past the rotated ones
        *b = 16 * p + 8;
    }
}

// x[0..7] = dims [a, a+8), x[8..15] = dims [b, b+8); pair j is (x[j], x[8+j])
// for halves and (x[2j], x[2j+1]) for interleaved pairs.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : 8 + j;
        const float xa = x[ia], xb = x[ib];
        x[ia] = xa * c[j] - xb * s[j];
        x[ib] = xb * c[j] + xa * s[j];
    }
}

// Cosines and sines of token t for frequencies 8p .. 8p + 7 (1 and 0 past the
// rotated ones).  The warp's lane groups (one per head it holds) work out a
// share each and exchange.
template <int D>
__device__ __forceinline__ void angles(const RopeArgs &a, int t, int lane, float (&c)[8],
                                       float (&s)[8])
{
    constexpr int LPH = D / 16, GROUPS = 32 / LPH, PER = GROUPS >= 8 ? 1 : 8 / GROUPS;
    const int p = lane % LPH, g = (lane / LPH) % (8 / PER);
    float mc[PER], ms[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = 8 * p + g * PER + e;
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
    for (int j = 0; j < 8; ++j) {
        const int src = (j / PER) * LPH + p;
        c[j] = __shfl_sync(0xffffffffu, mc[j % PER], src);
        s[j] = __shfl_sync(0xffffffffu, ms[j % PER], src);
    }
}

template <int D>
__device__ __forceinline__ float head_sum(float v)
{
#pragma unroll
    for (int off = 1; off < D / 16; off <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ void load_weight(const float *w, int da, int db, float (&o)[16])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        o[j] = w ? __ldg(w + da + j) : 1.f;
        o[8 + j] = w ? __ldg(w + db + j) : 1.f;
    }
}

// ------------------------------------------------------------ forward

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a)
{
    constexpr int LPH = D / 16, HPW = 32 / LPH;
    const int lane = threadIdx.x & 31;
    const int p = lane % LPH, g = lane / LPH;
    int da, db;
    lane_dims<INTER>(p, a.half, &da, &db);
    const int iq = (a.heads[0] + HPW - 1) / HPW, ik = (a.heads[1] + HPW - 1) / HPW;
    const int per = (iq + ik + a.segments - 1) / a.segments;
    const long long units = static_cast<long long>(a.tokens) * a.segments;
    const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += nwarps) {
        const int t = static_cast<int>(u / a.segments), seg = static_cast<int>(u % a.segments);
        const int i0 = seg * per, i1 = min(iq + ik, i0 + per);
        float c[8], s[8];
        angles<D>(a, t, lane, c, s);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int base = which ? iq : 0;
            const int e0 = max(i0 - base, 0), e1 = min(i1 - base, which ? ik : iq);
            if (e0 >= e1)
                continue;
            const int H = a.heads[which];
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.x[which]) +
                                       t * a.x_stride[which];
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.y[which]) + t * a.y_stride[which];
            const bool norm = a.weight[which] != nullptr;
            float w[16];
            load_weight(a.weight[which], da, db, w);
            for (int e = e0; e < e1; e += kUnroll) {
                uint4 ra[kUnroll], rb[kUnroll];
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const int h = (e + k) * HPW + g;
                    if (e + k < e1 && h < H) {
                        ra[k] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D + da));
                        rb[k] = __ldcs(reinterpret_cast<const uint4 *>(src + h * D + db));
                    } else {
                        ra[k] = rb[k] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const int h = (e + k) * HPW + g;
                    float x[16];
                    unpack8(ra[k], x);
                    unpack8(rb[k], x + 8);
                    if (norm) {
                        float q = 0.f;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            q = fmaf(x[j], x[j], q);
                        const float r = rsqrtf(head_sum<D>(q) * (1.f / D) + a.eps);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            x[j] = x[j] * r * w[j];
                    }
                    if (8 * p < a.half)
                        rotate<INTER>(x, c, s);
                    if (e + k < e1 && h < H) {
                        *reinterpret_cast<uint4 *>(dst + h * D + da) = pack8(x);
                        *reinterpret_cast<uint4 *>(dst + h * D + db) = pack8(x + 8);
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------ backward
//
// CTAs [0, ctas[0]) take the queries, the next ctas[1] the keys, each a fixed
// share of (token, head iteration) units, so the sums of dw run in a fixed
// order: per lane over its units, then over the warp's lane groups, the CTA's
// warps, and (second kernel) the CTAs.  No atomics.

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs a)
{
    constexpr int LPH = D / 16, HPW = 32 / LPH;
    __shared__ float s_dw[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = lane % LPH, g = lane / LPH;
    const int which = static_cast<int>(blockIdx.x) >= a.ctas[0];
    const int cta = blockIdx.x - (which ? a.ctas[0] : 0);
    const int H = a.heads[which];
    const int iters = (H + HPW - 1) / HPW;
    const bool norm = a.weight[which] != nullptr;
    int da, db;
    lane_dims<INTER>(p, a.half, &da, &db);
    float w[16], dw[16];
    load_weight(a.weight[which], da, db, w);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        dw[j] = 0.f;
    const long long nwarps = static_cast<long long>(a.ctas[which]) * kWarps;
    const int per = (iters + a.segments - 1) / a.segments;
    const long long units = static_cast<long long>(a.tokens) * a.segments;
    for (long long u = static_cast<long long>(cta) * kWarps + warp; u < units; u += nwarps) {
        const int t = static_cast<int>(u / a.segments), seg = static_cast<int>(u % a.segments);
        const int e0 = seg * per, e1 = min(iters, e0 + per);
        float c[8], s[8];
        angles<D>(a, t, lane, c, s);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = -s[j];
        const __nv_bfloat16 *px = static_cast<const __nv_bfloat16 *>(a.x[which]) +
                                  t * a.x_stride[which];
        const __nv_bfloat16 *pdy = static_cast<const __nv_bfloat16 *>(a.dy[which]) +
                                   t * a.dy_stride[which];
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.y[which]) + t * a.y_stride[which];
        for (int e = e0; e < e1; e += kUnroll) {
            uint4 xa[kUnroll], xb[kUnroll], ya[kUnroll], yb[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int h = (e + k) * HPW + g;
                xa[k] = xb[k] = ya[k] = yb[k] = make_uint4(0, 0, 0, 0);
                if (e + k < e1 && h < H) {
                    ya[k] = __ldcs(reinterpret_cast<const uint4 *>(pdy + h * D + da));
                    yb[k] = __ldcs(reinterpret_cast<const uint4 *>(pdy + h * D + db));
                    if (norm) {
                        xa[k] = __ldcs(reinterpret_cast<const uint4 *>(px + h * D + da));
                        xb[k] = __ldcs(reinterpret_cast<const uint4 *>(px + h * D + db));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int h = (e + k) * HPW + g;
                float y[16];
                unpack8(ya[k], y);
                unpack8(yb[k], y + 8);
                if (8 * p < a.half)
                    rotate<INTER>(y, c, s);
                if (norm) {
                    float x[16];
                    unpack8(xa[k], x);
                    unpack8(xb[k], x + 8);
                    float q = 0.f, d = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        q = fmaf(x[j], x[j], q);
                        d = fmaf(y[j] * w[j], x[j], d);
                    }
                    const float r = rsqrtf(head_sum<D>(q) * (1.f / D) + a.eps);
                    const float m = head_sum<D>(d) * (1.f / D) * r * r;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        dw[j] = fmaf(y[j] * r, x[j], dw[j]);
                        y[j] = r * (y[j] * w[j] - x[j] * m);
                    }
                }
                if (e + k < e1 && h < H) {
                    *reinterpret_cast<uint4 *>(dst + h * D + da) = pack8(y);
                    *reinterpret_cast<uint4 *>(dst + h * D + db) = pack8(y + 8);
                }
            }
        }
    }
    if (!norm)
        return;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
#pragma unroll
        for (int off = LPH; off < 32; off <<= 1)
            dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], off);
    }
    if (g == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s_dw[warp][da + j] = dw[j];
            s_dw[warp][db + j] = dw[8 + j];
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            v += s_dw[k][d];
        a.partial[static_cast<long long>(blockIdx.x) * D + d] = v;
    }
}

// dw[which][d] = sum of its CTAs' partial sums: eight slices of the CTAs per
// column, then the slices.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const RopeArgs a, const int D)
{
    constexpr int SLICES = 8, COLS = 1024 / SLICES;
    __shared__ float s[SLICES][COLS];
    const int which = blockIdx.y;
    const int d = blockIdx.x * COLS + threadIdx.x % COLS, slice = threadIdx.x / COLS;
    if (!a.dweight[which])
        return;
    const int c0 = which ? a.ctas[0] : 0, n = a.ctas[which];
    float v = 0.f;
    if (d < D)
        for (int i = slice; i < n; i += SLICES)
            v += a.partial[static_cast<long long>(c0 + i) * D + d];
    s[slice][threadIdx.x % COLS] = v;
    __syncthreads();
    if (slice == 0 && d < D) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < SLICES; ++i)
            v += s[i][threadIdx.x];
        a.dweight[which][d] = v;
    }
}

template <int D>
cudaError_t launch_fwd_d(RopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int HPW = 32 / (D / 16);
    const int iters = (a.heads[0] + HPW - 1) / HPW + (a.heads[1] + HPW - 1) / HPW;
    // One warp per token keeps the sines of a token to one warp; with fewer
    // tokens than warps that fill the GPU, a token's heads are spread out.
    const long long want = static_cast<long long>(sm_count) * 32;
    long long seg = (want + a.tokens - 1) / a.tokens;
    seg = seg < 1 ? 1 : (seg > iters ? iters : seg);
    a.segments = static_cast<int>(seg);
    const long long units = a.tokens * seg;
    long long grid = (units + kWarps - 1) / kWarps;
    if (grid > (1 << 20))
        grid = 1 << 20;
    if (a.interleaved)
        rope_fwd_kernel<D, true><<<static_cast<int>(grid), kThreads, 0, stream>>>(a);
    else
        rope_fwd_kernel<D, false><<<static_cast<int>(grid), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd_d(RopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int HPW = 32 / (D / 16);
    const int iq = (a.heads[0] + HPW - 1) / HPW, ik = (a.heads[1] + HPW - 1) / HPW;
    const int iters = iq > ik ? iq : ik;
    const long long want = static_cast<long long>(sm_count) * 32;
    long long seg = (want + a.tokens - 1) / a.tokens;
    seg = seg < 1 ? 1 : (seg > iters ? iters : seg);
    a.segments = static_cast<int>(seg);
    // CTAs in proportion to the two tensors' work, at most kRopeMaxCtas in all
    long long total = sm_count * 4;
    const long long need = (a.tokens * seg * 2 + kWarps - 1) / kWarps;
    total = total < need ? total : need;
    total = total > kRopeMaxCtas ? kRopeMaxCtas : (total < 2 ? 2 : total);
    long long cq = (total * iq + (iq + ik) / 2) / (iq + ik);
    cq = cq < 1 ? 1 : (cq > total - 1 ? total - 1 : cq);
    a.ctas[0] = static_cast<int>(cq);
    a.ctas[1] = static_cast<int>(total - cq);
    if (a.interleaved)
        rope_bwd_kernel<D, true><<<static_cast<int>(total), kThreads, 0, stream>>>(a);
    else
        rope_bwd_kernel<D, false><<<static_cast<int>(total), kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dweight[0] && !a.dweight[1]))
        return e;
    rope_dw_kernel<<<dim3((D + 127) / 128, 2), 1024, 0, stream>>>(a, D);
    return cudaGetLastError();
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
            rope_dw_kernel<<<dim3((head_dim + 127) / 128, 2), 1024, 0, stream>>>(a, head_dim);
        return cudaGetLastError();
    }
    switch (head_dim) {
    case 64: return launch_bwd_d<64>(a, sm_count, stream);
    case 128: return launch_bwd_d<128>(a, sm_count, stream);
    case 256: return launch_bwd_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
