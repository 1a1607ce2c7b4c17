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
// Bound: HBM (forward 4 bytes per element, backward 6), with the issue of
// instructions next: at the copy rate an SM has 350 issue slots per KB read
// forward.  A warp's turn is 1 KB of a tensor: 32 / (D/16) heads, 16
// dimensions per lane in two 16-byte pieces that contain both members of the
// lane's eight pairs, so the only exchange is the sum of the norm.  A warp
// takes one token after the other (or, when there are few, a share of a
// token's heads) and works out a token's sines and cosines once for all its
// heads.  Its turns are copied ahead into its own ring in shared memory with
// 16-byte asynchronous copies, across tokens, so the bytes in flight do not
// depend on registers.  fp32 work is on pairs of values (f32x2), and what a
// warp knows of its place comes from a shuffled warp number, so that it lives
// in uniform registers: the backward was bound by instructions that moved
// values about (191 us with 428 instructions per turn, 157 with 360).
// 32768 tokens of 40 heads of 128: forward 105 us (6.4 TB/s), backward 155
// (6.5 TB/s); loads into registers instead of the ring 113 and 188.  With few
// tokens per warp latency shows: 8649 tokens of 8 + 8 heads of 64 take the backward
// 18.5 us in a graph against 7.8 of bytes, for the chain table, position, sine at
// the head of every token and the second launch for the sums of dw.
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vfa {

namespace {

// Warps of a CTA, turns copied ahead, CTAs per SM (16 warps: with 24 the
// forward's reads and writes are spread over more rows, 108 -> 116 us).
template <bool BWD>
struct RopeCfg {
    static constexpr int WARPS = 4, AHEAD = BWD ? 4 : 8, CTAS = 4;
};

constexpr int kTurn = 1024;             // bytes of a turn of one tensor

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

// Eight pairs of dimensions: the first members at v[0..3], the second at
// v[4..7], two pairs per word.  Pair j is dims (a + j, b + j) for halves, (a +
// 2j, a + 2j + 1) for interleaved pairs (b = a + 8).
template <bool INTER>
__device__ __forceinline__ void unpack_pairs(const uint4 ra, const uint4 rb, f2 (&v)[8])
{
    const uint32_t w[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
    auto lo = [&](int i) { return __uint_as_float(w[i] << 16); };
    auto hi = [&](int i) { return __uint_as_float(w[i] & 0xffff0000u); };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = INTER ? f2_pack(lo(2 * j), lo(2 * j + 1)) : f2_pack(lo(j), hi(j));
        v[4 + j] = INTER ? f2_pack(hi(2 * j), hi(2 * j + 1)) : f2_pack(lo(4 + j), hi(4 + j));
    }
}

template <bool INTER>
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *pa, __nv_bfloat16 *pb, const f2 (&v)[8])
{
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = f2_unpack(v[j]), y = f2_unpack(v[4 + j]);
        if (INTER) {
            w[2 * j] = pack_bf16x2(x.x, y.x);
            w[2 * j + 1] = pack_bf16x2(x.y, y.y);
        } else {
            w[j] = pack_bf16x2(x.x, x.y);
            w[4 + j] = pack_bf16x2(y.x, y.y);
        }
    }
    *reinterpret_cast<uint4 *>(pa) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(pb) = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void rotate(f2 (&v)[8], const f2 (&c)[4], const f2 (&s)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f2 a = v[j], b = v[4 + j];
        v[j] = f2_sub(f2_mul(a, c[j]), f2_mul(b, s[j]));
        v[4 + j] = f2_fma(b, c[j], f2_mul(a, s[j]));
    }
}

// Cosines and sines of token t for frequencies 8p .. 8p + 7 (1 and 0 past the
// rotated ones).  The warp's lane groups (one per head it holds) work out a
// share each and exchange.
template <int D>
__device__ __forceinline__ void angles(const RopeArgs &a, int t, int lane, float (&c)[8],
                                       float (&s)[8])
{
    constexpr int LPH = D / 16, GROUPS = 32 / LPH, PER = 8 / GROUPS;
    const int p = lane % LPH, g = lane / LPH;
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

__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A warp's place in its work: turn e of token t (the query heads' turns first).
// Unit u covers turns [e, end) of a token; the warp takes units u, u + warps, ...
struct Turn {
    unsigned u;
    int t, e, end;

    __device__ __forceinline__ void unit(unsigned units, unsigned warps, unsigned segments, int per,
                                         int turns)
    {
        for (; u < units; u += warps) {
            t = static_cast<int>(u / segments);
            e = static_cast<int>(u % segments) * per;
            end = min(turns, e + per);
            if (e < end)
                return;
        }
    }
};

// Both directions.  Backward: a persistent grid whose warps take fixed units,
// so the sums of dw run in a fixed order: per lane over its turns, then over
// the warp's lane groups, the CTA's warps, and (second kernel) the CTAs.  No
// atomics.
template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(RopeCfg<BWD>::WARPS * 32, RopeCfg<BWD>::CTAS) rope_kernel(const RopeArgs a)
{
    constexpr int LPH = D / 16, HPW = 32 / LPH;
    constexpr int WARPS = RopeCfg<BWD>::WARPS, AHEAD = RopeCfg<BWD>::AHEAD;
    constexpr int STAGE = BWD ? 2 * kTurn : kTurn;
    extern __shared__ __align__(16) uint8_t ring[];     // [WARPS][AHEAD][STAGE]
    __shared__ __align__(16) float s_w[2][D];         // [which][quarter of a lane's 16][lane piece][4]
    grid_wait();
    if (BWD && (a.dweight[0] || a.dweight[1]))
        grid_release();                             // the sums of dw follow
    const int lane = threadIdx.x & 31;
    // (a shuffle's result is known to be the same in every lane: what follows from
    // it can live in uniform registers)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int p = lane % LPH, g = lane / LPH;
    for (int i = threadIdx.x; i < 2 * D; i += (WARPS * 32)) {
        const float *w = a.weight[i / D];
        const int quarter = i % D / (4 * LPH), q = i / 4 % LPH, j = quarter % 2 * 4 + i % 4;
        int da, db;
        lane_dims<INTER>(q, a.half, &da, &db);
        const int d = INTER ? da + 2 * j + quarter / 2 : (quarter < 2 ? da : db) + j;
        s_w[i / D][i % D] = w ? w[d] : 1.f;
    }
    __syncthreads();
    int da, db;
    lane_dims<INTER>(p, a.half, &da, &db);
    const bool turns_dims = 8 * p < a.half;
    const int iq = (a.heads[0] + HPW - 1) / HPW, turns = iq + (a.heads[1] + HPW - 1) / HPW;
    const unsigned segments = a.segments, units = static_cast<unsigned>(a.tokens) * segments;
    const unsigned warps = gridDim.x * WARPS;
    const int per = (turns + a.segments - 1) / a.segments;
    uint8_t *mine = ring + warp * AHEAD * STAGE;
    const uint32_t mine_u32 = smem_u32(mine) + lane * 16;

    Turn fill;
    fill.u = blockIdx.x * WARPS + warp;
    fill.unit(units, warps, segments, per, turns);
    Turn cur = fill;
    // Copies the next turn (or nothing, at the end) as one group.
    auto copy_turn = [&](int stage) {
        if (fill.u < units) {
            const int which = fill.e >= iq;
            const int first = (fill.e - (which ? iq : 0)) * (HPW * D) + lane * 8;
            const int left = a.heads[which] * D - first;        // elements of the row from here on
            const uint32_t dst = mine_u32 + stage * STAGE;
            if (!BWD || a.weight[which]) {          // a plain rotation's gradient needs no x
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.x[which]) +
                                           fill.t * a.x_stride[which] + first;
                if (left > 0)
                    copy16_async(dst, src);
                if (left > 256)
                    copy16_async(dst + 512, src + 256);
            }
            if (BWD) {
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.dy[which]) +
                                           fill.t * a.dy_stride[which] + first;
                if (left > 0)
                    copy16_async(dst + kTurn, src);
                if (left > 256)
                    copy16_async(dst + kTurn + 512, src + 256);
            }
            if (++fill.e == fill.end) {
                fill.u += warps;
                fill.unit(units, warps, segments, per, turns);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int k = 0; k < AHEAD; ++k)
        copy_turn(k);

    f2 dw[2][8];
    if (BWD) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[0][j] = dw[1][j] = 0;
    }
    f2 c2[4], s2[4];
    int stage = 0, t = -1;
    while (cur.u < units) {
        if (cur.t != t) {
            t = cur.t;
            float c[8], s[8];
            angles<D>(a, t, lane, c, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c2[j] = f2_pack(c[2 * j], c[2 * j + 1]);
                s2[j] = f2_pack(BWD ? -s[2 * j] : s[2 * j], BWD ? -s[2 * j + 1] : s[2 * j + 1]);
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        __syncwarp();
        const int which = cur.e >= iq;
        const int h = (cur.e - (which ? iq : 0)) * HPW + g;
        const bool live = h < a.heads[which];
        const bool norm = a.weight[which] != nullptr;
        const __nv_bfloat16 *sx = reinterpret_cast<const __nv_bfloat16 *>(mine + stage * STAGE) + g * D;
        f2 x[8], y[8];
        if (!BWD || norm)
            unpack_pairs<INTER>(*reinterpret_cast<const uint4 *>(sx + da),
                                *reinterpret_cast<const uint4 *>(sx + db), x);
        if (BWD) {
            const __nv_bfloat16 *sy = sx + kTurn / 2;
            unpack_pairs<INTER>(*reinterpret_cast<const uint4 *>(sy + da),
                                *reinterpret_cast<const uint4 *>(sy + db), y);
        }
        __syncwarp();                               // every lane has read the stage: refill it
        copy_turn(stage);
        stage = stage + 1 == AHEAD ? 0 : stage + 1;

        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.y[which]) + t * a.y_stride[which] + h * D;
        // words 2i, 2i + 1 of the weights, in the order of the pairs
        auto weights = [&](int i) {
            const float4 v = *reinterpret_cast<const float4 *>(&s_w[which][(i * LPH + p) * 4]);
            return make_ulonglong2(f2_pack(v.x, v.y), f2_pack(v.z, v.w));
        };
        if (!BWD) {
            if (norm) {
                f2 q = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q = f2_fma(x[j], x[j], q);
                const float r = rsqrtf(head_sum<D>(f2_sum(q)) * (1.f / D) + a.eps);
                const f2 r2 = f2_pack(r, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 w = weights(i);
                    x[2 * i] = f2_mul(f2_mul(x[2 * i], r2), w.x);
                    x[2 * i + 1] = f2_mul(f2_mul(x[2 * i + 1], r2), w.y);
                }
            }
            if (turns_dims)
                rotate(x, c2, s2);
            if (live)
                store_pairs<INTER>(dst + da, dst + db, x);
        } else {
            if (turns_dims)
                rotate(y, c2, s2);
            if (norm) {
                if (h - g + HPW > a.heads[which] && !live) {
                    // lanes past the heads hold whatever was there: no gradient, on rows that have
                    // a norm (with eps = 0 a zero row's r is infinite, and 0 r no number)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] = f2_pack(1.f, 1.f);
                        y[j] = 0;
                    }
                }
                f2 q = 0, d = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 w = weights(i);
                    q = f2_fma(x[2 * i], x[2 * i], q);
                    q = f2_fma(x[2 * i + 1], x[2 * i + 1], q);
                    d = f2_fma(f2_mul(y[2 * i], w.x), x[2 * i], d);
                    d = f2_fma(f2_mul(y[2 * i + 1], w.y), x[2 * i + 1], d);
                }
                const float r = rsqrtf(head_sum<D>(f2_sum(q)) * (1.f / D) + a.eps);
                const float m = -head_sum<D>(f2_sum(d)) * (1.f / D) * r * r;
                const f2 r2 = f2_pack(r, r), m2 = f2_pack(m, m);
                if (which) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        dw[1][j] = f2_fma(f2_mul(y[j], r2), x[j], dw[1][j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        dw[0][j] = f2_fma(f2_mul(y[j], r2), x[j], dw[0][j]);
                }
                // (u = g w once more: keeping it costs 16 registers, and more instructions
                // to move values about than it saves)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 w = weights(i);
                    y[2 * i] = f2_mul(r2, f2_fma(x[2 * i], m2, f2_mul(y[2 * i], w.x)));
                    y[2 * i + 1] = f2_mul(r2, f2_fma(x[2 * i + 1], m2, f2_mul(y[2 * i + 1], w.y)));
                }
            }
            if (live)
                store_pairs<INTER>(dst + da, dst + db, y);
        }
        if (++cur.e == cur.end) {
            cur.u += warps;
            cur.unit(units, warps, segments, per, turns);
        }
    }
    if (!BWD)
        return;
    // partial[cta][which][d], the warps' sums over the ring (no copy is in flight)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *s_dw = reinterpret_cast<float *>(ring);      // [WARPS][D]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!a.dweight[which])
            continue;
        float sum[16];                              // first members, then second members
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = f2_unpack(dw[which][j]);
            sum[2 * j] = v.x;
            sum[2 * j + 1] = v.y;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
#pragma unroll
            for (int off = LPH; off < 32; off <<= 1)
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
        }
        __syncthreads();                            // the ring, or the queries' sums, have been read
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s_dw[warp * D + (INTER ? da + 2 * j : da + j)] = sum[j];
                s_dw[warp * D + (INTER ? da + 2 * j + 1 : db + j)] = sum[8 + j];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += (WARPS * 32)) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k)
                v += s_dw[k * D + d];
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

template <int D, bool BWD>
cudaError_t launch_d(RopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int HPW = 32 / (D / 16);
    using C = RopeCfg<BWD>;
    constexpr int SMEM = C::WARPS * C::AHEAD * (BWD ? 2 : 1) * kTurn;
    static_assert(SMEM >= C::WARPS * D * static_cast<int>(sizeof(float)), "the ring holds the warps' dw");
    static_assert(SMEM + 2 * D * static_cast<int>(sizeof(float)) <= 48 * 1024, "no opt-in needed");
    a.segments = head_segments(a, (a.heads[0] + HPW - 1) / HPW + (a.heads[1] + HPW - 1) / HPW,
                               sm_count);
    const long long need = (static_cast<long long>(a.tokens) * a.segments + C::WARPS - 1) / C::WARPS;
    long long grid = static_cast<long long>(sm_count) * C::CTAS;
    grid = grid < need ? grid : need;
    grid = grid < kRopeMaxCtas ? grid : kRopeMaxCtas;
    a.ctas = static_cast<int>(grid);
    const auto kernel = a.interleaved ? rope_kernel<D, true, BWD> : rope_kernel<D, false, BWD>;
    const cudaError_t e = launch_dependent(kernel, dim3(a.ctas), C::WARPS * 32, SMEM, stream, a);
    if (e != cudaSuccess || !BWD || (!a.dweight[0] && !a.dweight[1]))
        return e;
    return launch_dependent(rope_dw_kernel, dim3(D / 32, 2), 1024, 0, stream, a, D);
}

}  // namespace

cudaError_t launch_rope_fwd(int head_dim, RopeArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.tokens == 0)
        return cudaSuccess;
    switch (head_dim) {
    case 64: return launch_d<64, false>(a, sm_count, stream);
    case 128: return launch_d<128, false>(a, sm_count, stream);
    case 256: return launch_d<256, false>(a, sm_count, stream);
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
    case 64: return launch_d<64, true>(a, sm_count, stream);
    case 128: return launch_d<128, true>(a, sm_count, stream);
    case 256: return launch_d<256, true>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
