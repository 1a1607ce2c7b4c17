// kv4.cu -- a paged K/V cache held in 4 bits: writing packed tokens into it,
// reading them back, and one-token grouped-query attention over it.
//
// Format.  Pages of 16 tokens; per page and kv head 18 D bytes: K codes
// (8 D), V codes (8 D), K scales (D), V scales (D).  Codes are E2M1 (0, 0.5,
// 1, 1.5, 2, 3, 4, 6 and a sign), scales E4M3, one per 16 consecutive
// dimensions of a token; value = descale * scale * code.  A code has 2
// significant bits and a scale 4, so with a power of two as descale a value
// has at most 6: it is exact in bf16 and in f16, and nothing after the
// quantisation rounds it again.  The order inside a page is the one the
// decode kernel's lanes read (below); every byte belongs to one token, so
// tokens are written independently.
//   K codes   token t, dim d: byte t D/2 + d/2, low nibble for even d
//   V codes   W = min(16, D/8) dims of a token and of its odd neighbour side by
//             side: c = d / W, byte ((t/8) (D/8W) + c/8) 32 W +
//             ((c%8) 4 + (t/2)%4) W + (t%2) W/2 + (d%W)/2
//   K scales  byte t D/16 + d/16
//   V scales  byte ((d/16) 4 + (t/2)%4) 4 + t%2 + 2 (t/8)
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f32x2.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vfa {

namespace {

constexpr int kPage = kKv4Page;
constexpr float kLn2 = 0.69314718055994531f;

// Offset in the V code area of the 16-dim group g of token t; for D = 64 the
// group is two runs of 4 bytes, 32 bytes apart.
template <int D>
__device__ __forceinline__ int v_code_at(int t, int g)
{
    if (D == 64)
        return (t >> 3) * 256 + (2 * g * 4 + ((t >> 1) & 3)) * 8 + (t & 1) * 4;
    return ((t >> 3) * (D / 128) + (g >> 3)) * 512 + ((g & 7) * 4 + ((t >> 1) & 3)) * 16 +
           (t & 1) * 8;
}

__device__ __forceinline__ int v_scale_at(int t, int g)
{
    return (g * 4 + ((t >> 1) & 3)) * 4 + (t & 1) + 2 * (t >> 3);
}

__device__ __forceinline__ void record(int32_t *status, int code)
{
    if (status)
        atomicCAS(status, 0, code);
}

// ------------------------------------------------------------ number formats

// Four bytes of two E2M1 codes each -> four f16x2 (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Eight floats -> eight E2M1 codes, nearest even, saturating; f[0] in the low nibble.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float *f)
{
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

// Two E4M3 codes (low byte first) -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two)
{
    uint32_t h;
    asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
        : "=r"(h)
        : "r"(two));
    return h;
}

__device__ __forceinline__ uint32_t f32_to_e4m3(float f)
{
    uint32_t r;
    asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %1, %2;\n\tcvt.u32.u16 %0, x;\n\t}"
        : "=r"(r)
        : "f"(0.f), "f"(f));
    return r & 0xffu;
}

__device__ __forceinline__ float f16_lo(uint32_t h)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

__device__ __forceinline__ float f16_hi(uint32_t h)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h >> 16)));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------ write, read
//
// A warp takes 32 / (D/16) consecutive packed tokens, D/16 lanes each (a lane
// holds one scale's 16 dims, so nothing is exchanged), and goes over the kv
// heads: the tokens' places are found side by side, and the V codes of
// neighbouring tokens, 8 bytes each, fill whole 32-byte sectors.  Bound: HBM,
// 2.5625 bytes per element.  85k tokens of 8 heads of 128: 75 us to write, 72
// to read back (89 and 89 with one token per warp).

// Page and row of packed token t; false where it has none (a padding row at
// or past cu[num_seqs], or bad tables, which are recorded).
__device__ __forceinline__ bool token_slot(const Kv4MoveArgs &a, int t, int *page, int *row)
{
    int lo = 0, hi = a.num_seqs;                 // cu[lo] <= t < cu[hi]
    if (t >= a.total || t >= __ldg(a.cu + hi))
        return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int c0 = __ldg(a.cu + lo);
    if (c0 > t || t >= __ldg(a.cu + lo + 1)) {
        record(a.status, VFA_ERR_BAD_SEQLENS);
        return false;
    }
    const int st = __ldg(a.start + lo);
    const long long pos = static_cast<long long>(st) + (t - c0);
    const bool in = st >= 0 && pos < static_cast<long long>(a.capacity) * kPage;
    const int p = in ? __ldg(a.tables + static_cast<long long>(lo) * a.capacity + pos / kPage) : -1;
    if (p < 0 || p >= a.num_blocks) {
        record(a.status, VFA_ERR_BAD_BLOCK);
        return false;
    }
    *page = p;
    *row = static_cast<int>(pos % kPage);
    return true;
}

// cu must start at 0, not decrease and not pass `total` (CTA 0 checks).
__device__ __forceinline__ void check_cu(const Kv4MoveArgs &a)
{
    bool bad = false;
    for (int s = threadIdx.x; s <= a.num_seqs; s += blockDim.x) {
        const int c = a.cu[s];
        bad |= s == 0 ? c != 0 : c < a.cu[s - 1];
        bad |= c > a.total;
    }
    if (bad)
        record(a.status, VFA_ERR_BAD_SEQLENS);
}

// 16 values -> scale byte and two code words.  x / scale decides at most
// which of two neighbouring codes is nearer.  With a power of two as descale
// x has 8 significant bits and scale * midpoint 7, so a quotient that is not
// exactly a midpoint is at least 2^-8 (relative) away from it; x * (1/scale)
// is within 2^-23, and rounding it to f16 (11 bits) restores exact midpoints
// and moves the others by at most 2^-11: the codes are those of the exact
// quotient.  The same holds for max / 6 against the midpoints of E4M3.
__device__ __forceinline__ void quantise16(const float (&x)[16], uint32_t *scale, uint32_t (&w)[2])
{
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        m = fmaxf(m, fabsf(x[j]));
    *scale = f32_to_e4m3(__fdiv_rn(m, 6.f));
    const float s = f16_lo(e4m3x2_to_f16(*scale));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    float y[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = pack_f16x2(x[2 * j] * r, x[2 * j + 1] * r);
        y[2 * j] = f16_lo(h);
        y[2 * j + 1] = f16_hi(h);
    }
    w[0] = f32_to_e2m1x8(y);
    w[1] = f32_to_e2m1x8(y + 8);
}

constexpr int kMoveWarps = 8;
constexpr int kMoveAhead = 2;           // kv heads of K and V loaded together

// A lane's 32 bytes as two 16-byte words, read or written by pairs of lanes so
// that every instruction touches whole 32-byte sectors: even lanes move the
// first halves of the pair's two runs, odd lanes the second halves.
struct PairBytes {
    uint4 lo, hi;                       // the lane's own 32 bytes

    // before a write, after a read: even lanes trade their neighbour's first
    // half for their own second half
    __device__ __forceinline__ void exchange(int lane)
    {
        const bool odd = lane & 1;
        uint4 give = odd ? lo : hi;
        give.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
        give.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
        give.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
        give.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
        if (odd)
            lo = give;
        else
            hi = give;
    }
};

// Byte offset, from the lane's own run, of the word it moves first; the other
// is 32 bytes on.
__device__ __forceinline__ int pair_offset(int lane) { return lane & 1 ? -16 : 0; }

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) kv4_write_kernel(const Kv4MoveArgs a)
{
    constexpr int GR = D / 16, TPW = 32 / GR;
    const int lane = threadIdx.x & 31;
    const int g = lane % GR;
    grid_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        check_cu(a);
    // this CTA's share of the kv heads (all of them but where tokens are few)
    const int per = (a.num_kv_heads + gridDim.y - 1) / gridDim.y;
    const int first_head = blockIdx.y * per, heads = min(a.num_kv_heads, first_head + per);
    const int po = pair_offset(lane);
    const long long warps = static_cast<long long>(gridDim.x) * kMoveWarps;
    for (long long t0 = (static_cast<long long>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5)) * TPW;
         t0 < a.total; t0 += warps * TPW) {
        const int t = static_cast<int>(t0) + lane / GR;
        int page = 0, row = 0;
        const bool has = token_slot(a, t, &page, &row);
        uint8_t *pg = static_cast<uint8_t *>(a.pool) +
                      static_cast<long long>(page) * a.num_kv_heads * kv4_head_page_bytes(D);
        const uint8_t *src[2] = {
            reinterpret_cast<const uint8_t *>(static_cast<const __nv_bfloat16 *>(a.k) +
                                              static_cast<long long>(t) * a.k_stride + g * 16) + po,
            reinterpret_cast<const uint8_t *>(static_cast<const __nv_bfloat16 *>(a.v) +
                                              static_cast<long long>(t) * a.v_stride + g * 16) + po};
        for (int h0 = first_head; h0 < heads; h0 += kMoveAhead) {
            PairBytes in[2][kMoveAhead];
#pragma unroll
            for (int i = 0; i < kMoveAhead; ++i)
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    in[which][i].lo = in[which][i].hi = make_uint4(0, 0, 0, 0);
                    if (has && h0 + i < heads) {
                        const uint8_t *q = src[which] + (h0 + i) * (2 * D);
                        in[which][i].lo = __ldcs(reinterpret_cast<const uint4 *>(q));
                        in[which][i].hi = __ldcs(reinterpret_cast<const uint4 *>(q + 32));
                    }
                }
#pragma unroll
            for (int i = 0; i < kMoveAhead; ++i)
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    PairBytes &r = in[which][i];
                    r.exchange(lane);
                    if (!has || h0 + i >= heads)
                        continue;
                    const float inv = which ? a.v_scale : a.k_scale;
                    const uint32_t rw[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w,
                                            r.hi.x, r.hi.y, r.hi.z, r.hi.w};
                    float x[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[2 * j] = __uint_as_float(rw[j] << 16) * inv;
                        x[2 * j + 1] = __uint_as_float(rw[j] & 0xffff0000u) * inv;
                    }
                    uint32_t scale, w[2];
                    quantise16(x, &scale, w);
                    uint8_t *hp = pg + (h0 + i) * kv4_head_page_bytes(D);
                    if (which == 0) {
                        *reinterpret_cast<uint2 *>(hp + row * (D / 2) + g * 8) = make_uint2(w[0], w[1]);
                        hp[16 * D + row * GR + g] = static_cast<uint8_t>(scale);
                    } else {
                        uint8_t *vp = hp + 8 * D + v_code_at<D>(row, g);
                        if (D == 64) {
                            *reinterpret_cast<uint32_t *>(vp) = w[0];
                            *reinterpret_cast<uint32_t *>(vp + 32) = w[1];
                        } else {
                            *reinterpret_cast<uint2 *>(vp) = make_uint2(w[0], w[1]);
                        }
                        hp[17 * D + v_scale_at(row, g)] = static_cast<uint8_t>(scale);
                    }
                }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) kv4_gather_kernel(const Kv4MoveArgs a)
{
    constexpr int GR = D / 16, TPW = 32 / GR;
    const int lane = threadIdx.x & 31;
    const int g = lane % GR;
    grid_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        check_cu(a);
    // this CTA's share of the kv heads (all of them but where tokens are few)
    const int per = (a.num_kv_heads + gridDim.y - 1) / gridDim.y;
    const int first_head = blockIdx.y * per, heads = min(a.num_kv_heads, first_head + per);
    const int po = pair_offset(lane);
    const long long warps = static_cast<long long>(gridDim.x) * kMoveWarps;
    for (long long t0 = (static_cast<long long>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5)) * TPW;
         t0 < a.total; t0 += warps * TPW) {
        const int t = static_cast<int>(t0) + lane / GR;
        int page = 0, row = 0;
        const bool has = token_slot(a, t, &page, &row);
        const uint8_t *pg = static_cast<const uint8_t *>(a.pool) +
                            static_cast<long long>(page) * a.num_kv_heads * kv4_head_page_bytes(D);
        uint8_t *dst[2] = {
            reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(a.k) +
                                        static_cast<long long>(t) * a.k_stride + g * 16) + po,
            reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(a.v) +
                                        static_cast<long long>(t) * a.v_stride + g * 16) + po};
        for (int h0 = first_head; h0 < heads; h0 += kMoveAhead) {
            uint2 code[2][kMoveAhead];
            uint32_t scale[2][kMoveAhead];
#pragma unroll
            for (int i = 0; i < kMoveAhead; ++i)
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    code[which][i] = make_uint2(0, 0);
                    scale[which][i] = 0;
                    if (has && h0 + i < heads) {
                        const uint8_t *hp = pg + (h0 + i) * kv4_head_page_bytes(D);
                        if (which == 0) {
                            code[0][i] = *reinterpret_cast<const uint2 *>(hp + row * (D / 2) + g * 8);
                            scale[0][i] = hp[16 * D + row * GR + g];
                        } else {
                            const uint8_t *vp = hp + 8 * D + v_code_at<D>(row, g);
                            if (D == 64) {
                                code[1][i].x = *reinterpret_cast<const uint32_t *>(vp);
                                code[1][i].y = *reinterpret_cast<const uint32_t *>(vp + 32);
                            } else {
                                code[1][i] = *reinterpret_cast<const uint2 *>(vp);
                            }
                            scale[1][i] = hp[17 * D + v_scale_at(row, g)];
                        }
                    }
                }
#pragma unroll
            for (int i = 0; i < kMoveAhead; ++i)
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    const float s = f16_lo(e4m3x2_to_f16(scale[which][i])) * (which ? a.v_scale : a.k_scale);
                    uint32_t lo[4], hi[4], o[8];
                    e2m1x8_to_f16(code[which][i].x, lo);
                    e2m1x8_to_f16(code[which][i].y, hi);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[j] = pack_bf16x2(f16_lo(lo[j]) * s, f16_hi(lo[j]) * s);
                        o[4 + j] = pack_bf16x2(f16_lo(hi[j]) * s, f16_hi(hi[j]) * s);
                    }
                    PairBytes out;
                    out.lo = make_uint4(o[0], o[1], o[2], o[3]);
                    out.hi = make_uint4(o[4], o[5], o[6], o[7]);
                    out.exchange(lane);
                    if (has && h0 + i < heads) {
                        uint8_t *q = dst[which] + (h0 + i) * (2 * D);
                        *reinterpret_cast<uint4 *>(q) = out.lo;
                        *reinterpret_cast<uint4 *>(q + 32) = out.hi;
                    }
                }
        }
    }
}

// ------------------------------------------------------------ decode
//
// Online softmax over the cached tokens of each sequence, the Hq / Hkv query
// heads of a kv head together: up to 8 as one tile of 8 columns, up to 16 as
// two that share the unpacked pages (16 heads of 128 on 8 kv heads, 64
// contexts of 4-8k: 167 us as two chunks of 8, 129 as two tiles); more are
// more head chunks, whose pages come from L2.  Two tiles are bound by latency,
// not by the second product: 239 registers leave eight warps per SM, which issue
// 1.7 instructions a cycle with no pipe above 35%, and wait most for the results
// of the instruction ahead.
//
// Bound: HBM for long batches, 1.125 bytes per dim and token of a kv head.  A
// call takes 14 us (17 for 64 sequences) plus its pages at 6.39 TB/s, 94% of
// the copy rate: the chain from counts over tables to the first pages, and the
// merge behind the last.  8 kv heads of 128, 4 query heads each: 256 sequences
// of 16-16k tokens 139 us (5.1 TB/s), four of 49-65k 52.8 us (4.9), 64 of 32k
// 390 us (6.1).  Unpacking comes close behind: 280 instructions per page and head,
// 2.2 of them a cycle and SM.
//
// Work.  Every sequence counts its pages (1 if empty) and kSeqUnits for its
// start and end (a query load, a merge of the warps, an output: about as long
// as kSeqUnits pages take a CTA); the batch's units in one row are cut into
// equal contiguous runs, one per CTA, so long and short contexts load every SM
// alike.  A run covers any number of sequences; a sequence whose pages lie in
// one run is finished there, the others leave partial states (m, l, o), merged
// in a fixed order by the CTA that takes the last ticket.  No CTA waits for
// another.
//
// Warp w takes every fourth group of NP of the run's pages (NP = 2, or 4 at D
// = 64: several at a time give a warp independent chains of products; with one
// the four long contexts take 64 us) and copies them ahead into its own ring of
// shared-memory stages with 16-byte asynchronous copies; it alone reads what it
// copied, so the ring needs no barrier, only its copy groups.  (Bulk copies
// held the issuing warp for about 500 cycles each: the four long contexts took
// 72 us with every warp issuing its own and 87 us from one producer warp.)  Per
// page, two products on mma.sync m16n8k16 (f16 in, fp32 accumulate):
//   S[16 tokens x 8 heads] = K Q^T    O^T[D x 8 heads] += V^T P
// The page's order gives every lane its A operands in whole 16-byte words: a
// lane of K's operand holds 32 consecutive dims of two tokens (two scales
// each), one of V's 16 dims of four tokens, whose codes are paired by token
// with two logic operations per eight codes.  Which dim is which k index of
// a product is free as long as Q agrees.
//
// Numbers.  K, V as f16: exact (see the format).  q is multiplied by a power
// of two per head that puts its largest element at 2^14: f16 then holds every
// bf16 bit of elements down to 2^-21 of the largest and is within 2^-39 of
// the largest below.  Weights are relative to a reference, the maximum when it
// was last taken: a warp takes it again (an exchange over its lanes and a
// rescaling) only when a weight would pass it by more than a factor 2^5, so
// most groups cost one vote.  References stay in units of the accumulators, whose
// difference is taken before the scale: it is exact near the maximum however
// large the logits are.  p is held as 2^10 p in f16, at most 2^15 (2^-11
// relative for p above 2^-24, 2^-35 absolute below), l sums the fp32 values,
// and the reference, l and o are fp32.  The roundings of p average out over the
// keys: 0.8 to 2.0 10^-4 of the output before its own rounding to bf16, 1.65 10^-3
// (2-norms; contexts of 150 to 65k tokens, normally distributed q, K and V).
constexpr int kConsumers = 4;
constexpr int kDecThreads = kConsumers * 32;
constexpr int kTile = 8;                // query heads of a tile (columns of a product)
constexpr int kSeqUnits = 24;           // units of a sequence besides its pages
constexpr int kMinRun = 24;             // units per CTA at least
constexpr int kMaxCtas = 1024;          // CTAs in all rows, where there are fewer rows
constexpr float kPShift = 10.f, kSlack = 5.f;    // log2
constexpr float kNoRef = -0x1p60f;      // below any finite accumulator (2^36 at most)

// Tiles of query heads a CTA takes: two where a kv head has more than eight
// (at D = 256 their accumulators would not fit the registers).
__host__ __device__ constexpr int head_tiles(int group, int head_dim)
{
    return group > kTile && head_dim <= 128 ? 2 : 1;
}

template <int D, int NT>
struct DecCfg {
    static constexpr int HEADS = NT * kTile;                    // of a CTA at most
    static constexpr int NP = D == 64 ? 4 : 2;                  // pages of a group
    static constexpr int PAGE = 18 * D;                         // bytes of a head page
    static constexpr int STAGE = NP * PAGE;                     // a stage holds a group
    static constexpr int WS = 2;                                // stages of a warp
    static constexpr int NS = WS * kConsumers;                  // stages of the CTA
    static constexpr int CTAS = D == 64 ? 5 - NT : D == 128 ? 4 - NT : 2;   // resident per SM
    // Merge areas: with two, a warp goes on to the next segment while others still
    // merge (the four long contexts: 54.0 -> 52.5 us with a sequence's 24 units; with
    // 20 of them 53.7); at D = 256 the second would cost the other CTA of the SM.
    static constexpr int AREAS = D == 256 ? 1 : 2;
    static constexpr int MT = D / 16;
    static constexpr int KW = D / 32;               // code words of one token per lane
    static constexpr int PART = HEADS * (D + 4);    // floats of a part: per head o, m, l
};

// 16 bytes from src + OFF to shared memory at dst + OFF.
template <int OFF>
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src),
                 "n"(OFF)
                 : "memory");
}

// The 16-byte pieces of NP pages in a row, 32 per turn and one per lane; p[i] is
// page i less the i pages before it.  A turn touches two pages at most.
template <int NP, int PIECES, int K = 0>
__device__ __forceinline__ void copy_pages(uint32_t dst, const uint8_t *const (&p)[NP], int lane)
{
    if constexpr (K < NP * PIECES) {
        constexpr int A = K / PIECES, B = (K + 31) / PIECES < NP ? (K + 31) / PIECES : NP - 1;
        if (K + 32 <= NP * PIECES || K + lane < NP * PIECES)
            copy16_async<K * 16>(dst, A == B || K + lane < B * PIECES ? p[A] : p[B]);
        copy_pages<NP, PIECES, K + 32>(dst, p, lane);
    }
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until all but the newest N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Pages of a sequence (1 if empty), and its token count (0 and *bad for an
// invalid one).
__device__ __forceinline__ int seq_pages(const Kv4DecodeArgs &a, int s, int *tokens, bool *bad)
{
    const int n = __ldg(a.counts + s);
    *bad = n < 0 || n > static_cast<long long>(a.capacity) * kPage;
    *tokens = *bad ? 0 : n;
    const int u = (*tokens + kPage - 1) / kPage;
    return u < 1 ? 1 : u;
}

// A place in the CTA's run [u0, u1): the segment of sequence s whose units
// start at `at` in the row (kSeqUnits, then its pages), the run's pages [j0,
// j1) of it, and (modulo 4) the groups of NP pages of the earlier segments,
// which decide the warp that takes its first group.
template <int NP>
struct RunCursor {
    int s, at, pages, tokens, j0, j1, base;
    bool bad;

    // The first segment with pages in the run from sequence s on; false if none.
    __device__ __forceinline__ bool enter(const Kv4DecodeArgs &a, int u0, int u1)
    {
        for (; at + kSeqUnits < u1; ++s) {
            pages = seq_pages(a, s, &tokens, &bad);
            const int p0 = at + kSeqUnits;
            j0 = max(0, u0 - p0);
            j1 = min(pages, u1 - p0);
            if (j0 < j1)
                return true;
            at = p0 + pages;
        }
        return false;
    }
    // First page of `warp`'s first group of the segment (at or past j1: none).
    __device__ __forceinline__ int first(int warp) const
    {
        return j0 + NP * ((warp - base) & (kConsumers - 1));
    }
    // The next segment; false at the end of the run.
    __device__ __forceinline__ bool next(const Kv4DecodeArgs &a, int u0, int u1)
    {
        base += (j1 - j0 + NP - 1) / NP;
        at += kSeqUnits + pages;
        ++s;
        return enter(a, u0, u1);
    }
};

// What the warps of a CTA leave at the end of a segment, besides their outputs.
template <int HEADS>
struct MergeArea {
    float m[kConsumers][HEADS], l[kConsumers][HEADS], scale[HEADS];
    int bad[kConsumers];
};

template <int D, int NT>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D, NT>::CTAS) kv4_decode_kernel(const Kv4DecodeArgs a)
{
    using C = DecCfg<D, NT>;
    constexpr int NP = C::NP, MT = C::MT, KW = C::KW, PART = C::PART;
    constexpr int STRIDE = NP * kConsumers;         // pages from a warp's group to its next
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ MergeArea<C::HEADS> merge[C::AREAS];
    __shared__ int s_scan[kDecThreads / 32];
    __shared__ int s_first, s_first_unit, s_last;

    grid_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.num_q_heads / a.num_kv_heads;
    const int chunks = (group + C::HEADS - 1) / C::HEADS;
    const int kh = blockIdx.y / chunks;
    const int h0 = kh * group + (blockIdx.y % chunks) * C::HEADS;   // first query head
    const int G = min(C::HEADS, (kh + 1) * group - h0);

    // Units before each thread's share of the sequences.
    const int per = (a.num_seqs + kDecThreads - 1) / kDecThreads;
    const int sa = min(a.num_seqs, tid * per), sb = min(a.num_seqs, sa + per);
    int mine = 0;
    for (int s = sa; s < sb; ++s) {
        int n;
        bool bad;
        mine += kSeqUnits + seq_pages(a, s, &n, &bad);
    }
    int x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += y;
    }
    if (lane == 31)
        s_scan[warp] = x;
    __syncthreads();
    int before = x - mine, total = 0;
#pragma unroll
    for (int i = 0; i < kDecThreads / 32; ++i) {
        before += i < warp ? s_scan[i] : 0;
        total += s_scan[i];
    }
    // This CTA's run [u0, u1) of the row of units.
    int run = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    run = run < kMinRun ? kMinRun : run;
    const long long u0l = static_cast<long long>(blockIdx.x) * run;
    if (u0l >= total)
        return;
    const int u0 = static_cast<int>(u0l), u1 = min(total, u0 + run);
    if (u0 >= before && u0 < before + mine) {
        int at = before;
        for (int s = sa; s < sb; ++s) {
            int n;
            bool bad;
            const int u = kSeqUnits + seq_pages(a, s, &n, &bad);
            if (u0 < at + u) {
                s_first = s;
                s_first_unit = at;
                break;
            }
            at += u;
        }
    }
    __syncthreads();
    const uint32_t page_bytes = static_cast<uint32_t>(a.num_kv_heads) * C::PAGE;
    const uint8_t *pool = a.pool + static_cast<size_t>(kh) * C::PAGE;

    // ---------------------------------------------------- copies
    // Fills of this warp's stages, WS groups ahead.  The ids of its next groups
    // in segment `fill`, up to 32 pages, are loaded and checked together: lane
    // l holds page l % NP of group l / NP.  Where there is no page (a last
    // group's rest, an empty sequence) or the id is bad, page 0 is copied in its
    // place and not used.  Every turn commits one group of copies, also where
    // there is nothing left to copy.
    RunCursor<NP> fill;
    fill.s = s_first;
    fill.at = s_first_unit;
    fill.base = 0;
    if (!fill.enter(a, u0, u1))
        return;                                     // (the whole CTA) no page in this run
    RunCursor<NP> seg = fill;
    int ahead = fill.first(warp), ids = 0, id_lane = 0, left = 0;
    uint32_t bad_ids = 0, bad_stages = 0;
    auto load_ids = [&]() {
        while (ahead >= fill.j1) {
            if (!fill.next(a, u0, u1))
                return;
            ahead = fill.first(warp);
        }
        left = min(32 / NP, (fill.j1 - ahead + STRIDE - 1) / STRIDE);
        const int j = ahead + (lane / NP) * STRIDE + lane % NP;
        const bool listed = j < fill.j1 && fill.tokens > 0;
        ids = listed ? __ldg(a.tables + static_cast<long long>(fill.s) * a.capacity + j) : 0;
        const bool bad = static_cast<unsigned>(ids) >= static_cast<unsigned>(a.num_blocks);
        bad_ids = __ballot_sync(0xffffffffu, bad && listed);
        ids = bad ? 0 : ids;
        id_lane = 0;
        ahead += 32 * kConsumers;
    };
    const uint32_t my_ring = smem_u32(dsm) + warp * C::WS * C::STAGE + lane * 16;
    const uint8_t *my_pool = pool + lane * 16;
    const bool pages_exist = a.num_blocks > 0;
    auto issue = [&](int ws) {
        if (left > 0) {
            const uint8_t *p[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i)
                p[i] = my_pool +
                       static_cast<uint64_t>(static_cast<uint32_t>(
                           __shfl_sync(0xffffffffu, ids, id_lane + i))) * page_bytes - i * C::PAGE;
            if (pages_exist)
                copy_pages<NP, C::PAGE / 16>(my_ring + ws * C::STAGE, p, lane);
            if (bad_ids >> id_lane & ((1u << NP) - 1)) {
                bad_stages |= 1u << ws;
                if (lane == 0)
                    record(a.status, VFA_ERR_BAD_BLOCK);
            }
            id_lane += NP;
            if (--left == 0)
                load_ids();
        }
        copy_commit();
    };
    load_ids();
#pragma unroll 1
    for (int k = 0; k < C::WS; ++k)
        issue(k);

    // ---------------------------------------------------- attention
    const int r = lane >> 2, t4 = lane & 3;
    float *const outs = reinterpret_cast<float *>(dsm + C::NS * C::STAGE);  // [AREAS][kConsumers][G][D]
    int ws = 0;                                     // stage of this warp's next group
    int area = 0;                                   // of this segment's merge
    bool first_segment = true;
    do {
        const int s = seg.s, n = seg.tokens, j0 = seg.j0, j1 = seg.j1;
        if (seg.bad && tid == 0)
            record(a.status, VFA_ERR_BAD_BLOCK);

        // Q^T operands: head r of each tile, dims as K's lanes hold them; the logit
        // scales of the heads of this lane's accumulators, 2 t4 and 2 t4 + 1.
        uint32_t qb[NT][MT][2];
        float sc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * kTile + r;
            const uint2 *qrow = reinterpret_cast<const uint2 *>(
                static_cast<const __nv_bfloat16 *>(a.q) +
                (static_cast<long long>(s) * a.num_q_heads + h0 + (h < G ? h : 0)) * D);
            uint2 raw[MT];
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                // dims of product j: piece j / 8 (128 dims), 4 dims from t4 * 32 (D = 64: t4 * 16)
                const int d = D == 64 ? t4 * 16 + 4 * j : (j >> 3) * 128 + t4 * 32 + 4 * (j & 7);
                raw[j] = __ldg(qrow + d / 4);
                const uint32_t w[2] = {raw[j].x, raw[j].y};
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                       fabsf(__uint_as_float(w[e] & 0xffff0000u))));
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // exponent of the largest element, kept where 2^(14 - e) is a normal float
            int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
            e = m > 0.f ? max(-100, min(127, e)) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
            const float down = ldexpf(1.f, e - 14);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const uint32_t w[2] = {raw[j].x, raw[j].y};
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    qb[nt][j][c] = h < G ? pack_f16x2(__uint_as_float(w[c] << 16) * up,
                                                      __uint_as_float(w[c] & 0xffff0000u) * up)
                                         : 0u;
            }
            // positive, or a masked -inf times it would be no number; finite, or the zero between
            // equal logits times it would (at FLT_MAX any other difference has weight zero)
            const float x = fminf(fmaxf(a.scale_log2 * down, FLT_MIN), FLT_MAX);
            sc[nt][0] = __shfl_sync(0xffffffffu, x, (2 * t4) * 4);
            sc[nt][1] = __shfl_sync(0xffffffffu, x, (2 * t4 + 1) * 4);
        }

        // per head: the reference, the logit that renews it (both before the scale), the sum
        float ref[NT][2], limit[NT][2], l_part[NT][2], o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ref[nt][0] = ref[nt][1] = kNoRef;
            limit[nt][0] = limit[nt][1] = -INFINITY;
            l_part[nt][0] = l_part[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[nt][mt][e] = 0.f;
        }
        bool bad = seg.bad;

        for (int j = seg.first(warp); j < j1; j += STRIDE) {
            copy_wait<C::WS - 1>();
            __syncwarp();                           // every lane's copies are there for every lane
            const uint8_t *stage = dsm + (warp * C::WS + ws) * C::STAGE;
            // tokens of the group that count, those of the run's pages
            const int valid = min(n - j * kPage, min(NP, j1 - j) * kPage);
            if (bad_stages) {
                bad |= (bad_stages >> ws) & 1u;
                bad_stages &= ~(1u << ws);
            }
            if (valid > 0 && !bad) {
                // S = K Q^T: an accumulator per page and tile
                float sacc[NT][NP][4];
                uint32_t kw[NP][2][KW], ks[NP][2];
#pragma unroll
                for (int c = 0; c < NP; ++c) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sacc[nt][c][e] = 0.f;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int tok = r + 8 * half;
                        const uint8_t *row = stage + c * C::PAGE + tok * (D / 2);
                        if constexpr (D == 64) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(row + t4 * 8);
                            kw[c][half][0] = v.x;
                            kw[c][half][1] = v.y;
                        } else {
#pragma unroll
                            for (int p = 0; p < KW / 4; ++p) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(row + p * 64 + t4 * 16);
                                kw[c][half][4 * p] = v.x;
                                kw[c][half][4 * p + 1] = v.y;
                                kw[c][half][4 * p + 2] = v.z;
                                kw[c][half][4 * p + 3] = v.w;
                            }
                        }
                        // the token's scales for this lane's dims, in order
                        const uint8_t *sp = stage + c * C::PAGE + 16 * D + tok * (D / 16);
                        if constexpr (D == 64) {
                            ks[c][half] = sp[t4] * 0x101u;
                        } else if constexpr (D == 128) {
                            ks[c][half] = *reinterpret_cast<const uint16_t *>(sp + 2 * t4);
                        } else {
                            ks[c][half] = *reinterpret_cast<const uint16_t *>(sp + 2 * t4) |
                                          (static_cast<uint32_t>(
                                               *reinterpret_cast<const uint16_t *>(sp + 8 + 2 * t4))
                                           << 16);
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    // one word: eight codes of 8 dims = products 2w, 2w + 1; one scale
                    const int si = D == 64 ? 0 : w / 2;         // index of the word's scale
#pragma unroll
                    for (int c = 0; c < NP; ++c) {
                        uint32_t c0[4], c1[4];
                        e2m1x8_to_f16(kw[c][0][w], c0);
                        e2m1x8_to_f16(kw[c][1][w], c1);
                        const uint32_t p0 = e4m3x2_to_f16(ks[c][0] >> (16 * (si / 2)));
                        const uint32_t p1 = e4m3x2_to_f16(ks[c][1] >> (16 * (si / 2)));
                        const uint32_t f0 = __byte_perm(p0, p0, si & 1 ? 0x3232 : 0x1010);
                        const uint32_t f1 = __byte_perm(p1, p1, si & 1 ? 0x3232 : 0x1010);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t af[4] = {hmul2(c0[2 * q], f0), hmul2(c1[2 * q], f1),
                                                    hmul2(c0[2 * q + 1], f0),
                                                    hmul2(c1[2 * q + 1], f1)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(sacc[nt][c], af, qb[nt][2 * w + q][0], qb[nt][2 * w + q][1]);
                        }
                    }
                }
                // tokens r (0, 1) and r + 8 (2, 3); heads 2 t4 (0, 2) and 2 t4 + 1 (1, 3) of the tile
                if (valid < NP * kPage) {
#pragma unroll
                    for (int c = 0; c < NP; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (c * kPage + r + 8 * (e >> 1) >= valid)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    sacc[nt][c][e] = -INFINITY;
                }
                uint32_t pb[NT][NP][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float top[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[h] = fmaxf(sacc[nt][0][h], sacc[nt][0][h + 2]);
#pragma unroll
                        for (int c = 1; c < NP; ++c)
                            top[h] = fmax3(top[h], sacc[nt][c][h], sacc[nt][c][h + 2]);
                    }
                    if (__any_sync(0xffffffffu, top[0] > limit[nt][0] || top[1] > limit[nt][1])) {
                        float f[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float y = top[h];
#pragma unroll
                            for (int off = 4; off <= 16; off <<= 1)
                                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
                            y = fmaxf(y, ref[nt][h]);
                            f[h] = ex2_approx((ref[nt][h] - y) * sc[nt][h]);
                            ref[nt][h] = y;
                            limit[nt][h] = __fadd_rd(y, __fdiv_rd(kSlack, sc[nt][h]));
                            l_part[nt][h] *= f[h];
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[nt][mt][0] *= f[0];
                            o[nt][mt][1] *= f[1];
                            o[nt][mt][2] *= f[0];
                            o[nt][mt][3] *= f[1];
                        }
                    }
                    const f2 r2 = f2_pack(ref[nt][0], ref[nt][1]), s2 = f2_pack(sc[nt][0], sc[nt][1]);
                    const f2 shift = f2_pack(kPShift, kPShift);
#pragma unroll
                    for (int c = 0; c < NP; ++c) {
                        const float2 x = f2_unpack(f2_fma(f2_sub(f2_pack(sacc[nt][c][0], sacc[nt][c][1]), r2),
                                                          s2, shift));
                        const float2 z = f2_unpack(f2_fma(f2_sub(f2_pack(sacc[nt][c][2], sacc[nt][c][3]), r2),
                                                          s2, shift));
                        const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                        const float p2 = ex2_approx(z.x), p3 = ex2_approx(z.y);
                        l_part[nt][0] += p0 + p2;
                        l_part[nt][1] += p1 + p3;
                        pb[nt][c][0] = movm_t(pack_f16x2(p0, p1));
                        pb[nt][c][1] = movm_t(pack_f16x2(p2, p3));
                    }
                }

                // O^T += V^T P
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const uint8_t *page = stage + c * C::PAGE;
#pragma unroll
                    for (int p = 0; p < (D == 256 ? 2 : 1); ++p) {
                        const int grp = D == 64 ? r >> 1 : r + 8 * p;
                        uint32_t vs = *reinterpret_cast<const uint32_t *>(page + 17 * D + (grp * 4 + t4) * 4);
                        if (valid < NP * kPage) {
                            // unused rows may hold any bytes: their scales count as zero
                            const int rest = valid - c * kPage;
                            vs &= (2 * t4 < rest ? 0x000000ffu : 0u) |
                                  (2 * t4 + 1 < rest ? 0x0000ff00u : 0u) |
                                  (2 * t4 + 8 < rest ? 0x00ff0000u : 0u) |
                                  (2 * t4 + 9 < rest ? 0xff000000u : 0u);
                        }
                        const uint32_t f0 = e4m3x2_to_f16(vs & 0xffffu), f1 = e4m3x2_to_f16(vs >> 16);
                        uint32_t even[2][2], odd[2][2];         // [token half][code word]
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if constexpr (D == 64) {
                                const uint2 v =
                                    *reinterpret_cast<const uint2 *>(page + 8 * D + half * 256 + lane * 8);
                                even[half][0] = v.x;
                                odd[half][0] = v.y;
                            } else {
                                const uint4 v = *reinterpret_cast<const uint4 *>(
                                    page + 8 * D + (half * (D / 128) + p) * 512 + lane * 16);
                                even[half][0] = v.x;
                                even[half][1] = v.y;
                                odd[half][0] = v.z;
                                odd[half][1] = v.w;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < (D == 64 ? 1 : 2); ++w) {
                            // codes of eight dims paired by token: (even, odd) per byte
                            uint32_t a0[4], a1[4], a2[4], a3[4];
                            const uint32_t M = 0x0f0f0f0fu;
                            e2m1x8_to_f16((even[0][w] & M) | ((odd[0][w] << 4) & ~M), a0);
                            e2m1x8_to_f16(((even[0][w] >> 4) & M) | (odd[0][w] & ~M), a1);
                            e2m1x8_to_f16((even[1][w] & M) | ((odd[1][w] << 4) & ~M), a2);
                            e2m1x8_to_f16(((even[1][w] >> 4) & M) | (odd[1][w] & ~M), a3);
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const uint32_t af[4] = {hmul2(a0[b], f0), hmul2(a1[b], f0),
                                                        hmul2(a2[b], f1), hmul2(a3[b], f1)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_f16(o[nt][8 * p + 4 * w + b], af, pb[nt][c][0], pb[nt][c][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();                           // every lane is done with the stage: refill it
            issue(ws);
            ws = ws + 1 == C::WS ? 0 : ws + 1;
        }

        // ------------------------------------------------ end of the segment
        MergeArea<C::HEADS> &mg = merge[area];
        float *s_o = outs + area * kConsumers * G * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1)
                    l_part[nt][h] += __shfl_xor_sync(0xffffffffu, l_part[nt][h], off);
                if (lane < 4) {
                    mg.m[warp][nt * kTile + 2 * lane + h] = ref[nt][h];
                    if (warp == 0)
                        mg.scale[nt * kTile + 2 * lane + h] = sc[nt][h];
                    mg.l[warp][nt * kTile + 2 * lane + h] = l_part[nt][h];
                }
            }
            // o[mt]: dims of run r: 16 (r + 8 p) + 2 b (D = 64: 8 r + 2 b) in c0, c1, the next in c2, c3
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int d = D == 64 ? r * 8 + 2 * mt : (r + 8 * (mt >> 3)) * 16 + 2 * (mt & 7);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int g = nt * kTile + 2 * t4 + h;
                    if (g < G)
                        *reinterpret_cast<float2 *>(&s_o[(warp * G + g) * D + d]) =
                            make_float2(o[nt][mt][h], o[nt][mt][2 + h]);
                }
            }
        }
        if (lane == 0)
            mg.bad[warp] = bad;
        __syncthreads();
        bad = mg.bad[0] || mg.bad[1] || mg.bad[2] || mg.bad[3];
        const bool whole = j0 == 0 && j1 == seg.pages;
        // The warps' states merged: four dims per thread and turn.
        float *part = a.part + (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * PART +
                      (first_segment ? 0 : PART);
        auto finish = [&](int g, int d, float4 v, float m, float l) {
            const long long out_row = static_cast<long long>(s) * a.num_q_heads + h0 + g;
            const float f = l == 0.f ? 0.f : a.descale_v / l;       // no token
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + out_row * D + d) =
                make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
            if (d == 0 && a.lse)
                a.lse[out_row] = l == 0.f ? -FLT_MAX : (m * mg.scale[g] - kPShift + __log2f(l)) * kLn2;
        };
        for (int e = 4 * tid; e < G * D; e += 4 * kDecThreads) {
            const int g = e / D, d = e % D;
            const float mt = fmaxf(fmaxf(mg.m[0][g], mg.m[1][g]), fmaxf(mg.m[2][g], mg.m[3][g]));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
                const float f = ex2_approx((mg.m[w][g] - mt) * mg.scale[g]);
                const float4 v = *reinterpret_cast<const float4 *>(&s_o[(w * G + g) * D + d]);
                acc.x = fmaf(v.x, f, acc.x);
                acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z);
                acc.w = fmaf(v.w, f, acc.w);
                l = fmaf(mg.l[w][g], f, l);
            }
            if (!whole) {
                float *q = part + g * (D + 4);
                __stcg(reinterpret_cast<float4 *>(q + d), acc);
                if (d == 0)                         // a sum is never negative
                    __stcg(reinterpret_cast<float2 *>(q + D), make_float2(mt, bad ? -1.f : l));
            } else if (!bad) {
                finish(g, d, acc, mt, l);
            }
        }
        if (!whole) {
            // runs with pages of this sequence
            const int p0 = seg.at + kSeqUnits;
            const int xa = p0 / run, parts = (p0 + seg.pages - 1) / run - xa + 1;
            int32_t *ticket = a.tickets + static_cast<long long>(s) * gridDim.y + blockIdx.y;
            __syncthreads();                        // every thread's part is written
            if (tid == 0) {
                __threadfence();
                s_last = atomicAdd(ticket, 1) == parts - 1;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                // run xa holds it in its second slot if it has pages of an earlier one
                const float *base = a.part + static_cast<long long>(blockIdx.y) * gridDim.x * 2 * PART;
                const int late = seg.at > xa * run;
                for (int e = 4 * tid; e < G * D; e += 4 * kDecThreads) {
                    const int g = e / D, d = e % D;
                    const float scale = mg.scale[g];
                    float mt = kNoRef, l = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    bool any_bad = false;
                    constexpr int B = 8;            // parts whose loads are in flight together
                    for (int x0 = 0; x0 < parts; x0 += B) {
                        float4 v[B];
                        float2 ml[B];
#pragma unroll
                        for (int x = 0; x < B; ++x) {
                            ml[x] = make_float2(kNoRef, 0.f);
                            v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (x0 + x < parts) {
                                const float *q = base + (static_cast<long long>(xa + x0 + x) * 2 +
                                                         (x0 + x == 0 ? late : 0)) * PART + g * (D + 4);
                                v[x] = __ldcg(reinterpret_cast<const float4 *>(q + d));
                                ml[x] = __ldcg(reinterpret_cast<const float2 *>(q + D));
                            }
                        }
                        float mn = mt;
#pragma unroll
                        for (int x = 0; x < B; ++x)
                            mn = fmaxf(mn, ml[x].x);
                        const float keep = ex2_approx((mt - mn) * scale);
                        mt = mn;
                        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
                        l *= keep;
#pragma unroll
                        for (int x = 0; x < B; ++x) {
                            const float f = ex2_approx((ml[x].x - mn) * scale);
                            any_bad |= ml[x].y < 0.f;
                            acc.x = fmaf(v[x].x, f, acc.x);
                            acc.y = fmaf(v[x].y, f, acc.y);
                            acc.z = fmaf(v[x].z, f, acc.z);
                            acc.w = fmaf(v[x].w, f, acc.w);
                            l = fmaf(ml[x].y, f, l);
                        }
                    }
                    if (!any_bad)
                        finish(g, d, acc, mt, l);
                }
                if (tid == 0)
                    *ticket = 0;                    // ready for the next call
            }
        }
        if constexpr (C::AREAS == 1)
            __syncthreads();                        // the area is free again
        else
            area ^= 1;      // (read again only behind the next segment's barrier)
        first_segment = false;
    } while (seg.next(a, u0, u1));
}

template <int D, int NT>
cudaError_t launch_decode_dn(const Kv4DecodeArgs &a, int sm_count, cudaStream_t stream)
{
    using C = DecCfg<D, NT>;
    const int group = a.num_q_heads / a.num_kv_heads;
    const int rows = a.num_kv_heads * ((group + C::HEADS - 1) / C::HEADS);
    const int heads = group < C::HEADS ? group : C::HEADS;
    const size_t smem = static_cast<size_t>(C::NS) * C::STAGE +
                        static_cast<size_t>(C::AREAS) * kConsumers * heads * D * sizeof(float);
    // the largest size any call needs, once per device
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(kv4_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::NS * C::STAGE +
                                     C::AREAS * kConsumers * C::HEADS * D *
                                         static_cast<int>(sizeof(float)));
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            attr_done[dev] = 1;
    }
    // as many CTAs as fit on the SMs; runs of at least kMinRun pages
    // (228 KB per SM; 2 KB covers a CTA's static and reserved shared memory)
    const long long by_smem = (228 * 1024) / (static_cast<long long>(smem) + 2048);
    const long long fit = (by_smem < C::CTAS ? by_smem : C::CTAS) * sm_count;
    const long long ctas = fit < kMaxCtas ? fit : kMaxCtas;
    long long parts = ctas / rows;
    const long long most = (static_cast<long long>(a.num_seqs) *
                                (kSeqUnits + (a.capacity > 0 ? a.capacity : 1)) +
                            kMinRun - 1) / kMinRun;
    parts = parts < most ? parts : most;
    // One CTA merges a sequence's parts, 8 per load latency: up to 256 runs where
    // a sequence may take them all, 8 per sequence where there are many (one kv
    // head, 64 contexts of 15-30k tokens of 128: 59 us with 256 runs, 51 with 456).
    const long long cap = 8LL * a.num_seqs > 256 ? 8LL * a.num_seqs : 256;
    parts = parts < 1 ? 1 : (parts > cap ? cap : parts);
    return launch_dependent(kv4_decode_kernel<D, NT>, dim3(static_cast<int>(parts), rows), kDecThreads,
                            smem, stream, a);
}

template <int D>
cudaError_t launch_decode_d(const Kv4DecodeArgs &a, int sm_count, cudaStream_t stream)
{
    if constexpr (D <= 128)
        if (head_tiles(a.num_q_heads / a.num_kv_heads, D) == 2)
            return launch_decode_dn<D, 2>(a, sm_count, stream);
    return launch_decode_dn<D, 1>(a, sm_count, stream);
}

// CTAs over the tokens; with too few tokens for every SM, CTAs share the kv
// heads too, kMoveAhead of them each at least.
dim3 move_grid(const Kv4MoveArgs &a, int head_dim, int sm_count)
{
    const int tokens = 32 / (head_dim / 16) * kMoveWarps;       // of a CTA
    long long x = (static_cast<long long>(a.total) + tokens - 1) / tokens;
    const long long most = 64LL * sm_count;
    x = x < most ? x : most;
    long long y = sm_count / x;
    const long long shares = (a.num_kv_heads + kMoveAhead - 1) / kMoveAhead;
    y = y < 1 ? 1 : (y < shares ? y : shares);
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

// The workspace: partial states, then the tickets.  Where the tickets start
// does not depend on the number of sequences, so a workspace made for a batch
// serves smaller ones too.
size_t part_bytes(int rows, int tiles, int head_dim)
{
    const size_t runs = rows > kMaxCtas ? rows : kMaxCtas;      // in all rows
    const size_t n = runs * 2 * tiles * kTile * (head_dim + 4) * sizeof(float);
    return (n + 255) & ~static_cast<size_t>(255);
}

}  // namespace

cudaError_t launch_kv4_write(int head_dim, const Kv4MoveArgs &a, int sm_count, cudaStream_t stream)
{
    const dim3 grid = move_grid(a, head_dim, sm_count);
    switch (head_dim) {
    case 64: return launch_dependent(kv4_write_kernel<64>, grid, kMoveWarps * 32, 0, stream, a);
    case 128: return launch_dependent(kv4_write_kernel<128>, grid, kMoveWarps * 32, 0, stream, a);
    case 256: return launch_dependent(kv4_write_kernel<256>, grid, kMoveWarps * 32, 0, stream, a);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv4_gather(int head_dim, const Kv4MoveArgs &a, int sm_count,
                              cudaStream_t stream)
{
    const dim3 grid = move_grid(a, head_dim, sm_count);
    switch (head_dim) {
    case 64: return launch_dependent(kv4_gather_kernel<64>, grid, kMoveWarps * 32, 0, stream, a);
    case 128: return launch_dependent(kv4_gather_kernel<128>, grid, kMoveWarps * 32, 0, stream, a);
    case 256: return launch_dependent(kv4_gather_kernel<256>, grid, kMoveWarps * 32, 0, stream, a);
    default: return cudaErrorInvalidValue;
    }
}

size_t kv4_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim)
{
    const int group = num_q_heads / num_kv_heads;
    const int tiles = head_tiles(group, head_dim);
    const int rows = num_kv_heads * ((group + tiles * kTile - 1) / (tiles * kTile));
    return part_bytes(rows, tiles, head_dim) + static_cast<size_t>(num_seqs) * rows * sizeof(int32_t);
}

cudaError_t launch_kv4_decode(int head_dim, Kv4DecodeArgs &a, void *workspace, int sm_count,
                              cudaStream_t stream)
{
    const int group = a.num_q_heads / a.num_kv_heads;
    const int tiles = head_tiles(group, head_dim);
    const int rows = a.num_kv_heads * ((group + tiles * kTile - 1) / (tiles * kTile));
    a.part = static_cast<float *>(workspace);
    a.tickets = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) +
                                            part_bytes(rows, tiles, head_dim));
    switch (head_dim) {
    case 64: return launch_decode_d<64>(a, sm_count, stream);
    case 128: return launch_decode_d<128>(a, sm_count, stream);
    case 256: return launch_decode_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
