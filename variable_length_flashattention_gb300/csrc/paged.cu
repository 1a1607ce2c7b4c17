// paged.cu -- attention of one new token per sequence over a paged bf16 cache,
// in one launch: sliding window, sinks, and the weight every cached token got.
//
// With n = counts[s] the query is the token at n - 1: it sees the tokens j < n
// with j >= n - 1 - window_left or j < sink_tokens.
//   out[s, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j)
// Online softmax over the pages that hold such tokens, the query heads of a kv
// head together, up to 8 as the columns of one tile; more are more head chunks,
// whose pages come from L2.
//
// Work.  The pages a sequence reads are its sinks' and its window's, in one
// row; kSeqUnits stand for its start and end.  The batch's units are cut into
// equal runs, one per CTA, so that long and short contexts load every SM alike;
// a sequence whose pages lie in one run is finished there, the others leave
// partial states (m, l, o), merged in a fixed order by the CTA that takes the
// last ticket.  No CTA waits for another.
//
// Warp w takes every fourth group of NP of the run's pages and copies them
// ahead into its own ring of shared-memory stages with 16-byte asynchronous
// copies (it alone reads what it copied: no barrier).  Rows of a page are
// swizzled by 16-byte chunk so that ldmatrix reads them without conflicts.  Per
// page, two products on mma.sync m16n8k16 (bf16 in, fp32 accumulate):
//   S[16 tokens x 8 heads] = K Q^T    O^T[D x 8 heads] += V^T P
// Weights are relative to a reference, the maximum when it was last taken,
// renewed when a weight would pass it by more than 2^kSlack; it stays in units
// of the accumulators, whose difference is taken before the scale.  p is
// rounded to bf16 for the second product (half a step, 2^-8); a third product
// with what the rounding leaves would make up for it and cost 0.5 to 3% (64 sequences of
// 1000-8000 tokens, 32 heads on 8 of 128: 181.1 us against 180; 256 of 1000 with a window of
// 255, 64 on 8: 79.2 against 76.5), for an error that the rounding of the output to
// bf16 has anyway; l, the reference and o are fp32.  What a page holds in hidden or unused slots does
// not matter: their logits are replaced, and their rows of V read as zeros.
//
// Key weights.  A token's weight needs the whole sum, which is there when its
// row of the batch ends.  The logits (4 bytes per token and query head; K and V
// are 4 D bytes per token and kv head) go to the workspace on the way, with m and l
// of every row, and a second kernel adds the weights of a kv head's query heads to
// the token's.
#include <cfloat>
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace vfa {

namespace {

constexpr int kPage = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 8;                // query heads of a CTA
constexpr int kSeqUnits = 12;           // units of a sequence besides its pages
constexpr int kMinRun = 12;             // units per CTA at least
constexpr int kMaxCtas = 1024;          // CTAs in all rows, where there are fewer rows
constexpr float kSlack = 8.f;           // log2
constexpr float kNoRef = -FLT_MAX;         // stands for a maximum that is not there yet
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
    static constexpr int NP = D == 64 ? 2 : 1;                  // pages of a group
    static constexpr int HALF = kPage * D * 2;                  // bytes of a page's K or V
    static constexpr int PAGE = 2 * HALF;
    static constexpr int STAGE = NP * PAGE;
    static constexpr int WS = D == 256 ? 2 : 3;                 // stages of a warp
    static constexpr int RING = kWarps * WS * STAGE;
    static constexpr int CTAS = D == 256 ? 1 : 2;               // resident per SM
    static constexpr int AREAS = D == 256 ? 1 : 2;              // merge areas
    static constexpr int MT = D / 16;
    static constexpr int PART = kTile * (D + 4);                // floats of a part
};

__device__ __forceinline__ void record(int32_t *status, int code)
{
    if (status)
        atomicCAS(status, 0, code);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What of a sequence is read: `pages` pages in a row (1 if it is empty), of
// which the first `sinks` are its first pages and the others those from
// sinks + skip on.
struct View {
    int tokens, lo, pages, sinks, skip;       // lo: the window's first token
    bool bad;

    __device__ __forceinline__ int page(int j) const { return j < sinks ? j : j + skip; }
};

__device__ __forceinline__ View view_of(const PagedDecodeArgs &a, int s)
{
    View v;
    const int n = __ldg(a.counts + s);
    v.bad = n < 0 || n > static_cast<long long>(a.capacity) * kPage;
    v.tokens = v.bad ? 0 : n;
    v.lo = a.window_left < 0 ? 0 : max(0, v.tokens - 1 - a.window_left);
    const int first = v.lo / kPage;
    v.sinks = min(first, (min(a.sink_tokens, v.tokens) + kPage - 1) / kPage);
    v.skip = first - v.sinks;
    v.pages = max(1, v.sinks + (v.tokens + kPage - 1) / kPage - first);
    return v;
}

// The tokens of page `page` that the query sees, one bit each.
__device__ __forceinline__ uint32_t visible(const PagedDecodeArgs &a, const View &v, int page)
{
    const int base = page * kPage;
    auto below = [&](int x) { return (1u << min(kPage, max(0, x - base))) - 1u; };
    return below(v.tokens) & (~below(v.lo) | below(a.sink_tokens));
}

// A place in the CTA's run [u0, u1): the segment of sequence s whose units
// start at `at` (kSeqUnits, then its pages), the run's pages [j0, j1) of it, and
// (modulo 4) the groups of NP pages of the earlier segments, which decide the warp
// that takes its first group.
template <int NP>
struct Cursor {
    View v;
    int s, at, j0, j1, base;

    // The first segment with pages in the run from sequence s on; false if none.
    __device__ __forceinline__ bool enter(const PagedDecodeArgs &a, int u0, int u1)
    {
        for (; at + kSeqUnits < u1; ++s) {
            v = view_of(a, s);
            const int p0 = at + kSeqUnits;
            j0 = max(0, u0 - p0);
            j1 = min(v.pages, u1 - p0);
            if (j0 < j1)
                return true;
            at = p0 + v.pages;
        }
        return false;
    }
    // First page of `warp`'s first group of the segment (at or past j1: none).
    __device__ __forceinline__ int first(int warp) const
    {
        return j0 + NP * ((warp - base) & (kWarps - 1));
    }
    // The next segment; false at the end of the run.
    __device__ __forceinline__ bool next(const PagedDecodeArgs &a, int u0, int u1)
    {
        base += (j1 - j0 + NP - 1) / NP;
        at += kSeqUnits + v.pages;
        ++s;
        return enter(a, u0, u1);
    }
};

// What the warps of a CTA leave at the end of a segment, besides their outputs.
struct MergeArea {
    float m[kWarps][kTile], l[kWarps][kTile];
    int bad[kWarps];
};

template <int D, bool LOGITS>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS) paged_decode_kernel(const PagedDecodeArgs a)
{
    using C = Cfg<D>;
    constexpr int NP = C::NP, MT = C::MT, PART = C::PART, WS = C::WS;
    constexpr int STRIDE = NP * kWarps;             // pages from a warp's group to its next
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ MergeArea merge[C::AREAS];
    __shared__ int s_scan[kWarps];
    __shared__ int s_first, s_first_unit, s_last;

    grid_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.num_q_heads / a.num_kv_heads;
    const int chunks = (group + kTile - 1) / kTile;
    const int kh = blockIdx.y / chunks;
    const int h0 = kh * group + (blockIdx.y % chunks) * kTile;      // first query head
    const int G = min(kTile, (kh + 1) * group - h0);

    // Units before each thread's share of the sequences.
    const int per = (a.num_seqs + kThreads - 1) / kThreads;
    const int sa = min(a.num_seqs, tid * per), sb = min(a.num_seqs, sa + per);
    int mine = 0;
    for (int s = sa; s < sb; ++s)
        mine += kSeqUnits + view_of(a, s).pages;
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
    for (int i = 0; i < kWarps; ++i) {
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
            const int u = kSeqUnits + view_of(a, s).pages;
            if (u0 < at + u) {
                s_first = s;
                s_first_unit = at;
                break;
            }
            at += u;
        }
    }
    __syncthreads();

    // ---------------------------------------------------- copies
    // Fills of this warp's stages, WS groups ahead.  The ids of its next groups
    // in segment `fill`, up to 32 pages, are loaded and checked together: lane l
    // holds page l % NP of group l / NP.  Where there is no page (a last group's
    // rest, an empty sequence) or the id is bad, page 0 is copied in its place
    // and not used.  Every turn commits one group of copies, also where there is
    // nothing left to copy.
    Cursor<NP> fill;
    fill.s = s_first;
    fill.at = s_first_unit;
    fill.base = 0;
    if (!fill.enter(a, u0, u1))
        return;                                     // (the whole CTA) no page in this run
    Cursor<NP> seg = fill;
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
        const bool listed = j < fill.j1 && fill.v.tokens > 0;
        ids = listed ? __ldg(a.tables + static_cast<long long>(fill.s) * a.capacity + fill.v.page(j)) : 0;
        const bool bad = static_cast<unsigned>(ids) >= static_cast<unsigned>(a.num_blocks);
        bad_ids = __ballot_sync(0xffffffffu, bad && listed);
        ids = bad ? 0 : ids;
        id_lane = 0;
        ahead += (32 / NP) * STRIDE;
    };
    // A lane copies chunk `chunk` of rows row0, row0 + ROWS, ... of K and of V.
    constexpr int CHUNKS = D / 8, ROWS = CHUNKS < 32 ? 32 / CHUNKS : 1, TURNS = kPage / ROWS;
    const int row0 = lane / CHUNKS, chunk = lane % CHUNKS;
    const size_t row_bytes = static_cast<size_t>(a.num_kv_heads) * D * 2;
    const size_t page_bytes = row_bytes * kPage;
    const size_t my_at = static_cast<size_t>(kh) * D * 2 + row0 * row_bytes + chunk * 16;
    const uint8_t *my_k = static_cast<const uint8_t *>(a.k_pool) + my_at;
    const uint8_t *my_v = static_cast<const uint8_t *>(a.v_pool) + my_at;
    const uint32_t my_ring = smem_u32(dsm) + warp * WS * C::STAGE;
    const bool pages_exist = a.num_blocks > 0;
    auto issue = [&](int ws) {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const size_t at = __shfl_sync(0xffffffffu, ids, id_lane + i) * page_bytes;
                const uint32_t dst = my_ring + ws * C::STAGE + i * C::PAGE;
                if (pages_exist) {
#pragma unroll
                    for (int t = 0; t < TURNS; ++t) {
                        const int row = row0 + t * ROWS;
                        const uint32_t to = dst + row * (D * 2) + ((chunk ^ (row & 7)) << 4);
                        copy16(to, my_k + at + t * ROWS * row_bytes);
                        copy16(to + C::HALF, my_v + at + t * ROWS * row_bytes);
                    }
                }
            }
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
    for (int k = 0; k < WS; ++k)
        issue(k);

    // ---------------------------------------------------- attention
    const int r = lane >> 2, t4 = lane & 3;
    float *const outs = reinterpret_cast<float *>(dsm + C::RING);      // [AREAS][kWarps][G][D]
    const float sc = a.scale_log2;
    // ldmatrix rows: lane L serves row L % 8 of 8x8 matrix L / 8
    const int mi = lane >> 3, mr = lane & 7;
    const int k_row = ((mi & 1) << 3) + mr, k_chunk = mi >> 1;          // K: A of S = K Q^T
    const int v_row = ((mi >> 1) << 3) + mr, v_chunk = mi & 1;          // V^T: A of O^T += V^T P
    int ws = 0;                                     // stage of this warp's next group
    int area = 0;                                   // of this segment's merge
    bool first_segment = true;
    do {
        const int s = seg.s, j0 = seg.j0, j1 = seg.j1;
        const View v = seg.v;
        if (v.bad && tid == 0)
            record(a.status, VFA_ERR_BAD_BLOCK);

        // Q^T operands: head r, columns 16 kt + 2 t4 + {0, 1} and + 8
        uint32_t qb[MT][2];
        {
            const uint32_t *qrow = reinterpret_cast<const uint32_t *>(
                static_cast<const __nv_bfloat16 *>(a.q) +
                (static_cast<long long>(s) * a.num_q_heads + h0 + (r < G ? r : 0)) * D);
#pragma unroll
            for (int kt = 0; kt < MT; ++kt) {
                qb[kt][0] = r < G ? __ldg(qrow + 8 * kt + t4) : 0u;
                qb[kt][1] = r < G ? __ldg(qrow + 8 * kt + 4 + t4) : 0u;
            }
        }
        // of this lane's heads, 2 t4 and 2 t4 + 1: the reference, the logit that renews it
        // (both before the scale), the sum
        float ref[2] = {kNoRef, kNoRef}, limit[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.f, 0.f};
        float o[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[mt][e] = 0.f;
        bool bad = v.bad;

        for (int j = seg.first(warp); j < j1; j += STRIDE) {
            copy_wait<WS - 1>();
            __syncwarp();                           // every lane's copies are there for every lane
            const uint32_t stage = my_ring + ws * C::STAGE;
            if (bad_stages) {
                bad |= (bad_stages >> ws) & 1u;
                bad_stages &= ~(1u << ws);
            }
            if (v.tokens > 0 && !bad) {
                uint32_t vis[NP];
#pragma unroll
                for (int c = 0; c < NP; ++c)
                    vis[c] = j + c < j1 ? visible(a, v, v.page(j + c)) : 0u;
                float sacc[NP][4];
#pragma unroll
                for (int c = 0; c < NP; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sacc[c][e] = 0.f;
#pragma unroll
                for (int kt = 0; kt < MT; ++kt)
#pragma unroll
                    for (int c = 0; c < NP; ++c) {
                        uint32_t af[4];
                        ldsm_x4(stage + c * C::PAGE + k_row * (D * 2) +
                                    (((2 * kt + k_chunk) ^ (k_row & 7)) << 4), af);
                        mma_bf16(sacc[c], af, qb[kt][0], qb[kt][1]);
                    }
                // tokens r (0, 1) and r + 8 (2, 3); heads 2 t4 (0, 2) and 2 t4 + 1 (1, 3)
                if constexpr (LOGITS) {
#pragma unroll
                    for (int c = 0; c < NP; ++c)
                        if (j + c < j1) {
                            float *row = a.logits +
                                         ((static_cast<long long>(s) * a.num_kv_heads + kh) * a.max_pages +
                                          j + c) * (kPage * group) + r * group + (h0 - kh * group) + 2 * t4;
                            if (2 * t4 < G) {
                                __stcg(row, sacc[c][0]);
                                __stcg(row + 8 * group, sacc[c][2]);
                            }
                            if (2 * t4 + 1 < G) {
                                __stcg(row + 1, sacc[c][1]);
                                __stcg(row + 8 * group + 1, sacc[c][3]);
                            }
                        }
                }
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    if (vis[c] != 0xffffu) {
                        const bool a0 = vis[c] >> r & 1u, a1 = vis[c] >> (r + 8) & 1u;
                        sacc[c][0] = a0 ? sacc[c][0] : -INFINITY;
                        sacc[c][1] = a0 ? sacc[c][1] : -INFINITY;
                        sacc[c][2] = a1 ? sacc[c][2] : -INFINITY;
                        sacc[c][3] = a1 ? sacc[c][3] : -INFINITY;
                    }
                    top[0] = fmax3(top[0], sacc[c][0], sacc[c][2]);
                    top[1] = fmax3(top[1], sacc[c][1], sacc[c][3]);
                }
                if (__any_sync(0xffffffffu, top[0] > limit[0] || top[1] > limit[1])) {
                    float f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float y = top[h];
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1)
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
                        y = fmaxf(y, ref[h]);
                        f[h] = ex2_approx((ref[h] - y) * sc);
                        ref[h] = y;
                        limit[h] = __fadd_rd(y, __fdiv_rd(kSlack, sc));
                        l_part[h] *= f[h];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[mt][0] *= f[0];
                        o[mt][1] *= f[1];
                        o[mt][2] *= f[0];
                        o[mt][3] *= f[1];
                    }
                }
                uint32_t pb[NP][2];
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const float p0 = ex2_approx((sacc[c][0] - ref[0]) * sc);
                    const float p1 = ex2_approx((sacc[c][1] - ref[1]) * sc);
                    const float p2 = ex2_approx((sacc[c][2] - ref[0]) * sc);
                    const float p3 = ex2_approx((sacc[c][3] - ref[1]) * sc);
                    l_part[0] += p0 + p2;
                    l_part[1] += p1 + p3;
                    pb[c][0] = movm_t(pack_bf16x2(p0, p1));
                    pb[c][1] = movm_t(pack_bf16x2(p2, p3));
                }
                // O^T += V^T P; a lane's operand holds tokens 2 t4, 2 t4 + 1 and those + 8
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    if (vis[c] == 0xffffu) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t af[4];
                            ldsm_x4_t(stage + c * C::PAGE + C::HALF + v_row * (D * 2) +
                                          (((2 * mt + v_chunk) ^ (v_row & 7)) << 4), af);
                            mma_bf16(o[mt], af, pb[c][0], pb[c][1]);
                        }
                    } else if (vis[c] != 0) {
                        const uint32_t two = vis[c] >> (2 * t4);
                        const uint32_t lo = (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
                        const uint32_t hi = (two & 0x100u ? 0xffffu : 0u) |
                                            (two & 0x200u ? 0xffff0000u : 0u);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t af[4];
                            ldsm_x4_t(stage + c * C::PAGE + C::HALF + v_row * (D * 2) +
                                          (((2 * mt + v_chunk) ^ (v_row & 7)) << 4), af);
                            af[0] &= lo;
                            af[1] &= lo;
                            af[2] &= hi;
                            af[3] &= hi;
                            mma_bf16(o[mt], af, pb[c][0], pb[c][1]);
                        }
                    }
                }
            }
            __syncwarp();                           // every lane is done with the stage: refill it
            issue(ws);
            ws = ws + 1 == WS ? 0 : ws + 1;
        }

        // ------------------------------------------------ end of the segment
        MergeArea &mg = merge[area];
        float *s_o = outs + area * kWarps * G * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1)
                l_part[h] += __shfl_xor_sync(0xffffffffu, l_part[h], off);
            if (lane < 4) {
                mg.m[warp][2 * lane + h] = ref[h];
                mg.l[warp][2 * lane + h] = l_part[h];
            }
        }
        // o[mt]: columns 16 mt + r (0, 1) and + 8 (2, 3); heads 2 t4 (0, 2), 2 t4 + 1 (1, 3)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int g = 2 * t4 + (e & 1);
                if (g < G)
                    s_o[(warp * G + g) * D + 16 * mt + r + ((e >> 1) << 3)] = o[mt][e];
            }
        if (lane == 0)
            mg.bad[warp] = bad;
        __syncthreads();
        bad = mg.bad[0] || mg.bad[1] || mg.bad[2] || mg.bad[3];
        const bool whole = j0 == 0 && j1 == v.pages;
        float *part = a.part + (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * PART +
                      (first_segment ? 0 : PART);
        auto finish = [&](int g, int d, float4 y, float m, float l, bool failed) {
            const long long out_row = static_cast<long long>(s) * a.num_q_heads + h0 + g;
            if (!failed) {
                const float f = l == 0.f ? 0.f : 1.f / l;           // no token
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + out_row * D + d) =
                    make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
            }
            if (d == 0) {
                if (a.lse && !failed)
                    a.lse[out_row] = l == 0.f ? -FLT_MAX : (m * sc + __log2f(l)) * kLn2;
                if constexpr (LOGITS)
                    a.ml[out_row] = make_float2(m, failed ? -1.f : l);
            }
        };
        for (int e = 4 * tid; e < G * D; e += 4 * kThreads) {
            const int g = e / D, d = e % D;
            const float mt = fmaxf(fmaxf(mg.m[0][g], mg.m[1][g]), fmaxf(mg.m[2][g], mg.m[3][g]));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx((mg.m[w][g] - mt) * sc);
                const float4 y = *reinterpret_cast<const float4 *>(&s_o[(w * G + g) * D + d]);
                acc.x = fmaf(y.x, f, acc.x);
                acc.y = fmaf(y.y, f, acc.y);
                acc.z = fmaf(y.z, f, acc.z);
                acc.w = fmaf(y.w, f, acc.w);
                l = fmaf(mg.l[w][g], f, l);
            }
            if (!whole) {
                float *q = part + g * (D + 4);
                __stcg(reinterpret_cast<float4 *>(q + d), acc);
                if (d == 0)                         // a sum is never negative
                    __stcg(reinterpret_cast<float2 *>(q + D), make_float2(mt, bad ? -1.f : l));
            } else {
                finish(g, d, acc, mt, l, bad);
            }
        }
        if (!whole) {
            // runs with pages of this sequence
            const int p0 = seg.at + kSeqUnits;
            const int xa = p0 / run, parts = (p0 + v.pages - 1) / run - xa + 1;
            // (a run holds the first pages of one such sequence at most)
            int32_t *ticket = a.tickets + static_cast<long long>(blockIdx.y) * gridDim.x + xa;
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
                for (int e = 4 * tid; e < G * D; e += 4 * kThreads) {
                    const int g = e / D, d = e % D;
                    float mt = kNoRef, l = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    bool any_bad = false;
                    constexpr int B = 8;            // parts whose loads are in flight together
                    for (int x0 = 0; x0 < parts; x0 += B) {
                        float4 y[B];
                        float2 ml[B];
#pragma unroll
                        for (int i = 0; i < B; ++i) {
                            ml[i] = make_float2(kNoRef, 0.f);
                            y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (x0 + i < parts) {
                                const float *q = base + (static_cast<long long>(xa + x0 + i) * 2 +
                                                         (x0 + i == 0 ? late : 0)) * PART + g * (D + 4);
                                y[i] = __ldcg(reinterpret_cast<const float4 *>(q + d));
                                ml[i] = __ldcg(reinterpret_cast<const float2 *>(q + D));
                            }
                        }
                        float mn = mt;
#pragma unroll
                        for (int i = 0; i < B; ++i)
                            mn = fmaxf(mn, ml[i].x);
                        const float keep = ex2_approx((mt - mn) * sc);
                        mt = mn;
                        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
                        l *= keep;
#pragma unroll
                        for (int i = 0; i < B; ++i) {
                            const float f = ex2_approx((ml[i].x - mn) * sc);
                            any_bad |= ml[i].y < 0.f;
                            acc.x = fmaf(y[i].x, f, acc.x);
                            acc.y = fmaf(y[i].y, f, acc.y);
                            acc.z = fmaf(y[i].z, f, acc.z);
                            acc.w = fmaf(y[i].w, f, acc.w);
                            l = fmaf(ml[i].y, f, l);
                        }
                    }
                    finish(g, d, acc, mt, l, any_bad);
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

// ------------------------------------------------------------ key weights
//
// weights_out = weights + the sum over a kv head's query heads of exp(logit) / l,
// one thread per visible token, CTAs (row, split) with row = (sequence, kv head).
// Bound: HBM, 8 bytes per token and kv head and 4 per query head.
// The heads' references and sums are the same for a CTA's tokens and wait in shared
// memory; a thread has kWeightTurns tokens' logits in flight.
constexpr int kWeightThreads = 256, kWeightTurns = 4, kWeightHeads = 64;

// The logits of a token's query heads, N at a time.
template <int N>
__device__ __forceinline__ void load_logits(const float *x, float (&v)[N])
{
    if constexpr (N == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4 *>(x));
        v[0] = y.x;
        v[1] = y.y;
        v[2] = y.z;
        v[3] = y.w;
    } else {
        v[0] = __ldcg(x);
    }
}

// N: query heads loaded together (4 where the group is a multiple of it).
template <int N>
__global__ void __launch_bounds__(kWeightThreads) paged_weights_kernel(const PagedDecodeArgs a)
{
    grid_wait();
    __shared__ float2 s_ml[kWeightHeads];               // reference, 1 / sum
    __shared__ int s_bad;
    const int s = blockIdx.x / a.num_kv_heads, kh = blockIdx.x % a.num_kv_heads;
    const int group = a.num_q_heads / a.num_kv_heads;
    const View v = view_of(a, s);
    const long long row = blockIdx.x;
    const float2 *ml = a.ml + static_cast<long long>(s) * a.num_q_heads + kh * group;
    const int end = v.tokens > 0 ? v.pages * kPage : 0;
    const int step = gridDim.y * kWeightThreads;
    if (blockIdx.y * kWeightThreads >= end)
        return;
    if (threadIdx.x == 0)
        s_bad = 0;
    __syncthreads();
    for (int h = threadIdx.x; h < group; h += kWeightThreads) {
        const float2 q = __ldcg(ml + h);
        if (q.y < 0.f)
            s_bad = 1;
        if (h < kWeightHeads)
            s_ml[h] = make_float2(q.x, 1.f / q.y);
    }
    __syncthreads();
    if (s_bad)
        return;
    for (int i0 = blockIdx.y * kWeightThreads + threadIdx.x; i0 < end; i0 += step * kWeightTurns) {
        float sum[kWeightTurns], old[kWeightTurns];
        long long at[kWeightTurns];
#pragma unroll
        for (int t = 0; t < kWeightTurns; ++t) {
            const int i = i0 + t * step, page = i < end ? v.page(i / kPage) : 0;
            at[t] = i < end && (visible(a, v, page) >> (i % kPage) & 1u)
                        ? row * a.weight_stride + page * kPage + i % kPage
                        : -1;
            old[t] = at[t] >= 0 ? a.weights[at[t]] : 0.f;
            sum[t] = 0.f;
        }
        for (int h = 0; h < group; h += N) {
            float x[kWeightTurns][N];
#pragma unroll
            for (int t = 0; t < kWeightTurns; ++t)
                if (at[t] >= 0)
                    load_logits<N>(a.logits + (row * a.max_pages * kPage + i0 + t * step) * group + h, x[t]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float2 q;
                if (h + e < kWeightHeads) {
                    q = s_ml[h + e];
                } else {
                    q = __ldcg(ml + h + e);
                    q.y = 1.f / q.y;
                }
#pragma unroll
                for (int t = 0; t < kWeightTurns; ++t)
                    if (at[t] >= 0)
                        sum[t] = fmaf(ex2_approx((x[t][e] - q.x) * a.scale_log2), q.y, sum[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < kWeightTurns; ++t)
            if (at[t] >= 0)
                a.weights_out[at[t]] = old[t] + sum[t];
    }
}

template <int D>
cudaError_t launch_d(const PagedDecodeArgs &a, int rows, int sm_count, cudaStream_t stream)
{
    using C = Cfg<D>;
    const int group = a.num_q_heads / a.num_kv_heads;
    const int heads = group < kTile ? group : kTile;
    const size_t smem = static_cast<size_t>(C::RING) +
                        static_cast<size_t>(C::AREAS) * kWarps * heads * D * sizeof(float);
    // the largest size any call needs, once per device
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !attr_done[dev]) {
        const int most = C::RING + C::AREAS * kWarps * kTile * D * static_cast<int>(sizeof(float));
        if ((e = cudaFuncSetAttribute(paged_decode_kernel<D, false>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(paged_decode_kernel<D, true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess)
            return e;
        if (dev < 64)
            attr_done[dev] = 1;
    }
    // as many CTAs as fit on the SMs (228 KB each; 2 KB covers a CTA's static and
    // reserved shared memory); runs of at least kMinRun units
    const long long by_smem = (228 * 1024) / (static_cast<long long>(smem) + 2048);
    const long long fit = (by_smem < C::CTAS ? by_smem : C::CTAS) * sm_count;
    const long long ctas = fit < kMaxCtas ? fit : kMaxCtas;
    long long parts = ctas / rows;
    const long long most = (static_cast<long long>(a.num_seqs) * (kSeqUnits + a.max_pages) + kMinRun - 1) /
                           kMinRun;
    parts = parts < most ? parts : most;
    // one CTA merges a sequence's parts, 8 per load latency
    const long long cap = 8LL * a.num_seqs > 256 ? 8LL * a.num_seqs : 256;
    parts = parts < 1 ? 1 : (parts > cap ? cap : parts);
    const dim3 grid(static_cast<int>(parts), rows);
    if (!a.weights)
        return launch_dependent(paged_decode_kernel<D, false>, grid, kThreads, smem, stream, a);
    if ((e = launch_dependent(paged_decode_kernel<D, true>, grid, kThreads, smem, stream, a)) != cudaSuccess)
        return e;
    // kWeightTurns tokens a thread, but CTAs for every SM where there are few
    const long long units = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
    const long long slots = static_cast<long long>(a.max_pages) * kPage;
    long long splits = (slots + kWeightTurns * kWeightThreads - 1) / (kWeightTurns * kWeightThreads);
    const long long fill = (8LL * sm_count + units - 1) / units;
    const long long all = (slots + kWeightThreads - 1) / kWeightThreads;
    splits = splits > fill ? splits : fill;
    splits = splits < all ? splits : all;
    splits = splits < 1 ? 1 : (splits > 65535 ? 65535 : splits);
    return launch_dependent(group % 4 == 0 ? paged_weights_kernel<4> : paged_weights_kernel<1>,
                            dim3(static_cast<unsigned>(units), static_cast<unsigned>(splits)),
                            kWeightThreads, 0, stream, a);
}

int head_rows(int num_q_heads, int num_kv_heads)
{
    return num_kv_heads * ((num_q_heads / num_kv_heads + kTile - 1) / kTile);
}

// The workspace: a ticket per run, which has to be zero between calls; partial states, two
// per run; m and l of every row, and the logits.  Where each starts depends on the heads
// alone, so that no call's scores reach into the tickets of another, whatever their
// sequences and capacities.
size_t runs_of(int rows) { return rows > kMaxCtas ? rows : kMaxCtas; }      // in all rows

size_t ticket_bytes(int rows)
{
    return (runs_of(rows) * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

size_t part_bytes(int rows, int head_dim)
{
    return (runs_of(rows) * 2 * kTile * (head_dim + 4) * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

// m and l of every row, and the logits.
size_t score_bytes(int num_seqs, int num_q_heads, int capacity)
{
    return (static_cast<size_t>(num_seqs) * num_q_heads *
                (sizeof(float2) + static_cast<size_t>(capacity) * kPage * sizeof(float)) +
            255) & ~static_cast<size_t>(255);
}

}  // namespace

size_t paged_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                    int capacity)
{
    const int rows = head_rows(num_q_heads, num_kv_heads);
    size_t n = ticket_bytes(rows) + part_bytes(rows, head_dim);
    if (capacity > 0)
        n += score_bytes(num_seqs, num_q_heads, capacity);
    return n;
}

cudaError_t launch_paged_decode(int head_dim, PagedDecodeArgs &a, void *workspace, int sm_count,
                                cudaStream_t stream)
{
    const int rows = head_rows(a.num_q_heads, a.num_kv_heads);
    uint8_t *p = static_cast<uint8_t *>(workspace);
    a.tickets = reinterpret_cast<int32_t *>(p);
    a.part = reinterpret_cast<float *>(p += ticket_bytes(rows));
    if (a.weights) {
        a.ml = reinterpret_cast<float2 *>(p += part_bytes(rows, head_dim));
        a.logits = reinterpret_cast<float *>(p + static_cast<size_t>(a.num_seqs) * a.num_q_heads * sizeof(float2));
    }
    // pages a sequence reads at most
    const long long window = a.window_left < 0 ? a.capacity : a.window_left / kPage + 2LL;
    const long long sinks = a.window_left < 0 ? 0 : (static_cast<long long>(a.sink_tokens) + kPage - 1) / kPage;
    a.max_pages = static_cast<int>(window + sinks < a.capacity ? window + sinks : a.capacity);
    a.max_pages = a.max_pages < 1 ? 1 : a.max_pages;
    switch (head_dim) {
    case 64: return launch_d<64>(a, rows, sm_count, stream);
    case 128: return launch_d<128>(a, rows, sm_count, stream);
    case 256: return launch_d<256>(a, rows, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
