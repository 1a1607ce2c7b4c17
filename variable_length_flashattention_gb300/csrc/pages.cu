// pages.cu -- the pages of paged K/V pools: extend, fork, free, truncate, compact, copy.
//
// State: refs[num_blocks] (users of a page, 0 = free), tables[num_seqs,
// capacity] (physical page of each logical page), counts[num_seqs] (tokens).
// A sequence of n tokens holds its first ceil(n / block_size) table entries.
// New pages are the free ones with the lowest ids, so every result is a
// function of the inputs alone, whatever order the threads run in.
//
// Extend, fork and compact need ranks among the free (or used) pages.  A pool
// of at most 32768 pages fits one CTA, a 32-page word of its use bits per
// thread: one kernel does all but the page data.  Larger pools take three:
//   count    one CTA per chunk of 4096 pages counts its used pages;
//   plan     one CTA checks the request and gives every new page its rank
//            (extend, fork); it is the only step that can refuse, before
//            anything but the workspace is written;
//   assign   one CTA per chunk: the chunk's first free rank is a sum over the
//            earlier chunks' counts, so the free pages of rank < N go to
//            their tables without a pass over the pool in one CTA;
//   copy     page data, 4 KB per warp and turn, every pool in one launch.
// Consecutive steps are launched with programmatic serialisation.
//
// Bound: HBM for the copied pages (2 bytes moved per byte), launch latency
// for the rest: with 1024 pages the one-CTA form takes an extension from three
// launches (9.9 us) to one (8.1), a fork from four to two; at 32768 pages the two
// forms are level (extension 10.2 us in one CTA, 10.3 to 12.3 of 32769 pages), which
// is where its CTA's words end too.  Of 500000 pages an extension takes 12 us, a
// fork of 256 rows of 4687 pages 23.  A compaction that moves 776 MB takes 245 us
// (6.3 TB/s, 93% of the copy rate).
#include <climits>

#include "internal.h"
#include "launch.cuh"

namespace vfa {

namespace {

constexpr int kChunk = 4096;
constexpr int kPlanThreads = 1024;
constexpr int kPer = kChunk / kPlanThreads;
constexpr int kPiece = 4096;            // bytes a warp copies per turn
constexpr int kSmallPool = 32 * kPlanThreads;   // pages one CTA ranks
constexpr int kSmallRows = 4096;        // rows (ranks) whose places one CTA keeps in shared memory

enum { H_N = 0, H_USED = 1 };

struct PageWs {
    int32_t *head;      // [64]: [H_N] pages to assign / move, [H_USED] used pages
    int32_t *chunk;     // [chunks] used pages per chunk
    int32_t *src, *dst; // [num_blocks] page copies
    int32_t *rank;      // [num_blocks] compact: index of the page's move, -1 none; fork: the
                        // pool's use bits when the call began, 32 pages a word
    int32_t *offs;      // [max(num_seqs, forks) + 1] first rank per sequence; fork: entry per rank
    int32_t *plan;      // [forks][4] parent, child, tokens, 0
    int32_t *mark;      // [num_seqs] fork: entry that claimed the child
};

__host__ __device__ inline int chunks_of(int num_blocks) { return (num_blocks + kChunk - 1) / kChunk; }

size_t carve(int32_t *ws, int num_blocks, int num_seqs, int forks, PageWs *w)
{
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 63) & ~static_cast<size_t>(63);
        return ws ? ws + o : nullptr;
    };
    PageWs r;
    r.head = take(64);
    r.chunk = take(chunks_of(num_blocks));
    r.src = take(num_blocks);
    r.dst = take(num_blocks);
    r.rank = take(num_blocks);
    r.offs = take(static_cast<size_t>(num_seqs > forks ? num_seqs : forks) + 1);
    r.plan = take(static_cast<size_t>(forks) * 4);
    r.mark = take(num_seqs);
    if (w)
        *w = r;
    return at * sizeof(int32_t);
}

__device__ __forceinline__ void record(int32_t *status, int code)
{
    if (status)
        atomicCAS(status, 0, code);
}

// Exclusive sum of v over the CTA's 1024 threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int *total, int *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off)
            x += y;
    }
    __syncthreads();                    // s_warp's readers of the previous call are done
    if (lane == 31)
        s_warp[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        const int w = s_warp[i];
        before += i < warp ? w : 0;
        sum += w;
    }
    *total = sum;
    return before + x - v;
}

// Sum over chunks [0, n) of the used counts.
__device__ __forceinline__ int used_before(const int32_t *chunk, int n, int *s_warp)
{
    int v = 0, total;
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        v += chunk[i];
    block_scan(v, &total, s_warp);
    return total;
}

// bits (nullable): the pages' use bits.
__global__ void __launch_bounds__(kPlanThreads) count_kernel(const int32_t *refs, int num_blocks,
                                                             int32_t *chunk, int32_t *bits)
{
    grid_wait();
    grid_release();
    __shared__ int s_warp[kPlanThreads / 32];
    int v = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const long long id = static_cast<long long>(blockIdx.x) * kChunk + k * kPlanThreads + threadIdx.x;
        const bool is_used = id < num_blocks && refs[id] > 0;
        v += is_used;
        if (bits) {
            const uint32_t word = __ballot_sync(0xffffffffu, is_used);
            if ((threadIdx.x & 31) == 0 && id < num_blocks)
                bits[id >> 5] = static_cast<int32_t>(word);
        }
    }
    block_scan(v, &total, s_warp);
    if (threadIdx.x == 0)
        chunk[blockIdx.x] = total;
}

// ------------------------------------------------------------ extend, fork

// The pages every row needs (offs[s]: before row s) and the verdict; token
// counts grow if there are enough.  Returns the pages to assign, 0 if refused.
__device__ __forceinline__ int plan_extend(const PageArgs &a, int used, int32_t *offs, int *s_warp)
{
    const long long room = static_cast<long long>(a.capacity) * a.block_size;
    long long carry = 0;
    bool bad = false;
    for (int s0 = 0; s0 < a.num_seqs; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        int need = 0;
        if (s < a.num_seqs) {
            const long long n = a.counts[s], add = a.add[s];
            if (n < 0 || add < 0 || n + add > room || n + add > INT_MAX)
                bad = true;
            else
                need = static_cast<int>((n + add + a.block_size - 1) / a.block_size -
                                        (n + a.block_size - 1) / a.block_size);
        }
        // a row needs at most `capacity` pages; past num_blocks the request fails anyway
        need = min(need, a.num_blocks + 1);
        // 1024 rows' needs can pass 32 bits: sum in two parts
        int lo, hi, tl, th;
        lo = block_scan(need & 0xffff, &tl, s_warp);
        hi = block_scan(need >> 16, &th, s_warp);
        const long long at = carry + lo + (static_cast<long long>(hi) << 16);
        if (s < a.num_seqs)
            offs[s] = at > a.num_blocks ? a.num_blocks : static_cast<int>(at);
        carry += tl + (static_cast<long long>(th) << 16);
    }
    bad = __syncthreads_or(bad);
    const bool room_ok = carry <= a.num_blocks - used;
    const bool ok = !bad && room_ok;
    if (threadIdx.x == 0) {
        offs[a.num_seqs] = ok ? static_cast<int>(carry) : 0;
        if (!ok)
            record(a.status, bad ? VFA_ERR_BAD_BLOCK : VFA_ERR_NO_PAGES);
    }
    if (ok)
        for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads)
            a.counts[s] += a.add[s];
    __syncthreads();
    return ok ? static_cast<int>(carry) : 0;
}

// Page `id` becomes the r-th new page.
__device__ __forceinline__ void place_extend(const PageArgs &a, const int32_t *offs, int r, int id)
{
    int lo = 0, hi = a.num_seqs;                    // the row s with offs[s] <= r < offs[s + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (offs[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    const int pages = static_cast<int>((static_cast<long long>(a.counts[lo]) + a.block_size - 1) /
                                       a.block_size);
    a.tables[static_cast<long long>(lo) * a.capacity + pages - offs[lo + 1] + r] = id;
    a.refs[id] = 1;
}

__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    grid_release();
    __shared__ int s_warp[kPlanThreads / 32];
    const int used = used_before(w.chunk, chunks_of(a.num_blocks), s_warp);
    const int n = plan_extend(a, used, w.offs, s_warp);
    if (threadIdx.x == 0)
        w.head[H_N] = n;
}

// The entries' plan (parent -1: nothing to do), the entry and the source page
// of every copy in order, and the verdict; children's token counts are set if
// there are enough pages.  Returns the copies, 0 if refused.
__device__ __forceinline__ int plan_fork(const PageArgs &a, const PageWs &w, int used, int *s_warp)
{
    const long long room = static_cast<long long>(a.capacity) * a.block_size;
    bool bad = false;
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const int c = a.children[i];
        if (a.parents[i] >= 0 && c >= 0 && c < a.num_seqs)
            w.mark[c] = -1;
    }
    __syncthreads();
    int carry = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int take = 0, total, tail = 0, p = -1, c = 0, n = 0;
        if (i < a.n) {
            p = a.parents[i];
            c = a.children[i];
            if (p >= 0) {
                if (p >= a.num_seqs || c < 0 || c >= a.num_seqs || a.counts[c] != 0 ||
                    atomicExch(&w.mark[c], i) != -1) {
                    bad = true;
                } else {
                    n = a.counts[p];
                    if (n < 0 || n > room) {
                        bad = true;
                    } else if (n % a.block_size) {
                        tail = a.tables[static_cast<long long>(p) * a.capacity + n / a.block_size];
                        if (tail < 0 || tail >= a.num_blocks || a.refs[tail] <= 0)
                            bad = true;
                        else
                            take = 1;
                    }
                }
            }
            w.plan[4 * i] = bad ? -1 : p;
            w.plan[4 * i + 1] = c;
            w.plan[4 * i + 2] = n;
        }
        const int r = carry + block_scan(take, &total, s_warp);
        if (take && r < a.num_blocks) {
            w.offs[r] = i;
            w.src[r] = tail;
        }
        carry += total;
    }
    bad = __syncthreads_or(bad);
    const bool ok = !bad && carry <= a.num_blocks - used;
    if (threadIdx.x == 0) {
        w.head[H_N] = ok ? carry : 0;
        if (!ok)
            record(a.status, bad ? VFA_ERR_BAD_BLOCK : VFA_ERR_NO_PAGES);
    }
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        if (!ok)
            w.plan[4 * i] = -1;
        else if (w.plan[4 * i] >= 0)
            a.counts[w.plan[4 * i + 1]] = w.plan[4 * i + 2];
    }
    __syncthreads();
    return ok ? carry : 0;
}

// Page `id` becomes the target of the r-th copy.
__device__ __forceinline__ void place_fork(const PageArgs &a, const PageWs &w, int r, int id)
{
    const int i = w.offs[r];
    w.dst[r] = id;
    a.tables[static_cast<long long>(w.plan[4 * i + 1]) * a.capacity +
             w.plan[4 * i + 2] / a.block_size] = id;
    a.refs[id] = 1;
}

// The full pages of entry i's parent are shared with its child.  Whether a page
// is in use is asked of the bits from before the call: this call's new pages
// have a reference already, or get it meanwhile from another CTA.
__device__ __forceinline__ void share_pages(const PageArgs &a, const PageWs &w, int i)
{
    const int p = w.plan[4 * i];
    if (p < 0)
        return;
    const int full = w.plan[4 * i + 2] / a.block_size;
    const int32_t *from = a.tables + static_cast<long long>(p) * a.capacity;
    int32_t *to = a.tables + static_cast<long long>(w.plan[4 * i + 1]) * a.capacity;
    for (int j = threadIdx.x; j < full; j += blockDim.x) {
        const int id = from[j];
        to[j] = id;
        if (id < 0 || id >= a.num_blocks || !(static_cast<uint32_t>(w.rank[id >> 5]) >> (id & 31) & 1))
            record(a.status, VFA_ERR_BAD_BLOCK);        // not a page in use: not counted
        else
            atomicAdd(&a.refs[id], 1);
    }
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    grid_release();
    __shared__ int s_warp[kPlanThreads / 32];
    plan_fork(a, w, used_before(w.chunk, chunks_of(a.num_blocks), s_warp), s_warp);
}

// CTAs [0, chunks): the chunk's free pages of rank < N go to their rows.
// FORK: CTA chunks + i shares the full pages of entry i's parent.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) assign_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    if (FORK && a.copies)
        grid_release();
    __shared__ int s_warp[kPlanThreads / 32];
    const int chunks = chunks_of(a.num_blocks);
    if (FORK && static_cast<int>(blockIdx.x) >= chunks) {
        share_pages(a, w, blockIdx.x - chunks);
        return;
    }
    const int n = w.head[H_N];
    if (n == 0)
        return;
    const int base = blockIdx.x * kChunk;
    const int first = base - used_before(w.chunk, blockIdx.x, s_warp);   // free pages below
    if (first >= n)
        return;
    const int id0 = base + threadIdx.x * kPer;
    bool is_free[kPer];
    int mine = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        is_free[k] = id0 + k < a.num_blocks && a.refs[id0 + k] <= 0;
        mine += is_free[k];
    }
    int r = first + block_scan(mine, &total, s_warp);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (!is_free[k])
            continue;
        if (r < n) {
            if (FORK)
                place_fork(a, w, r, id0 + k);
            else
                place_extend(a, w.offs, r, id0 + k);
        }
        ++r;
    }
}

// ------------------------------------------------------------ small pools
//
// Thread t's word of the pool's use bits (pages [32 t, 32 t + 32), past the end
// counted as used) and the number of used pages.
__device__ __forceinline__ uint32_t use_word(const PageArgs &a, uint32_t *s_bits, int *used, int *s_warp)
{
    const int lane = threadIdx.x & 31;
    const int words = (a.num_blocks + 31) / 32;
    constexpr int STEP = kPlanThreads / 32, U = 8;  // loads in flight per warp
    for (int w0 = threadIdx.x >> 5; w0 < words; w0 += U * STEP) {
        int ref[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int id = (w0 + u * STEP) * 32 + lane;
            ref[u] = id < a.num_blocks ? a.refs[id] : 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t bits = __ballot_sync(0xffffffffu, ref[u] > 0);
            if (lane == 0 && w0 + u * STEP < words)
                s_bits[w0 + u * STEP] = bits;
        }
    }
    __syncthreads();
    const uint32_t word = static_cast<int>(threadIdx.x) < words ? s_bits[threadIdx.x] : 0xffffffffu;
    int free;
    block_scan(__popc(~word), &free, s_warp);
    *used = a.num_blocks - free;
    return word;
}

// list[r] = the r-th free page, r < n.
__device__ __forceinline__ void list_free(uint32_t word, int n, int32_t *list, int *s_warp)
{
    int total;
    int r = block_scan(__popc(~word), &total, s_warp);
    for (uint32_t left = ~word; left && r < n; left &= left - 1, ++r)
        list[r] = threadIdx.x * 32 + __ffs(left) - 1;
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) extend_small_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    __shared__ uint32_t s_bits[kPlanThreads];
    __shared__ int s_warp[kPlanThreads / 32];
    __shared__ int32_t s_offs[kSmallRows + 1], s_list[kSmallRows];
    int used;
    const uint32_t word = use_word(a, s_bits, &used, s_warp);
    int32_t *offs = a.num_seqs <= kSmallRows ? s_offs : w.offs;
    const int n = plan_extend(a, used, offs, s_warp);
    int32_t *list = n <= kSmallRows ? s_list : w.dst;
    list_free(word, n, list, s_warp);
    for (int r = threadIdx.x; r < n; r += kPlanThreads)
        place_extend(a, offs, r, list[r]);
}

__global__ void __launch_bounds__(kPlanThreads) fork_small_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    grid_release();
    __shared__ uint32_t s_bits[kPlanThreads];
    __shared__ int s_warp[kPlanThreads / 32];
    int used;
    const uint32_t word = use_word(a, s_bits, &used, s_warp);
    if (static_cast<int>(threadIdx.x) < (a.num_blocks + 31) / 32)
        w.rank[threadIdx.x] = static_cast<int32_t>(s_bits[threadIdx.x]);
    const int n = plan_fork(a, w, used, s_warp);
    list_free(word, n, w.dst, s_warp);
    for (int r = threadIdx.x; r < n; r += kPlanThreads)
        place_fork(a, w, r, w.dst[r]);
}

// ------------------------------------------------------------ free

__global__ void __launch_bounds__(256) free_kernel(const PageArgs a)
{
    grid_wait();
    __shared__ int s_n;
    const int s = a.seqs[blockIdx.x];
    if (s < 0)
        return;                                     // a padding entry
    if (s >= a.num_seqs) {
        if (threadIdx.x == 0)
            record(a.status, VFA_ERR_BAD_BLOCK);
        return;
    }
    if (threadIdx.x == 0) {
        // the exchange makes a sequence listed twice release its pages once
        int n = atomicExch(&a.counts[s], 0);
        if (n < 0 || n > static_cast<long long>(a.capacity) * a.block_size) {
            record(a.status, VFA_ERR_BAD_BLOCK);
            a.counts[s] = n;
            n = 0;
        }
        s_n = n;
    }
    __syncthreads();
    const int pages = static_cast<int>((static_cast<long long>(s_n) + a.block_size - 1) / a.block_size);
    for (int j = threadIdx.x; j < pages; j += blockDim.x) {
        const int id = a.tables[static_cast<long long>(s) * a.capacity + j];
        if (id < 0 || id >= a.num_blocks) {
            record(a.status, VFA_ERR_BAD_BLOCK);
        } else if (atomicSub(&a.refs[id], 1) <= 0) {
            atomicAdd(&a.refs[id], 1);
            record(a.status, VFA_ERR_BAD_BLOCK);
        }
    }
}

// ------------------------------------------------------------ truncate
//
// The rows are judged by the references from before the call (a page that is cut in
// two must not be another row's as well), one thread each; then every row that
// shrinks gives up its pages.  One CTA does both where that is little to do
// (a launch is 4 us of the host's time, and the call's time is the host's);
// otherwise two launches, the second with some CTAs per row.

// Row s judged: its pages [ws[2 s], ws[2 s + 1]) are to go.
__device__ __forceinline__ void plan_truncate(const PageArgs &a, int s)
{
    const int n = a.counts[s], m = a.new_counts[s];
    const bool valid = n >= 0 && n <= static_cast<long long>(a.capacity) * a.block_size;
    bool ok = m >= 0 && m < n && valid;
    bool bad = m >= 0 && m != n && !ok;
    if (ok && m % a.block_size != 0) {
        const int id = a.tables[static_cast<long long>(s) * a.capacity + m / a.block_size];
        if (id >= 0 && id < a.num_blocks && a.refs[id] > 1) {
            ok = false;
            bad = true;
        }
    }
    if (bad)
        record(a.status, VFA_ERR_BAD_BLOCK);
    auto pages = [&](int x) {
        return static_cast<int>((static_cast<long long>(x) + a.block_size - 1) / a.block_size);
    };
    a.ws[2 * s] = ok ? pages(m) : 0;
    a.ws[2 * s + 1] = ok ? pages(n) : 0;
    a.counts_out[s] = ok ? m : n;
}

// Pages first, first + step, ... of row s's that go.
__device__ __forceinline__ void drop_pages(const PageArgs &a, int s, int first, int step)
{
    const int end = a.ws[2 * s + 1];
    for (int j = a.ws[2 * s] + first; j < end; j += step) {
        const int id = a.tables[static_cast<long long>(s) * a.capacity + j];
        if (id < 0 || id >= a.num_blocks) {
            record(a.status, VFA_ERR_BAD_BLOCK);
        } else if (atomicSub(&a.refs_out[id], 1) <= 0) {
            atomicAdd(&a.refs_out[id], 1);
            record(a.status, VFA_ERR_BAD_BLOCK);
        }
    }
}

__global__ void __launch_bounds__(256) truncate_plan_kernel(const PageArgs a)
{
    grid_wait();
    grid_release();
    const int first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    if (a.refs_out != a.refs)
        for (int i = first; i < a.num_blocks; i += step)
            a.refs_out[i] = a.refs[i];
    for (int s = first; s < a.num_seqs; s += step)
        plan_truncate(a, s);
}

__global__ void __launch_bounds__(256) truncate_kernel(const PageArgs a)
{
    grid_wait();
    drop_pages(a, blockIdx.x, blockIdx.y * blockDim.x + threadIdx.x, gridDim.y * blockDim.x);
}

__global__ void __launch_bounds__(kPlanThreads) truncate_small_kernel(const PageArgs a)
{
    grid_wait();
    for (int s = threadIdx.x; s < a.num_seqs; s += kPlanThreads)
        plan_truncate(a, s);
    if (a.refs_out != a.refs)
        for (int i = threadIdx.x; i < a.num_blocks; i += kPlanThreads)
            a.refs_out[i] = a.refs[i];
    __threadfence();
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int s = warp; s < a.num_seqs; s += kPlanThreads / 32)
        drop_pages(a, s, lane, 32);
}

// ------------------------------------------------------------ compact
//
// With U used pages, the used pages at or above U move, in ascending order,
// to the free pages below U: as many, and no page is both source and target.

__global__ void __launch_bounds__(kPlanThreads) compact_rank_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    grid_release();
    __shared__ int s_warp[kPlanThreads / 32];
    const int chunks = chunks_of(a.num_blocks);
    const int U = used_before(w.chunk, chunks, s_warp);
    // used pages below U: whole chunks, then the chunk that holds U
    const int cu = U / kChunk;
    int below = used_before(w.chunk, min(cu, chunks), s_warp);
    {
        int v = 0, total;
        for (int id = cu * kChunk + threadIdx.x; id < U; id += kPlanThreads)
            v += a.refs[id] > 0;
        block_scan(v, &total, s_warp);
        below += total;
    }
    const int id0 = blockIdx.x * kChunk + threadIdx.x * kPer;
    bool is_used[kPer];
    int mine = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        is_used[k] = id0 + k < a.num_blocks && a.refs[id0 + k] > 0;
        mine += is_used[k];
    }
    int before = used_before(w.chunk, blockIdx.x, s_warp);
    before += block_scan(mine, &total, s_warp);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int id = id0 + k;
        if (id < a.num_blocks) {
            int r = -1;
            if (is_used[k] && id >= U) {
                r = before - below;
                w.src[r] = id;
            } else if (!is_used[k] && id < U) {
                r = id - before;
                w.dst[r] = id;
            }
            w.rank[id] = r;
        }
        before += is_used[k];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        w.head[H_N] = U - below;
        w.head[H_USED] = U;
        *a.num_used = U;
    }
}

__global__ void __launch_bounds__(kPlanThreads) compact_small_kernel(const PageArgs a, const PageWs w)
{
    grid_wait();
    grid_release();
    __shared__ uint32_t s_bits[kPlanThreads];
    __shared__ int s_warp[kPlanThreads / 32];
    int U, total, below;
    const uint32_t word = use_word(a, s_bits, &U, s_warp);
    const int id0 = threadIdx.x * 32;
    // (pages past the pool's end have set bits, but no page of the pool is above them)
    __shared__ int s_before[kPlanThreads];              // used pages below the word
    s_before[threadIdx.x] = block_scan(__popc(word), &total, s_warp);
    {
        const int part = U - id0;                   // pages of this word below U
        const uint32_t mask = part <= 0 ? 0u : part >= 32 ? 0xffffffffu : (1u << part) - 1;
        block_scan(__popc(word & mask), &below, s_warp);
    }
    for (int id = threadIdx.x; id < a.num_blocks; id += kPlanThreads) {
        const uint32_t bits = s_bits[id >> 5];
        const int before = s_before[id >> 5] + __popc(bits & ((1u << (id & 31)) - 1));
        const bool is_used = bits >> (id & 31) & 1;
        int r = -1;
        if (is_used && id >= U) {
            r = before - below;
            w.src[r] = id;
        } else if (!is_used && id < U) {
            r = id - before;
            w.dst[r] = id;
        }
        w.rank[id] = r;
    }
    if (threadIdx.x == 0) {
        w.head[H_N] = U - below;
        w.head[H_USED] = U;
        *a.num_used = U;
    }
}

// Tables and reference counts after the moves (part, parts: this CTA's share).
__device__ __forceinline__ void compact_apply(const PageArgs &a, const PageWs &w, int part,
                                              int parts)
{
    const int U = w.head[H_USED];
    const long long stride = static_cast<long long>(parts) * blockDim.x;
    const long long t0 = static_cast<long long>(part) * blockDim.x + threadIdx.x;
    for (long long id = t0; id < a.num_blocks; id += stride) {
        const int r = w.rank[id];
        if (id < U && r >= 0) {                     // takes over a moved page's users
            const int from = w.src[r];
            a.refs_out[id] = a.refs[from];
            a.refs_out[from] = 0;
        } else if (r < 0) {
            a.refs_out[id] = a.refs[id];
        }
    }
    const long long entries = static_cast<long long>(a.num_seqs) * a.capacity;
    for (long long e = t0; e < entries; e += stride) {
        const int s = static_cast<int>(e / a.capacity);
        const long long n = a.counts[s];
        if (n < 0 || n > static_cast<long long>(a.capacity) * a.block_size) {
            record(a.status, VFA_ERR_BAD_BLOCK);
            continue;
        }
        if (e % a.capacity >= (n + a.block_size - 1) / a.block_size)
            continue;
        int id = a.tables[e];
        if (id < 0 || id >= a.num_blocks) {
            record(a.status, VFA_ERR_BAD_BLOCK);
        } else {
            const int r = w.rank[id];
            if ((id < U) == (r >= 0))               // listed, but nobody counts as its user
                record(a.status, VFA_ERR_BAD_BLOCK);
            else if (r >= 0)
                id = w.dst[r];
        }
        a.tables_out[e] = id;
    }
}

// ------------------------------------------------------------ copy
//
// blockIdx.y < pools: warps copy pieces of that pool's pages.  blockIdx.y ==
// pools, meanwhile: COMPACT rewrites tables and counts, SHARE shares a fork's
// full pages.
enum { COPY_ONLY, COPY_COMPACT, COPY_SHARE };

template <int ROLE>
__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ PagePools p,
                                                   const int32_t *src, const int32_t *dst,
                                                   const int32_t *n_dev, int n_host, int num_blocks,
                                                   int32_t *status, const PageArgs a,
                                                   const PageWs w)
{
    grid_wait();
    if (ROLE != COPY_ONLY && static_cast<int>(blockIdx.y) == p.n) {
        if (ROLE == COPY_COMPACT)
            compact_apply(a, w, blockIdx.x, gridDim.x);
        else
            for (int i = blockIdx.x; i < a.n; i += gridDim.x)
                share_pages(a, w, i);
        return;
    }
    const int n = n_dev ? *n_dev : n_host;
    const int bytes = p.page_bytes[blockIdx.y];
    uint8_t *base = p.ptr[blockIdx.y];
    const int pieces = (bytes + kPiece - 1) / kPiece;
    const int lane = threadIdx.x & 31;
    const long long items = static_cast<long long>(n) * pieces;
    const long long nwarps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    for (long long it = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
         it < items; it += nwarps) {
        const int pair = static_cast<int>(it / pieces), piece = static_cast<int>(it % pieces);
        const int from = src[pair], to = dst[pair];
        if (!n_dev && from < 0)
            continue;                               // a padding entry of the caller's list
        if (from < 0 || from >= num_blocks || to < 0 || to >= num_blocks) {
            if (lane == 0)
                record(status, VFA_ERR_BAD_BLOCK);
            continue;
        }
        const uint8_t *s = base + static_cast<long long>(from) * bytes;
        uint8_t *d = base + static_cast<long long>(to) * bytes;
        uint4 v[kPiece / 512];
#pragma unroll
        for (int k = 0; k < kPiece / 512; ++k) {
            const int o = piece * kPiece + k * 512 + lane * 16;
            if (o < bytes)
                v[k] = __ldcs(reinterpret_cast<const uint4 *>(s + o));
        }
#pragma unroll
        for (int k = 0; k < kPiece / 512; ++k) {
            const int o = piece * kPiece + k * 512 + lane * 16;
            if (o < bytes)
                __stcs(reinterpret_cast<uint4 *>(d + o), v[k]);
        }
    }
}

// CTAs per pool: about eight CTAs of eight warps on every SM in all, and no
// more warps than `max_pairs` pages have pieces.
int copy_ctas(const PagePools &p, long long max_pairs, int sm_count)
{
    int pieces = 1;
    for (int i = 0; i < p.n; ++i)
        pieces = pieces > (p.page_bytes[i] + kPiece - 1) / kPiece
                     ? pieces
                     : (p.page_bytes[i] + kPiece - 1) / kPiece;
    long long g = (8LL * sm_count + p.n - 1) / (p.n > 0 ? p.n : 1);
    const long long need = (max_pairs * pieces + 7) / 8;
    g = g < need ? g : need;
    return static_cast<int>(g < 1 ? 1 : g);
}

}  // namespace

size_t page_workspace_bytes(int num_blocks, int num_seqs, int num_forks)
{
    return carve(nullptr, num_blocks, num_seqs, num_forks, nullptr);
}

cudaError_t launch_pages_extend(const PageArgs &a, cudaStream_t stream)
{
    PageWs w;
    carve(a.ws, a.num_blocks, a.num_seqs, 0, &w);
    if (a.num_blocks <= kSmallPool)
        return launch_dependent(extend_small_kernel, dim3(1), kPlanThreads, 0, stream, a, w);
    const int chunks = chunks_of(a.num_blocks);
    cudaError_t e;
    if ((e = launch_dependent(count_kernel, dim3(chunks), kPlanThreads, 0, stream, a.refs,
                              a.num_blocks, w.chunk, static_cast<int32_t *>(nullptr))) ||
        (e = launch_dependent(extend_plan_kernel, dim3(1), kPlanThreads, 0, stream, a, w)) ||
        (e = launch_dependent(assign_kernel<false>, dim3(chunks), kPlanThreads, 0, stream, a, w)))
        return e;
    return cudaSuccess;
}

cudaError_t launch_pages_fork(const PageArgs &a, const PagePools &p, int sm_count,
                              cudaStream_t stream)
{
    PageWs w;
    carve(a.ws, a.num_blocks, a.num_seqs, a.n, &w);
    cudaError_t e;
    if (a.num_blocks <= kSmallPool) {
        if ((e = launch_dependent(fork_small_kernel, dim3(1), kPlanThreads, 0, stream, a, w)))
            return e;
        const int ctas = copy_ctas(p, a.n, sm_count);
        return launch_dependent(copy_kernel<COPY_SHARE>, dim3(ctas > a.n ? ctas : a.n, p.n + 1), 256, 0,
                                stream, p, w.src, w.dst, w.head + H_N, 0, a.num_blocks, a.status, a,
                                w);
    }
    const int chunks = chunks_of(a.num_blocks);
    PageArgs b = a;
    b.copies = p.n > 0;
    if ((e = launch_dependent(count_kernel, dim3(chunks), kPlanThreads, 0, stream, a.refs,
                              a.num_blocks, w.chunk, w.rank)) ||
        (e = launch_dependent(fork_plan_kernel, dim3(1), kPlanThreads, 0, stream, a, w)) ||
        (e = launch_dependent(assign_kernel<true>, dim3(chunks + a.n), kPlanThreads, 0, stream, b, w)))
        return e;
    if (p.n == 0)
        return cudaSuccess;
    return launch_dependent(copy_kernel<COPY_ONLY>, dim3(copy_ctas(p, a.n, sm_count), p.n), 256, 0,
                            stream, p, w.src, w.dst, w.head + H_N, 0, a.num_blocks, a.status, a, w);
}

cudaError_t launch_pages_free(const PageArgs &a, cudaStream_t stream)
{
    return launch_dependent(free_kernel, dim3(a.n), 256, 0, stream, a);
}

cudaError_t launch_pages_truncate(const PageArgs &a, int sm_count, cudaStream_t stream)
{
    // rows with few pages and a pool that a CTA copies in a few turns
    // (64 rows of 68 pages: 27 us with the eviction ahead of it, 32 in two launches; 8 rows of
    // 2048 pages: 104 and 71)
    if (a.num_seqs <= kPlanThreads && a.capacity <= 256 &&
        static_cast<long long>(a.num_seqs) * a.capacity <= 16384 &&
        (a.refs_out == a.refs || a.num_blocks <= 16384))
        return launch_dependent(truncate_small_kernel, dim3(1), kPlanThreads, 0, stream, a);
    const int n = a.refs_out != a.refs && a.num_blocks > a.num_seqs ? a.num_blocks : a.num_seqs;
    const int ctas = (n + 255) / 256;
    // a page per thread, as long as that takes no more CTAs than run side by side
    const int most = (a.capacity + 255) / 256, room = 8 * sm_count / a.num_seqs;
    const int shares = most < room ? most : (room < 1 ? 1 : room);
    const cudaError_t e = launch_dependent(truncate_plan_kernel, dim3(ctas < 4 * sm_count ? ctas : 4 * sm_count),
                                           256, 0, stream, a);
    return e != cudaSuccess ? e : launch_dependent(truncate_kernel, dim3(a.num_seqs, shares), 256, 0, stream,
                                                   a);
}

cudaError_t launch_pages_compact(const PageArgs &a, const PagePools &p, int sm_count,
                                 cudaStream_t stream)
{
    PageWs w;
    carve(a.ws, a.num_blocks, a.num_seqs, 0, &w);
    const int chunks = chunks_of(a.num_blocks);
    cudaError_t e;
    if (a.num_blocks <= kSmallPool) {
        if ((e = launch_dependent(compact_small_kernel, dim3(1), kPlanThreads, 0, stream, a, w)))
            return e;
    } else if ((e = launch_dependent(count_kernel, dim3(chunks), kPlanThreads, 0, stream, a.refs,
                                     a.num_blocks, w.chunk, static_cast<int32_t *>(nullptr))) ||
               (e = launch_dependent(compact_rank_kernel, dim3(chunks), kPlanThreads, 0, stream, a,
                                     w))) {
        return e;
    }
    return launch_dependent(copy_kernel<COPY_COMPACT>,
                            dim3(copy_ctas(p, a.num_blocks / 2 + 1, sm_count), p.n + 1), 256, 0,
                            stream, p, w.src, w.dst, w.head + H_N, 0, a.num_blocks, a.status, a, w);
}

cudaError_t launch_pages_copy(const PagePools &p, const int32_t *src, const int32_t *dst, int n,
                              int num_blocks, int32_t *status, int sm_count, cudaStream_t stream)
{
    PageArgs a = {};
    PageWs w = {};
    return launch_dependent(copy_kernel<COPY_ONLY>, dim3(copy_ctas(p, n, sm_count), p.n), 256, 0,
                            stream, p, src, dst, static_cast<const int32_t *>(nullptr), n,
                            num_blocks, status, a, w);
}

}  // namespace vfa
