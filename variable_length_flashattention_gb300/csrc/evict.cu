// evict.cu -- tokens of little weight leave a paged cache.
//
// Per sequence and kv head, of n tokens b stay: the first positions (sinks), the
// last (recent), and of the others those with the largest accumulated weight, ties
// by the lowest slot.  Nothing but kept tokens past slot b moves: in ascending
// order they go to the free slots below b, in ascending order, so no slot is read
// and written and all moves run side by side.  Slots then hold tokens out of order;
// `positions` says which token of the sequence a slot holds, for slots below
// history[s][0]; later slots were appended since and hold the tokens slot +
// history[s][1].
//
// Two kernels:
//   select   a cluster of up to 8 CTAs per (sequence, kv head), each with a run of the
//            slots.  Every slot has a key, an unsigned integer in the order of the
//            weights, the largest for tokens that stay whatever their weight: the
//            b largest keys stay, ties by the lowest slot.  The border key is
//            found by its bits, 11, 11 and 10 at a time from the top, by counting
//            the keys that share the bits so far, until all of those stay; every CTA
//            of a cluster adds up its share of the counts.  Then every warp takes a run
//            of slots: ballots give the ranks of ties, free slots and movers, sums over
//            warps and CTAs their starts.  Weights and positions are rewritten here.
//            One CTA per row whose keys were formed anew from the weights for every
//            count took 41 us for 64 sequences of 1056 tokens on 8 kv heads and 57 for 8 of
//            4000-32768.  Keys in shared memory, loads in batches and the scan by all
//            threads brought the first, whose rows have one CTA still, to 21, those and
//            clusters the second to 34, and one barrier per sum (two buffers of sums in
//            turn) instead of two that to 32.  The CTAs of a row go by the table's
//            width, which the host knows, not by the row's tokens, which it does not:
//            the 64 sequences take 19 us with their moves in tables of 128 pages, 39 in
//            256, 116 in 2048 (clusters of eight CTAs, four or five words of slots each);
//   move     the rows of K and V by the lists, 16 bytes per thread, and the
//            sequences' new state.
// Bound: HBM, 8 D bytes per moved token and kv head, and 12 to 16 bytes per token for weights
// and positions; for small rows the chain of the select kernel's counts.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace vfa {

namespace {

constexpr int kPage = 16;
constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMostCtas = 8;            // of a cluster
constexpr int kTurns = 4;               // slots a thread has loads in flight for
constexpr int kSmemKeys = 4096;         // keys a CTA keeps in shared memory
constexpr uint32_t kStays = 0xffffffffu;    // the key of a token that stays whatever its weight
constexpr int kMoveThreads = 256;

__device__ __forceinline__ void record(int32_t *status, int code)
{
    if (status)
        atomicCAS(status, 0, code);
}

// What is asked of a sequence.
struct Plan {
    int n, b, known, gone;        // tokens, tokens that stay, stored positions, evicted before
    int sinks;                    // positions below stay
    long long recent;             // positions from here on stay
    bool bad;

    // the position of slot j, p its stored one
    __device__ __forceinline__ int position(int j, int p) const { return j < known ? p : j + gone; }
    __device__ __forceinline__ bool safe(int pos) const { return pos < sinks || pos >= recent; }
};

__device__ __forceinline__ Plan plan_of(const EvictArgs &a, int s)
{
    Plan p;
    p.n = a.counts[s];
    p.known = a.history[2 * s];
    p.gone = a.history[2 * s + 1];
    const int budget = a.budgets[s];
    p.bad = p.n < 0 || p.n > static_cast<long long>(a.capacity) * kPage || p.known < 0 ||
            p.known > p.n || p.gone < 0 || static_cast<long long>(p.n) + p.gone > 0x7fffffffll;
    p.b = budget < 0 || budget > p.n ? p.n : budget;
    p.sinks = min(a.sink_tokens, p.b);
    p.recent = static_cast<long long>(p.n) + p.gone - min(a.recent_tokens, p.b - p.sinks);
    return p;
}

// Weights in the order of unsigned integers below kStays; any NaN is the largest.
__device__ __forceinline__ uint32_t order_of(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);          // -0 is 0
    if (w != w)
        return kStays - 1;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What the CTAs of a cluster tell each other: their sums of three values.
struct Shared {
    int bins[kBins];
    int warp[3][kSelWarps];
    int sums[2][3][kMostCtas];          // of every CTA, by rank; calls take the two in turn
    int digit, left, exact, bad;
};

// Sums ahead of this warp, in the order of ranks and warps, of N values per warp (its lane
// 0's); total[i] gets the cluster's.  Everybody calls it, with a `call` that counts up: the
// sums of a call are written where those of the one before the last were read.
template <int N>
__device__ __forceinline__ void warp_starts(cg::cluster_group &cluster, Shared &sh, int &call,
                                            const int (&v)[N], int (&start)[N], int (&total)[N])
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    __syncthreads();
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            sh.warp[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        start[i] = total[i] = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            start[i] += w < warp ? sh.warp[i][w] : 0;
            total[i] += sh.warp[i][w];
        }
    }
    if (ctas == 1)
        return;
    const int half = call++ & 1;
    if (threadIdx.x < ctas)
#pragma unroll
        for (int i = 0; i < N; ++i)
            cluster.map_shared_rank(&sh, threadIdx.x)->sums[half][i][rank] = total[i];
    cluster.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        total[i] = 0;
        for (int c = 0; c < ctas; ++c) {
            start[i] += c < rank ? sh.sums[half][i][c] : 0;
            total[i] += sh.sums[half][i][c];
        }
    }
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a)
{
    grid_wait();
    grid_release();
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Shared sh;
    extern __shared__ uint32_t s_keys[];
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int row = blockIdx.x / ctas, s = row / a.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Plan p = plan_of(a, s);
    // This CTA's slots, whole words of 32.
    const int words = p.bad ? 0 : (p.n + 31) / 32, share = (words + ctas - 1) / ctas;
    const int c0 = min(words, rank * share), c1 = min(words, c0 + share);
    const int j0 = c0 * 32, j1 = min(p.n, c1 * 32);
    // pages that are none, or that a move would write although another row has them, among
    // those of its slots
    bool bad = p.bad;
    if (!bad) {
        const int written = p.b < p.n ? (p.b + kPage - 1) / kPage : 0;
        for (int j = j0 / kPage + tid; j * kPage < j1; j += kSelThreads) {
            const int id = a.tables[static_cast<long long>(s) * a.capacity + j];
            bad |= id < 0 || id >= a.num_blocks || (j < written && a.refs[id] != 1);
        }
    }
    bad = __syncthreads_or(bad);
    if (ctas > 1) {
        // the row is refused as a whole
        if (tid == 0)
            sh.bad = 0;
        cluster.sync();
        if (bad && tid < ctas)
            cluster.map_shared_rank(&sh, tid)->bad = 1;
        cluster.sync();
        bad = sh.bad;
    }
    if (bad) {
        if (tid == 0 && rank == 0) {
            a.moves[row] = -1;
            record(a.status, VFA_ERR_BAD_BLOCK);
        }
        return;
    }
    const long long at = static_cast<long long>(row) * a.capacity * kPage;
    const float *w = a.weights + at;
    const int32_t *pos = a.positions + at;
    float *w_out = a.weights_out + at;
    int32_t *pos_out = a.positions_out + at;
    uint32_t *bits = a.bits + static_cast<long long>(row) * ((a.capacity + 1) / 2);
    int32_t *to = a.lists + at, *from = to + static_cast<long long>(a.capacity) * (kPage / 2);
    auto position = [&](int j) { return p.position(j, j < p.known ? pos[j] : 0); };
    int moves = 0, call = 0;
    if (p.b < p.n) {
        // Keys: in shared memory, or (long runs) where the lists will be.
        uint32_t *keys = c1 - c0 <= kSmemKeys / 32 ? s_keys - j0 : reinterpret_cast<uint32_t *>(to);
        for (int j = j0 + tid; j < j1; j += kSelThreads * kTurns) {
            uint32_t k[kTurns];
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
                const int i = j + t * kSelThreads;
                k[t] = i < j1 ? (p.safe(position(i)) ? kStays : order_of(w[i])) : 0u;
            }
#pragma unroll
            for (int t = 0; t < kTurns; ++t)
                if (j + t * kSelThreads < j1)
                    keys[j + t * kSelThreads] = k[t];
        }
        // The border: the b-th largest key, and how many of those that equal it stay.
        // (Where all keys that share the border's bits so far stay, none has to be
        // told apart any more: the border is just below them.)
        uint32_t border = 0, known_bits = 0;
        int left = p.b;
        if (left > 0) {
            for (int turn = 0; turn < 3; ++turn) {
                const int shift = turn == 0 ? 21 : (turn == 1 ? 10 : 0);
                const uint32_t mask = turn == 2 ? 1023u : 2047u;
                for (int i = tid; i < kBins; i += kSelThreads)
                    sh.bins[i] = 0;
                __syncthreads();
                for (int j = j0 + tid; j < j1; j += kSelThreads) {
                    const uint32_t k = keys[j];
                    if ((k & known_bits) == border)
                        atomicAdd(&sh.bins[k >> shift & mask], 1);
                }
                if (ctas > 1)
                    cluster.sync();
                else
                    __syncthreads();
                // Every CTA adds up its share of the bins, from the top: rank r's and thread
                // t's are the `per` bins from 2047 - (r * threads + t) * per down.
                const int per = kBins / kSelThreads / ctas, top = kBins - 1 - (rank * kSelThreads + tid) * per;
                int mine[kBins / kSelThreads], sum = 0;
#pragma unroll
                for (int i = 0; i < kBins / kSelThreads; ++i)
                    mine[i] = 0;
                for (int c = 0; c < ctas; ++c) {
                    const int *bins = cluster.map_shared_rank(&sh, c)->bins;
#pragma unroll
                    for (int i = 0; i < kBins / kSelThreads; ++i)
                        if (i < per)
                            mine[i] += bins[top - i];
                }
#pragma unroll
                for (int i = 0; i < kBins / kSelThreads; ++i)
                    sum += mine[i];
                int x = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o)
                        x += y;
                }
                const int in_warp[1] = {__shfl_sync(0xffffffffu, x, 31)};
                int start[1], total[1];
                warp_starts<1>(cluster, sh, call, in_warp, start, total);
                int before = start[0] + x - sum;
                if (before < left && left <= before + sum) {
                    int digit = top, count = 0;
#pragma unroll
                    for (int i = 0; i < kBins / kSelThreads; ++i)
                        if (i < per && count == 0) {
                            if (left <= before + mine[i]) {
                                count = mine[i];
                            } else {
                                before += mine[i];
                                --digit;
                            }
                        }
                    for (int c = 0; c < ctas; ++c) {
                        Shared *other = cluster.map_shared_rank(&sh, c);
                        other->digit = digit;
                        other->left = left - before;
                        other->exact = count == left - before;
                    }
                }
                if (ctas > 1)
                    cluster.sync();
                else
                    __syncthreads();
                border |= static_cast<uint32_t>(sh.digit) << shift;
                known_bits |= mask << shift;
                left = sh.left;
                if (sh.exact && border > 0) {
                    border -= 1;
                    left = 0;
                    break;
                }
            }
        }
        // Warps take runs of the CTA's words.
        const int per = (c1 - c0 + kSelWarps - 1) / kSelWarps;
        const int w0 = min(c1, c0 + warp * per), w1 = min(c1, w0 + per);
        const bool any = p.b > 0;
        int ties[1] = {0}, rank_of[1], all[1];
        for (int i = w0; i < w1; ++i) {
            const int j = i * 32 + lane;
            ties[0] += __popc(__ballot_sync(0xffffffffu, any && j < j1 && keys[j] == border));
        }
        warp_starts<1>(cluster, sh, call, ties, rank_of, all);
        int counts[2] = {0, 0}, start[2], total[2];         // free slots, movers
        for (int i = w0; i < w1; ++i) {
            const int j = i * 32 + lane;
            const uint32_t k = j < j1 ? keys[j] : 0u;
            const bool tie = any && j < j1 && k == border;
            const uint32_t t = __ballot_sync(0xffffffffu, tie);
            const bool keep = (any && j < j1 && k > border) ||
                              (tie && rank_of[0] + __popc(t & ((1u << lane) - 1)) < left);
            rank_of[0] += __popc(t);
            const uint32_t word = __ballot_sync(0xffffffffu, keep);
            if (lane == 0)
                bits[i] = word;
            const uint32_t low = __ballot_sync(0xffffffffu, j < p.b);
            counts[0] += __popc(~word & low);
            counts[1] += __popc(word & ~low);
        }
        // (behind this nobody of the cluster reads keys: the lists may be written)
        warp_starts<2>(cluster, sh, call, counts, start, total);
        moves = total[0];
        int h = start[0], m = start[1];
        for (int i = w0; i < w1; ++i) {
            const int j = i * 32 + lane;
            const uint32_t word = bits[i], low = __ballot_sync(0xffffffffu, j < p.b);
            const uint32_t hb = ~word & low, mb = word & ~low, below = (1u << lane) - 1;
            if (hb >> lane & 1u)
                to[h + __popc(hb & below)] = j;
            if (mb >> lane & 1u)
                from[m + __popc(mb & below)] = j;
            h += __popc(hb);
            m += __popc(mb);
        }
        // the lists are there for every CTA of the cluster
        if (ctas > 1)
            cluster.sync();
        else
            __syncthreads();
    }
    // Weights and positions: slots that stay, then those that are filled, then
    // (weights) zeros for the tokens to come.
    const bool copy_w = w_out != w, copy_p = pos_out != pos;
    const int first = rank * kSelThreads + tid, step = ctas * kSelThreads;
    for (int j = first; j < p.b; j += step * kTurns) {
        bool stay[kTurns];
        float wv[kTurns];
        int pv[kTurns];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int i = j + t * step;
            stay[t] = i < p.b && (p.b == p.n || (__ldcg(bits + i / 32) >> (i % 32) & 1u));
            wv[t] = i < p.b && copy_w ? w[i] : 0.f;
            pv[t] = i < p.b ? position(i) : 0;
        }
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int i = j + t * step;
            if (stay[t] && copy_w)
                w_out[i] = wv[t];
            if (stay[t] && (copy_p || i >= p.known))
                pos_out[i] = pv[t];
        }
    }
    for (int i = first; i < moves; i += step * kTurns) {
        int j[kTurns], pv[kTurns];
        float wv[kTurns];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            j[t] = -1;
            if (i + t * step < moves) {
                const int f = __ldcg(from + i + t * step);
                j[t] = __ldcg(to + i + t * step);
                wv[t] = w[f];
                pv[t] = position(f);
            }
        }
#pragma unroll
        for (int t = 0; t < kTurns; ++t)
            if (j[t] >= 0) {
                w_out[j[t]] = wv[t];
                pos_out[j[t]] = pv[t];
            }
    }
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    for (int j = max(p.b, j0) + tid; j < j1; j += kSelThreads)
        w_out[j] = 0.f;
    if (tid == 0 && rank == 0)
        a.moves[row] = moves;
}

// CTAs (row, share of its moves): 16 bytes of K or V per thread and turn.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a)
{
    grid_wait();
    const int row = blockIdx.x, s = row / a.num_kv_heads, kh = row % a.num_kv_heads;
    const int moves = a.moves[row];
    if (kh == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        const Plan p = plan_of(a, s);
        const bool refused = moves < 0;
        if (!refused) {
            a.history_out[2 * s] = p.b;
            a.history_out[2 * s + 1] = p.gone + p.n - p.b;
        } else if (a.history_out != a.history) {
            a.history_out[2 * s] = p.known;
            a.history_out[2 * s + 1] = p.gone;
        }
        a.kept[s] = refused ? p.n : p.b;
    }
    const int32_t *table = a.tables + static_cast<long long>(s) * a.capacity;
    const int32_t *to = a.lists + static_cast<long long>(row) * a.capacity * kPage;
    const int32_t *from = to + static_cast<long long>(a.capacity) * (kPage / 2);
    constexpr int CH = D / 8, PER = 2 * CH;                // 16-byte pieces of a row; of a move
    constexpr int MOVES = kMoveThreads / PER > 0 ? kMoveThreads / PER : 1, TURNS = 4;
    const int piece = threadIdx.x % PER, ch = piece % CH;
    uint8_t *pool = static_cast<uint8_t *>(piece < CH ? a.k_pool : a.v_pool);
    const size_t row_bytes = static_cast<size_t>(a.num_kv_heads) * D * 2;
    auto place = [&](int slot) {
        return pool + (static_cast<size_t>(__ldg(table + slot / kPage)) * kPage + slot % kPage) * row_bytes +
               kh * (D * 2) + ch * 16;
    };
    for (int i0 = blockIdx.y * (MOVES * TURNS) + threadIdx.x / PER; i0 < moves;
         i0 += gridDim.y * (MOVES * TURNS)) {
        uint4 v[TURNS];
        uint8_t *dst[TURNS];
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const int i = i0 + t * MOVES;
            if (i < moves) {
                v[t] = __ldcs(reinterpret_cast<const uint4 *>(place(from[i])));
                dst[t] = place(to[i]);
            }
        }
#pragma unroll
        for (int t = 0; t < TURNS; ++t)
            if (i0 + t * MOVES < moves)
                *reinterpret_cast<uint4 *>(dst[t]) = v[t];
    }
}

template <int D>
cudaError_t launch_d(const EvictArgs &a, int sm_count, cudaStream_t stream)
{
    const long long rows = static_cast<long long>(a.num_seqs) * a.num_kv_heads;
    // CTAs of a row: one for each 2048 slots, up to a cluster's eight
    const long long slots = static_cast<long long>(a.capacity) * kPage;
    int ctas = 1;
    while (ctas < kMostCtas && ctas * 2048LL < slots)
        ctas *= 2;
    const long long share = (slots / 32 + ctas) / ctas * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (share < kSmemKeys ? share : kSmemKeys) * sizeof(uint32_t);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess)
        return e;
    // CTAs for every SM; a row has capacity * 8 moves at most
    constexpr int per = (kMoveThreads / (D / 4) > 0 ? kMoveThreads / (D / 4) : 1) * 4;
    const long long most = (static_cast<long long>(a.capacity) * (kPage / 2) + per - 1) / per;
    long long y = (16LL * sm_count + rows - 1) / rows;
    y = y < most ? y : most;
    return launch_dependent(evict_move_kernel<D>, dim3(static_cast<unsigned>(rows),
                                                       static_cast<unsigned>(y < 1 ? 1 : y)),
                            kMoveThreads, 0, stream, a);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t evict_workspace_bytes(int num_seqs, int num_kv_heads, int capacity)
{
    const size_t rows = static_cast<size_t>(num_seqs) * num_kv_heads;
    return round256(rows * sizeof(int32_t)) + round256(rows * ((capacity + 1) / 2) * sizeof(uint32_t)) +
           rows * capacity * kPage * sizeof(int32_t);
}

cudaError_t launch_evict(int head_dim, EvictArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    const size_t rows = static_cast<size_t>(a.num_seqs) * a.num_kv_heads;
    uint8_t *p = static_cast<uint8_t *>(workspace);
    a.moves = reinterpret_cast<int32_t *>(p);
    p += round256(rows * sizeof(int32_t));
    a.bits = reinterpret_cast<uint32_t *>(p);
    p += round256(rows * ((a.capacity + 1) / 2) * sizeof(uint32_t));
    a.lists = reinterpret_cast<int32_t *>(p);
    switch (head_dim) {
    case 64: return launch_d<64>(a, sm_count, stream);
    case 128: return launch_d<128>(a, sm_count, stream);
    case 256: return launch_d<256>(a, sm_count, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace vfa
