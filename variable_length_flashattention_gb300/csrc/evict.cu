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
//   select   one CTA per (sequence, kv head).  The border weight is found by its
//            bits, 11, 11 and 10 at a time from the top, by counting the weights
//            that share the bits so far (weights map to unsigned integers of the
//            same order).  Then every warp takes a run of slots: ballots give the
//            ranks of ties, free slots and movers, sums over the warps their
//            starts.  Weights and positions are rewritten here;
//   move     the rows of K and V by the lists, 16 bytes per thread, and the
//            sequences' new state.
// Bound: HBM, 8 D bytes per moved token and kv head, and 12 to 16 bytes per token for weights
// and positions.
#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"

namespace vfa {

namespace {

constexpr int kPage = 16;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
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

// Weights in the order of unsigned integers; any NaN is the largest.
__device__ __forceinline__ uint32_t order_of(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);          // -0 is 0
    if (w != w)
        return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the CTA's warps of one value per warp (its lane 0's).
__device__ __forceinline__ int warp_start(int v, int *s_warp, int *total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0)
        s_warp[warp] = v;
    __syncthreads();
    int x = s_warp[lane], y = x;                           // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o)
            y += z;
    }
    *total = __shfl_sync(0xffffffffu, y, 31);
    return __shfl_sync(0xffffffffu, y - x, warp);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a)
{
    static_assert(kSelWarps == 32, "one lane per warp in warp_start");
    grid_wait();
    grid_release();
    __shared__ int s_bins[kBins];
    __shared__ int s_warp[kSelWarps];
    __shared__ int s_digit, s_left;
    const int row = blockIdx.x, s = row / a.num_kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Plan p = plan_of(a, s);
    // pages that are none, or that a move would write although another row has them
    bool bad = p.bad;
    if (!bad) {
        const int pages = (p.n + kPage - 1) / kPage, written = p.b < p.n ? (p.b + kPage - 1) / kPage : 0;
        for (int j = tid; j < pages; j += kSelThreads) {
            const int id = a.tables[static_cast<long long>(s) * a.capacity + j];
            bad |= id < 0 || id >= a.num_blocks || (j < written && a.refs[id] != 1);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
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

    int moves = 0;
    if (p.b < p.n) {
        // Tokens that stay whatever their weight, and how many others do.
        int safe = 0;
        for (int j = tid; j < p.n; j += kSelThreads)
            safe += p.safe(position(j));
        int total;
        warp_start(__reduce_add_sync(0xffffffffu, safe), s_warp, &total);
        // More than may stay (stored positions that are not one per token): the lowest
        // slots of them do.
        const bool crowd = total > p.b;
        int left = crowd ? p.b : p.b - total;
        // The border: the left-th largest weight of the others, and how many of that
        // weight stay.
        uint32_t border = 0, known_bits = 0;
        if (left > 0 && !crowd) {
            for (int turn = 0; turn < 3; ++turn) {
                const int shift = turn == 0 ? 21 : (turn == 1 ? 10 : 0);
                const uint32_t mask = turn == 2 ? 1023u : 2047u;
                __syncthreads();
                for (int i = tid; i < kBins; i += kSelThreads)
                    s_bins[i] = 0;
                __syncthreads();
                for (int j = tid; j < p.n; j += kSelThreads) {
                    const uint32_t k = order_of(w[j]);
                    if ((k & known_bits) == border && !p.safe(position(j)))
                        atomicAdd(&s_bins[k >> shift & mask], 1);
                }
                __syncthreads();
                // thread t holds the two bins 2047 - 2t, 2046 - 2t: a scan from the top
                const int hi = s_bins[kBins - 1 - 2 * tid], lo = s_bins[kBins - 2 - 2 * tid];
                int x = hi + lo;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o)
                        x += y;
                }
                int all;
                const int before = warp_start(__shfl_sync(0xffffffffu, x, 31), s_warp, &all) + x - hi - lo;
                if (before < left && left <= before + hi) {
                    s_digit = kBins - 1 - 2 * tid;
                    s_left = left - before;
                } else if (before + hi < left && left <= before + hi + lo) {
                    s_digit = kBins - 2 - 2 * tid;
                    s_left = left - before - hi;
                }
                __syncthreads();
                border |= static_cast<uint32_t>(s_digit) << shift;
                known_bits |= mask << shift;
                left = s_left;
            }
        }
        const bool any = left > 0 && !crowd;    // a border exists
        // Warps take runs of slots, whole words of 32.
        const int words = (p.n + 31) / 32, per = (words + kSelWarps - 1) / kSelWarps;
        const int w0 = min(words, warp * per), w1 = min(words, w0 + per);
        int ties = 0;
        for (int i = w0; i < w1; ++i) {
            const int j = i * 32 + lane;
            const bool tie = j < p.n && (crowd ? p.safe(position(j))
                                               : any && order_of(w[j]) == border && !p.safe(position(j)));
            ties += __popc(__ballot_sync(0xffffffffu, tie));
        }
        int rank = warp_start(ties, s_warp, &total);
        int holes = 0, movers = 0;
        for (int i = w0; i < w1; ++i) {
            const int j = i * 32 + lane;
            bool keep = false, tie = false;
            if (j < p.n) {
                const uint32_t k = order_of(w[j]);
                const bool safe_one = p.safe(position(j));
                keep = !crowd && (safe_one || (any && k > border));
                tie = crowd ? safe_one : any && !keep && k == border;
            }
            const uint32_t t = __ballot_sync(0xffffffffu, tie);
            keep |= tie && rank + __popc(t & ((1u << lane) - 1)) < left;
            rank += __popc(t);
            const uint32_t word = __ballot_sync(0xffffffffu, keep);
            if (lane == 0)
                bits[i] = word;
            const uint32_t low = __ballot_sync(0xffffffffu, j < p.b);
            holes += __popc(~word & low);
            movers += __popc(word & ~low);
        }
        const int hole0 = warp_start(holes, s_warp, &moves), mover0 = warp_start(movers, s_warp, &total);
        int h = hole0, m = mover0;
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
        __syncthreads();
    }
    // Weights and positions: slots that stay, then those that are filled, then
    // (weights) zeros for the tokens to come.
    const bool copy_w = w_out != w, copy_p = pos_out != pos;
    for (int j = tid; j < p.b; j += kSelThreads) {
        const bool stay = p.b == p.n || (bits[j / 32] >> (j % 32) & 1u);
        if (stay && copy_w)
            w_out[j] = w[j];
        if (stay && (copy_p || j >= p.known))
            pos_out[j] = position(j);
    }
    for (int i = tid; i < moves; i += kSelThreads) {
        const int j = to[i], f = from[i];
        w_out[j] = w[f];
        pos_out[j] = position(f);
    }
    __syncthreads();
    for (int j = p.b + tid; j < p.n; j += kSelThreads)
        w_out[j] = 0.f;
    if (tid == 0)
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
    cudaError_t e = launch_dependent(evict_select_kernel, dim3(static_cast<unsigned>(rows)), kSelThreads, 0,
                                     stream, a);
    if (e != cudaSuccess)
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
