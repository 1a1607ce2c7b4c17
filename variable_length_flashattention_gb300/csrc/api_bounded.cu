// api_bounded.cu -- C ABI entry points of the operators of a bounded cache
// (one-launch paged decode, accumulated key weights, eviction): argument checks
// and launches.  Nothing here allocates or frees device memory.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "internal.h"

namespace {

vfa_status fail(vfa_status st, const char *fmt, ...)
{
    char msg[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return vfa::set_error(st, msg);
}

vfa_status launched(cudaError_t e, const char *what)
{
    if (e == cudaSuccess)
        return VFA_OK;
    return fail(VFA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_head_dim(int d) { return d == 64 || d == 128 || d == 256; }

constexpr int kMaxBlocks = 1 << 26;
constexpr int kMaxHeads = 65535;
constexpr int kMaxCapacity = 1 << 26;           // no more pages than a pool; slots and steps fit 32 bits

vfa_status check_workspace(const void *workspace, size_t bytes, size_t need)
{
    if (!workspace || !aligned(workspace, 256))
        return fail(VFA_ERR_INVALID_ARG, "workspace must be a non-null, 256-byte aligned pointer");
    if (bytes < need)
        return fail(VFA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", bytes, need);
    return VFA_OK;
}

// What the operators over a paged bf16 cache have in common.
vfa_status check_cache(const void *k_pool, const void *v_pool, int num_blocks, const int32_t *tables,
                       int capacity, const int32_t *token_counts, int num_seqs, int num_kv_heads,
                       int head_dim, const int32_t *device_status)
{
    if (!k_pool || !v_pool || !tables || !token_counts)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (num_blocks < 0 || capacity < 0 || num_seqs < 1 || num_kv_heads < 1)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument");
    if (!supported_head_dim(head_dim))
        return fail(VFA_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128, 256)", head_dim);
    if (num_blocks > kMaxBlocks)
        return fail(VFA_ERR_UNSUPPORTED, "num_blocks %d above 2^26 not supported", num_blocks);
    if (num_kv_heads > kMaxHeads)
        return fail(VFA_ERR_UNSUPPORTED, "%d kv heads, at most %d", num_kv_heads, kMaxHeads);
    if (capacity > kMaxCapacity)
        return fail(VFA_ERR_UNSUPPORTED, "capacity %d above 2^26 pages not supported", capacity);
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(tables, 4) ||
        !aligned(token_counts, 4) || !aligned(device_status, 4))
        return fail(VFA_ERR_INVALID_ARG, "pools must be 16-byte aligned, int32 arrays 4-byte");
    return VFA_OK;
}

}  // namespace

extern "C" {

size_t vfa_paged_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                        int capacity)
{
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        !supported_head_dim(head_dim) || capacity < 0 || capacity > kMaxCapacity)
        return 0;
    return vfa::paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, capacity);
}

vfa_status vfa_paged_decode(const void *q, const void *k_pool, const void *v_pool, int num_blocks,
                            const int32_t *tables, int capacity, const int32_t *token_counts,
                            int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int window_left, int sink_tokens, float softmax_scale, void *out,
                            float *lse, const float *key_weights, float *key_weights_out,
                            int32_t *device_status, void *workspace, size_t workspace_bytes,
                            vfa_stream_t stream)
{
    vfa_status st = check_cache(k_pool, v_pool, num_blocks, tables, capacity, token_counts, num_seqs,
                                num_kv_heads, head_dim, device_status);
    if (st)
        return st;
    if (!q || !out || (key_weights && !key_weights_out))
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(VFA_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d",
                    num_q_heads, num_kv_heads);
    if (sink_tokens < 0)
        return fail(VFA_ERR_INVALID_ARG, "sink_tokens %d is negative", sink_tokens);
    if (!std::isfinite(softmax_scale))
        return fail(VFA_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(key_weights, 4) ||
        !aligned(key_weights_out, 4))
        return fail(VFA_ERR_INVALID_ARG, "q and out must be 16-byte aligned, f32 arrays 4-byte");
    // the kernel counts pages, and some per sequence besides, in 32 bits
    if (static_cast<long long>(num_seqs) * (static_cast<long long>(capacity) + 64) > (1LL << 30) ||
        static_cast<long long>(num_kv_heads) * ((num_q_heads / num_kv_heads + 7) / 8) > 65535 ||
        static_cast<long long>(num_seqs) * num_kv_heads > INT_MAX)
        return fail(VFA_ERR_UNSUPPORTED, "num_seqs * capacity or the head count too large");
    if ((st = check_workspace(workspace, workspace_bytes,
                              vfa::paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads,
                                                                head_dim, key_weights ? capacity : 0))))
        return st;
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::PagedDecodeArgs a = {};
    a.q = q;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.tables = tables;
    a.counts = token_counts;
    a.out = out;
    a.lse = lse;
    a.weights = capacity > 0 ? key_weights : nullptr;       // no slots, no weights
    a.weights_out = key_weights_out;
    a.weight_stride = static_cast<long long>(capacity) * 16;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.num_blocks = num_blocks;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.window_left = window_left < 0 ? -1 : window_left;
    a.sink_tokens = window_left < 0 ? 0 : sink_tokens;
    // positive, or a masked -inf times it would be no number; finite, or the zero between
    // equal logits times it would
    const double scale_log2 =
        (softmax_scale > 0.f ? static_cast<double>(softmax_scale) : 1.0 / std::sqrt(double(head_dim))) *
        1.4426950408889634;
    a.scale_log2 = scale_log2 > FLT_MAX ? FLT_MAX
                                        : (scale_log2 < FLT_MIN ? FLT_MIN : static_cast<float>(scale_log2));
    return launched(vfa::launch_paged_decode(head_dim, a, workspace, sms,
                                             reinterpret_cast<cudaStream_t>(stream)),
                    "paged decode launch");
}

size_t vfa_varlen_key_weights_workspace_bytes(int batch, int total_q, int total_k, int max_seqlen_q,
                                              int num_heads)
{
    if (batch < 1 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || num_heads < 1)
        return 0;
    return vfa::key_weights_workspace_bytes(batch, total_q, total_k, max_seqlen_q, num_heads);
}

vfa_status vfa_varlen_key_weights(const void *q, const void *k, const float *lse,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                  int total_q, int total_k, int max_seqlen_q, int batch,
                                  int num_heads, int num_kv_heads, int head_dim,
                                  float softmax_scale, int causal, int window_left,
                                  int sink_tokens, const float *key_weights,
                                  float *key_weights_out, int64_t row_stride, void *workspace,
                                  size_t workspace_bytes, vfa_stream_t stream)
{
    if (!q || !k || !lse || !cu_seqlens_q || !cu_seqlens_k || !key_weights || !key_weights_out)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (batch < 1 || num_heads < 1 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || row_stride < 0)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument (batch %d, heads %d, totals %d/%d)", batch,
                    num_heads, total_q, total_k);
    if (num_kv_heads < 1 || num_heads % num_kv_heads != 0)
        return fail(VFA_ERR_INVALID_ARG, "num_heads %d is not a multiple of num_kv_heads %d", num_heads,
                    num_kv_heads);
    if (causal < 0 || causal > 2)
        return fail(VFA_ERR_INVALID_ARG, "causal must be 0, 1 (top-left) or 2 (bottom-right)");
    if (window_left >= 0 && causal == 0)
        return fail(VFA_ERR_INVALID_ARG, "a sliding window needs a causal mode");
    if (sink_tokens < 0)
        return fail(VFA_ERR_INVALID_ARG, "sink_tokens %d is negative", sink_tokens);
    if (!supported_head_dim(head_dim))
        return fail(VFA_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128, 256)", head_dim);
    if (!(softmax_scale >= 0.f) || softmax_scale > FLT_MAX)
        return fail(VFA_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0 (got %g)",
                    static_cast<double>(softmax_scale));
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) ||
        !aligned(cu_seqlens_k, 4) || !aligned(key_weights, 4) || !aligned(key_weights_out, 4))
        return fail(VFA_ERR_INVALID_ARG, "q and k must be 16-byte aligned, the others 4-byte");
    // tensors as the forward takes them, and a unit count of 32 bits
    const long long pairs = static_cast<long long>(total_k) / 256 + batch;
    const long long chunks = static_cast<long long>(max_seqlen_q) / 1024 + 1;
    if (static_cast<long long>(total_q) * num_heads > (1LL << 31) ||
        static_cast<long long>(total_k) * num_heads > (1LL << 31) || num_kv_heads > kMaxHeads ||
        static_cast<double>(pairs) * static_cast<double>(chunks) * num_heads > double(1LL << 30))
        return fail(VFA_ERR_UNSUPPORTED, "tensor too large");
    vfa_status st = check_workspace(
        workspace, workspace_bytes,
        vfa::key_weights_workspace_bytes(batch, total_q, total_k, max_seqlen_q, num_heads));
    if (st)
        return st;
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::KeyWeightArgs a = {};
    if ((st = vfa::encode_tile_map(&a.tm_q, q, total_q, num_heads, head_dim,
                                   vfa::key_weights_rows(head_dim))) ||
        (st = vfa::encode_tile_map(&a.tm_k, k, total_k, num_kv_heads, head_dim, 128)))
        return st;
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.lse = lse;
    a.weights = key_weights;
    a.weights_out = key_weights_out;
    a.weight_stride = row_stride;
    a.batch = batch;
    a.total_q = total_q;
    a.total_k = total_k;
    a.max_seqlen_q = max_seqlen_q;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    // positive and finite, as in the forward: a masked -inf times it would be no number
    a.scale_log2 = std::fmax(std::fmin(softmax_scale * 1.4426950408889634f, FLT_MAX), FLT_MIN);
    a.causal = causal;
    a.window_left = window_left < 0 ? -1 : window_left;
    a.sink_tokens = window_left < 0 ? 0 : sink_tokens;
    return launched(vfa::launch_key_weights(head_dim, a, workspace, sms,
                                            reinterpret_cast<cudaStream_t>(stream)),
                    "key weights launch");
}

size_t vfa_cache_evict_workspace_bytes(int num_seqs, int num_kv_heads, int capacity)
{
    if (num_seqs < 1 || num_kv_heads < 1 || num_kv_heads > kMaxHeads || capacity < 0 ||
        capacity > kMaxCapacity)
        return 0;
    return vfa::evict_workspace_bytes(num_seqs, num_kv_heads, capacity);
}

vfa_status vfa_cache_evict(void *k_pool, void *v_pool, const int32_t *refcounts, int num_blocks,
                           const int32_t *tables, int capacity, const int32_t *token_counts,
                           const int32_t *budgets, int num_seqs, int num_kv_heads, int head_dim,
                           const float *key_weights, const int32_t *positions,
                           const int32_t *history, int sink_tokens, int recent_tokens,
                           float *key_weights_out, int32_t *positions_out, int32_t *history_out,
                           int32_t *kept, void *workspace, size_t workspace_bytes,
                           int32_t *device_status, vfa_stream_t stream)
{
    vfa_status st = check_cache(k_pool, v_pool, num_blocks, tables, capacity, token_counts, num_seqs,
                                num_kv_heads, head_dim, device_status);
    if (st)
        return st;
    if (!refcounts || !budgets || !key_weights || !positions || !history || !key_weights_out ||
        !positions_out || !history_out || !kept)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (sink_tokens < 0 || recent_tokens < 0)
        return fail(VFA_ERR_INVALID_ARG, "sink_tokens and recent_tokens must not be negative");
    if (!aligned(refcounts, 4) || !aligned(budgets, 4) || !aligned(key_weights, 4) ||
        !aligned(positions, 4) || !aligned(history, 4) || !aligned(key_weights_out, 4) ||
        !aligned(positions_out, 4) || !aligned(history_out, 4) || !aligned(kept, 4))
        return fail(VFA_ERR_INVALID_ARG, "arrays must be 4-byte aligned");
    if (static_cast<long long>(num_seqs) * num_kv_heads > (1 << 27))      // clusters of up to 8 CTAs
        return fail(VFA_ERR_UNSUPPORTED, "num_seqs * num_kv_heads too large");
    if ((st = check_workspace(workspace, workspace_bytes,
                              vfa::evict_workspace_bytes(num_seqs, num_kv_heads, capacity))))
        return st;
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::EvictArgs a = {};
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.refs = refcounts;
    a.tables = tables;
    a.counts = token_counts;
    a.budgets = budgets;
    a.weights = key_weights;
    a.positions = positions;
    a.history = history;
    a.weights_out = key_weights_out;
    a.positions_out = positions_out;
    a.history_out = history_out;
    a.kept = kept;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.num_blocks = num_blocks;
    a.num_kv_heads = num_kv_heads;
    a.sink_tokens = sink_tokens;
    a.recent_tokens = recent_tokens;
    return launched(vfa::launch_evict(head_dim, a, workspace, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "eviction launch");
}

}  // extern "C"
