// api_serving.cu -- C ABI entry points of the operators around attention
// (query / key norm and rotation, the 4-bit paged cache, page operations):
// argument checks and launches.  Nothing here allocates or frees device
// memory.
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
constexpr int kMaxHeads = 65535;            // a token's or a page's bytes stay within 32 bits
constexpr int kMaxPageBytes = INT_MAX - 4095;       // the copy counts a page's pieces in 32 bits

// ---------------------------------------------------------------- norm, rotation

vfa_status check_rope(const vfa::RopeArgs &a, int rotary_dim, int head_dim, const void *const *tensors,
                      const int64_t *strides, const int *heads, int n)
{
    if (a.tokens < 0 || a.heads[0] < 1 || a.heads[1] < 1)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument (tokens %d, heads %d / %d)", a.tokens,
                    a.heads[0], a.heads[1]);
    if (!supported_head_dim(head_dim))
        return fail(VFA_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128, 256)", head_dim);
    if (a.heads[0] > kMaxHeads || a.heads[1] > kMaxHeads)
        return fail(VFA_ERR_UNSUPPORTED, "%d / %d heads, at most %d", a.heads[0], a.heads[1], kMaxHeads);
    if (rotary_dim < 0 || rotary_dim > head_dim)
        return fail(VFA_ERR_INVALID_ARG, "rotary_dim %d outside [0, head_dim]", rotary_dim);
    if (rotary_dim % 16 != 0)
        return fail(VFA_ERR_UNSUPPORTED, "rotary_dim %d not supported (multiples of 16)", rotary_dim);
    if (rotary_dim > 0 && ((a.tokens > 0 && (!a.positions || !a.table)) || a.num_axes < 1))
        return fail(VFA_ERR_INVALID_ARG, "a rotation needs positions, a table and an axis");
    if (!(a.eps >= 0.f) || a.eps > FLT_MAX)
        return fail(VFA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    for (int i = 0; i < n; ++i) {
        if (!tensors[i] && a.tokens > 0)
            return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
        if (!aligned(tensors[i], 16))
            return fail(VFA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
        if (strides[i] % 8 != 0 || strides[i] < static_cast<int64_t>(heads[i]) * head_dim)
            return fail(VFA_ERR_INVALID_ARG,
                        "token strides must be multiples of 8 and at least heads * head_dim");
    }
    if (!aligned(a.positions, 4) || !aligned(a.table, 16) || !aligned(a.weight[0], 4) ||
        !aligned(a.weight[1], 4))
        return fail(VFA_ERR_INVALID_ARG,
                    "positions and weights must be 4-byte aligned, the table 16-byte");
    return VFA_OK;
}

void rope_args(vfa::RopeArgs *a, const void *q, const void *k, int64_t q_stride, int64_t k_stride,
               const int32_t *positions, int num_axes, const uint64_t *table, int rotary_dim,
               int interleaved, const float *q_weight, const float *k_weight, float eps, int tokens,
               int num_q_heads, int num_kv_heads)
{
    *a = vfa::RopeArgs{};
    a->x[0] = q;
    a->x[1] = k;
    a->x_stride[0] = q_stride;
    a->x_stride[1] = k_stride;
    a->positions = positions;
    a->num_axes = num_axes;
    a->table = table;
    a->half = rotary_dim / 2;
    a->interleaved = interleaved != 0;
    a->weight[0] = q_weight;
    a->weight[1] = k_weight;
    a->eps = eps;
    a->tokens = tokens;
    a->heads[0] = num_q_heads;
    a->heads[1] = num_kv_heads;
}

// ---------------------------------------------------------------- 4-bit cache

bool power_of_two(float x)
{
    int e;
    return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e - 1 >= -64 && e - 1 <= 64;
}

vfa_status check_kv4(const void *pool, int num_blocks, const int32_t *tables, int capacity,
                     int num_seqs, int num_kv_heads, int head_dim, float descale_k,
                     float descale_v)
{
    if (!pool || !tables)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (num_blocks < 0 || capacity < 0 || num_seqs < 1 || num_kv_heads < 1)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument");
    if (!supported_head_dim(head_dim))
        return fail(VFA_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128, 256)", head_dim);
    if (num_blocks > kMaxBlocks)
        return fail(VFA_ERR_UNSUPPORTED, "num_blocks %d above 2^26 not supported", num_blocks);
    if (num_kv_heads > kMaxHeads)
        return fail(VFA_ERR_UNSUPPORTED, "%d kv heads, at most %d", num_kv_heads, kMaxHeads);
    if (!power_of_two(descale_k) || !power_of_two(descale_v))
        return fail(VFA_ERR_INVALID_ARG,
                    "descale_k and descale_v must be powers of two in [2^-64, 2^64]");
    if (!aligned(pool, 16) || !aligned(tables, 4))
        return fail(VFA_ERR_INVALID_ARG, "the pool must be 16-byte aligned, tables 4-byte");
    return VFA_OK;
}

vfa_status kv4_move(bool write, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                    int total, const void *pool, int num_blocks, const int32_t *tables,
                    int capacity, const int32_t *cu_seqlens, const int32_t *start_positions,
                    int num_seqs, int num_kv_heads, int head_dim, float descale_k,
                    float descale_v, int32_t *device_status, vfa_stream_t stream)
{
    vfa_status st = check_kv4(pool, num_blocks, tables, capacity, num_seqs, num_kv_heads, head_dim,
                              descale_k, descale_v);
    if (st)
        return st;
    if (total < 0)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument (total %d)", total);
    if (((!k || !v) && total > 0) || !cu_seqlens || !start_positions)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_seqlens, 4) ||
        !aligned(start_positions, 4) || !aligned(device_status, 4))
        return fail(VFA_ERR_INVALID_ARG, "k and v must be 16-byte aligned, int32 arrays 4-byte");
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < row || v_stride < row)
        return fail(VFA_ERR_INVALID_ARG,
                    "token strides must be multiples of 8 and at least num_kv_heads * head_dim");
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    if (total == 0)
        return VFA_OK;
    vfa::Kv4MoveArgs a;
    a.k = const_cast<void *>(k);
    a.v = const_cast<void *>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.pool = const_cast<void *>(pool);
    a.tables = tables;
    a.cu = cu_seqlens;
    a.start = start_positions;
    a.status = device_status;
    a.total = total;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.num_blocks = num_blocks;
    a.num_kv_heads = num_kv_heads;
    a.k_scale = write ? 1.f / descale_k : descale_k;
    a.v_scale = write ? 1.f / descale_v : descale_v;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return write ? launched(vfa::launch_kv4_write(head_dim, a, sms, s), "4-bit cache write launch")
                 : launched(vfa::launch_kv4_gather(head_dim, a, sms, s), "4-bit cache gather launch");
}

// ---------------------------------------------------------------- pages

vfa_status check_pages(const void *refcounts, int num_blocks, const void *tables, int capacity,
                       const void *token_counts, int num_seqs, int block_size,
                       const void *device_status)
{
    if (!refcounts || !tables || !token_counts)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (num_blocks < 1 || capacity < 1 || num_seqs < 1 || block_size < 1)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument");
    if (num_blocks > kMaxBlocks)
        return fail(VFA_ERR_UNSUPPORTED, "num_blocks %d above 2^26 not supported", num_blocks);
    if (!aligned(refcounts, 4) || !aligned(tables, 4) || !aligned(token_counts, 4) ||
        !aligned(device_status, 4))
        return fail(VFA_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    return VFA_OK;
}

vfa_status check_page_workspace(const void *workspace, size_t bytes, int num_blocks, int num_seqs,
                                int num_forks)
{
    if (!workspace || !aligned(workspace, 16))
        return fail(VFA_ERR_INVALID_ARG, "workspace must be a non-null, 16-byte aligned pointer");
    const size_t need = vfa::page_workspace_bytes(num_blocks, num_seqs, num_forks);
    if (bytes < need)
        return fail(VFA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", bytes, need);
    return VFA_OK;
}

vfa_status page_pools(void *const *pools, const int *page_bytes, int num_pools, vfa::PagePools *p)
{
    if (num_pools < 0 || (num_pools > 0 && (!pools || !page_bytes)))
        return fail(VFA_ERR_INVALID_ARG, "bad pool list");
    if (num_pools > vfa::kMaxPagePools)
        return fail(VFA_ERR_UNSUPPORTED, "%d pools, at most %d in one call", num_pools,
                    vfa::kMaxPagePools);
    *p = vfa::PagePools{};
    p->n = num_pools;
    for (int i = 0; i < num_pools; ++i) {
        if (!pools[i] || !aligned(pools[i], 16) || page_bytes[i] < 16 || page_bytes[i] % 16 != 0)
            return fail(VFA_ERR_INVALID_ARG,
                        "pool %d must be 16-byte aligned with pages of a multiple of 16 bytes", i);
        if (page_bytes[i] > kMaxPageBytes)
            return fail(VFA_ERR_UNSUPPORTED, "pool %d has pages of %d bytes, at most %d", i,
                        page_bytes[i], kMaxPageBytes);
        p->ptr[i] = static_cast<uint8_t *>(pools[i]);
        p->page_bytes[i] = page_bytes[i];
    }
    return VFA_OK;
}

}  // namespace

extern "C" {

vfa_status vfa_qk_norm_rope_fwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride,
                                const int32_t *positions, int num_axes, const uint64_t *table,
                                int rotary_dim, int interleaved, const float *q_weight,
                                const float *k_weight, float eps, int tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, void *q_out, void *k_out,
                                int64_t q_out_stride, int64_t k_out_stride, vfa_stream_t stream)
{
    vfa::RopeArgs a;
    rope_args(&a, q, k, q_stride, k_stride, positions, num_axes, table, rotary_dim, interleaved,
              q_weight, k_weight, eps, tokens, num_q_heads, num_kv_heads);
    a.y[0] = q_out;
    a.y[1] = k_out;
    a.y_stride[0] = q_out_stride;
    a.y_stride[1] = k_out_stride;
    const void *tensors[4] = {q, k, q_out, k_out};
    const int64_t strides[4] = {q_stride, k_stride, q_out_stride, k_out_stride};
    const int heads[4] = {num_q_heads, num_kv_heads, num_q_heads, num_kv_heads};
    vfa_status st = check_rope(a, rotary_dim, head_dim, tensors, strides, heads, 4);
    if (st)
        return st;
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    return launched(vfa::launch_rope_fwd(head_dim, a, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "norm and rotation launch");
}

size_t vfa_qk_norm_rope_bwd_workspace_bytes(int head_dim)
{
    if (!supported_head_dim(head_dim))
        return 0;
    return static_cast<size_t>(vfa::kRopeMaxCtas) * 2 * head_dim * sizeof(float);
}

vfa_status vfa_qk_norm_rope_bwd(const void *q, const void *k, int64_t q_stride, int64_t k_stride,
                                const void *dq_out, const void *dk_out, int64_t dq_out_stride,
                                int64_t dk_out_stride, const int32_t *positions, int num_axes,
                                const uint64_t *table, int rotary_dim, int interleaved,
                                const float *q_weight, const float *k_weight, float eps,
                                int tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                void *dq, void *dk, int64_t dq_stride, int64_t dk_stride,
                                float *dq_weight, float *dk_weight, void *workspace,
                                size_t workspace_bytes, vfa_stream_t stream)
{
    vfa::RopeArgs a;
    rope_args(&a, q, k, q_stride, k_stride, positions, num_axes, table, rotary_dim, interleaved,
              q_weight, k_weight, eps, tokens, num_q_heads, num_kv_heads);
    a.dy[0] = dq_out;
    a.dy[1] = dk_out;
    a.dy_stride[0] = dq_out_stride;
    a.dy_stride[1] = dk_out_stride;
    a.y[0] = dq;
    a.y[1] = dk;
    a.y_stride[0] = dq_stride;
    a.y_stride[1] = dk_stride;
    a.dweight[0] = q_weight ? dq_weight : nullptr;
    a.dweight[1] = k_weight ? dk_weight : nullptr;
    const void *tensors[6] = {q, k, dq_out, dk_out, dq, dk};
    const int64_t strides[6] = {q_stride, k_stride, dq_out_stride, dk_out_stride, dq_stride,
                                dk_stride};
    const int heads[6] = {num_q_heads, num_kv_heads, num_q_heads, num_kv_heads, num_q_heads,
                          num_kv_heads};
    vfa_status st = check_rope(a, rotary_dim, head_dim, tensors, strides, heads, 6);
    if (st)
        return st;
    if ((q_weight && !dq_weight) || (k_weight && !dk_weight))
        return fail(VFA_ERR_INVALID_ARG, "a weight's gradient has nowhere to go (null pointer)");
    if (q_weight || k_weight) {
        const size_t need = vfa_qk_norm_rope_bwd_workspace_bytes(head_dim);
        if (!workspace || !aligned(workspace, 16))
            return fail(VFA_ERR_INVALID_ARG,
                        "workspace must be a non-null, 16-byte aligned pointer");
        if (workspace_bytes < need)
            return fail(VFA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes",
                        workspace_bytes, need);
        if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4))
            return fail(VFA_ERR_INVALID_ARG, "weight gradients must be 4-byte aligned");
    }
    a.partial = static_cast<float *>(workspace);
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    return launched(vfa::launch_rope_bwd(head_dim, a, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "norm and rotation backward launch");
}

size_t vfa_kv4_block_bytes(int num_kv_heads, int head_dim)
{
    if (num_kv_heads < 1 || num_kv_heads > kMaxHeads || !supported_head_dim(head_dim))
        return 0;
    return static_cast<size_t>(num_kv_heads) * vfa::kv4_head_page_bytes(head_dim);
}

vfa_status vfa_kv4_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                         int total, void *pool, int num_blocks, const int32_t *tables,
                         int capacity, const int32_t *cu_seqlens, const int32_t *start_positions,
                         int num_seqs, int num_kv_heads, int head_dim, float descale_k,
                         float descale_v, int32_t *device_status, vfa_stream_t stream)
{
    return kv4_move(true, k, v, k_stride, v_stride, total, pool, num_blocks, tables, capacity,
                    cu_seqlens, start_positions, num_seqs, num_kv_heads, head_dim, descale_k,
                    descale_v, device_status, stream);
}

vfa_status vfa_kv4_gather(void *k, void *v, int64_t k_stride, int64_t v_stride, int total,
                          const void *pool, int num_blocks, const int32_t *tables, int capacity,
                          const int32_t *cu_seqlens, const int32_t *start_positions, int num_seqs,
                          int num_kv_heads, int head_dim, float descale_k, float descale_v,
                          int32_t *device_status, vfa_stream_t stream)
{
    return kv4_move(false, k, v, k_stride, v_stride, total, pool, num_blocks, tables, capacity,
                    cu_seqlens, start_positions, num_seqs, num_kv_heads, head_dim, descale_k,
                    descale_v, device_status, stream);
}

size_t vfa_kv4_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                      int head_dim)
{
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        !supported_head_dim(head_dim))
        return 0;
    return vfa::kv4_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim);
}

vfa_status vfa_kv4_decode(const void *q, const void *pool, int num_blocks, const int32_t *tables,
                          int capacity, const int32_t *token_counts, int num_seqs,
                          int num_q_heads, int num_kv_heads, int head_dim, float descale_k,
                          float descale_v, float softmax_scale, void *out, float *lse,
                          int32_t *device_status, void *workspace, size_t workspace_bytes,
                          vfa_stream_t stream)
{
    vfa_status st = check_kv4(pool, num_blocks, tables, capacity, num_seqs, num_kv_heads, head_dim,
                              descale_k, descale_v);
    if (st)
        return st;
    if (!q || !token_counts || !out)
        return fail(VFA_ERR_INVALID_ARG, "null pointer argument");
    if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(VFA_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d",
                    num_q_heads, num_kv_heads);
    if (!std::isfinite(softmax_scale))
        return fail(VFA_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(token_counts, 4) || !aligned(lse, 4) ||
        !aligned(device_status, 4))
        return fail(VFA_ERR_INVALID_ARG, "q and out must be 16-byte aligned, the others 4-byte");
    // the kernel counts pages, and some per sequence besides, in 32 bits
    if (static_cast<long long>(num_seqs) * (static_cast<long long>(capacity) + 64) > (1LL << 30) ||
        static_cast<long long>(num_kv_heads) * ((num_q_heads / num_kv_heads + 7) / 8) > 65535)
        return fail(VFA_ERR_UNSUPPORTED, "num_seqs * capacity or the head count too large");
    if (!workspace || !aligned(workspace, 256))
        return fail(VFA_ERR_INVALID_ARG, "workspace must be a non-null, 256-byte aligned pointer");
    const size_t need = vfa::kv4_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim);
    if (workspace_bytes < need)
        return fail(VFA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes,
                    need);
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::Kv4DecodeArgs a = {};
    a.q = q;
    a.pool = static_cast<const uint8_t *>(pool);
    a.tables = tables;
    a.counts = token_counts;
    a.out = out;
    a.lse = lse;
    a.status = device_status;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.num_blocks = num_blocks;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    const double scale_log2 =
        (softmax_scale > 0.f ? static_cast<double>(softmax_scale) : 1.0 / std::sqrt(double(head_dim))) *
        descale_k * 1.4426950408889634;
    a.scale_log2 = scale_log2 > FLT_MAX ? INFINITY : static_cast<float>(scale_log2);
    a.descale_v = descale_v;
    return launched(vfa::launch_kv4_decode(head_dim, a, workspace, sms,
                                           reinterpret_cast<cudaStream_t>(stream)),
                    "4-bit cache decode launch");
}

size_t vfa_pages_workspace_bytes(int num_blocks, int num_seqs, int num_forks)
{
    if (num_blocks < 1 || num_blocks > kMaxBlocks || num_seqs < 1 || num_forks < 0 ||
        num_forks > kMaxBlocks)
        return 0;
    return vfa::page_workspace_bytes(num_blocks, num_seqs, num_forks);
}

vfa_status vfa_pages_extend(int32_t *refcounts, int num_blocks, int32_t *tables, int capacity,
                            int32_t *token_counts, int num_seqs, const int32_t *add_tokens,
                            int block_size, void *workspace, size_t workspace_bytes,
                            int32_t *device_status, vfa_stream_t stream)
{
    vfa_status st = check_pages(refcounts, num_blocks, tables, capacity, token_counts, num_seqs,
                                block_size, device_status);
    if (st || (st = check_page_workspace(workspace, workspace_bytes, num_blocks, num_seqs, 0)))
        return st;
    if (!add_tokens || !aligned(add_tokens, 4))
        return fail(VFA_ERR_INVALID_ARG, "add_tokens must be a non-null, aligned pointer");
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::PageArgs a = {};
    a.refs = refcounts;
    a.tables = tables;
    a.counts = token_counts;
    a.add = add_tokens;
    a.status = device_status;
    a.ws = static_cast<int32_t *>(workspace);
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.block_size = block_size;
    return launched(vfa::launch_pages_extend(a, reinterpret_cast<cudaStream_t>(stream)),
                    "page extend launch");
}

vfa_status vfa_pages_fork(int32_t *refcounts, int num_blocks, int32_t *tables, int capacity,
                          int32_t *token_counts, int num_seqs, const int32_t *parents,
                          const int32_t *children, int num_forks, void *const *pools,
                          const int *page_bytes, int num_pools, int block_size, void *workspace,
                          size_t workspace_bytes, int32_t *device_status, vfa_stream_t stream)
{
    vfa::PagePools p;
    vfa_status st = check_pages(refcounts, num_blocks, tables, capacity, token_counts, num_seqs,
                                block_size, device_status);
    if (st || (st = page_pools(pools, page_bytes, num_pools, &p)))
        return st;
    if (num_forks < 0 || (num_forks > 0 && (!parents || !children)) || !aligned(parents, 4) ||
        !aligned(children, 4))
        return fail(VFA_ERR_INVALID_ARG, "parents and children must be non-null, aligned pointers");
    if (num_forks > kMaxBlocks)
        return fail(VFA_ERR_UNSUPPORTED, "num_forks %d above 2^26 not supported", num_forks);
    if ((st = check_page_workspace(workspace, workspace_bytes, num_blocks, num_seqs, num_forks)))
        return st;
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    if (num_forks == 0)
        return VFA_OK;
    vfa::PageArgs a = {};
    a.refs = refcounts;
    a.tables = tables;
    a.counts = token_counts;
    a.parents = parents;
    a.children = children;
    a.status = device_status;
    a.ws = static_cast<int32_t *>(workspace);
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.block_size = block_size;
    a.n = num_forks;
    return launched(vfa::launch_pages_fork(a, p, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "page fork launch");
}

vfa_status vfa_pages_free(int32_t *refcounts, int num_blocks, const int32_t *tables, int capacity,
                          int32_t *token_counts, int num_seqs, const int32_t *seqs, int n,
                          int block_size, int32_t *device_status, vfa_stream_t stream)
{
    vfa_status st = check_pages(refcounts, num_blocks, tables, capacity, token_counts, num_seqs,
                                block_size, device_status);
    if (st)
        return st;
    if (n < 0 || (n > 0 && !seqs) || !aligned(seqs, 4))
        return fail(VFA_ERR_INVALID_ARG, "seqs must be a non-null, aligned pointer");
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    if (n == 0)
        return VFA_OK;
    vfa::PageArgs a = {};
    a.refs = refcounts;
    a.tables = const_cast<int32_t *>(tables);
    a.counts = token_counts;
    a.seqs = seqs;
    a.status = device_status;
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.block_size = block_size;
    a.n = n;
    return launched(vfa::launch_pages_free(a, reinterpret_cast<cudaStream_t>(stream)),
                    "page free launch");
}

vfa_status vfa_pages_truncate(const int32_t *refcounts, int num_blocks, const int32_t *tables,
                              int capacity, const int32_t *token_counts, int num_seqs,
                              const int32_t *new_counts, int block_size, int32_t *refcounts_out,
                              int32_t *token_counts_out, void *workspace, size_t workspace_bytes,
                              int32_t *device_status, vfa_stream_t stream)
{
    vfa_status st = check_pages(refcounts, num_blocks, tables, capacity, token_counts, num_seqs,
                                block_size, device_status);
    if (st)
        return st;
    if (!new_counts || !refcounts_out || !token_counts_out || !aligned(new_counts, 4) ||
        !aligned(refcounts_out, 4) || !aligned(token_counts_out, 4))
        return fail(VFA_ERR_INVALID_ARG,
                    "new_counts and the outputs must be non-null, aligned pointers");
    const size_t need = 2 * static_cast<size_t>(num_seqs) * sizeof(int32_t);
    if (!workspace || !aligned(workspace, 16))
        return fail(VFA_ERR_INVALID_ARG, "workspace must be a non-null, 16-byte aligned pointer");
    if (workspace_bytes < need)
        return fail(VFA_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::PageArgs a = {};
    a.refs = const_cast<int32_t *>(refcounts);
    a.refs_out = refcounts_out;
    a.tables = const_cast<int32_t *>(tables);
    a.counts = const_cast<int32_t *>(token_counts);
    a.counts_out = token_counts_out;
    a.new_counts = new_counts;
    a.status = device_status;
    a.ws = static_cast<int32_t *>(workspace);
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.block_size = block_size;
    return launched(vfa::launch_pages_truncate(a, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "page truncate launch");
}

vfa_status vfa_pages_compact(const int32_t *refcounts, int num_blocks, const int32_t *tables,
                             int capacity, const int32_t *token_counts, int num_seqs,
                             void *const *pools, const int *page_bytes, int num_pools,
                             int block_size, int32_t *refcounts_out, int32_t *tables_out,
                             int32_t *num_used, void *workspace, size_t workspace_bytes,
                             int32_t *device_status, vfa_stream_t stream)
{
    vfa::PagePools p;
    vfa_status st = check_pages(refcounts, num_blocks, tables, capacity, token_counts, num_seqs,
                                block_size, device_status);
    if (st || (st = page_pools(pools, page_bytes, num_pools, &p)) ||
        (st = check_page_workspace(workspace, workspace_bytes, num_blocks, num_seqs, 0)))
        return st;
    if (!refcounts_out || !tables_out || !num_used || !aligned(refcounts_out, 4) ||
        !aligned(tables_out, 4) || !aligned(num_used, 4))
        return fail(VFA_ERR_INVALID_ARG, "outputs must be non-null, aligned pointers");
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    vfa::PageArgs a = {};
    a.refs = const_cast<int32_t *>(refcounts);
    a.refs_out = refcounts_out;
    a.tables = const_cast<int32_t *>(tables);
    a.tables_out = tables_out;
    a.counts = const_cast<int32_t *>(token_counts);
    a.num_used = num_used;
    a.status = device_status;
    a.ws = static_cast<int32_t *>(workspace);
    a.num_blocks = num_blocks;
    a.num_seqs = num_seqs;
    a.capacity = capacity;
    a.block_size = block_size;
    return launched(vfa::launch_pages_compact(a, p, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "page compact launch");
}

vfa_status vfa_pages_copy(void *const *pools, const int *page_bytes, int num_pools,
                          const int32_t *src, const int32_t *dst, int n, int num_blocks,
                          int32_t *device_status, vfa_stream_t stream)
{
    vfa::PagePools p;
    vfa_status st = page_pools(pools, page_bytes, num_pools, &p);
    if (st)
        return st;
    if (n < 0 || (n > 0 && (!src || !dst)) || !aligned(src, 4) || !aligned(dst, 4) ||
        !aligned(device_status, 4))
        return fail(VFA_ERR_INVALID_ARG, "src and dst must be non-null, aligned pointers");
    if (num_blocks < 1)
        return fail(VFA_ERR_INVALID_ARG, "bad size argument");
    int sms;
    if ((st = vfa::device_sm_count(&sms)))
        return st;
    if (n == 0 || num_pools == 0)
        return VFA_OK;
    return launched(vfa::launch_pages_copy(p, src, dst, n, num_blocks, device_status, sms,
                                           reinterpret_cast<cudaStream_t>(stream)),
                    "page copy launch");
}

}  // extern "C"
