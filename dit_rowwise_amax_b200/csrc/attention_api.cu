// C-ABI entry points of the attention operators (declared and documented in
// include/fp8dit.h): rotary positions, the key / value cache's append and
// attention over it. Arguments are checked here; nothing is computed on the
// host but the launch's size and the rotary frequencies in turns.
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace fp8dit {
namespace {

fp8dit_status invalid(const char* msg) {
    set_error("invalid argument: %s", msg);
    return FP8DIT_ERR_INVALID_ARG;
}
fp8dit_status unsupported(const char* msg) {
    set_error("unsupported shape: %s", msg);
    return FP8DIT_ERR_UNSUPPORTED_SHAPE;
}
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxTokens = 1ll << 30;
constexpr int32_t kMaxHeads = 65535;

// nullptr: fine; else what is wrong with x as [tokens, heads > 0, dim].
const char* heads_problem(const fp8dit_heads& x, int dim) {
    if (x.ptr == nullptr || !aligned(x.ptr, 16)) return "a tensor's pointer must be non-null and 16-byte aligned";
    if (x.reserved != 0) return "reserved fields must be 0";
    if (x.token_stride % 8 != 0 || x.head_stride % 8 != 0 || x.head_stride < dim || x.token_stride < dim)
        return "token and head strides must be multiples of 8 and at least dim";
    return nullptr;
}
HeadsView view(const fp8dit_heads& x) { return HeadsView{x.ptr, x.token_stride, x.head_stride, x.heads}; }

fp8dit_status check_cache(const fp8dit_kv_cache* c, KvCacheView* v) {
    if (!c) return invalid("null cache");
    if (c->head_dim != 64 && c->head_dim != 128) return unsupported("head_dim must be 64 or 128");
    if (c->block_tokens != 16 && c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128)
        return unsupported("block_tokens must be 16, 32, 64 or 128");
    if (c->n_blocks <= 0 || c->kv_heads <= 0) return invalid("n_blocks and kv_heads must be > 0");
    if (c->kv_heads > kMaxHeads) return unsupported("too many kv heads");
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return invalid("the cache's codes must be non-null and 16-byte aligned");
    if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return invalid("the cache's scales must be non-null and 4-byte aligned");
    const int log2 = c->block_tokens == 16 ? 4 : c->block_tokens == 32 ? 5 : c->block_tokens == 64 ? 6 : 7;
    *v = KvCacheView{c->k, c->v, c->k_scale, c->v_scale, c->n_blocks, c->kv_heads, c->head_dim, log2};
    return FP8DIT_OK;
}

fp8dit_status check_batch(const fp8dit_kv_batch* b, const KvCacheView& c, KvBatchView* v) {
    if (!b) return invalid("null batch");
    if (b->n_requests < 0 || b->total_tokens < 0 || b->max_new < 0 || b->max_kv < 0 || b->table_width < 0)
        return invalid("the batch's counts must be >= 0");
    if (b->n_requests > 65535 || b->total_tokens > kMaxTokens || b->max_new > kMaxTokens || b->max_kv > kMaxTokens)
        return unsupported("too many requests or tokens");
    if ((int64_t)b->max_kv > ((int64_t)b->table_width << c.block_log2))
        return invalid("max_kv exceeds table_width * block_tokens");
    if (b->n_requests > 0 && b->total_tokens > 0 && b->max_new > 0) {
        if (!b->kv_lens || !b->offsets || !aligned(b->kv_lens, 4) || !aligned(b->offsets, 4))
            return invalid("kv_lens and offsets must be non-null and 4-byte aligned");
        if (b->max_kv > 0 && (!b->block_table || !aligned(b->block_table, 4)))
            return invalid("block_table must be non-null and 4-byte aligned");
    }
    *v = KvBatchView{b->block_table, b->kv_lens, b->offsets, b->total_tokens,
                     b->n_requests, b->table_width, b->max_new,
                     b->max_kv};
    return FP8DIT_OK;
}

bool nothing(const KvBatchView& b) { return b.n == 0 || b.total == 0 || b.max_new == 0; }

// Query heads over a cache, and the bound that keeps the plan's numbers in 32 bits.
fp8dit_status check_q_heads(int32_t q_heads, const KvCacheView& c, const KvBatchView& b) {
    if (q_heads <= 0 || q_heads % c.heads != 0) return invalid("q's heads must be a multiple of the cache's");
    if (q_heads > kMaxHeads) return unsupported("too many query heads");
    if (!nothing(b) && (int64_t)b.max_new * q_heads > INT32_MAX) return unsupported("max_new x heads too large");
    return FP8DIT_OK;
}

}  // namespace
}  // namespace fp8dit

using namespace fp8dit;

fp8dit_status fp8_rotary_axes(const fp8dit_heads* q, const fp8dit_heads* k, const fp8dit_heads* q_out,
                              const fp8dit_heads* k_out, int64_t M, int32_t dim, const void* positions,
                              fp8dit_pos_dtype pos_dtype, const double* freqs, const int32_t* axis_dims,
                              int32_t n_axes, int32_t interleaved, fp8dit_stream_t stream) {
    clear_error();
    if (!q || !k || !q_out || !k_out) return invalid("null tensor description (k with heads = 0 if there is none)");
    if (M < 0) return invalid("M must be >= 0");
    if (M > kMaxTokens) return unsupported("M too large");
    if (dim <= 0 || dim % 8 != 0 || dim > FP8DIT_ROTARY_MAX_DIM)
        return unsupported("dim must be a positive multiple of 8 up to 256");
    if (n_axes < 1 || n_axes > FP8DIT_ROTARY_MAX_AXES) return unsupported("n_axes must be 1 .. 4");
    if (pos_dtype != FP8DIT_POS_I32 && pos_dtype != FP8DIT_POS_F32) return invalid("pos_dtype");
    if (!freqs || !axis_dims) return invalid("null freqs or axis_dims");
    RotaryArgs a{};
    for (int i = 0; i < n_axes; ++i) {
        if (axis_dims[i] <= 0 || axis_dims[i] % 2 != 0 || axis_dims[i] > dim)
            return unsupported("every axis needs a positive even number of elements");
        if (2 * a.pairs + axis_dims[i] > dim) return unsupported("the axes' elements exceed dim");
        for (int j = 0; j < axis_dims[i] / 2; ++j) {
            if (!std::isfinite(freqs[a.pairs])) return invalid("freqs must be finite");
            a.turns[a.pairs] = freqs[a.pairs] / 6.283185307179586476925;
            a.axis[a.pairs++] = (uint8_t)i;
        }
    }
    if (!interleaved && a.pairs % 4 != 0) return unsupported("split halves need a multiple of 8 rotated elements");
    if (q->heads < 0 || k->heads < 0 || q->heads > kMaxHeads / 2 || k->heads > kMaxHeads / 2)
        return invalid("head counts must be >= 0 and below 32768");
    if (q->heads != q_out->heads || k->heads != k_out->heads) return invalid("an output's heads differ from its input's");
    if (M == 0 || q->heads + k->heads == 0) return FP8DIT_OK;
    for (const fp8dit_heads* x : {q, q_out, k, k_out})
        if (x->heads > 0)
            if (const char* msg = heads_problem(*x, dim)) return invalid(msg);
    if (!positions || !aligned(positions, 4)) return invalid("positions must be non-null and 4-byte aligned");
    const DeviceInfo* dev = device_info();
    if (!dev) return FP8DIT_ERR_CUDA;
    a.q = view(*q), a.k = view(*k), a.qo = view(*q_out), a.ko = view(*k_out);
    a.pos = positions;
    a.M = M;
    a.n_axes = n_axes, a.pos_float = pos_dtype == FP8DIT_POS_F32, a.interleaved = interleaved != 0;
    a.dim = dim;
    a.units = interleaved ? dim / 8 : a.pairs / 4 + (dim - 2 * a.pairs) / 8;
    cudaError_t e = launch_rotary(a, (cudaStream_t)stream, dev);
    return e == cudaSuccess ? FP8DIT_OK : cuda_fail(e, "rotary launch");
}

fp8dit_status fp8_kv_cache_append(const fp8dit_kv_cache* cache, const fp8dit_heads* k, const fp8dit_heads* v,
                                  const fp8dit_kv_batch* batch, fp8dit_stream_t stream) {
    clear_error();
    KvAppendArgs a{};
    fp8dit_status st = check_cache(cache, &a.c);
    if (st == FP8DIT_OK) st = check_batch(batch, a.c, &a.b);
    if (st != FP8DIT_OK) return st;
    if (!k || !v) return invalid("null tensor description");
    if (k->heads != a.c.heads || v->heads != a.c.heads) return invalid("k and v need the cache's number of heads");
    if (nothing(a.b)) return FP8DIT_OK;
    for (const fp8dit_heads* x : {k, v})
        if (const char* msg = heads_problem(*x, a.c.dim)) return invalid(msg);
    const int64_t T = 1ll << a.c.block_log2;
    const int64_t touched = (a.b.max_new + T - 2) / T + 1;
    if (touched * a.b.n > INT32_MAX) return unsupported("n_requests x max_new too large");
    const DeviceInfo* dev = device_info();
    if (!dev) return FP8DIT_ERR_CUDA;
    a.k = view(*k), a.v = view(*v);
    a.touched = (int32_t)touched;
    a.err = DevErr{dev->err_word, kDefaultWaitLimitNs};
    cudaError_t e = launch_kv_append(a, (cudaStream_t)stream);
    return e == cudaSuccess ? FP8DIT_OK : cuda_fail(e, "cache append launch");
}

size_t fp8_kv_cache_attention_workspace_size(const fp8dit_kv_cache* cache, const fp8dit_kv_batch* batch,
                                             int32_t q_heads) {
    clear_error();
    KvCacheView c{};
    KvBatchView b{};
    if (check_cache(cache, &c) != FP8DIT_OK || check_batch(batch, c, &b) != FP8DIT_OK ||
        check_q_heads(q_heads, c, b) != FP8DIT_OK || nothing(b))
        return 0;
    const DeviceInfo* dev = device_info();
    return dev ? kv_attn_plan(c, b, q_heads, dev->num_sms).ws_bytes : 0;
}

fp8dit_status fp8_kv_cache_attention_plan(const fp8dit_kv_cache* cache, const fp8dit_kv_batch* batch, int32_t q_heads,
                                          int32_t* rows_per_tile, int32_t* key_ranges) {
    clear_error();
    KvCacheView c{};
    KvBatchView b{};
    fp8dit_status st = check_cache(cache, &c);
    if (st == FP8DIT_OK) st = check_batch(batch, c, &b);
    if (st == FP8DIT_OK) st = check_q_heads(q_heads, c, b);
    if (st != FP8DIT_OK) return st;
    KvAttnPlan plan{};
    if (!nothing(b)) {
        const DeviceInfo* dev = device_info();
        if (!dev) return FP8DIT_ERR_CUDA;
        plan = kv_attn_plan(c, b, q_heads, dev->num_sms);
    }
    if (rows_per_tile) *rows_per_tile = plan.rows_per_tile;
    if (key_ranges) *key_ranges = plan.splits;
    return FP8DIT_OK;
}

fp8dit_status fp8_kv_cache_attention(const fp8dit_kv_cache* cache, const fp8dit_heads* q, const fp8dit_kv_batch* batch,
                                     const fp8dit_heads* out, float* lse, float scale, int32_t causal,
                                     void* workspace, size_t ws_bytes, fp8dit_stream_t stream) {
    clear_error();
    KvAttnArgs a{};
    fp8dit_status st = check_cache(cache, &a.c);
    if (st == FP8DIT_OK) st = check_batch(batch, a.c, &a.b);
    if (st != FP8DIT_OK) return st;
    if (!q || !out) return invalid("null tensor description");
    if ((st = check_q_heads(q->heads, a.c, a.b)) != FP8DIT_OK) return st;
    if (out->heads != q->heads) return invalid("out's heads differ from q's");
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!(scale > 0.0f) || !std::isfinite(scale_log2)) return invalid("scale must be > 0 and finite, times log2(e) too");
    if (causal < 0) return invalid("causal must be >= 0");
    if (nothing(a.b)) return FP8DIT_OK;
    for (const fp8dit_heads* x : {q, out})
        if (const char* msg = heads_problem(*x, a.c.dim)) return invalid(msg);
    if (!aligned(lse, 4)) return invalid("lse must be 4-byte aligned");
    const DeviceInfo* dev = device_info();
    if (!dev) return FP8DIT_ERR_CUDA;
    const KvAttnPlan plan = kv_attn_plan(a.c, a.b, q->heads, dev->num_sms);
    if ((int64_t)a.b.n * plan.row_tiles * plan.splits * (plan.tensor ? a.c.heads : 1) > INT32_MAX)
        return unsupported("too many row tiles");
    if (plan.ws_bytes > 0) {
        if (!workspace || !aligned(workspace, 16)) return invalid("this call needs a 16-byte aligned workspace");
        if (ws_bytes < plan.ws_bytes) return invalid("workspace smaller than fp8_kv_cache_attention_workspace_size");
        a.part_o = static_cast<float*>(workspace);
        a.part_sum = reinterpret_cast<float2*>(a.part_o + (size_t)plan.splits * (size_t)a.b.total * (size_t)q->heads * (size_t)a.c.dim);
    }
    a.q = view(*q), a.out = view(*out);
    a.lse = lse;
    a.scale_log2 = scale_log2;
    a.q_most = std::min(119, 126 + std::ilogb(scale_log2));
    a.group = q->heads / a.c.heads;
    a.frame = causal;
    a.err = DevErr{dev->err_word, kDefaultWaitLimitNs};
    cudaError_t e = launch_kv_attention(plan, a, (cudaStream_t)stream);
    return e == cudaSuccess ? FP8DIT_OK : cuda_fail(e, "cache attention launch");
}
