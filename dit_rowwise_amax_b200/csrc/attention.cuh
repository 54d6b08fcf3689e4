// What the rotary, cache and attention kernels share: their launch arguments,
// the checks of lengths and block indices that live in device memory, and the
// E4M3 -> bf16 decoding of cached codes.
#pragma once

#include <cuda_bf16.h>

#include "fp8dit_internal.cuh"

namespace fp8dit {

// ------------------------------------------------------------- arguments
struct HeadsView {
    uint16_t* ptr;
    int64_t token_stride, head_stride;
    int32_t heads;
};

struct RotaryArgs {
    HeadsView q, k, qo, ko;
    const void* pos;
    int64_t M;
    int32_t n_axes, pos_float, interleaved;
    int32_t dim, pairs;       // pairs = rotated elements / 2
    int32_t units;            // 4-pair (or 8-element copy) units of a head
    int32_t heads_per_thread;
    double turns[FP8DIT_ROTARY_MAX_DIM / 2];  // freqs / (2 pi)
    uint8_t axis[FP8DIT_ROTARY_MAX_DIM / 2];
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t stream, const DeviceInfo* dev);

struct KvCacheView {
    uint8_t *k, *v;
    float *ks, *vs;
    int32_t n_blocks, heads, dim;
    int32_t block_log2;  // tokens per block = 1 << block_log2
};

struct KvBatchView {
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* offsets;
    int64_t total;
    int32_t n, width, max_new, max_kv;
};

struct KvAppendArgs {
    KvCacheView c;
    KvBatchView b;
    HeadsView k, v;
    int32_t touched;  // blocks that max_new tokens reach at most
    DevErr err;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);

struct KvAttnArgs {
    KvCacheView c;
    KvBatchView b;
    HeadsView q, out;
    float* lse;         // [total, q heads] or null
    float scale_log2;   // softmax scale * log2(e)
    int32_t group;      // query heads per kv head
    int32_t frame;      // causal granularity, 0: none
    int32_t splits;     // key ranges per (row tile, kv head)
    int32_t chunk;      // keys per range (a multiple of 128 when splits > 1)
    int32_t row_tiles;  // row tiles per request (rows = new tokens x group)
    float* part_o;      // splits > 1: [splits][total * q heads][dim], normalised
    float* part_lse;    // splits > 1: [splits][total * q heads], log2 units; -inf: no key seen
    DevErr err;
};

// How an attention call is cut; a function of host-side sizes only.
struct KvAttnPlan {
    int32_t rows_per_tile, row_tiles, splits, chunk;
    bool tensor;  // the tcgen05 kernel
    size_t ws_bytes;
};
KvAttnPlan kv_attn_plan(const KvCacheView& c, const KvBatchView& b, int q_heads, int num_sms);
cudaError_t launch_kv_attn_tiles(const KvAttnArgs& a, cudaStream_t stream);  // 256-row tiles, tcgen05
cudaError_t launch_kv_attention(const KvAttnPlan& plan, KvAttnArgs& a, cudaStream_t stream);

// ------------------------------------------------------------ device side
#if defined(__CUDACC__)

struct Request {
    int32_t first;  // its first row in q / k / v / out
    int32_t n;      // its new tokens (0: nothing to do)
    int32_t len;    // its tokens in the cache, the new ones included
};

// Request b's numbers, checked against the bounds the launch was sized for.
__device__ __forceinline__ Request load_request(const KvBatchView& v, int b, const DevErr& err, bool needs_start) {
    const int32_t o0 = v.offsets[b], o1 = v.offsets[b + 1], len = v.kv_lens[b];
    Request r{o0, o1 - o0, len};
    const bool ok = o0 >= 0 && o1 >= o0 && o1 <= v.total && o1 - o0 <= v.max_new && len >= 0 && len <= v.max_kv &&
                    !(needs_start && len < o1 - o0);
    if (!ok) {
        if (threadIdx.x == 0) atomicOr(err.word, kDevErrIndex);
        r.n = 0;
        r.len = 0;
    }
    return r;
}

// Keys that a query at position pos (from the end: len - n + i, may be
// negative) sees of len.
__device__ __forceinline__ int32_t key_limit(int32_t pos, int32_t len, int32_t frame) {
    if (frame == 0) return len;
    if (pos < 0) return 0;
    const int64_t end = ((int64_t)(pos / frame) + 1) * frame;
    return end < len ? (int32_t)end : len;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// E4M3 codes as bf16 bit patterns: moving a code's sign to bit 15 and its
// exponent and mantissa to bits 10..4 gives code x 2^-120 exactly, subnormal
// codes included (bf16's subnormals continue E4M3's), in three instructions
// for two codes: a byte permute that spreads two bytes to 16-bit lanes with
// their sign above them, a shift and a mask. The NaN codes come out as +-480,
// so bytes that nothing has written never turn into a NaN.
constexpr uint32_t kCodeMask = 0x87f087f0u;
__device__ __forceinline__ uint32_t spread_codes(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return (d << 4) & kCodeMask;
}
// Selector of spread_codes: byte i for the low lane and byte j for the high
// one, 0..3 of a, 4..7 of b (bit 3 of a selector digit repeats the byte's sign).
__host__ __device__ constexpr uint32_t spread_sel(uint32_t i, uint32_t j) {
    return i | (i | 8) << 4 | j << 8 | (j | 8) << 12;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The factor pair that takes spread codes to code x S, S = 2^n, -120 <= n <=
// 120: 2^(120 + n) is a bf16 up to n = 7; above, the rest is a second factor
// (1 otherwise).
struct CodeScale {
    uint32_t m;     // 2^(120 + min(n, 7)), twice
    uint32_t rest;  // 2^max(n - 7, 0), twice
};
constexpr uint32_t kBf16One2 = 0x3f803f80u;
__device__ __forceinline__ CodeScale code_scale(float s) {
    const int e = (int)((__float_as_uint(s) >> 23) & 0xff);  // n + 127, 7 .. 247
    const int lo = e < 134 ? e : 134;
    const uint32_t m = (uint32_t)(lo + 120) << 7;   // biased exponent in a bf16
    const uint32_t r = (uint32_t)(127 + e - lo) << 7;
    return CodeScale{m | m << 16, r | r << 16};
}

#endif  // __CUDACC__

}  // namespace fp8dit
