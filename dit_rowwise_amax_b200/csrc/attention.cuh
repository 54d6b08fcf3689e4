// What the rotary, cache and attention kernels share: their launch arguments,
// the checks of lengths and block indices that live in device memory, and the
// decoding of cached codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
    int32_t units;            // threads per token: units of a head
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
    int32_t q_most;     // bound of q's exponent: scale_log2 / 2^q_most is a normal number
    int32_t group;      // query heads per kv head
    int32_t frame;      // causal granularity, 0: none
    int32_t splits;     // key ranges per (row tile, kv head)
    int32_t chunk;      // keys per range (a multiple of 128 when splits > 1)
    int32_t tail_last;  // 1: the last row tile is a short one and is launched last
    int32_t row_tiles;  // row tiles per request (rows = new tokens x group)
    float* part_o;      // splits > 1: [splits][total * q heads][dim], normalised
    float2* part_sum;   // splits > 1: [splits][total * q heads], reference m (log2 units; -inf: no key seen) and sum of 2^(s - m)
    DevErr err;
};

// How an attention call is cut; a function of host-side sizes only.
struct KvAttnPlan {
    int32_t rows_per_tile, row_tiles, splits, chunk;
    bool tensor;  // the tcgen05 kernel
    bool tail_last;
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
        if (threadIdx.x + threadIdx.y == 0) atomicOr(err.word, kDevErrIndex);
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

// Two E4M3 codes (the low 16 bits) -> two fp16, exact.
__device__ __forceinline__ uint32_t decode2(uint32_t codes) {
    uint32_t d;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(d) : "r"(codes));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// fp16 and the ranges. The attention kernels multiply in fp16: every E4M3 code
// is exact there and decoding is one instruction for two codes (four to bf16).
// q is brought to [2^14, 2^15) by a power of two per row (q_exponent, from the
// row's largest |q|), undone in the score; what lies 2^-38 below the row's
// largest is lost, as in any fp32 sum of products. The exponent's bounds: the
// largest bf16 still comes below 2^15, rows below 2^-105 keep 2^119, or less
// (KvAttnArgs::q_most) where the softmax scale over it would not be a normal
// number: such rows' scores are then below 2^-5.
__device__ __forceinline__ int q_exponent(uint32_t amax_bf16_bits, int most) {
    return max(-113, min(most, 14 + 127 - (int)(amax_bf16_bits >> 7)));
}
// A score's factor: softmax scale over q's, times K's block scale. Not 0, so a
// masked score of -inf stays one; not infinite, so a product of 0 stays 0.
__device__ __forceinline__ float score_factor(float c, float k_scale) { return fminf(fmaxf(c * k_scale, 0x1p-126f), 0x1.fp127f); }
__device__ __forceinline__ float pow2f(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }  // -126 .. 127
// log2 of a block's scale (a power of two).
__device__ __forceinline__ int scale_log2_of(float s) { return (int)(__float_as_uint(s) >> 23) - 127; }

// The softmax's references are lazy: they only move when a score exceeds them by
// kLazy (log2 units). P goes into the product as 2^(kLift + score - reference),
// at most 2^15 in fp16 (largest 65504), so that weights are normal numbers down
// to 2^-21 of the reference's and count at all down to 2^-32: what a row of n
// keys loses to the rounding of its small weights stays below n 2^-32 (without
// the lift n 2^-25, 3% at a million keys).
constexpr float kLazy = 8.0f, kLift = 7.0f;

constexpr float kLog2ToNat = 0.6931471805599453f;

#endif  // __CUDACC__

}  // namespace fp8dit
