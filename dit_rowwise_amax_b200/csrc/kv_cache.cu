// Appending keys and values to the E4M3 cache (one power-of-two scale per
// block of tokens and head).
//
// Per (block, head): amax over the new tokens, S = 2^n with the smallest n >=
// -120 such that amax <= 448 S; a block that already holds tokens of its
// request keeps the larger of its scale and S and, when it grows, has its
// other codes brought over; the new codes are RNEsat(x / S), an exact product
// with 2^-n followed by one rounding.
//
// Bound: HBM, 2 bytes read and 1 written per element. A row of threads owns
// one block and head of K or of V, so the amax and the codes need one read: a
// thread keeps 64 of the block's elements (eight 16-byte loads in flight) in
// registers between the two steps. That is 16 (16 x 64 elements) to 256
// threads; small blocks put as many heads into a CTA as give it 256, whose
// slices of a token lie side by side. 32760 tokens, 16 heads of 128: 64 us,
// 6.3 TB/s (four loads per thread 73.6 us, two 171); seven requests' 10160 new
// tokens, blocks of 16 x 64, 12 heads: 33.6 us with one head per CTA, 13.3 with
// whole warps per head, 11.3 so.
#include <algorithm>

#include "attention.cuh"
#include "fp8_codec.cuh"

namespace fp8dit {
namespace {

constexpr int kVecs = 8;  // 16-byte loads (8 elements) per thread

// Exponent n of the scale that |x| <= amax (a non-negative bf16's bits) needs:
// 448 = 1.75 x 2^8, so n = exponent - 8, one more if the mantissa is above 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
    const int n = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
    return n < -120 ? -120 : n > 120 ? 120 : n;  // exponent field 0 (zero, subnormals) ends at -120
}

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
    __shared__ uint32_t warp_max[8];
    pdl_wait();
    pdl_trigger();
    const int T = 1 << a.c.block_log2;
    const int b = blockIdx.x / a.touched, j = blockIdx.x - b * a.touched;
    const int h = blockIdx.y * blockDim.y + threadIdx.y;
    const bool leader = threadIdx.x + threadIdx.y == 0;
    const bool is_v = blockIdx.z != 0;
    const Request r = load_request(a.b, b, a.err, true);
    const int start = r.len - r.n;
    const int blk = (start >> a.c.block_log2) + j;
    const int base = blk << a.c.block_log2;
    if (r.n == 0 || base >= r.len) return;
    const int page = a.b.table[(int64_t)b * a.b.width + blk];
    if (page < 0 || page >= a.c.n_blocks) {
        if (leader) atomicOr(a.err.word, kDevErrIndex);
        return;
    }
    const HeadsView& in = is_v ? a.v : a.k;
    // Threads of a head past the last one go along to the barrier.
    const bool works = h < a.c.heads;
    const int64_t slot = (int64_t)page * a.c.heads + (works ? h : 0);
    uint8_t* codes = (is_v ? a.c.v : a.c.k) + slot * T * D;
    float* scale = (is_v ? a.c.vs : a.c.ks) + slot;
    const int lo = max(start - base, 0), hi = min(r.len - base, T);  // the block's new rows
    const uint16_t* src = in.ptr + ((int64_t)r.first + base - start) * in.token_stride + h * in.head_stride;

    constexpr int VPR = D / 8;  // vectors per row
    uint4 v[kVecs];
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = i * blockDim.x + threadIdx.x, row = at / VPR, col = at % VPR;
        v[i] = make_uint4(0, 0, 0, 0);
        if (works && row >= lo && row < hi)
            v[i] = *reinterpret_cast<const uint4*>(src + (int64_t)row * in.token_stride + col * 8);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m2 = absmax8(v[i], m2);
    uint32_t m = fold_halves(m2);
    for (int z = min(16, (int)blockDim.x / 2); z > 0; z >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, z));
    const int warps = blockDim.x / 32;  // of this head (0: half a one)
    if (warps > 1 && (threadIdx.x & 31) == 0) warp_max[threadIdx.y * warps + (threadIdx.x >> 5)] = m;
    // The block's old scale is read by every thread before any may replace it.
    const bool held = lo > 0;
    const float old = held ? *scale : 0.0f;
    __syncthreads();
    if (!works) return;
    if (warps > 1)
        for (int w = 0; w < warps; ++w) m = max(m, warp_max[threadIdx.y * warps + w]);
    const int need = scale_exponent(m);
    int n = need;
    if (held) {
        const int n_old = scale_log2_of(old);
        n = max(need, min(max(n_old, -120), 120));
        if (n != n_old) {
            // ratio = 2^(n_old - n): below 2^-126 every code becomes a zero anyway.
            const float ratio = n_old - n < -126 ? 0.0f : pow2f(n_old - n);
            for (int at = threadIdx.x; at < T * VPR; at += blockDim.x) {
                if (at >= lo * VPR && at < hi * VPR) continue;  // the new rows
                uint2* p = reinterpret_cast<uint2*>(codes) + at;
                uint2 w = *p;
                uint32_t* ww = &w.x;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2_raw f0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(ww[k] & 0xffffu), __NV_E4M3);
                    const __half2_raw f1 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(ww[k] >> 16), __NV_E4M3);
                    const float2 x0 = __half22float2(__half2(f0)), x1 = __half22float2(__half2(f1));
                    ww[k] = quant4(x0.x * ratio, x0.y * ratio, x1.x * ratio, x1.y * ratio);
                }
                *p = w;
            }
        }
    }
    const float inv = pow2f(-n);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int at = i * blockDim.x + threadIdx.x, row = at / VPR;
        if (row < lo || row >= hi) continue;
        uint2 o;
        o.x = quant4(bf16_lo(v[i].x) * inv, bf16_hi(v[i].x) * inv, bf16_lo(v[i].y) * inv, bf16_hi(v[i].y) * inv);
        o.y = quant4(bf16_lo(v[i].z) * inv, bf16_hi(v[i].z) * inv, bf16_lo(v[i].w) * inv, bf16_hi(v[i].w) * inv);
        reinterpret_cast<uint2*>(codes)[at] = o;
    }
    if (threadIdx.x == 0) *scale = pow2f(n);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
    const int threads = (a.c.dim << a.c.block_log2) / (8 * kVecs);
    int per_cta = std::min(a.c.heads, std::max(1, 256 / threads));
    if (threads == 16) per_cta += per_cta & 1;  // whole warps
    const dim3 grid((unsigned)((int64_t)a.b.n * a.touched), (unsigned)((a.c.heads + per_cta - 1) / per_cta), 2);
    const dim3 block(threads, per_cta);
    return a.c.dim == 64 ? launch_pdl(kv_append_kernel<64>, grid, block, 0, stream, 1, a)
                         : launch_pdl(kv_append_kernel<128>, grid, block, 0, stream, 1, a);
}

}  // namespace fp8dit
