// Rotary positions with several axes (time, height, width, ...) on q and k.
//
// Pair i of a head turns by angle = positions[m, axis(i)] * freqs[i]:
//     (x, y) -> (x cos - y sin, x sin + y cos).
// The angle is held in turns (freqs / 2 pi, from the host, in double): double
// product, minus its nearest integer, then fp32 sinpi / cospi of twice that.
// A position p costs an angle error of about p * freq * 2^-53 turns instead of
// the p * freq * 2^-24 of an fp32 product, which at frame 5000 is visible in
// bf16.
//
// Bound: HBM, 2 + 2 bytes per element (32760 tokens, 16 + 16 heads of 128:
// 92 us, 5.8 TB/s). A thread owns four pairs of one token (16 bytes in
// interleaved order, two times 8 in split order), takes their four sines and
// cosines once and applies them to several heads of q and k, so the
// double-precision work is shared by the heads; the number of heads per thread
// shrinks when there are few tokens, so that a decoding step still fills the
// GPU. (Angles taken once per token into shared memory instead: 116 us, the
// threads' integer divisions and shared reads bound it.) Elements that are
// only copied go the pairs' way in split order, four and four, so a warp that
// has both does not load twice in turn (96 of 128 rotated, 24 + 8 heads, 4099
// tokens: 17.1 us; copied eight by eight, loaded in turn: 24.0).
#include "attention.cuh"
#include "fp8_codec.cuh"

namespace fp8dit {
namespace {

constexpr int kThreads = 256;

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    __shared__ double turns[FP8DIT_ROTARY_MAX_DIM / 2];
    __shared__ uint8_t axis[FP8DIT_ROTARY_MAX_DIM / 2];
    for (int i = threadIdx.x; i < a.pairs; i += kThreads) {
        turns[i] = a.turns[i];
        axis[i] = a.axis[i];
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t m = idx / a.units;
    if (m >= a.M) return;
    const int u = (int)(idx - m * a.units);
    // Interleaved: unit u is elements 8u .. 8u + 7 (pairs 4u ..; pairs past the
    // last one stand still). Split: unit u < pairs / 4 is elements 4u .. 4u + 3
    // and the same + pairs; the others copy what follows 2 * pairs, 4 elements
    // of its first half and 4 of its second.
    const bool copy = !INTERLEAVED && u >= a.pairs / 4;
    const int lo = INTERLEAVED ? 8 * u : copy ? 2 * a.pairs + 4 * (u - a.pairs / 4) : 4 * u;
    const int apart = copy ? a.dim / 2 - a.pairs : a.pairs;  // split: from the first four to the second
    float c[4], s[4];
    if (!copy) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = 1.0f;
            s[j] = 0.0f;
            const int p = 4 * u + j;
            if (p < a.pairs) {
                const int64_t at = m * a.n_axes + axis[p];
                const double pos = a.pos_float ? (double)static_cast<const float*>(a.pos)[at]
                                               : (double)static_cast<const int32_t*>(a.pos)[at];
                double t = pos * turns[p];
                t -= rint(t);
                sincospif(2.0f * (float)t, &s[j], &c[j]);
            }
        }
    }
    const int heads = a.q.heads + a.k.heads;
    const int h0 = blockIdx.y * a.heads_per_thread;
    const int h1 = min(h0 + a.heads_per_thread, heads);
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool is_q = h < a.q.heads;
        const HeadsView& in = is_q ? a.q : a.k;
        const HeadsView& out = is_q ? a.qo : a.ko;
        const int hh = is_q ? h : h - a.q.heads;
        const uint16_t* src = in.ptr + m * in.token_stride + hh * in.head_stride + lo;
        uint16_t* dst = out.ptr + m * out.token_stride + hh * out.head_stride + lo;
        if constexpr (INTERLEAVED) {
            uint4 v = *reinterpret_cast<const uint4*>(src);
            uint32_t* w = &v.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (4 * u + j >= a.pairs) continue;  // a copy stays one, infinities included
                const float x = bf16_lo(w[j]), y = bf16_hi(w[j]);
                w[j] = pack_bf16x2(fmaf(x, c[j], -(y * s[j])), fmaf(x, s[j], y * c[j]));
            }
            *reinterpret_cast<uint4*>(dst) = v;
        } else {
            uint2 x2 = *reinterpret_cast<const uint2*>(src);
            uint2 y2 = *reinterpret_cast<const uint2*>(src + apart);
            uint32_t* xw = &x2.x;
            uint32_t* yw = &y2.x;
            if (!copy) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float x0 = bf16_lo(xw[j]), x1 = bf16_hi(xw[j]), y0 = bf16_lo(yw[j]), y1 = bf16_hi(yw[j]);
                    const float c0 = c[2 * j], c1 = c[2 * j + 1], s0 = s[2 * j], s1 = s[2 * j + 1];
                    xw[j] = pack_bf16x2(fmaf(x0, c0, -(y0 * s0)), fmaf(x1, c1, -(y1 * s1)));
                    yw[j] = pack_bf16x2(fmaf(x0, s0, y0 * c0), fmaf(x1, s1, y1 * c1));
                }
            }
            *reinterpret_cast<uint2*>(dst) = x2;
            *reinterpret_cast<uint2*>(dst + apart) = y2;
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& args, cudaStream_t stream, const DeviceInfo* dev) {
    RotaryArgs a = args;
    const int heads = a.q.heads + a.k.heads;
    // Up to 16 heads share a thread's angles, fewer while that would leave the
    // GPU's 2048 threads per SM idle.
    const int64_t threads = a.M * a.units;
    int64_t hpt = threads * heads / ((int64_t)dev->num_sms * 2048);
    a.heads_per_thread = (int32_t)(hpt < 1 ? 1 : hpt > 16 ? 16 : hpt);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads),
                    (unsigned)((heads + a.heads_per_thread - 1) / a.heads_per_thread));
    return a.interleaved ? launch_pdl(rotary_kernel<true>, grid, dim3(kThreads), 0, stream, 1, a)
                         : launch_pdl(rotary_kernel<false>, grid, dim3(kThreads), 0, stream, 1, a);
}

}  // namespace fp8dit
