// Attention over the E4M3 cache for many query rows: sm_100a tensor cores.
//
// One CTA takes up to 256 rows (new tokens x the query heads of one kv head,
// two tiles of 128), one kv head and one range of keys, and walks the range in
// tiles of 128 keys:
//     S = Q K^T        tcgen05.mma, Q and K in shared memory, S in TMEM
//     P = 2^(c S - m)  a thread per row: TMEM -> registers -> bf16 -> TMEM
//     O += P V         tcgen05.mma, P from TMEM, V in shared memory, O in TMEM
// one pass over the keys, with a running maximum and sum per row. The tensor
// cores multiply bf16 (q is bf16, and code x S is exact in bf16), so the
// cached codes are decoded on the way.
//
// Warp roles (16 warps, one CTA per SM):
//   0-3, 4-7   softmax of row tile 0 and 1: a thread owns a row. While one
//              tile's softmax runs, the tensor cores work on the other's.
//   8-11       decode a raw tile of codes into the 128-byte-swizzled bf16
//              layout the MMAs read (K: row = key, K-major; V: the same bytes
//              read MN-major, so neither is transposed).
//   12         looks block indices up and bulk-copies the blocks' codes
//              (untiled: a block and head is one contiguous piece).
//   13         issues the MMAs (one thread), owns TMEM.
// Shared memory at dim 128: Q 64 KB, two decoded K and two V tiles 128 KB, two
// raw tiles 32 KB. TMEM: S (P over it) 2 x 128 columns, O 2 x dim columns.
//
// Bound: per 256 x 128 tile at dim 128 the MMAs take 2048 cycles and so do the
// 32768 exponentials at 16 per cycle; decoding adds about a third of a warp
// instruction per key byte to the issue slots. Loads are far below HBM.
//
// The running maximum is lazy: a row's reference moves, and O is rescaled,
// only when a score exceeds it by 8 (log2 units), so after the first tiles O
// stays in TMEM untouched by the softmax threads; p is at most 2^8.
//
// Every wait is bounded; an expired one raises the error word and the CTA's
// abort flag, lets copies and MMAs land, frees TMEM and returns.
#include "attention.cuh"
#include "fp8_codec.cuh"

namespace fp8dit {
namespace {

constexpr int kRows = 128;  // rows of a tile = TMEM lanes
constexpr int kKeys = 128;  // keys of a tile
constexpr int kThreads = 512;
constexpr float kLazy = 8.0f;
constexpr float kNegInf = -__builtin_huge_valf();

// Registers per thread by role: 2 x 128 x 184 + 128 x 96 + 128 x 48 = 512 x 128.
constexpr int kRegsSoftmax = 184, kRegsConvert = 96, kRegsOther = 48;
static_assert(256 * kRegsSoftmax + 128 * kRegsConvert + 128 * kRegsOther <= kThreads * 128, "register split");

struct Bars {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t raw_full[2], raw_empty[2];  // [0]: K tiles, [1]: V tiles
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    uint32_t bad[8];       // bad blocks of K tile j, bit per block, at j % 8
    CodeScale scale[2][8]; // [K, V][block of the raw tile]
};

template <int D>
struct Tile {
    static constexpr int HALF = kKeys * 128;           // 64 dims of 128 rows: 16 KB
    static constexpr int BYTES = HALF * (D / 64);      // a bf16 tile of 128 rows
    static constexpr int RAW = kKeys * D;
    static constexpr int SMEM = 1024 + 2 * BYTES + 4 * BYTES + 2 * RAW + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(sizeof(Bars) <= 1024, "barrier area");
    static_assert(SMEM <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ f32x2_t f2_add(f32x2_t a, f32x2_t b) {
    f32x2_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// What the roles of a CTA agree on.
struct Work {
    int b, head, split, r0, rows;  // first row and rows of the request
    int k0;                        // first key of the range
    int n[2], n_max;               // key tiles of each row tile
    Request r;
};

// ------------------------------------------------------------ load codes
template <int D>
__device__ __forceinline__ void load_role(const KvAttnArgs& a, const Work& w, Bars* sm, uint8_t* raw, int lane) {
    const int tlog = a.c.block_log2, T = 1 << tlog, per_tile = kKeys >> tlog;
    const int32_t* table = a.b.table + (int64_t)w.b * a.b.width;
    const int blocks = (w.r.len + T - 1) >> tlog;  // blocks the request has
    const uint32_t bytes = (uint32_t)T * D;
    volatile int* abort = &sm->abort;
    int at = (w.k0 >> tlog) + lane;
    int page = lane < per_tile && at < blocks ? table[at] : 0;
    int done = 0;  // raw tiles issued, K and V alternating
    for (int j = 0; j < w.n_max; ++j) {
        const bool have = lane < per_tile && at < blocks;
        const bool ok = have && page >= 0 && page < a.c.n_blocks;
        const int64_t slot = ok ? (int64_t)page * a.c.heads + w.head : 0;
        const uint32_t bad = __ballot_sync(0xffffffffu, have && !ok);
        const int count = __popc(__ballot_sync(0xffffffffu, ok));
        float s[2] = {0.0f, 0.0f};
        if (ok) {
            s[0] = a.c.ks[slot];
            s[1] = a.c.vs[slot];
        }
        at += per_tile;
        page = lane < per_tile && at < blocks ? table[at] : 0;
        bool fail = false;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sm->raw_empty[v], (uint32_t)(j & 1) ^ 1u, abort, a.err))) {
                fail = true;
                break;
            }
            if (lane < per_tile) sm->scale[v][lane] = ok ? code_scale(s[v]) : CodeScale{0u, kBf16One2};
            if (lane == 0 && v == 0) {
                sm->bad[j & 7] = bad;
                if (bad) atomicOr(a.err.word, kDevErrIndex);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sm->raw_full[v], (uint32_t)count * bytes);
            __syncwarp();
            if (ok)
                bulk_load_g2s(raw + v * Tile<D>::RAW + lane * bytes, (v ? a.c.v : a.c.k) + slot * (int64_t)bytes, bytes,
                              &sm->raw_full[v]);
            ++done;
        }
        if (fail) break;
    }
    if (*abort) {  // let the copies in flight land
        for (int i = max(0, done - 2); i < done; ++i)
            mbar_wait_bounded(&sm->raw_full[i & 1], (uint32_t)(i >> 1) & 1u, nullptr, a.err);
    }
}

// ---------------------------------------------------------- decode codes
// 16 codes -> 16 bf16 (two 16-byte pieces of a swizzled row).
__device__ __forceinline__ void decode16(const uint4& w, const CodeScale& c, uint4& lo, uint4& hi) {
    uint32_t o[8];
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = mul_bf16x2(spread_codes(in[i], in[i], spread_sel(0, 1)), c.m);
        o[2 * i + 1] = mul_bf16x2(spread_codes(in[i], in[i], spread_sel(2, 3)), c.m);
    }
    if (c.rest != kBf16One2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], c.rest);
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D>
__device__ __forceinline__ void convert_role(const KvAttnArgs& a, const Work& w, Bars* sm, const uint8_t* raw,
                                             uint8_t* tiles, int t) {
    constexpr int VPR = D / 16;  // 16-byte raw vectors per row
    const int tlog = a.c.block_log2;
    const int lane = t & 31;
    volatile int* abort = &sm->abort;
    for (int j = 0; j < w.n_max; ++j) {
        const int st = j & 1;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint64_t* full = v ? &sm->v_full[st] : &sm->k_full[st];
            uint64_t* empty = v ? &sm->v_empty[st] : &sm->k_empty[st];
            bool ok = mbar_wait_bounded(&sm->raw_full[v], (uint32_t)(j & 1), abort, a.err);
            ok = ok && mbar_wait_bounded(empty, (uint32_t)((j >> 1) & 1) ^ 1u, abort, a.err);
            if (!__all_sync(0xffffffffu, ok)) return;
            const uint4* src = reinterpret_cast<const uint4*>(raw + v * Tile<D>::RAW);
            uint8_t* dst = tiles + (2 * v + st) * Tile<D>::BYTES;
#pragma unroll 4
            for (int it = 0; it < VPR; ++it) {
                const int i = it * 128 + t, row = i / VPR, c16 = i % VPR;
                const CodeScale cs = sm->scale[v][row >> tlog];
                uint4 lo, hi;
                decode16(src[i], cs, lo, hi);
                uint8_t* p = dst + (c16 >> 2) * Tile<D>::HALF + row * 128;
                const int x = row & 7, c = (c16 & 3) * 2;
                // Lanes of the two 64-dim halves write their pieces in opposite
                // order: the eight lanes of a phase then cover all banks.
                const bool swap = (c16 >> 2) & 1;
                *reinterpret_cast<uint4*>(p + (((c + (swap ? 1 : 0)) ^ x) << 4)) = swap ? hi : lo;
                *reinterpret_cast<uint4*>(p + (((c + (swap ? 0 : 1)) ^ x) << 4)) = swap ? lo : hi;
            }
            fence_proxy_async_smem();  // before the MMAs (and the next raw copy) touch it
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&sm->raw_empty[v]);
            }
        }
    }
}

// ------------------------------------------------------------------ MMAs
template <int D>
__device__ __forceinline__ void mma_role(const KvAttnArgs& a, const Work& w, Bars* sm, const uint8_t* q,
                                         const uint8_t* tiles, uint32_t tmem) {
    constexpr uint32_t kIdescS = umma_idesc_bf16_f32(128, kKeys);
    constexpr uint32_t kIdescO = umma_idesc_bf16_f32(128, D) | (1u << 16);  // B (V) is MN-major
    volatile int* abort = &sm->abort;
    const uint32_t q_addr = smem_u32(q), t_addr = smem_u32(tiles);
    const int nt = w.n[1] > 0 || w.rows - w.r0 > kRows ? 2 : 1;
    auto scores = [&](int i, int j) {
        const uint32_t qa = q_addr + i * Tile<D>::BYTES, ka = t_addr + (j & 1) * Tile<D>::BYTES;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = (s >> 2) * Tile<D>::HALF + (s & 3) * 32;
            mma_bf16(tmem + i * kKeys, umma_desc_kmajor_sw128(qa + off), umma_desc_kmajor_sw128(ka + off), kIdescS, s > 0);
        }
        mma_commit(&sm->s_full[i]);
    };
    auto output = [&](int i, int j) {
        const uint32_t va = t_addr + (2 + (j & 1)) * Tile<D>::BYTES;
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
            mma_bf16_tmem_a(tmem + 2 * kKeys + i * D, tmem + i * kKeys + s * 8,
                            umma_desc_mnmajor_sw128(va + s * 2048, Tile<D>::HALF), kIdescO, j > 0 || s > 0);
    };
    bool ok = true;
    for (int i = 0; i < nt && ok; ++i) ok = mbar_wait_bounded(&sm->q_full[i], 0, abort, a.err);
    if (ok && w.n_max > 0) {
        ok = mbar_wait_bounded(&sm->k_full[0], 0, abort, a.err);
        if (ok) {
            tc_fence_after();
            for (int i = 0; i < 2; ++i)
                if (w.n[i] > 0) scores(i, 0);
            mma_commit(&sm->k_empty[0]);
        }
    }
    for (int j = 0; j < w.n_max && ok; ++j) {
        ok = mbar_wait_bounded(&sm->v_full[j & 1], (uint32_t)(j >> 1) & 1u, abort, a.err);
        const bool more = j + 1 < w.n_max;
        bool k_ready = false;
        for (int i = 0; i < 2 && ok; ++i) {
            if (j < w.n[i]) {
                ok = mbar_wait_bounded(&sm->p_full[i], (uint32_t)j & 1u, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                output(i, j);
                if (j + 1 == w.n[i]) mma_commit(&sm->o_full[i]);
            }
            if (i == 1 || w.n[1] <= j) mma_commit(&sm->v_empty[j & 1]);
            if (j + 1 < w.n[i]) {
                if (!k_ready) ok = mbar_wait_bounded(&sm->k_full[(j + 1) & 1], (uint32_t)((j + 1) >> 1) & 1u, abort, a.err);
                if (!ok) break;
                k_ready = true;
                tc_fence_after();
                scores(i, j + 1);
            }
            if (w.n[1] <= j) break;
        }
        if (ok && more) mma_commit(&sm->k_empty[(j + 1) & 1]);
    }
    // Every MMA and every arrival on this CTA's barriers lands before it ends.
    mma_commit(&sm->drain);
    mbar_wait_bounded(&sm->drain, 0, nullptr, a.err);
}

// --------------------------------------------------------------- softmax
template <int D>
__device__ __forceinline__ void softmax_role(const KvAttnArgs& a, const Work& w, Bars* sm, uint8_t* q, uint32_t tmem,
                                             int i, int t) {
    const int lane = t & 31;
    const int row = w.r0 + i * kRows + t;
    const bool in = row < w.rows;
    const int token = in ? row / a.group : 0, qh = w.head * a.group + (in ? row % a.group : 0);
    // Rows past the last one compute on zeros and are not written.
    const int limit = in ? key_limit(w.r.len - w.r.n + token, w.r.len, a.frame) : INT32_MAX;
    volatile int* abort = &sm->abort;
    {
        const uint16_t* src = a.q.ptr + (int64_t)(w.r.first + token) * a.q.token_stride + (int64_t)qh * a.q.head_stride;
        uint8_t* dst = q + i * Tile<D>::BYTES + t * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(src + c * 8);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * Tile<D>::HALF + (((c & 7) ^ (t & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->q_full[i]);
    }
    const uint32_t lanes = (uint32_t)(t >> 5) << 21;  // this warp's TMEM lanes: (t / 32) * 32 << 16
    const uint32_t s_addr = tmem + lanes + i * kKeys, o_addr = tmem + lanes + 2 * kKeys + i * D;
    const float c = a.scale_log2;
    float m = kNegInf, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < w.n[i]; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm->s_full[i], (uint32_t)j & 1u, abort, a.err));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(s_addr + 32 * k, s[k]);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_tie32(s[k]);
        const int seen = limit - (w.k0 + j * kKeys);  // this row sees columns below it
        const uint32_t bad = *(volatile uint32_t*)&sm->bad[j & 7];
        if (__any_sync(0xffffffffu, seen < kKeys) || bad) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (32 * k + x >= seen || (bad >> ((32 * k + x) >> a.c.block_log2) & 1u)) s[k][x] = __float_as_uint(kNegInf);
        }
        float top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            top[k] = __uint_as_float(s[k][0]);
#pragma unroll
            for (int x = 1; x < 32; ++x) top[k] = fmaxf(top[k], __uint_as_float(s[k][x]));
        }
        const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (__any_sync(0xffffffffu, (tile_top - m) * c > kLazy)) {
            const float to = fmaxf(m, tile_top);
            const float f = to == kNegInf ? 1.0f : ex2_approx((m - to) * c);
            m = to;
            l *= f;
            if (j > 0) {  // O of the earlier tiles is complete: S came after it
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(o_addr + 16 * k, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                    tmem_st_32x32b_x16(o_addr + 16 * k, o);
                }
            }
        }
        const float mc = m == kNegInf ? 0.0f : -m * c;
        const f32x2_t c2 = f2_pack(c, c), mc2 = f2_pack(mc, mc);
        f32x2_t sum[2] = {f2_pack(l, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const int k = 2 * h + (x >> 4), y = (2 * x) & 31;
                const float2 e = f2_unpack(
                    f2_fma(f2_pack(__uint_as_float(s[k][y]), __uint_as_float(s[k][y + 1])), c2, mc2));
                const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
                sum[x & 1] = f2_add(sum[x & 1], f2_pack(p0, p1));
                p[x] = pack2(p0, p1);
            }
            tmem_st_32x32b_x32(s_addr + 32 * h, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full[i]);
        const float2 t2 = f2_unpack(f2_add(sum[0], sum[1]));
        l = t2.x + t2.y;
    }
    if (w.n[i] > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm->o_full[i], 0, abort, a.err));
    if (!ok) return;
    tc_fence_after();
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const int64_t tok = w.r.first + token;
    const int64_t flat = tok * a.q.heads + qh;
    const int64_t part = (int64_t)w.split * a.b.total * a.q.heads + flat;
    const float lse = m == kNegInf ? kNegInf : m * c + lg2_approx(l);
    if (in) {
        if (a.splits > 1)
            a.part_lse[part] = lse;
        else if (a.lse)
            a.lse[flat] = lse * 0.6931471805599453f;
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        if (w.n[i] > 0) {
            tmem_ld_32x32b_x32(o_addr + 32 * k, o);
            tmem_wait_ld();
            tmem_tie32(o);
        } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0;
        }
        if (!in) continue;
        if (a.splits > 1) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + 32 * k);
#pragma unroll
            for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(__uint_as_float(o[4 * x]) * inv, __uint_as_float(o[4 * x + 1]) * inv,
                                     __uint_as_float(o[4 * x + 2]) * inv, __uint_as_float(o[4 * x + 3]) * inv);
        } else {
            uint4* dst = reinterpret_cast<uint4*>(a.out.ptr + tok * a.out.token_stride + (int64_t)qh * a.out.head_stride + 32 * k);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t y[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    y[z] = pack2(__uint_as_float(o[8 * x + 2 * z]) * inv, __uint_as_float(o[8 * x + 2 * z + 1]) * inv);
                dst[x] = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_tiles(const __grid_constant__ KvAttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* q = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* tiles = q + 2 * Tile<D>::BYTES;  // K stages 0, 1, V stages 0, 1
    uint8_t* raw = tiles + 4 * Tile<D>::BYTES;
    Bars* sm = reinterpret_cast<Bars*>(raw + 2 * Tile<D>::RAW);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();

    // Blocks in launch order: heads fastest, then requests, key ranges, and the
    // row tiles from the last (which under a causal mask sees most) to the first.
    Work w;
    int64_t id = blockIdx.x;
    w.head = (int)(id % a.c.heads);
    id /= a.c.heads;
    w.b = (int)(id % a.b.n);
    id /= a.b.n;
    w.split = (int)(id % a.splits);
    const int tile = a.row_tiles - 1 - (int)(id / a.splits);
    w.r = load_request(a.b, w.b, a.err, false);
    w.rows = w.r.n * a.group;
    w.r0 = tile * 2 * kRows;
    w.k0 = w.split * a.chunk;
    if (w.r0 >= w.rows || (w.split > 0 && w.k0 >= w.r.len)) return;
    w.n_max = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = min(w.r0 + (i + 1) * kRows, w.rows) - 1;
        int keys = 0;
        if (w.r0 + i * kRows < w.rows)
            keys = min(key_limit(w.r.len - w.r.n + last / a.group, w.r.len, a.frame), w.k0 + a.chunk) - w.k0;
        w.n[i] = keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
        w.n_max = max(w.n_max, w.n[i]);
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->q_full[i], 4);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->p_full[i], 4);
            mbar_init(&sm->o_full[i], 1);
            mbar_init(&sm->raw_full[i], 1);
            mbar_init(&sm->raw_empty[i], 4);
            mbar_init(&sm->k_full[i], 4);
            mbar_init(&sm->k_empty[i], 1);
            mbar_init(&sm->v_full[i], 4);
            mbar_init(&sm->v_empty[i], 1);
        }
        mbar_init(&sm->drain, 1);
        sm->abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 13) {
        tmem_alloc(&sm->tmem, Tile<D>::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem;

    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        const int i = warp >> 2;
        if (w.r0 + i * kRows < w.rows) softmax_role<D>(a, w, sm, q, tmem, i, threadIdx.x & 127);
    } else if (warp < 12) {
        regs_dec<kRegsConvert>();
        convert_role<D>(a, w, sm, raw, tiles, threadIdx.x & 127);
    } else {
        regs_dec<kRegsOther>();
        if (warp == 12)
            load_role<D>(a, w, sm, raw, lane);
        else if (warp == 13 && lane == 0)
            mma_role<D>(a, w, sm, q, tiles, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, Tile<D>::TMEM_COLS);
    }
}

template <int D>
cudaError_t launch_for(const KvAttnArgs& a, cudaStream_t stream) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(kv_attn_tiles<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<D>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_done[dev] = true;
    }
    const int64_t ctas = (int64_t)a.c.heads * a.b.n * a.splits * a.row_tiles;
    return launch_pdl(kv_attn_tiles<D>, dim3((unsigned)ctas), dim3(kThreads), Tile<D>::SMEM, stream, 1, a);
}

}  // namespace

cudaError_t launch_kv_attn_tiles(const KvAttnArgs& a, cudaStream_t stream) {
    return a.c.dim == 64 ? launch_for<64>(a, stream) : launch_for<128>(a, stream);
}

}  // namespace fp8dit
