// Attention over the E4M3 cache for many query rows: sm_100a tensor cores.
//
// One CTA takes up to 256 rows (new tokens x the query heads of one kv head,
// two tiles of 128), one kv head and one range of keys, and walks the range in
// tiles of 128 keys:
//     S = Q K^T        tcgen05.mma, Q and K in shared memory, S in TMEM
//     P = 2^(c S - m)  two threads per row: TMEM -> registers -> bf16 -> TMEM
//     O += P V         tcgen05.mma, P from TMEM, V in shared memory, O in TMEM
// one pass over the keys, with a running maximum and sum per row. The tensor
// cores multiply bf16 (q is bf16, and code x S is exact in bf16), so the
// cached codes are decoded on the way.
//
// Warp roles (24 warps, one CTA per SM):
//   0-7, 8-15  softmax of row tile 0 and 1: two threads share a row, 64 keys
//              each; the warp with the same rows is four warps further on, and
//              the two exchange their maxima through shared memory. While one
//              tile's softmax runs, the tensor cores work on the other's.
//   16-19      decode a raw tile of codes into the 128-byte-swizzled bf16
//              layout the MMAs read (K: row = key, K-major; V: the same bytes
//              read MN-major, so neither is transposed).
//   20         looks block indices up and bulk-copies the blocks' codes
//              (untiled: a block and head is one contiguous piece).
//   21         issues the MMAs (one thread), owns TMEM.
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
constexpr int kThreads = 768;
constexpr float kLazy = 8.0f;
constexpr float kNegInf = -__builtin_huge_valf();

// Registers per thread by role, out of the launch's 768 x 80.
constexpr int kRegsSoftmax = 88, kRegsConvert = 88, kRegsOther = 40;
static_assert(512 * kRegsSoftmax + 128 * kRegsConvert + 128 * kRegsOther <= kThreads * 80, "register split");

// What the roles of a CTA agree on.
struct Work {
    int b, head, split, r0, rows;  // first row and rows of the request
    int k0;                        // first key of the range
    int n[2], n_max;               // key tiles of each row tile
    Request r;
};

struct Bars {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t raw_full[4], raw_empty[4];  // first and second 64 keys of K, of V
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    uint32_t bad[8];       // bad blocks of K tile j, bit per block, at j % 8
    CodeScale scale[4][4]; // [raw stage][block of its 64 keys]
    int failed[16];        // softmax warp w saw an expired wait
    Work work;             // kept here, not in every thread's registers
};
struct Tops {
    float v[2][2][kRows];  // [row tile][half of the keys][row]: maxima, at the end sums
};

template <int D>
struct Tile {
    static constexpr int HALF = kKeys * 128;           // 64 dims of 128 rows: 16 KB
    static constexpr int BYTES = HALF * (D / 64);      // a bf16 tile of 128 rows
    static constexpr int RAW = 64 * D;                 // a raw stage: 64 keys' codes
    static constexpr int SMEM = 2 * BYTES + 4 * BYTES + 4 * RAW + (int)sizeof(Tops) + 1024;
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

// ------------------------------------------------------------ load codes
template <int D>
__device__ __forceinline__ void load_role(const KvAttnArgs& a, const Work& w, Bars* sm, uint8_t* raw, int lane) {
    const int tlog = a.c.block_log2, T = 1 << tlog, per_tile = kKeys >> tlog;
    const int32_t* table = a.b.table + (int64_t)w.b * a.b.width;
    const int blocks = (w.r.len + T - 1) >> tlog;  // blocks the request has
    const int rows = min(T, 64);  // rows of a copy: a block, or half of one of 128
    const uint32_t bytes = (uint32_t)rows * D;
    volatile int* abort = &sm->abort;
    int at = (w.k0 >> tlog) + lane;
    int page = lane < per_tile && at < blocks ? table[at] : 0;
    int done = 0;  // raw stages filled
    for (int j = 0; j < w.n_max; ++j) {
        const bool have = lane < per_tile && at < blocks;
        const bool ok = have && page >= 0 && page < a.c.n_blocks;
        const int64_t slot = ok ? (int64_t)page * a.c.heads + w.head : 0;
        const uint32_t bad = __ballot_sync(0xffffffffu, have && !ok);
        float s[2] = {0.0f, 0.0f};
        if (ok) {
            s[0] = a.c.ks[slot];
            s[1] = a.c.vs[slot];
        }
        at += per_tile;
        page = lane < per_tile && at < blocks ? table[at] : 0;
        bool fail = false;
        for (int st = 0; st < 4; ++st) {  // K's two halves, V's two halves
            const int v = st >> 1, half = st & 1;
            const bool mine = T == 128 ? lane == 0 : lane < per_tile && ((lane << tlog) >> 6) == half;
            const int count = __popc(__ballot_sync(0xffffffffu, mine && ok));
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sm->raw_empty[st], (uint32_t)(j & 1) ^ 1u, abort, a.err))) {
                fail = true;
                break;
            }
            const int key = (lane << tlog) & 63;  // first key of this lane's copy in the stage
            if (mine) sm->scale[st][key >> tlog] = ok ? code_scale(v ? s[1] : s[0]) : CodeScale{0u, kBf16One2};
            if (lane == 0 && st == 0) {
                sm->bad[j & 7] = bad;
                if (bad) atomicOr(a.err.word, kDevErrIndex);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sm->raw_full[st], (uint32_t)count * bytes);
            __syncwarp();
            if (mine && ok)
                bulk_load_g2s(raw + st * Tile<D>::RAW + key * D,
                              (v ? a.c.v : a.c.k) + ((slot << tlog) + (T == 128 ? 64 * half : 0)) * D, bytes,
                              &sm->raw_full[st]);
            ++done;
        }
        if (fail) break;
    }
    if (*abort) {  // let the copies in flight land
        for (int i = max(0, done - 4); i < done; ++i)
            mbar_wait_bounded(&sm->raw_full[i & 3], (uint32_t)(i >> 2) & 1u, nullptr, a.err);
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
        const int buf = j & 1;
#pragma unroll 1
        for (int st = 0; st < 4; ++st) {
            const int v = st >> 1, half = st & 1;
            uint64_t* full = v ? &sm->v_full[buf] : &sm->k_full[buf];
            uint64_t* empty = v ? &sm->v_empty[buf] : &sm->k_empty[buf];
            bool ok = mbar_wait_bounded(&sm->raw_full[st], (uint32_t)(j & 1), abort, a.err);
            if (half == 0) ok = ok && mbar_wait_bounded(empty, (uint32_t)((j >> 1) & 1) ^ 1u, abort, a.err);
            if (!__all_sync(0xffffffffu, ok)) return;
            const uint4* src = reinterpret_cast<const uint4*>(raw + st * Tile<D>::RAW);
            uint8_t* dst = tiles + (2 * v + buf) * Tile<D>::BYTES + half * (64 * 128);
            uint4 in[VPR / 2];
#pragma unroll
            for (int it = 0; it < VPR / 2; ++it) in[it] = src[it * 128 + t];
#pragma unroll
            for (int it = 0; it < VPR / 2; ++it) {
                const int i = it * 128 + t, row = i / VPR, c16 = i % VPR;
                const CodeScale cs = sm->scale[st][row >> tlog];
                uint4 lo, hi;
                decode16(in[it], cs, lo, hi);
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
                if (half == 1) mbar_arrive(full);
                mbar_arrive(&sm->raw_empty[st]);
            }
        }
    }
}

// ------------------------------------------------------------------ MMAs
// The whole warp walks through this, one lane issues.
template <int D>
__device__ __forceinline__ void mma_role(const KvAttnArgs& a, Bars* sm, const uint8_t* q, const uint8_t* tiles,
                                         uint32_t tmem) {
    constexpr uint32_t kIdescS = umma_idesc_bf16_f32(128, kKeys);
    constexpr uint32_t kIdescO = umma_idesc_bf16_f32(128, D) | (1u << 16);  // B (V) is MN-major
    volatile int* abort = &sm->abort;
    const uint32_t lead = elect_one();
    // Broadcast from one lane: known to be the same in the whole warp.
    const int n0 = __shfl_sync(0xffffffffu, sm->work.n[0], 0), n1 = __shfl_sync(0xffffffffu, sm->work.n[1], 0);
    const int n_max = max(n0, n1);
    const bool two = __shfl_sync(0xffffffffu, sm->work.rows - sm->work.r0, 0) > kRows;
    const uint64_t q_desc = umma_desc_kmajor_sw128(smem_u32(q)), k_desc = umma_desc_kmajor_sw128(smem_u32(tiles));
    const uint64_t v_desc = umma_desc_mnmajor_sw128(smem_u32(tiles) + 2 * Tile<D>::BYTES, Tile<D>::HALF);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, a.err));
        tc_fence_after();
        return ok;
    };
    auto scores = [&](int i, int j) {
        const uint64_t qd = q_desc + i * (Tile<D>::BYTES >> 4), kd = k_desc + (j & 1) * (Tile<D>::BYTES >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            constexpr int kHalf = Tile<D>::HALF >> 4;
            const int off = (s >> 2) * kHalf + (s & 3) * 2;  // in 16-byte units
            mma_bf16_warp(lead, tmem + i * kKeys, qd + off, kd + off, kIdescS, s > 0);
        }
        mma_commit_warp(lead, &sm->s_full[i]);
    };
    auto output = [&](int i, int j) {
        const uint64_t vd = v_desc + (j & 1) * (Tile<D>::BYTES >> 4);
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
            mma_bf16_tmem_a_warp(lead, tmem + 2 * kKeys + i * D, tmem + i * kKeys + s * 8, vd + s * (2048 >> 4), kIdescO,
                                 j > 0 || s > 0);
    };
    bool ok = wait(&sm->q_full[0], 0);
    if (ok && two) ok = wait(&sm->q_full[1], 0);
    if (ok && n_max > 0) {
        ok = wait(&sm->k_full[0], 0);
        if (ok) {
            if (n0 > 0) scores(0, 0);
            if (n1 > 0) scores(1, 0);
            mma_commit_warp(lead, &sm->k_empty[0]);
        }
    }
    for (int j = 0; j < n_max && ok; ++j) {
        const int next = j + 1;
        ok = wait(&sm->v_full[j & 1], (uint32_t)(j >> 1) & 1u);
        if (ok && next < n_max) ok = wait(&sm->k_full[next & 1], (uint32_t)(next >> 1) & 1u);
        if (!ok) break;
        if (j < n0) {
            ok = wait(&sm->p_full[0], (uint32_t)j & 1u);
            if (!ok) break;
            output(0, j);
            if (next == n0) mma_commit_warp(lead, &sm->o_full[0]);
            if (next < n0) scores(0, next);
        }
        if (j < n1) {
            ok = wait(&sm->p_full[1], (uint32_t)j & 1u);
            if (!ok) break;
            output(1, j);
            if (next == n1) mma_commit_warp(lead, &sm->o_full[1]);
            mma_commit_warp(lead, &sm->v_empty[j & 1]);
            if (next < n1) scores(1, next);
        } else {
            mma_commit_warp(lead, &sm->v_empty[j & 1]);
        }
        if (next < n_max) mma_commit_warp(lead, &sm->k_empty[next & 1]);
    }
    // Every MMA and every arrival on this CTA's barriers lands before it ends.
    mma_commit_warp(lead, &sm->drain);
    mbar_wait_bounded(&sm->drain, 0, nullptr, a.err);
}

// --------------------------------------------------------------- softmax
// Thread t of 128 (a row of row tile i), half h of the keys and of dim.
template <int D>
__device__ __forceinline__ void softmax_role(const KvAttnArgs& a, const Work& w, Bars* sm, Tops* tops, uint8_t* q,
                                             uint32_t tmem, int i, int h, int t) {
    const int lane = t & 31, warp = 8 * i + 4 * h + (t >> 5), partner = warp ^ 4;
    const uint32_t pair = 1u + 4 * i + (t >> 5);  // named barrier of the two warps that share rows
    const int row = w.r0 + i * kRows + t;
    const bool in = row < w.rows;
    // Rows past the last one compute on zeros and are not written.
    const int limit = in ? key_limit(w.r.len - w.r.n + row / a.group, w.r.len, a.frame) : INT32_MAX;
    volatile int* abort = &sm->abort;
    {
        const int token = in ? row / a.group : 0, qh = w.head * a.group + (in ? row % a.group : 0);
        const uint16_t* src = a.q.ptr + (int64_t)(w.r.first + token) * a.q.token_stride + (int64_t)qh * a.q.head_stride;
        uint8_t* dst = q + i * Tile<D>::BYTES + t * 128;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const int c = h * (D / 16) + k;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(src + c * 8);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * Tile<D>::HALF + (((c & 7) ^ (t & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->q_full[i]);
    }
    const uint32_t lanes = (uint32_t)(t >> 5) << 21;  // this warp's TMEM lanes: (t / 32) * 32 << 16
    const uint32_t s_addr = tmem + lanes + i * kKeys, o_addr = tmem + lanes + 2 * kKeys + i * D + h * (D / 2);
    const float c = a.scale_log2;
    float m = kNegInf, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < w.n[i]; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm->s_full[i], (uint32_t)j & 1u, abort, a.err));
        uint32_t s[2][32];
        float tile_top = kNegInf;
        if (ok) {
            tc_fence_after();
            tmem_ld_32x32b_x32(s_addr + 64 * h, s[0]);
            tmem_ld_32x32b_x32(s_addr + 64 * h + 32, s[1]);
            tmem_wait_ld();
            tmem_tie32(s[0]);
            tmem_tie32(s[1]);
            const int seen = limit - (w.k0 + j * kKeys) - 64 * h;  // this row sees columns below it
            const uint32_t bad = *(volatile uint32_t*)&sm->bad[j & 7];
            if (__any_sync(0xffffffffu, seen < 64) || bad) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (32 * k + x >= seen || (bad >> ((64 * h + 32 * k + x) >> a.c.block_log2) & 1u))
                            s[k][x] = __float_as_uint(kNegInf);
            }
            float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int x = 0; x < 32; x += 2)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    top[2 * k] = fmaxf(top[2 * k], __uint_as_float(s[k][x]));
                    top[2 * k + 1] = fmaxf(top[2 * k + 1], __uint_as_float(s[k][x + 1]));
                }
            tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            tops->v[i][h][t] = tile_top;
        } else if (lane == 0) {
            *(volatile int*)&sm->failed[warp] = 1;
        }
        // Both warps have read their scores (P will overwrite them) and come
        // here whatever their waits said, so neither is left alone.
        named_barrier_sync(pair, 64);
        if (!ok || *(volatile int*)&sm->failed[partner]) {
            ok = false;
            break;
        }
        tile_top = fmaxf(tile_top, *(volatile float*)&tops->v[i][h ^ 1][t]);
        if (__any_sync(0xffffffffu, (tile_top - m) * c > kLazy)) {
            const float to = fmaxf(m, tile_top);
            const float f = to == kNegInf ? 1.0f : ex2_approx((m - to) * c);
            m = to;
            l *= f;
            if (j > 0) {  // O of the earlier tiles is complete: S came after it
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
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
        for (int k = 0; k < 2; ++k) {
            uint32_t p[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float2 e =
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[k][2 * x]), __uint_as_float(s[k][2 * x + 1])), c2, mc2));
                const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
                sum[x & 1] = f2_add(sum[x & 1], f2_pack(p0, p1));
                p[x] = pack2(p0, p1);
            }
            tmem_st_32x32b_x16(s_addr + 32 * h + 16 * k, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full[i]);
        const float2 t2 = f2_unpack(f2_add(sum[0], sum[1]));
        l = t2.x + t2.y;
    }
    if (w.n[i] > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sm->o_full[i], 0, abort, a.err));
    // The row's sum over both halves (the last maxima have been read).
    if (ok)
        tops->v[i][h][t] = l;
    else if (lane == 0)
        *(volatile int*)&sm->failed[warp] = 1;
    named_barrier_sync(pair, 64);
    if (!ok || *(volatile int*)&sm->failed[partner]) return;
    l += *(volatile float*)&tops->v[i][h ^ 1][t];
    tc_fence_after();
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    // Taken again rather than kept in registers through the loop.
    const int token = in ? row / a.group : 0, qh = w.head * a.group + (in ? row % a.group : 0);
    const int64_t tok = w.r.first + token;
    const int64_t flat = tok * a.q.heads + qh;
    const int64_t part = (int64_t)w.split * a.b.total * a.q.heads + flat;
    if (in && h == 0) {
        const float lse = m == kNegInf ? kNegInf : m * c + lg2_approx(l);
        if (a.splits > 1)
            a.part_lse[part] = lse;
        else if (a.lse)
            a.lse[flat] = lse * 0.6931471805599453f;
    }
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
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
        const int d = h * (D / 2) + 32 * k;
        if (a.splits > 1) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + d);
#pragma unroll
            for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(__uint_as_float(o[4 * x]) * inv, __uint_as_float(o[4 * x + 1]) * inv,
                                     __uint_as_float(o[4 * x + 2]) * inv, __uint_as_float(o[4 * x + 3]) * inv);
        } else {
            uint4* dst = reinterpret_cast<uint4*>(a.out.ptr + tok * a.out.token_stride + (int64_t)qh * a.out.head_stride + d);
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
    // Dynamic shared memory starts on a 1024-byte boundary (there is no static
    // one); the swizzled tiles rely on it, so it is checked.
    extern __shared__ __align__(1024) uint8_t q[];
    uint8_t* tiles = q + 2 * Tile<D>::BYTES;  // K stages 0, 1, V stages 0, 1
    uint8_t* raw = tiles + 4 * Tile<D>::BYTES;
    Tops* tops = reinterpret_cast<Tops*>(raw + 4 * Tile<D>::RAW);
    Bars* sm = reinterpret_cast<Bars*>(tops + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (smem_u32(q) & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err.word, kDevErrTimeout);
        return;
    }

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
            mbar_init(&sm->q_full[i], 8);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->p_full[i], 8);
            mbar_init(&sm->o_full[i], 1);
            mbar_init(&sm->k_full[i], 4);
            mbar_init(&sm->k_empty[i], 1);
            mbar_init(&sm->v_full[i], 4);
            mbar_init(&sm->v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm->raw_full[i], 1);
            mbar_init(&sm->raw_empty[i], 4);
        }
        mbar_init(&sm->drain, 1);
        sm->abort = 0;
        for (int i = 0; i < 16; ++i) sm->failed[i] = 0;
        sm->work = w;
        fence_mbarrier_init();
    }
    if (warp == 21) {
        tmem_alloc(&sm->tmem, Tile<D>::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm->tmem, 0);

    if (warp < 16) {
        regs_inc<kRegsSoftmax>();
        const int i = warp >> 3;
        if (sm->work.r0 + i * kRows < sm->work.rows)
            softmax_role<D>(a, sm->work, sm, tops, q, tmem, i, (warp >> 2) & 1, threadIdx.x & 127);
    } else if (warp < 20) {
        regs_inc<kRegsConvert>();
        convert_role<D>(a, sm->work, sm, raw, tiles, threadIdx.x & 127);
    } else {
        regs_dec<kRegsOther>();
        if (warp == 20)
            load_role<D>(a, sm->work, sm, raw, lane);
        else if (warp == 21)
            mma_role<D>(a, sm, q, tiles, tmem);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 21) {
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
