// Attention over the E4M3 cache for many query rows: sm_100a tensor cores.
//
// One CTA takes up to 256 rows (new tokens x the query heads of one kv head),
// one kv head and one range of keys, and walks the range in tiles of 128 keys
// with two slots, each 128 rows with a score tile S and an output O in TMEM:
//     S = Q K^T        tcgen05.mma, Q and K in shared memory, S in TMEM
//     P = 2^(7 + c S - m)  a thread per row: TMEM -> registers -> fp16 -> TMEM
//     O += P V         tcgen05.mma, P from TMEM, V in shared memory, O in TMEM
// one pass over the keys, with a running maximum and sum per row. With more
// than 128 rows the slots are two row tiles that share every key tile; with
// fewer both slots hold the same rows and take the even and the odd key tiles
// (dual), and their results are joined at the end. Either way one slot's
// softmax runs while the tensor cores work for the other.
//
// The products are fp16 (attention.cuh says why). K's block scale multiplies
// the scores; V is decoded as code x 2^(n - r), n its block's scale exponent
// and r the largest one the CTA has met so far, so O is in units of 2^(m + r)
// and is brought along when either grows. That is exact while n >= r - 14, and
// r counts blocks that the mask hides from a row. So from the first tile on
// after which the exponents met lie more than 14 apart, V is decoded as its
// codes ("wide" tiles) and n goes into P's exponent, with a reference per row for
// O's unit from the keys that the row sees, and the softmax's sum takes a second
// exponential (careful_tile, in a loop of its own: 2.6 times as long, 1560 rows x
// 16 heads over 32760 keys 1120 us instead of 430; 2^14 between two blocks'
// largest values is rare). Blocks with the smallest scale 2^-120, which blocks of
// zeros have, do not count for the distance.
//
// Warp roles (16 warps, one CTA per SM):
//   0-3, 4-7   softmax of slot 0 and 1, a thread per row. P is handed over in
//              two halves, so the first half's product runs under the second
//              half's exponentials.
//   8-11       decode 64 keys' codes at a time into the 128-byte-swizzled fp16
//              layout the MMAs read (K: row = key, K-major; V: the same bytes
//              read MN-major, so neither is transposed).
//   12         looks block indices and scales up and bulk-copies the codes
//              (untiled: a block and head is one contiguous piece).
//   13         issues the MMAs (the converged warp, one lane), owns TMEM.
// Shared memory at dim 128: Q 64 KB, two decoded K and two V tiles 128 KB,
// four raw stages 32 KB. TMEM: S (P over it) 2 x 128 columns, O 2 x dim.
//
// Bound: per 256 x 128 tile at dim 128 the MMAs take 2048 cycles and so do the
// 32768 exponentials at 16 per cycle, and shared memory carries about 2560
// cycles' worth (raw codes in, decoded tiles out, MMA operands). Measured: 3550
// cycles per tile with a CTA's start and end (128 tiles), 68% of the tensor
// pipe; 4096 queries x 8 heads over 16384 tokens 1.1 PFLOP/s, 6240 queries x
// 16 heads over 32760 tokens in frames of 1560 1.45 ms (1.07 PFLOP/s at
// sustained clocks), 32760 queries over as many tokens 6.6 to 7.4 ms (1.33 to
// 1.19 PFLOP/s). At dim 64 a tile takes as long (1.78 us as against 1.90): there
// the softmax's own time bounds it. Loads are far below HBM.
//
// The running maximum is lazy (attention.cuh), so after the first tiles O stays
// in TMEM untouched by the softmax threads.
//
// Every wait is bounded; an expired one raises the error word and the CTA's
// abort flag, lets copies and MMAs land, frees TMEM and returns. Warps that
// share a named barrier reach it whatever their waits said.
#include "attention.cuh"
#include "fp8_codec.cuh"

namespace fp8dit {
namespace {

constexpr int kRows = 128;  // rows of a slot = TMEM lanes
constexpr int kKeys = 128;  // keys of a tile
constexpr int kThreads = 512;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kSpread = 14;      // exponents of V's scales that one unit covers exactly
constexpr int kWide = 1000;  // in place of r: a wide tile

// Registers per thread by role, out of the launch's 512 x 128. The softmax holds
// a row's 128 scores: with 168 registers it spilled and was 6% slower, and with
// eight decoding warps there are no more to give it (4% slower at 176).
constexpr int kRegsSoftmax = 200, kRegsConvert = 64, kRegsOther = 48;
static_assert(256 * kRegsSoftmax + 128 * kRegsConvert + 128 * kRegsOther <= kThreads * 128, "register split");

// What the roles of a CTA agree on.
struct Work {
    Request r;
    int b, head, split, r0, rows;  // first row; rows of the request
    int k0;                        // first key of the range
    int n[2];                      // key tiles of each slot
    int tiles;                     // key tiles to decode
    int dual;                      // the slots hold the same rows
};

constexpr int kRing = 8;  // what the loader tells the softmax per key tile; the two are never 8 tiles apart

struct Bars {
    uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2];  // p_full: [slot][half of the keys]
    uint64_t raw_full[4], raw_empty[4];  // first and second 64 keys of K, of V
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t drain;
    alignas(16) float k_scale[kRing][kKeys / 16];  // of every 16 keys (read as float4)
    uint32_t bad[kRing];               // bad blocks, bit per block
    int v_ref[kRing];                // exponent r that V is decoded with, or kWide
    float v_exp[kRing][kKeys / 16];    // n of every 16 keys
    uint32_t v_mul[2][4];              // 2^(n - r) (wide: 1) as fp16, twice: [half of the tile][block]; 0: V counts as 0
    uint32_t tmem;
    int abort;
    int failed[8];  // softmax warp w saw an expired wait
    Work work;       // kept here, not in every thread's registers
};
template <int D>
struct Tile {
    static constexpr int HALF = kKeys * 128;       // 64 dims of 128 rows: 16 KB
    static constexpr int BYTES = HALF * (D / 64);  // an fp16 tile of 128 rows
    static constexpr int RAW = 64 * D;             // a raw stage: 64 keys' codes
    static constexpr int SMEM = 2 * BYTES + 4 * BYTES + 4 * RAW + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(sizeof(Bars) <= 1024, "barrier area");
    static_assert(SMEM <= 232448, "shared memory budget");
};

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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// mbar_wait_bounded for kernels with many waiting warps: after a first try each
// further one may sleep in hardware for up to 20 us. Measured against polling
// without the hint, at sustained (power-limited) clocks: 1% faster.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, const DevErr& err) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if (abort != nullptr && *abort) return false;
        if (globaltimer_ns() - t0 > err.limit_ns) {
            if (abort != nullptr) *abort = 1;
            atomicOr(err.word, kDevErrTimeout);
            return false;
        }
    }
}

// ------------------------------------------------------------ load codes
template <int D>
__device__ __forceinline__ void load_role(const KvAttnArgs& a, Bars* sm, uint8_t* raw, int lane) {
    const Work& w = sm->work;
    const int tlog = a.c.block_log2, T = 1 << tlog, per_tile = kKeys >> tlog;
    const int32_t* table = a.b.table + (int64_t)w.b * a.b.width;
    const int blocks = (w.r.len + T - 1) >> tlog;  // blocks the request has
    const int head = w.head, tiles = w.tiles;
    const uint32_t bytes = (uint32_t)min(T, 64) * D;  // a copy: a block, or half of one of 128
    volatile int* abort = &sm->abort;
    // Lane l < per_tile has the tile's block l. Block indices are fetched two
    // tiles ahead of the copies, scales one.
    int at = (w.k0 >> tlog) + lane;
    auto fetch_page = [&]() {
        const int p = lane < per_tile && at < blocks ? table[at] : -1;
        const bool have = lane < per_tile && at < blocks;
        at += per_tile;
        return have ? (p >= 0 && p < a.c.n_blocks ? p : -2) : -1;  // -1: past the end, -2: bad
    };
    auto fetch_scale = [&](const float* s, int page) {
        return page >= 0 ? s[(int64_t)page * a.c.heads + head] : 1.0f;
    };
    int page = fetch_page(), next = fetch_page();
    float sk = fetch_scale(a.c.ks, page), sv = fetch_scale(a.c.vs, page);
    int v_ref = -120, v_low = 120;  // of the exponents met so far, all and those above -120
    // One raw stage: K's two halves, V's two halves.
    auto mine = [&](int st) { return T == 128 ? lane == 0 : lane < per_tile && ((lane << tlog) >> 6) == (st & 1); };
    const int key = (lane << tlog) & 63;  // first key of this lane's copy in its stage
    auto copy = [&](int st) {
        if (!mine(st) || page < 0) return;
        const int64_t slot = (int64_t)page * a.c.heads + head;
        bulk_load_g2s(raw + st * Tile<D>::RAW + key * D,
                      (st >> 1 ? a.c.v : a.c.k) + ((slot << tlog) + (T == 128 ? 64 * (st & 1) : 0)) * D, bytes,
                      &sm->raw_full[st]);
    };
    // The first tile's copies do not wait for its scales (the barriers count
    // bytes that land before they are announced, too).
    if (tiles > 0)
        for (int st = 0; st < 4; ++st) copy(st);
    int done = 0;  // raw stages announced
    for (int g = 0; g < tiles; ++g) {
        const int after = fetch_page();
        const float nk = fetch_scale(a.c.ks, next), nv = fetch_scale(a.c.vs, next);
        const uint32_t bad = __ballot_sync(0xffffffffu, page == -2);
        const int n = scale_log2_of(sv);
        v_ref = max(v_ref, __reduce_max_sync(0xffffffffu, page >= 0 ? n : -120));
        v_low = min(v_low, __reduce_min_sync(0xffffffffu, page >= 0 && n > -120 ? n : 120));
        const bool wide = v_ref - v_low > kSpread;  // from here on: v_ref only grows, v_low only falls
        const int e = wide ? 0 : n - v_ref;
        uint32_t mul = page < 0 || e < -24 ? 0u : e >= -14 ? (uint32_t)(15 + e) << 10 : 1u << (24 + e);
        mul |= mul << 16;
        const float sk16 = __shfl_sync(0xffffffffu, sk, (lane << 4 >> tlog) & 31);
        const float n16 = __shfl_sync(0xffffffffu, (float)n, (lane << 4 >> tlog) & 31);
        bool fail = false;
        for (int st = 0; st < 4; ++st) {
            const int count = __popc(__ballot_sync(0xffffffffu, mine(st) && page >= 0));
            if (g > 0) {
                if (!__all_sync(0xffffffffu,
                                wait_for(&sm->raw_empty[st], (uint32_t)(g & 1) ^ 1u, abort, a.err))) {
                    fail = true;
                    break;
                }
                copy(st);
            }
            if (st >= 2 && mine(st)) sm->v_mul[st & 1][key >> tlog] = mul;
            if (st == 0) {
                if (lane < kKeys / 16) {
                    sm->k_scale[g % kRing][lane] = sk16;
                    sm->v_exp[g % kRing][lane] = n16;
                }
                if (lane == 0) {
                    sm->bad[g % kRing] = bad;
                    sm->v_ref[g % kRing] = wide ? kWide : v_ref;
                    if (bad) atomicOr(a.err.word, kDevErrIndex);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sm->raw_full[st], (uint32_t)count * bytes);
            ++done;
        }
        if (fail) break;
        page = next, next = after, sk = nk, sv = nv;
    }
    if (*abort) {  // let the copies in flight land
        for (int i = max(0, done - 4); i < done; ++i)
            wait_for(&sm->raw_full[i & 3], (uint32_t)(i >> 2) & 1u, nullptr, a.err);
    }
}

// ---------------------------------------------------------- decode codes
template <int D>
__device__ __forceinline__ void convert_role(const KvAttnArgs& a, Bars* sm, const uint8_t* raw, uint8_t* tiles, int t) {
    // Thread t turns 16 codes (16 bytes) of a raw row into two 16-byte pieces
    // of a swizzled fp16 row, kIters times per stage, kRowStep rows apart. At
    // dim 128 a quarter of a warp reads the first half of one row and the
    // second half of the next: both that read and the writes then cover all
    // banks once.
    constexpr int kIters = D / 32, kRowStep = 2048 / D;
    const int row = D == 128 ? 2 * (t >> 4) + (((t >> 2) ^ (t >> 3)) & 1) : t >> 2;
    const int c16 = D == 128 ? t & 7 : t & 3;
    const uint8_t* src = raw + row * D + c16 * 16;
    const int piece = (c16 & 3) * 2;
    const int to = (c16 >> 2) * Tile<D>::HALF + row * 128;
    uint8_t* dst0 = tiles + to + ((piece ^ (row & 7)) << 4);
    uint8_t* dst1 = tiles + to + (((piece + 1) ^ (row & 7)) << 4);
    const int tlog = a.c.block_log2;
    const int lane = t & 31;
    const int n = sm->work.tiles;
    const int keys = sm->work.r.len - sm->work.k0;  // keys from the range's start on
    volatile int* abort = &sm->abort;
    for (int g = 0; g < n; ++g) {
        const int buf = g & 1;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint64_t* full = v ? &sm->v_full[buf] : &sm->k_full[buf];
            uint64_t* empty = v ? &sm->v_empty[buf] : &sm->k_empty[buf];
            // Not unrolled: the roles' loops share the instruction caches (7% slower).
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int st = 2 * v + half;
                bool ok = wait_for(&sm->raw_full[st], (uint32_t)(g & 1), abort, a.err);
                if (half == 0) ok = ok && wait_for(empty, (uint32_t)((g >> 1) & 1) ^ 1u, abort, a.err);
                if (!__all_sync(0xffffffffu, ok)) return;
                const int at = (2 * v + buf) * Tile<D>::BYTES + half * (64 * 128);
                uint4 in[kIters];
                uint32_t mul[kIters];
#pragma unroll
                for (int it = 0; it < kIters; ++it) {
                    in[it] = *reinterpret_cast<const uint4*>(src + st * Tile<D>::RAW + it * kRowStep * D);
                    if (v) mul[it] = sm->v_mul[half][(row + it * kRowStep) >> tlog];
                }
                if (v) {
                    // Rows without a token may hold NaN codes, which a p of 0 keeps
                    // (K's only reach scores that are masked).
                    const int valid = keys - g * kKeys - half * 64;
                    if (valid < 64 || *(volatile uint32_t*)&sm->bad[g % kRing]) {
#pragma unroll
                        for (int it = 0; it < kIters; ++it)
                            if (row + it * kRowStep >= valid || mul[it] == 0) in[it] = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int it = 0; it < kIters; ++it) {
                    uint32_t o[8];
                    const uint32_t x[4] = {in[it].x, in[it].y, in[it].z, in[it].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[2 * k] = decode2(x[k]);
                        o[2 * k + 1] = decode2(x[k] >> 16);
                    }
                    if (v) {
                        const __half2 m = *reinterpret_cast<const __half2*>(&mul[it]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&o[k]), m);
                            o[k] = *reinterpret_cast<const uint32_t*>(&y);
                        }
                    }
                    *reinterpret_cast<uint4*>(dst0 + at + it * kRowStep * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst1 + at + it * kRowStep * 128) = make_uint4(o[4], o[5], o[6], o[7]);
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
}

// ------------------------------------------------------------------ MMAs
// The whole warp walks through this, one lane issues.
template <int D>
__device__ __forceinline__ void mma_role(const KvAttnArgs& a, Bars* sm, const uint8_t* q, const uint8_t* tiles,
                                         uint32_t tmem) {
    constexpr uint32_t kIdescS = umma_idesc_f16_f32(128, kKeys);
    constexpr uint32_t kIdescO = umma_idesc_f16_f32(128, D) | (1u << 16);  // B (V) is MN-major
    volatile int* abort = &sm->abort;
    const uint32_t lead = elect_one();
    // Broadcast from one lane: known to be the same in the whole warp.
    const int n0 = __shfl_sync(0xffffffffu, sm->work.n[0], 0), n1 = __shfl_sync(0xffffffffu, sm->work.n[1], 0);
    const bool dual = __shfl_sync(0xffffffffu, sm->work.dual, 0) != 0;
    const int rounds = max(n0, n1);
    const uint64_t q_desc = umma_desc_kmajor_sw128(smem_u32(q)), k_desc = umma_desc_kmajor_sw128(smem_u32(tiles));
    const uint64_t v_desc = umma_desc_mnmajor_sw128(smem_u32(tiles) + 2 * Tile<D>::BYTES, Tile<D>::HALF);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, wait_for(bar, parity, abort, a.err));
        tc_fence_after();
        return ok;
    };
    auto k_full = [&](int g) { return wait(&sm->k_full[g & 1], (uint32_t)(g >> 1) & 1u); };
    auto v_full = [&](int g) { return wait(&sm->v_full[g & 1], (uint32_t)(g >> 1) & 1u); };
    // S of slot i = Q (row tile qt) K^T (key tile g).
    auto scores = [&](int i, int qt, int g) {
        const uint64_t qd = q_desc + qt * (Tile<D>::BYTES >> 4), kd = k_desc + (g & 1) * (Tile<D>::BYTES >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            constexpr int kHalf = Tile<D>::HALF >> 4;
            const int off = (s >> 2) * kHalf + (s & 3) * 2;  // in 16-byte units
            mma_f16_warp(lead, tmem + i * kKeys, qd + off, kd + off, kIdescS, s > 0);
        }
        mma_commit_warp(lead, &sm->s_full[i]);
    };
    // O of slot i += P V (key tile g, the slot's tile j), as P's halves come.
    auto output = [&](int i, int j, int g) {
        const uint64_t vd = v_desc + (g & 1) * (Tile<D>::BYTES >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!wait(&sm->p_full[i][half], (uint32_t)j & 1u)) return false;
#pragma unroll
            for (int s = 4 * half; s < 4 * half + 4; ++s)
                mma_f16_tmem_a_warp(lead, tmem + 2 * kKeys + i * D, tmem + i * kKeys + s * 8, vd + s * (2048 >> 4),
                                    kIdescO, j > 0 || s > 0);
        }
        return true;
    };
    bool ok = wait(&sm->q_full[0], 0);
    if (dual) {
        // Slot i has the tiles 2 j + i, alone; tile g is in buffer g & 1 = i.
        for (int i = 0; i < 2 && ok; ++i) {
            if ((i ? n1 : n0) == 0) break;
            ok = k_full(i);
            if (!ok) break;
            scores(i, 0, i);
            mma_commit_warp(lead, &sm->k_empty[i]);
        }
        for (int j = 0; j < rounds && ok; ++j) {
#pragma unroll 1
            for (int i = 0; i < 2 && ok; ++i) {
                const int n = i ? n1 : n0, g = 2 * j + i;
                if (j >= n) break;
                ok = v_full(g) && output(i, j, g);
                if (!ok) break;
                if (j + 1 == n) mma_commit_warp(lead, &sm->o_full[i]);
                mma_commit_warp(lead, &sm->v_empty[i]);
                if (j + 1 < n) {
                    ok = k_full(g + 2);
                    if (!ok) break;
                    scores(i, 0, g + 2);
                    mma_commit_warp(lead, &sm->k_empty[i]);
                }
            }
        }
    } else {
        // Both slots use every key tile; slot 0 may have fewer of them.
        ok = ok && wait(&sm->q_full[1], 0);
        if (ok && rounds > 0) ok = k_full(0);
        if (ok && rounds > 0) {
            if (n0 > 0) scores(0, 0, 0);
            scores(1, 1, 0);
            mma_commit_warp(lead, &sm->k_empty[0]);
        }
        for (int j = 0; j < rounds && ok; ++j) {
            const int next = j + 1;
            ok = v_full(j);
            if (ok && next < n1) ok = k_full(next);
            if (!ok) break;
            if (j < n0) {
                ok = output(0, j, j);
                if (!ok) break;
                if (next == n0) mma_commit_warp(lead, &sm->o_full[0]);
                if (next < n0) scores(0, 0, next);
            }
            ok = output(1, j, j);
            if (!ok) break;
            if (next == n1) mma_commit_warp(lead, &sm->o_full[1]);
            mma_commit_warp(lead, &sm->v_empty[j & 1]);
            if (next < n1) {
                scores(1, 1, next);
                mma_commit_warp(lead, &sm->k_empty[next & 1]);
            }
        }
    }
    // Every MMA and every arrival on this CTA's barriers lands before it ends.
    mma_commit_warp(lead, &sm->drain);
    wait_for(&sm->drain, 0, nullptr, a.err);
}

// --------------------------------------------------------------- softmax
// This warp's 32 rows of O times a factor per row.
template <int D>
__device__ __forceinline__ void scale_rows(uint32_t o_addr, float by) {
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(o_addr + 16 * k, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * by);
        tmem_st_32x32b_x16(o_addr + 16 * k, o);
    }
}

// A tile of slot i for which the usual loop is not exact: a wide one, or scores
// so large that a score's product and the rounded reference lie more than the
// room in P's range apart. 16 keys at a time: the scores are read from TMEM once
// for the references and once for the weights, and a chunk's P goes into
// columns whose scores have been read. Keys from `seen` on and bad blocks are
// masked. O is in units of 2^(m + v): v follows the largest score (over m) plus
// exponent of V that the row has seen; the first time it is what the tiles
// before used, which may lie kSpread above that. Scores only meet as
// differences, which are exact where they matter.
template <int D>
__device__ __forceinline__ void careful_tile(Bars* sm, int i, int ring, int block_log2, uint32_t s_addr, uint32_t o_addr, float c,
                                             int seen, uint32_t bad, bool have_o, bool first, int lane, float& m, float& l,
                                             float& v) {
    const int r = *(volatile int*)&sm->v_ref[ring];
    auto unit = [&](int k) { return r == kWide ? sm->v_exp[ring][k] : (float)r; };
    float s[16];
    auto scores = [&](int k) {
        uint32_t x[16];
        tmem_ld_32x32b_x16(s_addr + 16 * k, x);
        tmem_wait_ld16(x);
        const int end = bad >> (16 * k >> block_log2) & 1u ? 0 : seen - 16 * k;
        const float f = score_factor(c, sm->k_scale[ring][k]);
#pragma unroll
        for (int y = 0; y < 16; ++y) s[y] = y < end ? __fmul_rn(__uint_as_float(x[y]), f) : kNegInf;
    };
    float t[8], top = kNegInf;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        scores(k);
        t[k] = s[0];
#pragma unroll
        for (int x = 1; x < 16; ++x) t[k] = fmaxf(t[k], s[x]);
        top = fmaxf(top, t[k]);
    }
    const float to = fmaxf(m, top);
    const bool any = to != kNegInf;  // else the row has seen nothing yet: O is 0
    float scale_o = 1.0f;
    if (any) {
        const float down = m - to;
        float next = (first ? v - kSpread : v) + down;
#pragma unroll
        for (int k = 0; k < 8; ++k) next = fmaxf(next, (t[k] - to) + unit(k));
        l *= ex2_approx(down);
        scale_o = ex2_approx(v + down - next);
        v = next, m = to;
    }
    if (have_o) scale_rows<D>(o_addr, scale_o);
    const float ref = any ? m : 0.0f;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
        scores(k);
        const float more = unit(k) - v;
        float sum = 0.0f;
        uint32_t p[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float d0 = (s[2 * x] - ref) + kLift, d1 = (s[2 * x + 1] - ref) + kLift;
            sum += ex2_approx(d0) + ex2_approx(d1);
            p[x] = pack_f16x2(ex2_approx(d0 + more), ex2_approx(d1 + more));
        }
        tmem_st_32x32b_x8(s_addr + 8 * k, p);
        l += sum;
        if ((k & 3) == 3) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->p_full[i][k >> 2]);
        }
    }
}

// Thread t of 128: a row of slot i.
template <int D>
__device__ __forceinline__ void softmax_role(const KvAttnArgs& a, Bars* sm, uint8_t* q, uint8_t* tiles, uint32_t tmem,
                                             int i, int t) {
    const Work& w = sm->work;
    const int lane = t & 31, warp = 4 * i + (t >> 5);
    const bool dual = w.dual != 0;
    const int row = w.r0 + (dual ? 0 : i * kRows) + t;
    const bool in = row < w.rows;
    // Rows past the last one compute on zeros and are not written.
    const int limit = (in ? key_limit(w.r.len - w.r.n + row / a.group, w.r.len, a.frame) : w.r.len) - w.k0;
    volatile int* abort = &sm->abort;
    // Q, a warp its 32 rows: D / 8 lanes read a row (16 bytes each), so every
    // load is whole lines, and agree on its largest |q|.
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    float c = 0.0f;  // softmax scale * log2(e) / q's scale, of this thread's row
    {
        const int token = in ? row / a.group : 0, qh = w.head * a.group + (in ? row % a.group : 0);
        const int64_t own = in ? (int64_t)(w.r.first + token) * a.q.token_stride + (int64_t)qh * a.q.head_stride : -1;
        const int part = lane % kLanes;
        uint4 v[kLanes];
#pragma unroll
        for (int k = 0; k < kLanes; ++k) {
            const int64_t at = __shfl_sync(0xffffffffu, own, k * kAtOnce + lane / kLanes);
            v[k] = make_uint4(0, 0, 0, 0);
            if (at >= 0) v[k] = *reinterpret_cast<const uint4*>(a.q.ptr + at + part * 8);
        }
        // Step by step over all rows: each step is a chain of dependent shuffles.
        uint32_t top[kLanes];
#pragma unroll
        for (int k = 0; k < kLanes; ++k) top[k] = fold_halves(absmax8(v[k], 0));
#pragma unroll
        for (int z = 1; z < kLanes; z <<= 1)
#pragma unroll
            for (int k = 0; k < kLanes; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], z));
        uint32_t mine = 0;
#pragma unroll
        for (int k = 0; k < kLanes; ++k) {
            const uint32_t x = __shfl_sync(0xffffffffu, top[k], (lane % kAtOnce) * kLanes);
            if (lane / kAtOnce == k) mine = x;
        }
        c = a.scale_log2 * pow2f(-q_exponent(mine, a.q_most));
        if (!dual || i == 0) {
#pragma unroll
            for (int k = 0; k < kLanes; ++k) {
                const float f = pow2f(q_exponent(top[k], a.q_most));
                const int r = (t & 96) + k * kAtOnce + lane / kLanes;
                uint32_t* y = &v[k].x;
#pragma unroll
                for (int z = 0; z < 4; ++z) y[z] = pack_f16x2(bf16_lo(y[z]) * f, bf16_hi(y[z]) * f);
                *reinterpret_cast<uint4*>(q + i * Tile<D>::BYTES + r * 128 + (part >> 3) * Tile<D>::HALF +
                                          (((part & 7) ^ (r & 7)) << 4)) = v[k];
            }
        }
        if (!dual || i == 0) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->q_full[i]);
        }
    }
    const uint32_t lanes = (uint32_t)(t >> 5) << 21;  // this warp's TMEM lanes: (t / 32) * 32 << 16
    const uint32_t s_addr = tmem + lanes + i * kKeys, o_addr = tmem + lanes + 2 * kKeys + i * D;
    const int n = w.n[i];
    // P and l are in units of 2^(m - kLift), O in units of 2^(m - kLift + r_now). m
    // is a largest score itself, not rounded: its own weight is then exact in P,
    // which counts where few keys have most of a row's weight (the error of 26
    // rows over 32760 keys, scores spread over several units, halves).
    // A tile's weights add up by themselves (small ones would be lost beside a
    // large l) and meet l one turn later: 1.3% faster than at the tile's end.
    float m = kNegInf, l = 0.0f, recent = 0.0f;
    int r_now = -120;
    bool ok = true;
    int j = 0;
    for (; j < n; ++j) {
        const int g = dual ? 2 * j + i : j;
        ok = __all_sync(0xffffffffu, wait_for(&sm->s_full[i], (uint32_t)j & 1u, abort, a.err));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(s_addr + 32 * k, s[k]);
        float f[8];  // score factors of 16 keys each
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 ks = *reinterpret_cast<const float4*>(&sm->k_scale[g % kRing][4 * k]);
            f[4 * k] = score_factor(c, ks.x), f[4 * k + 1] = score_factor(c, ks.y);
            f[4 * k + 2] = score_factor(c, ks.z), f[4 * k + 3] = score_factor(c, ks.w);
        }
        l += recent;
        const int seen = limit - g * kKeys;  // this row sees columns below it
        const uint32_t bad = *(volatile uint32_t*)&sm->bad[g % kRing];
        const int r = *(volatile int*)&sm->v_ref[g % kRing];
        const bool mask = __any_sync(0xffffffffu, seen < kKeys) || bad;
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_tie32(s[k]);
        if (__builtin_expect(mask, 0)) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (32 * k + x >= seen) s[k][x] = __float_as_uint(kNegInf);
            if (bad) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int x = 0; x < 32; x += 16)
                        if (bad >> ((32 * k + x) >> a.c.block_log2) & 1u) {
#pragma unroll
                            for (int y = 0; y < 16; ++y) s[k][x + y] = __float_as_uint(kNegInf);
                        }
            }
        }
        float tile_top = kNegInf;
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            const uint32_t* y = &s[z >> 1][(z & 1) * 16];
            float u0 = max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
            float u1 = max3(__uint_as_float(y[3]), __uint_as_float(y[4]), __uint_as_float(y[5]));
#pragma unroll
            for (int x = 6; x < 14; x += 4) {
                u0 = max3(u0, __uint_as_float(y[x]), __uint_as_float(y[x + 1]));
                u1 = max3(u1, __uint_as_float(y[x + 2]), __uint_as_float(y[x + 3]));
            }
            u0 = max3(u0, __uint_as_float(y[14]), __uint_as_float(y[15]));
            tile_top = fmaxf(tile_top, fmaxf(u0, u1) * f[z]);
        }
        if (__builtin_expect(__any_sync(0xffffffffu, tile_top > m + kLazy) || r != r_now, 0)) {
            // From here on the careful way: wide (as are all tiles behind it), or
            // scores of 2^22 and more.
            if (r == kWide || __any_sync(0xffffffffu, fabsf(tile_top) > 0x1p22f && tile_top != kNegInf)) {
                recent = 0.0f;
                break;
            }
            const float to = fmaxf(m, tile_top);
            const float down = to == kNegInf ? 1.0f : ex2_approx(m - to);
            const float fo = down * ex2_approx((float)(r_now - r));
            m = to;
            l *= down;
            r_now = r;
            if (j > 0) scale_rows<D>(o_addr, fo);  // O of the earlier tiles is complete: S came after it
        }
        const float neg = m == kNegInf ? 0.0f : kLift - m;
        const f32x2_t neg2 = f2_pack(neg, neg);
        f32x2_t sum[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int k = 2 * half; k < 2 * half + 2; ++k) {
                uint32_t p[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float fx = f[2 * k + (x >> 3)];
                    const float2 e = f2_unpack(
                        f2_fma(f2_pack(__uint_as_float(s[k][2 * x]), __uint_as_float(s[k][2 * x + 1])), f2_pack(fx, fx), neg2));
                    const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
                    sum[x & 1] = f2_add(sum[x & 1], f2_pack(p0, p1));
                    p[x] = pack_f16x2(p0, p1);
                }
                tmem_st_32x32b_x16(s_addr + 16 * k, p);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->p_full[i][half]);
        }
        const float2 t2 = f2_unpack(f2_add(sum[0], sum[1]));
        recent = t2.x + t2.y;
    }
    l += recent;
    float v_ref = (float)r_now;  // O's unit over l's, log2
    for (bool first = true; ok && j < n; ++j, first = false) {
        const int g = dual ? 2 * j + i : j;
        ok = __all_sync(0xffffffffu, wait_for(&sm->s_full[i], (uint32_t)j & 1u, abort, a.err));
        if (!ok) break;
        tc_fence_after();
        careful_tile<D>(sm, i, g % kRing, a.c.block_log2, s_addr, o_addr, c, limit - g * kKeys,
                        *(volatile uint32_t*)&sm->bad[g % kRing], j > 0, first, lane, m, l, v_ref);
    }
    // The slot's O; without a key tile the slot's Q, whose buffer takes the rows
    // on their way out: every warp of the slot has to have written its own.
    if (ok) ok = __all_sync(0xffffffffu, wait_for(n > 0 ? &sm->o_full[i] : &sm->q_full[dual ? 0 : i], 0, abort, a.err));
    tc_fence_after();

    // Dual: slot 1 leaves its results in the buffers that only it has used (K's
    // and V's second; [4 dims][row] float4), slot 0 joins them.
    auto other = [&](int d4) {
        uint8_t* base = tiles + (d4 < D / 8 ? 1 : 3) * Tile<D>::BYTES;
        return reinterpret_cast<float4*>(base) + (d4 < D / 8 ? d4 : d4 - D / 8) * kRows + t;
    };
    float* meta = reinterpret_cast<float*>(q + Tile<D>::BYTES);  // reference, sum, unit
    if (dual) {
        if (i == 1 && ok) {
            meta[t] = m;
            meta[kRows + t] = l;
            meta[2 * kRows + t] = v_ref;
            if (n > 0) {
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(o_addr + 16 * k, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *other(4 * k + x) = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                                        __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
                }
            }
        }
        if (!ok && lane == 0) *(volatile int*)&sm->failed[warp] = 1;
        named_barrier_sync(1, 256);  // reached whatever the waits said
        if (i == 1) return;
        if (*(volatile int*)&sm->failed[warp + 4]) ok = false;
    }
    if (!ok) return;
    // out = (O own + O' theirs) 2^unit / l, O' of the other slot. The larger of
    // the two slots' units 2^(m + v_ref) is the common one, so no factor exceeds
    // one, whatever block scales either slot has met.
    float own = 1.0f, theirs = 0.0f, unit = v_ref;
    if (dual && w.n[1] > 0) {
        const float mo = meta[t], to = fmaxf(m, mo);
        if (to != kNegInf) {
            const float x = ex2_approx(m - to), y = ex2_approx(mo - to), vo = meta[2 * kRows + t];
            const float ahead = (m - mo) + (v_ref - vo);
            own = ex2_approx(fminf(ahead, 0.0f)), theirs = ex2_approx(fminf(-ahead, 0.0f));
            unit = ahead >= 0.0f ? unit + (m - to) : vo + (mo - to);
            l = l * x + meta[kRows + t] * y;
        }
        m = to;
    }
    // 2^unit may be 2^-120: half of it in front of the division, half behind.
    const bool some = l > 0.0f || l != l;
    const float half = some ? ex2_approx(0.5f * unit) : 0.0f, inv = some ? half / l : 0.0f;
    own *= half, theirs *= half;
    // Taken again rather than kept in registers through the loop.
    const int token = in ? row / a.group : 0, qh = w.head * a.group + (in ? row % a.group : 0);
    const int64_t tok = w.r.first + token;
    const int64_t flat = tok * a.q.heads + qh;
    const int64_t part = (int64_t)w.split * a.b.total * a.q.heads + flat;
    if (in) {
        if (a.splits > 1)
            a.part_sum[part] = make_float2(m, l * (1.0f / (1 << (int)kLift)));
        else if (a.lse)
            a.lse[flat] = m == kNegInf ? kNegInf : kLog2ToNat * (m - kLift + lg2_approx(l));
    }
    // Through the slot's Q buffer (all four warps have written it, every product
    // with it is done), so that rows leave in whole lines: 16-byte pieces,
    // swizzled by the row. fp32 partials take two passes of half the dims.
    uint8_t* stage = q + i * Tile<D>::BYTES;
    const bool partial = a.splits > 1;
    const int64_t own_at = !in ? -1 : partial ? part * D : tok * a.out.token_stride + (int64_t)qh * a.out.head_stride;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            const int k = pass * (D / 32) + kk;
            uint32_t o[16];
            if (n > 0) {
                tmem_ld_32x32b_x16(o_addr + 16 * k, o);
                tmem_wait_ld16(o);
            } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = 0;
            }
            float y[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) y[x] = __uint_as_float(o[x]) * own;
            if (theirs != 0.0f) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float4 z = *other(4 * k + x);
                    y[4 * x] = fmaf(z.x, theirs, y[4 * x]);
                    y[4 * x + 1] = fmaf(z.y, theirs, y[4 * x + 1]);
                    y[4 * x + 2] = fmaf(z.z, theirs, y[4 * x + 2]);
                    y[4 * x + 3] = fmaf(z.w, theirs, y[4 * x + 3]);
                }
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) y[x] *= inv;
            auto put = [&](int piece, uint4 x) {
                *reinterpret_cast<uint4*>(stage + t * (2 * D) + ((piece ^ (t & 7)) << 4)) = x;
            };
            if (partial) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    put(4 * kk + x, make_uint4(__float_as_uint(y[4 * x]), __float_as_uint(y[4 * x + 1]),
                                               __float_as_uint(y[4 * x + 2]), __float_as_uint(y[4 * x + 3])));
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    put(2 * k + x,
                        make_uint4(pack_bf16x2(y[8 * x], y[8 * x + 1]), pack_bf16x2(y[8 * x + 2], y[8 * x + 3]),
                                   pack_bf16x2(y[8 * x + 4], y[8 * x + 5]), pack_bf16x2(y[8 * x + 6], y[8 * x + 7])));
            }
        }
        if (!partial && pass == 0) continue;
        __syncwarp();
#pragma unroll 8
        for (int k = 0; k < kLanes; ++k) {
            const int r = k * kAtOnce + lane / kLanes, piece = lane % kLanes;
            const int64_t at = __shfl_sync(0xffffffffu, own_at, r);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + ((t & 96) + r) * (2 * D) + ((piece ^ (r & 7)) << 4));
            if (at < 0) continue;
            if (partial)
                *reinterpret_cast<uint4*>(a.part_o + at + pass * (D / 2) + piece * 4) = x;
            else
                *reinterpret_cast<uint4*>(a.out.ptr + at + piece * 8) = x;
        }
        __syncwarp();
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_tiles(const __grid_constant__ KvAttnArgs a) {
    // Dynamic shared memory starts on a 1024-byte boundary (there is no static
    // one); the swizzled tiles rely on it, so it is checked.
    extern __shared__ __align__(1024) uint8_t q[];
    uint8_t* tiles = q + 2 * Tile<D>::BYTES;  // K buffers 0, 1, V buffers 0, 1
    uint8_t* raw = tiles + 4 * Tile<D>::BYTES;
    Bars* sm = reinterpret_cast<Bars*>(raw + 4 * Tile<D>::RAW);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (smem_u32(q) & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.err.word, kDevErrTimeout);
        return;
    }

    // CTAs in launch order: heads fastest, then key ranges, then a request's row
    // tiles from the last (which under a causal mask sees most) to the first, a
    // short last one at its end, then the requests, longest cache first (up to
    // 32 of them): what takes longest begins first. (Requests of 1209 .. 6001
    // tokens with row tiles outermost: 237 us, so: 223.)
    Work w;
    uint32_t id = blockIdx.x;
    w.head = (int)(id % (uint32_t)a.c.heads);
    id /= (uint32_t)a.c.heads;
    w.split = (int)(id % (uint32_t)a.splits);
    id /= (uint32_t)a.splits;
    const int place = (int)(id % (uint32_t)a.row_tiles) + a.tail_last;
    const int tile = place == a.row_tiles ? place - 1 : a.row_tiles - 1 - place;
    w.b = (int)(id / (uint32_t)a.row_tiles);
    if (a.b.n > 1 && a.b.n <= 32) {
        const int len = lane < a.b.n ? a.b.kv_lens[lane] : INT32_MIN;
        int before = 0;  // requests that go before this lane's
        for (int k = 0; k < a.b.n; ++k) {
            const int other = __shfl_sync(0xffffffffu, len, k);
            before += other > len || (other == len && k < lane);
        }
        w.b = __ffs(__ballot_sync(0xffffffffu, lane < a.b.n && before == w.b)) - 1;
    }
    w.r = load_request(a.b, w.b, a.err, false);
    w.rows = w.r.n * a.group;
    w.r0 = tile * 2 * kRows;
    w.k0 = w.split * a.chunk;
    if (w.r0 >= w.rows || (w.split > 0 && w.k0 >= w.r.len)) return;
    w.dual = w.rows - w.r0 <= kRows;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = min(w.r0 + (w.dual ? 1 : i + 1) * kRows, w.rows) - 1;
        const int keys = min(key_limit(w.r.len - w.r.n + last / a.group, w.r.len, a.frame), w.k0 + a.chunk) - w.k0;
        w.n[i] = keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
    }
    w.tiles = w.n[1];
    if (w.dual) {
        w.n[0] = (w.tiles + 1) / 2;
        w.n[1] = w.tiles / 2;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->q_full[i], 4);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->p_full[i][0], 4);
            mbar_init(&sm->p_full[i][1], 4);
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
        for (int i = 0; i < 8; ++i) sm->failed[i] = 0;
        sm->work = w;
        fence_mbarrier_init();
    }
    if (warp == 13) {
        tmem_alloc(&sm->tmem, Tile<D>::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm->tmem, 0);

    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        softmax_role<D>(a, sm, q, tiles, tmem, warp >> 2, threadIdx.x & 127);
    } else if (warp < 12) {
        regs_dec<kRegsConvert>();
        convert_role<D>(a, sm, raw, tiles, threadIdx.x & 127);
    } else {
        regs_dec<kRegsOther>();
        if (warp == 12)
            load_role<D>(a, sm, raw, lane);
        else if (warp == 13)
            mma_role<D>(a, sm, q, tiles, tmem);
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
