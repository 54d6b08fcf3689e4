// Attention over the E4M3 cache for few query rows, and the join of split
// key ranges.
//
// A request's rows are its new tokens times the query heads that share a kv
// head; one CTA takes a tile of up to 16 rows, one kv head and one range of
// keys, so a cached byte is read once for the whole group of heads. Its four
// warps walk the range in granules of 16 keys (always inside one block: a
// block is 16 tokens or more), each with its own running references, sums and
// output, which are joined through shared memory at the end.
//
// Mathematics, per granule and warp (mma.sync m16n8k16, fp16 -> fp32):
//     S^T = K Q^T      A = 16 keys x dim, B = 8 query rows per column tile
//     P^T = 2^(7 + t - v)  t = s - mu + log2 S_V: the score plus V's block scale
//     O^T += V^T P^T   A = dim x 16 keys, B = P^T
// Keys and values are the A operands so that 8 rows fill a column tile (the
// 16-row A side would be half empty at a group of 8 or fewer). Both products
// leave the order of their inner index free, which lets a thread use 16-byte
// loads straight from the cache as its fragments: for K the 16 bytes at
// dim 16 tig (+ 64) of keys gid and gid + 8, with Q permuted the same way;
// for V the 16 bytes at dim 16 gid of keys 2 tig, 2 tig + 1, 2 tig + 8,
// 2 tig + 9, whose bytes a permute pairs across keys. P^T comes out of S^T by
// an 8 x 8 transpose in registers (movmatrix).
//
// The products are fp16 (attention.cuh says why; decoding to bf16 this kernel
// issued 520 instructions per granule instead of 376 and was bound by them).
// K's scale multiplies the score; V's is in the exponent of P, with a
// reference v of its own (over mu, the scores'), so P is exact to 2^-32 of the
// row's largest contribution however V's scales differ. The softmax sum takes a
// second exponential 2^(s - mu), in fp32. Scores only meet as differences, so
// their size does not matter.
//
// Both references are lazy (attention.cuh), so the usual granule needs one vote
// and no shuffles.
//
// Bound: HBM, 2 bytes per token, kv head and dim. 32 requests of 100 .. 16001
// tokens, 8 kv heads of 128, 4 query heads each: 104 us, 5.1 TB/s; alone and
// with equal lengths of 8000 the kernel reads 5.7 TB/s (87% of a copy).
#include <algorithm>

#include "attention.cuh"
#include "fp8_codec.cuh"


namespace fp8dit {
namespace {

constexpr int kWarps = 4;
constexpr int kGranule = 16;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMostRanges = 64;  // of keys, that a call is cut into

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A warp's ring of granules in shared memory, filled by cp.async two granules
// ahead: 8 KB of loads in flight per warp (dim 128) without registers to hold
// them. (One granule ahead in registers, the GPU waited on loads 60% of the
// time: 4.2 TB/s.) 16-byte pieces are swizzled within 128-byte lines so that
// the fragments' reads are free of bank conflicts.
constexpr int kStages = 3;

template <int D>
struct Ring {
    static constexpr int BYTES = kGranule * D;  // a granule's K or V codes
    uint8_t k[kStages][BYTES], v[kStages][BYTES];
};
struct Header {
    float ks, vs;
    int ok;  // the block index is valid
    int pad;
};

// Byte offset of 16-byte piece c of a granule's row r.
template <int D>
__device__ __forceinline__ int piece(int r, int c) {
    const int line = D == 128 ? r : r >> 1;
    const int p = D == 128 ? c : (r & 1) * 4 + c;
    // K's reads pair rows 2 i, 2 i + 1; V's take rows 0, 2, 4, 6 (+ 1) at once.
    const int sw = D == 128 ? (((r ^ (r >> 2)) & 1) << 2) | (r & 2) : (line & 3) << 1;
    return line * 128 + ((p ^ sw) << 4);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__device__ __forceinline__ void load_granule(Ring<D>& ring, Header* hdr, int stage, const KvAttnArgs& a, int page,
                                             int head, int row, int lane) {
    const bool ok = page >= 0 && page < a.c.n_blocks;
    if (lane == 0) {
        hdr[stage].ok = ok;
        if (!ok) atomicOr(a.err.word, kDevErrIndex);
    }
    if (!ok) return;
    const int64_t slot = (int64_t)page * a.c.heads + head;
    const int64_t at = ((slot << a.c.block_log2) + row) * D + lane * 16;
    constexpr int kPieces = D / 16;  // per row
#pragma unroll
    for (int i = 0; i < kGranule * kPieces / 32; ++i) {
        const int p = i * 32 + lane;
        const int to = piece<D>(p / kPieces, p % kPieces);
        cp_async16(ring.k[stage] + to, a.c.k + at + i * 512);
        cp_async16(ring.v[stage] + to, a.c.v + at + i * 512);
    }
    if (lane == 0) cp_async4(&hdr[stage].ks, a.c.ks + slot);
    if (lane == 1) cp_async4(&hdr[stage].vs, a.c.vs + slot);
}

template <int D, int NT>
struct RowsSmem {
    float v[kWarps][8 * NT], mu[kWarps][8 * NT], l[kWarps][8 * NT];
    float o[kWarps][8 * NT][D + 4];
};

// The warps' common references of row q: mu, and top for the rest of O's exponent.
template <int D, int NT>
__device__ __forceinline__ void common(const RowsSmem<D, NT>& sm, int q, float& mu, float& top) {
    mu = sm.mu[0][q];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mu = fmaxf(mu, sm.mu[w][q]);
    top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, (sm.mu[w][q] - mu) + sm.v[w][q]);  // NaN without a key: left out
}

// A warp's running state: per lane the columns (query rows) 2 tig, 2 tig + 1 of
// every column tile.
template <int D, int NT>
struct RowsState {
    uint32_t q[NT][D / 16][2];  // scaled fp16 Q^T fragments
    float cq[NT][2];            // softmax scale * log2(e) / q's scale
    int limit[NT][2];           // keys the row sees
    float mu[NT][2], v[NT][2];  // references: scores', and of score over mu plus V's exponent
    float l[NT][2], o[NT][D / 16][4];
};

template <int D, int NT>
__device__ __forceinline__ void attend_granule(RowsState<D, NT>& st, const uint8_t* kc, const uint8_t* vc,
                                               const Header& h, int key, int least, int len, int gid, int tig) {
    if (!h.ok) return;
    const float ks = h.ks, vs = h.vs;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(kc + piece<D>(gid, 4 * c + tig));
        const uint4 y4 = *reinterpret_cast<const uint4*>(kc + piece<D>(gid + 8, 4 * c + tig));
        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = decode2(x[i]), a1 = decode2(y[i]), a2 = decode2(x[i] >> 16), a3 = decode2(y[i] >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_16816(s[nt], a0, a1, a2, a3, st.q[nt][4 * c + i][0], st.q[nt][4 * c + i][1]);
        }
    }
    // V's codes: keys 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9, D / 8 dims from gid (D / 8).
    uint32_t v[4][D / 32];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 2 * tig + (r & 1) + 8 * (r >> 1);
        if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vc + piece<D>(row, gid));
            v[r][0] = w.x, v[r][1] = w.y, v[r][D / 32 - 2] = w.z, v[r][D / 32 - 1] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vc + piece<D>(row, gid >> 1) + (gid & 1) * 8);
            v[r][0] = w.x, v[r][1] = w.y;
        }
    }
    // V's scale is a power of two: its log2 is its exponent.
    const float ev = (float)scale_log2_of(vs);
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float f0 = score_factor(st.cq[nt][0], ks), f1 = score_factor(st.cq[nt][1], ks);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] *= i & 1 ? f1 : f0;
    }
    if (key + kGranule > least) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (key + gid + 8 * (i >> 1) >= st.limit[nt][i & 1]) s[nt][i] = kNegInf;
        // Rows behind the last token may hold NaN codes, which a p of 0 keeps.
        if (key + kGranule > len) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (key + 2 * tig + (r & 1) + 8 * (r >> 1) >= len) {
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) v[r][w] = 0;
                }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float t = fmaxf(s[nt][i], s[nt][i + 2]) - st.mu[nt][i];
            over |= t > kLazy || t + ev > st.v[nt][i] + kLazy;
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float t = fmaxf(s[nt][i], s[nt][i + 2]);
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                const float mu = fmaxf(st.mu[nt][i], t);
                const bool none = mu == kNegInf;  // nothing seen yet
                const float down = none ? 0.0f : st.mu[nt][i] - mu, was = st.v[nt][i] + down;
                const float v = none ? was : fmaxf(was, (t - mu) + ev);
                st.l[nt][i] *= ex2_approx(down);
                const float c = ex2_approx(was - v);
                st.mu[nt][i] = mu;
                st.v[nt][i] = v;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    st.o[nt][d][i] *= c;
                    st.o[nt][d][i + 2] *= c;
                }
            }
    }
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // A row that has seen nothing yet has a reference of -inf; its scores are too.
            const float mu = st.mu[nt][i] == kNegInf ? 0.0f : st.mu[nt][i], more = (ev + kLift) - st.v[nt][i];
            const float d0 = s[nt][i] - mu, d1 = s[nt][i + 2] - mu;
            st.l[nt][i] += ex2_approx(d0) + ex2_approx(d1);
            e[i] = ex2_approx(d0 + more);
            e[i + 2] = ex2_approx(d1 + more);
        }
        p[nt][0] = transpose_8x8(pack_f16x2(e[0], e[1]));
        p[nt][1] = transpose_8x8(pack_f16x2(e[2], e[3]));
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        // Bytes of two keys side by side, two dims per word.
        const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
        const uint32_t a[2][4] = {{decode2(x0), decode2(x0 >> 16), decode2(y0), decode2(y0 >> 16)},
                                  {decode2(x1), decode2(x1 >> 16), decode2(y1), decode2(y1 >> 16)}};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_16816(st.o[nt][2 * w + half], a[half][0], a[half][1], a[half][2], a[half][3], p[nt][0], p[nt][1]);
    }
}

// The rings while the keys are walked, the warps' results afterwards.
template <int D, int NT>
constexpr int kRowsSmem = kWarps * (sizeof(Ring<D>) + kStages * sizeof(Header)) > sizeof(RowsSmem<D, NT>)
                              ? kWarps * (sizeof(Ring<D>) + kStages * sizeof(Header))
                              : sizeof(RowsSmem<D, NT>);

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 4 : 3) kv_attn_rows(const __grid_constant__ KvAttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    RowsSmem<D, NT>& sm = *reinterpret_cast<RowsSmem<D, NT>*>(smem);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int split = blockIdx.x % a.splits;
    const int tile = (blockIdx.x / a.splits) % a.row_tiles;
    const int b = blockIdx.x / a.splits / a.row_tiles;
    const int head = blockIdx.y;
    const Request r = load_request(a.b, b, a.err, false);
    const int rows = r.n * a.group;  // row -> token row / group, query head head * group + row % group
    const int r0 = tile * 8 * NT;
    if (r0 >= rows) return;
    // Keys that the tile's rows see at most / at least (limits grow with the token).
    const int t_first = r0 / a.group, t_last = (min(r0 + 8 * NT, rows) - 1) / a.group;
    const int most = key_limit(r.len - r.n + t_last, r.len, a.frame);
    const int least = key_limit(r.len - r.n + t_first, r.len, a.frame);
    const int k0 = split * a.chunk;
    const int k1 = min(most, k0 + a.chunk);
    if (k0 >= r.len && split > 0) return;  // not read by the join either

    const int32_t* table = a.b.table + (int64_t)b * a.b.width;
    const int bmask = (1 << a.c.block_log2) - 1;
    constexpr int kStep = kWarps * kGranule;
    int key = k0 + warp * kGranule;
    Ring<D>& ring = reinterpret_cast<Ring<D>*>(smem)[warp];
    Header* hdr = reinterpret_cast<Header*>(smem + kWarps * sizeof(Ring<D>)) + warp * kStages;
    // Granules load[0 .. kStages - 1) are on their way before the first is computed.
    int page = key < k1 ? table[key >> a.c.block_log2] : 0;
    int load = key;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        const int now = page;
        if (load + kStep < k1) page = table[(load + kStep) >> a.c.block_log2];
        if (load < k1) load_granule<D>(ring, hdr, i, a, now, head, load & bmask, lane);
        cp_async_commit();
        load += kStep;
    }

    RowsState<D, NT> st;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = r0 + nt * 8 + gid;
        const bool in = row < rows;
        const uint16_t* qp = a.q.ptr;
        if (in)
            qp += (int64_t)(r.first + row / a.group) * a.q.token_stride +
                  (int64_t)(head * a.group + row % a.group) * a.q.head_stride + tig * 16;
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            uint2 w = make_uint2(0, 0);
            if (in) w = *reinterpret_cast<const uint2*>(qp + (s >> 2) * 64 + (s & 3) * 4);
            st.q[nt][s][0] = w.x;
            st.q[nt][s][1] = w.y;
            top = absmax2(w.x, absmax2(w.y, top));
        }
        top = fold_halves(top);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = q_exponent(top, a.q_most);
        const float f = pow2f(e), back = pow2f(-e);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w = st.q[nt][s][i];
                st.q[nt][s][i] = pack_f16x2(bf16_lo(w) * f, bf16_hi(w) * f);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            st.cq[nt][i] = a.scale_log2 * __shfl_sync(0xffffffffu, back, (2 * tig + i) * 4);
            const int lr = r0 + nt * 8 + 2 * tig + i;
            st.limit[nt][i] = lr < rows ? key_limit(r.len - r.n + lr / a.group, r.len, a.frame) : 0;
            st.mu[nt][i] = kNegInf;
            st.v[nt][i] = 0.0f;
            st.l[nt][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[nt][i][0] = st.o[nt][i][1] = st.o[nt][i][2] = st.o[nt][i][3] = 0.0f;
    }

    int stage = 0;
    for (; key < k1; key += kStep) {
        cp_async_wait<kStages - 2>();
        __syncwarp();  // every lane's pieces of this granule; the one before has been read
        const int to = stage == 0 ? kStages - 1 : stage - 1;
        if (load < k1) {
            const int now = page;
            if (load + kStep < k1) page = table[(load + kStep) >> a.c.block_log2];
            load_granule<D>(ring, hdr, to, a, now, head, load & bmask, lane);
        }
        cp_async_commit();
        load += kStep;
        attend_granule<D, NT>(st, ring.k[stage], ring.v[stage], hdr[stage], key, least, r.len, gid, tig);
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings' memory becomes sm

    // Join the warps: per row the common references, then the scaled sums.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float l = st.l[nt][i];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (gid == 0) {
                const int q = nt * 8 + 2 * tig + i;
                sm.v[warp][q] = st.v[nt][i];
                sm.mu[warp][q] = st.mu[nt][i];
                sm.l[warp][q] = l;
            }
        }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = nt * 8 + 2 * tig + i;
            float mu, top;
            common<D, NT>(sm, q, mu, top);
            const float c = st.mu[nt][i] == kNegInf ? 0.0f : ex2_approx((st.mu[nt][i] - mu) + st.v[nt][i] - top);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                // Row gid of column tile d is dim gid (D / 8) + 2 d, row gid + 8 the next one.
                float2 x = make_float2(st.o[nt][d][i] * c, st.o[nt][d][i + 2] * c);
                *reinterpret_cast<float2*>(&sm.o[warp][q][gid * (D / 8) + 2 * d]) = x;
            }
        }
    __syncthreads();
    const int64_t total_rows = (int64_t)a.b.total * a.q.heads;
    for (int at = threadIdx.x; at < 8 * NT * (D / 4); at += 32 * kWarps) {
        const int q = at / (D / 4), d = (at % (D / 4)) * 4;
        const int row = r0 + q;
        if (row >= rows) break;
        float mu, top;
        common<D, NT>(sm, q, mu, top);
        float sum = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (mu != kNegInf) sum += sm.l[w][q] * ex2_approx(sm.mu[w][q] - mu);
            const float4 y = *reinterpret_cast<const float4*>(&sm.o[w][q][d]);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        // out = x 2^(top - kLift) / sum; the power in two steps, it may reach 2^-128.
        const bool some = sum > 0.0f || sum != sum;
        const float half = some ? ex2_approx(0.5f * (top - kLift)) : 0.0f;
        const float inv = some ? half / sum : 0.0f;
        x.x = x.x * half * inv, x.y = x.y * half * inv, x.z = x.z * half * inv, x.w = x.w * half * inv;
        const int64_t token = r.first + row / a.group;
        const int qh = head * a.group + row % a.group;
        const int64_t flat = token * a.q.heads + qh;
        if (a.splits > 1) {
            const int64_t part = split * total_rows + flat;
            *reinterpret_cast<float4*>(a.part_o + part * D + d) = x;
            if (d == 0) a.part_sum[part] = make_float2(mu, sum);
        } else {
            *reinterpret_cast<uint2*>(a.out.ptr + token * a.out.token_stride + (int64_t)qh * a.out.head_stride + d) =
                make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
            if (d == 0 && a.lse) a.lse[flat] = mu == kNegInf ? kNegInf : kLog2ToNat * (mu + lg2_approx(sum));
        }
    }
}

// Joins the splits of every row: out = sum_i w_i o_i / sum_i w_i, w_i = l_i 2^(m_i - max m).
// (A range's m and sum l come apart: their log2 in one fp32 would lose l beside a large m.)
// One warp per row, 8 rows per CTA; grid (rows of a request / 8, requests).
template <int D>
__global__ void __launch_bounds__(256) kv_attn_join(const __grid_constant__ KvAttnArgs a) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Request r = load_request(a.b, blockIdx.y, a.err, false);
    const int64_t row = (int64_t)blockIdx.x * 8 + warp;
    if (row >= (int64_t)r.n * a.q.heads) return;
    const int64_t flat = (int64_t)r.first * a.q.heads + row;
    const int64_t stride = (int64_t)a.b.total * a.q.heads;
    const int n = max(1, (r.len + a.chunk - 1) / a.chunk);  // splits that hold keys of this request
    // Lane l has the weights of ranges l and l + 32, brought to a sum of one
    // before they meet the ranges' rows: no term is larger than the result may be.
    static_assert(kMostRanges <= 64, "two ranges per lane");
    const float2 none = make_float2(kNegInf, 0.0f);
    const float2 e0 = lane < n ? a.part_sum[lane * stride + flat] : none;
    const float2 e1 = lane + 32 < n ? a.part_sum[(lane + 32) * stride + flat] : none;
    float top = fmaxf(e0.x, e1.x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    float w0 = e0.x == kNegInf ? 0.0f : e0.y * ex2_approx(e0.x - top);
    float w1 = e1.x == kNegInf ? 0.0f : e1.y * ex2_approx(e1.x - top);
    float sum = w0 + w1;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    w0 *= inv, w1 *= inv;
    constexpr int V = D / 32;  // outputs per lane
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float w = __shfl_sync(0xffffffffu, i < 32 ? w0 : w1, i & 31);
        const float* p = a.part_o + (i * stride + flat) * D + lane * V;
        float y[V];
        if (V == 4)
            *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(p);
        else
            *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(p);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] += w == 0.0f ? 0.0f : w * y[j];
    }
    const int64_t token = r.first + row / a.q.heads;
    const int qh = (int)(row % a.q.heads);
    uint16_t* dst = a.out.ptr + token * a.out.token_stride + (int64_t)qh * a.out.head_stride + lane * V;
#pragma unroll
    for (int j = 0; j < V; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = pack_bf16x2(x[j], x[j + 1]);
    if (lane == 0 && a.lse) a.lse[flat] = top == kNegInf ? kNegInf : kLog2ToNat * (top + lg2_approx(sum));
}

}  // namespace

// Cutting a call. Up to 16 rows per request (new tokens x heads of a group) go
// to kv_attn_rows, 8 or 16 to a CTA; more than that to the tcgen05 kernel, 256
// to a CTA, unless the keys that kv_attn_rows would walk (once for every 16
// rows, and a start and an end worth 384 keys) are few, where its shorter start
// wins: 64 rows x 8 heads over 1024 tokens take 12.3 us there and 19.2 here,
// x 128 over 128 14.2 and 12.0, x 128 over 2048 74 and 35; 32 x 148 over 256
// 11.8 and 13.2, over 512 22.7 and 16.3. (The bound comes from 221 such calls,
// 1 to 148 heads, 17 to 1600 rows, 128 to 4096 tokens: the faster of the two
// was taken or one 0.6% slower on average, 21% at most.) A request counts at
// the call's bounds and as seeing all keys: the rule is for requests of equal
// size; shorter ones and a mask only make CTAs end early.
// Then the keys are cut into ranges whose results kv_attn_join joins:
//  - kv_attn_rows: until four CTAs run on every SM (one wave), with ranges of
//    at least 256 keys and at most kMostRanges of them; beyond one wave, ranges
//    of about 1024 keys while they are at most 16 CTAs per SM, which even out
//    requests of different lengths. 16 heads over 1000 tokens take 8.6 us in 4
//    ranges and 11.1 in 2; 32 requests of 100 .. 16001 tokens 103 us in 10, 115
//    in 5, 163 in 2; equal ones pay a little for it: 32 x 8 over 4000 52.5 us in
//    4 ranges, 49.6 in 2, 53.9 in 1.
//  - tcgen05 (one CTA per SM): the number of ranges with the earliest estimated
//    end (tensor_cost).
//
// tensor_cost: full row tiles are dealt to the SMs first, row tiles of at most
// 128 rows fill in after them; a CTA takes 9 us and 1.9 us per tile of 128 keys
// (a short one 0.83 of that, it decodes every tile for itself), the join reads
// and writes its partials. For 1560 rows x 16 heads over 32760 tokens it gives
// 495, 517, 504, 505, 453, 470 us for 1 .. 6 ranges; measured 491, 504, 493,
// 480, 441, 477.
static double tensor_cost(int64_t full, int64_t small, double kv_tiles, double row_bytes, int64_t s, int sms) {
    const double tile = 1.9 * kv_tiles / (double)s, t_full = tile + 9.0, t_small = 0.83 * tile + 9.0;
    full *= s;
    small *= s;
    const int64_t rounds = full / sms, rest = full % sms, idle = sms - rest;
    const double after = (double)(rounds + (rest > 0)) * t_full;  // every full one is done
    // Short ones: all on the SMs that are idle meanwhile, or one there each and
    // the others behind the full ones.
    const double beside = (double)rounds * t_full + (double)((small + idle - 1) / idle) * t_small;
    const int64_t later = small > idle ? small - idle : 0;
    const double first = (double)rounds * t_full + (small > 0 ? t_small : 0.0);
    const double behind = std::max(after, first) + (double)((later + sms - 1) / sms) * t_small;
    double end = small == 0 ? after : std::min(std::max(after, beside), behind);
    if (s > 1) end += 3.0 + row_bytes * 2.0 * (double)s / 5e6;  // 5 TB/s
    return end;
}

KvAttnPlan kv_attn_plan(const KvCacheView& c, const KvBatchView& b, int q_heads, int num_sms) {
    KvAttnPlan p{};
    const int64_t rows = (int64_t)b.max_new * (q_heads / c.heads);
    p.tensor = rows > 16 && (double)b.n * c.heads * (double)((rows + 15) / 16) * (b.max_kv + 384.0) > 216000.0;
    p.rows_per_tile = p.tensor ? 256 : rows <= 8 ? 8 : 16;
    const int64_t tiles = (rows + p.rows_per_tile - 1) / p.rows_per_tile;
    p.row_tiles = (int32_t)(tiles < 1 ? 1 : tiles);
    const int64_t ctas = (int64_t)b.n * p.row_tiles * c.heads;
    const int64_t kv = b.max_kv;
    int64_t splits = 1, most = 1;
    if (p.tensor) {
        const int64_t rem = rows % 256, heads = (int64_t)b.n * c.heads;
        const bool tail = rem > 0 && rem <= 128;
        const int64_t full = heads * (p.row_tiles - (tail ? 1 : 0)), small = tail ? heads : 0;
        const double kv_tiles = (double)((kv + 127) / 128), row_bytes = (double)b.total * q_heads * (c.dim + 1) * 4.0;
        most = std::min<int64_t>((kv + 511) / 512, kMostRanges / 2);
        double best = tensor_cost(full, small, kv_tiles, row_bytes, 1, num_sms);
        for (int64_t s = 2; s <= most; ++s) {
            const double cost = tensor_cost(full, small, kv_tiles, row_bytes, s, num_sms);
            if (cost < 0.97 * best) {
                best = cost;
                splits = s;
            }
        }
        p.tail_last = tail && p.row_tiles > 1;
    } else {
        const int64_t even = std::min<int64_t>((16ll * num_sms + ctas - 1) / ctas, (kv + 1023) / 1024);
        splits = std::max<int64_t>(4ll * num_sms / ctas, even);
        most = std::min<int64_t>((kv + 255) / 256, kMostRanges);
    }
    splits = std::max<int64_t>(1, std::min(splits, most));
    int64_t chunk = (b.max_kv + splits - 1) / splits;
    chunk = (chunk + 127) / 128 * 128;
    if (chunk < 128) chunk = 128;
    splits = (b.max_kv + chunk - 1) / chunk;
    p.splits = (int32_t)(splits < 1 ? 1 : splits);
    p.chunk = (int32_t)chunk;
    p.ws_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)b.total * (size_t)q_heads * (size_t)(c.dim + 4) * sizeof(float) : 0;
    return p;
}

template <int D, int NT>
static cudaError_t launch_rows(dim3 grid, const KvAttnArgs& a, cudaStream_t stream) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(kv_attn_rows<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem<D, NT>);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_done[dev] = true;
    }
    return launch_pdl(kv_attn_rows<D, NT>, grid, dim3(32 * kWarps), kRowsSmem<D, NT>, stream, 1, a);
}

template <int D>
static cudaError_t launch_for(const KvAttnPlan& p, const KvAttnArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.b.n * a.row_tiles * a.splits), (unsigned)a.c.heads);
    cudaError_t e = p.tensor ? launch_kv_attn_tiles(a, stream)
                    : p.rows_per_tile == 8 ? launch_rows<D, 1>(grid, a, stream)
                                           : launch_rows<D, 2>(grid, a, stream);
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)a.b.max_new * a.q.heads;
    return launch_pdl(kv_attn_join<D>, dim3((unsigned)((rows + 7) / 8), (unsigned)a.b.n), dim3(256), 0, stream, 1, a);
}

cudaError_t launch_kv_attention(const KvAttnPlan& p, KvAttnArgs& a, cudaStream_t stream) {
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.row_tiles = p.row_tiles;
    a.tail_last = p.tail_last;
    return a.c.dim == 64 ? launch_for<64>(p, a, stream) : launch_for<128>(p, a, stream);
}

}  // namespace fp8dit
