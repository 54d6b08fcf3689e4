// Attention over the E4M3 cache for few query rows, and the join of split
// key ranges.
//
// A request's rows are its new tokens times the query heads that share a kv
// head; one CTA takes a tile of up to 16 rows, one kv head and one range of
// keys, so a cached byte is read once for the whole group of heads. Its four
// warps walk the range in granules of 16 keys (always inside one block: a
// block is 16 tokens or more), each with its own running maximum, sum and
// output, which are joined through shared memory at the end.
//
// Mathematics, per granule and warp (mma.sync m16n8k16, bf16 -> fp32):
//     S^T = K Q^T      A = 16 keys x dim, B = 8 query rows per column tile
//     P^T = 2^(S^T - m)
//     O^T += V^T P^T   A = dim x 16 keys, B = P^T
// Keys and values are the A operands so that 8 rows fill a column tile (the
// 16-row A side would be half empty at a group of 8 or fewer). Both products
// leave the order of their inner index free, which lets a thread use 16-byte
// loads straight from the cache as its fragments: for K the 16 bytes at
// dim 16 tig (+ 64) of keys gid and gid + 8, with Q permuted the same way;
// for V the 16 bytes at dim 16 gid of keys 2 tig, 2 tig + 1, 2 tig + 8,
// 2 tig + 9, whose bytes are paired across keys by the permute that decodes
// them. P^T comes out of S^T by an 8 x 8 transpose in registers (movmatrix).
// Decoded codes are multiplied by 2^120 S, which is exact: the products are
// those of q and of what the cache holds.
//
// The maximum is lazy: rows keep a reference m that only moves when a score
// exceeds it by 8 (in log2 units), so the usual granule needs one vote and no
// shuffles; p is at most 2^8.
//
// Bound: HBM, 2 bytes per token, kv head and dim; a granule's loads are issued
// one granule ahead (4 KB in flight per warp at dim 128).
#include "attention.cuh"
#include "fp8_codec.cuh"

namespace fp8dit {
namespace {

constexpr int kWarps = 4;
constexpr int kGranule = 16;
constexpr float kLazy = 8.0f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// One granule's codes and scales as this lane needs them.
template <int D>
struct Granule {
    uint32_t k[2][D / 16];  // keys gid, gid + 8: D / 16 words of 4 codes
    uint32_t v[4][D / 32];  // keys 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9: D / 32 words
    float ks, vs;
    bool ok;  // its block index is valid
};

template <int D>
__device__ __forceinline__ void load_granule(Granule<D>& g, const KvAttnArgs& a, int page, int head, int row, int gid,
                                             int tig) {
    g.ok = page >= 0 && page < a.c.n_blocks;
    if (!g.ok) {
        if ((threadIdx.x & 31) == 0) atomicOr(a.err.word, kDevErrIndex);
        page = 0;
    }
    const int64_t slot = (int64_t)page * a.c.heads + head;
    const int64_t at = ((slot << a.c.block_log2) + row) * D;
    g.ks = a.c.ks[slot];
    g.vs = a.c.vs[slot];
    const uint8_t* kp = a.c.k + at + tig * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            const uint4 w = *reinterpret_cast<const uint4*>(kp + (gid + 8 * r) * D + 64 * h);
            g.k[r][4 * h] = w.x, g.k[r][4 * h + 1] = w.y, g.k[r][4 * h + 2] = w.z, g.k[r][4 * h + 3] = w.w;
        }
    const uint8_t* vp = a.c.v + at + gid * (D / 8);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint8_t* p = vp + (2 * tig + (r & 1) + 8 * (r >> 1)) * D;
        if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            g.v[r][0] = w.x, g.v[r][1] = w.y, g.v[r][D / 32 - 2] = w.z, g.v[r][D / 32 - 1] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            g.v[r][0] = w.x, g.v[r][1] = w.y;
        }
    }
}

template <int D, int NT>
struct RowsSmem {
    float m[kWarps][8 * NT], l[kWarps][8 * NT];
    float o[kWarps][8 * NT][D + 4];
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps) kv_attn_rows(const __grid_constant__ KvAttnArgs a) {
    __shared__ RowsSmem<D, NT> sm;
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
    if (a.splits > 1 && k0 >= r.len && split > 0) return;  // not read by the join either

    uint32_t qf[NT][D / 16][2];
    int limit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = r0 + nt * 8 + gid;
        const bool in = row < rows;
        const uint16_t* qp = a.q.ptr;
        if (in)
            qp += (int64_t)(r.first + row / a.group) * a.q.token_stride +
                  (int64_t)(head * a.group + row % a.group) * a.q.head_stride + tig * 16;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            uint2 w = make_uint2(0, 0);
            if (in) w = *reinterpret_cast<const uint2*>(qp + (s >> 2) * 64 + (s & 3) * 4);
            qf[nt][s][0] = w.x;
            qf[nt][s][1] = w.y;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int lr = r0 + nt * 8 + 2 * tig + i;
            limit[nt][i] = lr < rows ? key_limit(r.len - r.n + lr / a.group, r.len, a.frame) : 0;
        }
    }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = kNegInf;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
    }

    const int32_t* table = a.b.table + (int64_t)b * a.b.width;
    const int bmask = (1 << a.c.block_log2) - 1;
    constexpr int kStep = kWarps * kGranule;
    int key = k0 + warp * kGranule;
    Granule<D> next;
    int page = key < k1 ? table[key >> a.c.block_log2] : 0;
    if (key < k1) load_granule<D>(next, a, page, head, key & bmask, gid, tig);
    page = key + kStep < k1 ? table[(key + kStep) >> a.c.block_log2] : 0;
    for (; key < k1; key += kStep) {
        const Granule<D> g = next;
        if (key + kStep < k1) load_granule<D>(next, a, page, head, (key + kStep) & bmask, gid, tig);
        if (key + 2 * kStep < k1) page = table[(key + 2 * kStep) >> a.c.block_log2];
        if (!g.ok) continue;

        const CodeScale ck = code_scale(g.ks);
        const bool big_k = ck.rest != kBf16One2;
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint32_t x = g.k[0][i], y = g.k[1][i];
            uint32_t a0 = mul_bf16x2(spread_codes(x, x, spread_sel(0, 1)), ck.m);
            uint32_t a1 = mul_bf16x2(spread_codes(y, y, spread_sel(0, 1)), ck.m);
            uint32_t a2 = mul_bf16x2(spread_codes(x, x, spread_sel(2, 3)), ck.m);
            uint32_t a3 = mul_bf16x2(spread_codes(y, y, spread_sel(2, 3)), ck.m);
            if (big_k) {
                a0 = mul_bf16x2(a0, ck.rest), a1 = mul_bf16x2(a1, ck.rest);
                a2 = mul_bf16x2(a2, ck.rest), a3 = mul_bf16x2(a3, ck.rest);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(s[nt], a0, a1, a2, a3, qf[nt][i][0], qf[nt][i][1]);
        }
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nt][i] *= a.scale_log2;
                if (key + kGranule > least && key + gid + 8 * (i >> 1) >= limit[nt][i & 1]) s[nt][i] = kNegInf;
                over |= s[nt][i] > m[nt][i & 1] + kLazy;
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
                    const float to = fmaxf(m[nt][i], t);
                    const float c = to == kNegInf ? 1.0f : ex2_approx(m[nt][i] - to);
                    m[nt][i] = to;
                    l[nt][i] *= c;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        o[nt][d][i] *= c;
                        o[nt][d][i + 2] *= c;
                    }
                }
        }
        uint32_t p[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ref = m[nt][i & 1] == kNegInf ? 0.0f : m[nt][i & 1];
                s[nt][i] = ex2_approx(s[nt][i] - ref);
                l[nt][i & 1] += s[nt][i];
            }
            p[nt][0] = transpose_8x8(pack2(s[nt][0], s[nt][1]));
            p[nt][1] = transpose_8x8(pack2(s[nt][2], s[nt][3]));
        }
        const CodeScale cs = code_scale(g.vs);
        const bool big = cs.rest != kBf16One2;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t e0 = spread_sel(2 * half, 2 * half + 4), e1 = spread_sel(2 * half + 1, 2 * half + 5);
                uint32_t a0 = mul_bf16x2(spread_codes(g.v[0][w], g.v[1][w], e0), cs.m);
                uint32_t a1 = mul_bf16x2(spread_codes(g.v[0][w], g.v[1][w], e1), cs.m);
                uint32_t a2 = mul_bf16x2(spread_codes(g.v[2][w], g.v[3][w], e0), cs.m);
                uint32_t a3 = mul_bf16x2(spread_codes(g.v[2][w], g.v[3][w], e1), cs.m);
                if (big) {
                    a0 = mul_bf16x2(a0, cs.rest), a1 = mul_bf16x2(a1, cs.rest);
                    a2 = mul_bf16x2(a2, cs.rest), a3 = mul_bf16x2(a3, cs.rest);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][2 * w + half], a0, a1, a2, a3, p[nt][0], p[nt][1]);
            }
    }

    // Join the warps: per row the common reference, then the scaled sums.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
            l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
            if (gid == 0) {
                sm.m[warp][nt * 8 + 2 * tig + i] = m[nt][i];
                sm.l[warp][nt * 8 + 2 * tig + i] = l[nt][i];
            }
        }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = nt * 8 + 2 * tig + i;
            float top = sm.m[0][q];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.m[w][q]);
            const float c = top == kNegInf ? 0.0f : ex2_approx(m[nt][i] - top);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                // Row gid of column tile d is dim gid (D / 8) + 2 d, row gid + 8 the next one.
                float2 x = make_float2(o[nt][d][i] * c, o[nt][d][i + 2] * c);
                *reinterpret_cast<float2*>(&sm.o[warp][q][gid * (D / 8) + 2 * d]) = x;
            }
        }
    __syncthreads();
    const int64_t total_rows = (int64_t)a.b.total * a.q.heads;
    for (int at = threadIdx.x; at < 8 * NT * (D / 4); at += 32 * kWarps) {
        const int q = at / (D / 4), d = (at % (D / 4)) * 4;
        const int row = r0 + q;
        if (row >= rows) break;
        float top = sm.m[0][q];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.m[w][q]);
        float sum = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (top != kNegInf) sum += sm.l[w][q] * ex2_approx(sm.m[w][q] - top);
            const float4 y = *reinterpret_cast<const float4*>(&sm.o[w][q][d]);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        const int64_t token = r.first + row / a.group;
        const int qh = head * a.group + row % a.group;
        const int64_t flat = token * a.q.heads + qh;
        if (a.splits > 1) {
            const int64_t part = split * total_rows + flat;
            *reinterpret_cast<float4*>(a.part_o + part * D + d) = x;
            if (d == 0) a.part_lse[part] = top == kNegInf ? kNegInf : top + lg2_approx(sum);
        } else {
            *reinterpret_cast<uint2*>(a.out.ptr + token * a.out.token_stride + (int64_t)qh * a.out.head_stride + d) =
                make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
            if (d == 0 && a.lse) a.lse[flat] = top == kNegInf ? kNegInf : 0.6931471805599453f * (top + lg2_approx(sum));
        }
    }
}

// Joins the splits of every row: out = sum_i 2^(lse_i - m) o_i / sum_i 2^(lse_i - m).
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
    float top = kNegInf;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, a.part_lse[i * stride + flat]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    constexpr int V = D / 32;  // outputs per lane
    float x[V], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float lse = a.part_lse[i * stride + flat];
        if (lse == kNegInf) continue;
        const float w = ex2_approx(lse - top);
        sum += w;
        const float* p = a.part_o + (i * stride + flat) * D + lane * V;
        float y[V];
        if (V == 4)
            *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(p);
        else
            *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(p);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] += w * y[j];
    }
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int64_t token = r.first + row / a.q.heads;
    const int qh = (int)(row % a.q.heads);
    uint16_t* dst = a.out.ptr + token * a.out.token_stride + (int64_t)qh * a.out.head_stride + lane * V;
#pragma unroll
    for (int j = 0; j < V; j += 2) *reinterpret_cast<uint32_t*>(dst + j) = pack2(x[j] * inv, x[j + 1] * inv);
    if (lane == 0 && a.lse) a.lse[flat] = top == kNegInf ? kNegInf : 0.6931471805599453f * (top + lg2_approx(sum));
}

}  // namespace

// Cutting a call: up to 16 rows per request go to kv_attn_rows (8 or 16 rows
// per CTA), more to the tcgen05 kernel (256). Then, while the CTAs would not
// fill the GPU (four per SM, or one), the keys are cut into ranges of at least
// 256 (512).
KvAttnPlan kv_attn_plan(const KvCacheView& c, const KvBatchView& b, int q_heads, int num_sms) {
    KvAttnPlan p{};
    const int64_t rows = (int64_t)b.max_new * (q_heads / c.heads);
    p.tensor = rows > 16;
    p.rows_per_tile = rows <= 8 ? 8 : rows <= 16 ? 16 : 256;
    const int64_t tiles = (rows + p.rows_per_tile - 1) / p.rows_per_tile;
    p.row_tiles = (int32_t)(tiles < 1 ? 1 : tiles);
    const int64_t ctas = (int64_t)b.n * p.row_tiles * c.heads;
    const int64_t fill = p.tensor ? num_sms : 4ll * num_sms;
    const int64_t least = p.tensor ? 512 : 256;
    int64_t splits = fill / ctas;
    const int64_t most = (b.max_kv + least - 1) / least;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    int64_t chunk = (b.max_kv + splits - 1) / splits;
    chunk = (chunk + 127) / 128 * 128;
    if (chunk < 128) chunk = 128;
    splits = (b.max_kv + chunk - 1) / chunk;
    p.splits = (int32_t)(splits < 1 ? 1 : splits);
    p.chunk = (int32_t)chunk;
    p.ws_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)b.total * (size_t)q_heads * (size_t)(c.dim + 4) * sizeof(float) : 0;
    return p;
}

template <int D>
static cudaError_t launch_for(const KvAttnPlan& p, const KvAttnArgs& a, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.b.n * a.row_tiles * a.splits), (unsigned)a.c.heads);
    cudaError_t e = p.tensor ? launch_kv_attn_tiles(a, stream)
                    : p.rows_per_tile == 8
                        ? launch_pdl(kv_attn_rows<D, 1>, grid, dim3(32 * kWarps), 0, stream, 1, a)
                        : launch_pdl(kv_attn_rows<D, 2>, grid, dim3(32 * kWarps), 0, stream, 1, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t rows = (int64_t)a.b.max_new * a.q.heads;
    return launch_pdl(kv_attn_join<D>, dim3((unsigned)((rows + 7) / 8), (unsigned)a.b.n), dim3(256), 0, stream, 1, a);
}

cudaError_t launch_kv_attention(const KvAttnPlan& p, KvAttnArgs& a, cudaStream_t stream) {
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.row_tiles = p.row_tiles;
    return a.c.dim == 64 ? launch_for<64>(p, a, stream) : launch_for<128>(p, a, stream);
}

}  // namespace fp8dit
