/*
 * fp8dit — FP8 linear layer of a diffusion / video DiT on B200 (sm_100a).
 *
 * The path (from "从 BF16 到 FP8：HunyuanVideo1.5推理优化复盘", section 三.1):
 *
 *     BF16 activation -> dynamic per-token FP8 quant -> FP8 GEMM
 *                     -> scale / bias / output dtype
 *
 * with weights quantised per output channel ahead of time (section 二),
 * one quantised activation shared by the Q, K and V projections (section
 * 三.4), an entry that takes an already-quantised (fp8, scale) activation
 * (sections 三.3 and 三.5), and the backend / tile choice bound once when a
 * layer is created (section 三.3). The companion step converts whole weight
 * tensors to float8_e4m3fn or float8_e5m2 with one scale each ("Quantize
 * Model to FP8 Format", inputs model_state_dict and fp8_format).
 *
 * Quantisation recipe ("ComfyUI自定义节点开发适配Stable Diffusion 3.5 FP8技术要点",
 * section "FP8：不只是精度减半", steps 1-4), read for FP8:
 *     amax = max |x|                      (over a row, a channel or a tensor)
 *     S    = fp32(amax) / fmax            IEEE fp32 division; S = 1 if amax == 0
 *     q    = RNEsat(fp32(x) / S)          IEEE fp32 division, then round to the
 *                                         nearest FP8 code (ties to even
 *                                         mantissa), |.| > fmax clamps to fmax
 *     x   ~= decode(q) * S                (the stored scale is S)
 * fmax = 448 for E4M3FN, 57344 for E5M2.
 *
 * Conventions for every entry point
 *  - bf16 tensors are passed as uint16_t bit patterns, FP8 tensors as uint8_t
 *    codes (OCP E4M3FN / E5M2), scales as fp32. All tensors are row-major;
 *    "K-major" means the reduction index is the contiguous one.
 *  - Every tensor pointer is a DEVICE pointer on the current device unless a
 *    parameter says "host". The caller owns all memory: inputs, outputs,
 *    scratch and workspace. The library owns only linear handles.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and enqueue work only after every argument has been validated.
 *    An argument error returns a status and enqueues nothing. There is no
 *    fallback path: a shape the kernels cannot take is an error.
 *  - Device-side bounded waits that expire, and lengths, offsets and block
 *    indices in device memory that lie outside their range, set a per-device
 *    error word; fp8dit_device_error() reads and clears it.
 *  - On any status other than FP8DIT_OK, fp8dit_last_error_string() (per
 *    thread) describes the failure.
 *  - CUDA graphs: the quantisers, the linear entry points (single, multi,
 *    weight-only, fused, stream-K), the per-tensor conversion, the rotary
 *    positions and the key / value cache's append and attention only enqueue
 *    kernels (and, per-tensor, a memset), so they can be captured into a
 *    graph and replayed; each replay reads whatever the captured buffers hold
 *    then. Make the first fp8_act_quantize_rowwise call on a device (it builds
 *    its activation tables and synchronises once) and the first
 *    fp8_scaled_linear_noalloc call on a device before capturing.
 *    fp8_scaled_linear_host uses its own copy streams and is not meant for
 *    capture.
 */
#ifndef FP8DIT_H
#define FP8DIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8DIT_OK = 0,
    FP8DIT_ERR_INVALID_ARG = 1,       /* null / misaligned pointer, negative size, bad format */
    FP8DIT_ERR_UNSUPPORTED_SHAPE = 2, /* K % 16 != 0, N % 8 != 0, size beyond the kernels' range */
    FP8DIT_ERR_EMPTY = 3,             /* per-tensor conversion with nothing to convert */
    FP8DIT_ERR_CUDA = 4,              /* a CUDA runtime / driver call failed */
    FP8DIT_ERR_TIMEOUT = 5,           /* a bounded device wait expired */
    FP8DIT_ERR_INDEX = 6              /* a kernel met a length, offset or block index outside its range */
} fp8dit_status;

typedef enum { FP8DIT_E4M3FN = 0, FP8DIT_E5M2 = 1 } fp8dit_format;

/* Same type as cudaStream_t; the header does not need the CUDA headers. */
typedef struct CUstream_st* fp8dit_stream_t;

/* Opaque handle of one FP8 linear layer (see fp8_linear_create). */
typedef struct fp8dit_linear_s* fp8dit_linear;

/*
 * Per-token (rowwise) quantisation of a bf16 activation.
 * ("从 BF16 到 FP8", section 三.1: dynamic per-token FP8 quant; recipe above.)
 *   x     [M, K] bf16, row stride ldx elements (ldx >= K, ldx % 8 == 0), 16-byte aligned.
 *   q     [M, K] FP8 codes of format fmt, row stride ldq bytes (ldq >= K, ldq % 16 == 0),
 *         16-byte aligned.
 *   scale [M] fp32: S of each row.
 * Requires K % 16 == 0 and K > 0, M >= 0 (M == 0 is a no-op). Any K that is a
 * multiple of 16 is accepted. Inputs must be finite.
 */
fp8dit_status fp8_quantize_rowwise(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                   fp8dit_format fmt, uint8_t* q, int64_t ldq, float* scale,
                                   fp8dit_stream_t stream);

/* Activations a producer kernel can apply before quantising. */
typedef enum {
    FP8DIT_ACT_GELU_ERF = 1,  /* x Phi(x) = x/2 (1 + erf(x / sqrt 2)) */
    FP8DIT_ACT_GELU_TANH = 2, /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
    FP8DIT_ACT_SILU = 3       /* x / (1 + exp(-x)) */
} fp8dit_activation;

/*
 * Producer fusion ("从 BF16 到 FP8", section 三.5): the GELU / SiLU in front of
 * FFN-down emits the (FP8 tensor, per-token scale) pair directly instead of a
 * bf16 tensor that a separate pass then quantises.
 *   h     [M, K] bf16 (the FFN-up output), row stride ldh elements (ldh % 8 == 0), 16-byte aligned.
 *   g     = bf16_rne(act(h)): act evaluated in double (CUDA's double erfc / exp,
 *         every other step an IEEE double operation) and rounded once to bf16,
 *         ties to even; stored to gout [M, K] (row stride ldg, 16-byte aligned)
 *         when gout != NULL.
 *   q, scale: the rowwise recipe applied to g, E4M3FN codes (the GEMM's input).
 * Same shape rules as fp8_quantize_rowwise. The first call on a device builds
 * a 128 KB table per activation (bf16(act(x)) for all 65536 bf16 x, in static
 * device memory) and synchronises `stream` once; make that first call before
 * any stream capture.
 */
fp8dit_status fp8_act_quantize_rowwise(const uint16_t* h, int64_t M, int64_t K, int64_t ldh,
                                       fp8dit_activation act, uint8_t* q, int64_t ldq, float* scale,
                                       uint16_t* gout, int64_t ldg, fp8dit_stream_t stream);

/*
 * Per-output-channel quantisation of a bf16 weight W [N, K] (K contiguous):
 * the rowwise recipe applied to each of the N rows, producing the K-major
 * FP8 weight the GEMM consumes with no transpose ("从 BF16 到 FP8", section
 * 二: parameters quantised per channel ahead of time; section 三.1: B must
 * stay column-major, never transposed and made contiguous).
 *   w [N, K] bf16 contiguous; qw [N, K] codes contiguous; sw [N] fp32.
 * Requires N > 0, K > 0, K % 16 == 0.
 */
fp8dit_status fp8_quantize_weight_per_channel(const uint16_t* w, int64_t N, int64_t K,
                                              fp8dit_format fmt, uint8_t* qw, float* sw,
                                              fp8dit_stream_t stream);

/* Element types a per-tensor conversion reads (a state-dict's floating dtypes). */
typedef enum {
    FP8DIT_SRC_BF16 = 0, /* bfloat16 bit patterns (the default: a zeroed field) */
    FP8DIT_SRC_F16 = 1,  /* IEEE binary16 bit patterns */
    FP8DIT_SRC_F32 = 2   /* IEEE binary32 */
} fp8dit_src_dtype;

/* One tensor of a per-tensor conversion. Pointers are device pointers. */
typedef struct {
    const void* src;   /* numel values of src_dtype, contiguous, 16-byte aligned */
    int64_t numel;     /* >= 0, any size */
    uint8_t* dst;      /* numel FP8 codes, 16-byte aligned */
    float* scale;      /* one fp32: S of the tensor (left untouched when numel == 0) */
    int32_t src_dtype; /* fp8dit_src_dtype of src */
    int32_t reserved;  /* must be 0 */
} fp8dit_tensor_desc;

/* Bytes of device workspace fp8_quantize_weight_per_tensor needs for n tensors. */
size_t fp8_quantize_weight_per_tensor_workspace_size(int32_t n_tensors);

/*
 * Per-tensor conversion of a weight set (a state-dict's tensors) to FP8 with
 * one amax scale per tensor ("Quantize Model to FP8 Format": model_state_dict
 * in, quantised state-dict out in float8_e4m3fn or float8_e5m2). Each tensor
 * may be bf16, fp16 or fp32 (its src_dtype); every value is exact in fp32, so
 * the recipe above applies unchanged: amax = max |x|, S = amax / fmax and
 * q = RNEsat(x / S), both IEEE fp32 divisions.
 *   tensors   HOST array of n_tensors descriptors; it may be freed on return.
 *   workspace DEVICE scratch of at least
 *             fp8_quantize_weight_per_tensor_workspace_size(n_tensors) bytes,
 *             16-byte aligned; its contents on entry do not matter. It must not
 *             be used by another call that runs at the same time on the GPU.
 * Errors: FP8DIT_ERR_EMPTY when n_tensors == 0 or every numel is 0 (the page's
 * "Invalid input." and "No tensor converted to <fp8_format>." outcomes).
 */
fp8dit_status fp8_quantize_weight_per_tensor(const fp8dit_tensor_desc* tensors, int32_t n_tensors,
                                             fp8dit_format fmt, void* workspace, size_t ws_bytes,
                                             fp8dit_stream_t stream);

/*
 * Create an FP8 linear layer y = (A W^T) * sa * sw + bias with E4M3FN
 * operands, fp32 accumulation and bf16 output. The tile plan for every
 * M-bucket and the weight's TMA descriptors are built here, once
 * ("从 BF16 到 FP8", section 三.3: backend chosen from weight shape, device
 * and bias contract at construction, forward does no such checks).
 *   qw   [N, K] E4M3FN codes, K contiguous (from fp8_quantize_weight_per_channel).
 *   sw   [N] fp32 per-channel scales.
 *   bias [N] bf16, or NULL for no bias.
 * The handle BORROWS qw, sw and bias: they must stay valid and unchanged
 * until fp8_linear_destroy. device is the CUDA device that holds them.
 * Requires N % 8 == 0, K % 16 == 0; qw, sw and bias 16-byte aligned.
 */
fp8dit_status fp8_linear_create(int64_t N, int64_t K, const uint8_t* qw, const float* sw,
                                const uint16_t* bias, int device, fp8dit_linear* out);

fp8dit_status fp8_linear_destroy(fp8dit_linear h);

/*
 * Optional stream-K workspace for a layer. When a layer's 256 x 256 output
 * tiles would keep the CTA pairs busy for less than 3/4 of the waves of a
 * tile-per-pair schedule (a nearly empty last wave: e.g. 150 tiles on 74
 * pairs) and a tile has at least 8 k-blocks of 128, each pair instead takes
 * an equal share of the layer's k-blocks; a tile split between two pairs is
 * finished by whichever of the two gets there second, from the fp32 partial
 * the other has stored in this workspace; neither waits for the other, so the
 * launch does not need all of its pairs resident at once. Results stay
 * deterministic (the two parts are added once, in fp32, whichever side
 * finishes) but differ in rounding from the plain schedule.
 * The same workspace enables split-K for few tiles and a long K: when the
 * 128 x 128 tiles of a small-M call fill at most half of the SMs and K has at
 * least 48 k-blocks of 128 (K >= 6144; e.g. text tokens through an FFN-down
 * weight), each tile is cut into up to 8 pieces of at least 6 k-blocks on
 * separate CTAs; every piece stores its fp32 partial and the piece that
 * arrives last adds all of them in piece order for the whole tile
 * (deterministic, rounding differs from the plain schedule). No piece waits
 * for another, so split-K launches need not have all their CTAs resident at
 * once and may share the GPU with other kernels.
 * fp8_weight_only_linear splits the same way from 32 k-blocks of 64 (K >=
 * 2048; K >= 4096 above 64 rows). fp8_scaled_linear_multi uses the workspace
 * of its first layer. Without a workspace, or for other shapes (the
 * FFN shapes among them), the plain schedule is used.
 *   fp8_linear_workspace_size: bytes needed on the layer's device (~38 MB on
 *     148 SMs), the same for every M.
 *   fp8_linear_set_workspace: attach caller-owned DEVICE memory (256-byte
 *     aligned, at least that size) or detach with NULL, while no call that
 *     uses the layer is in flight. Attaching clears the workspace's flags
 *     and counters (synchronously); every launch leaves them cleared, so
 *     stream-ordered launches and replays of a captured CUDA graph need no
 *     host reset. After a call whose device error word reports
 *     FP8DIT_ERR_TIMEOUT, attach the workspace again before reusing it (an
 *     interrupted launch can leave a flag or a count behind). The
 *     workspace may be attached to several layers whose calls run one after
 *     another on the GPU; calls that overlap on the GPU must not share a
 *     workspace.
 */
size_t fp8_linear_workspace_size(fp8dit_linear h);
fp8dit_status fp8_linear_set_workspace(fp8dit_linear h, void* workspace, size_t bytes);
/* Bytes at the start of the workspace that hold its flags and counters: zero
 * after attaching and between launches (the rest holds fp32 partials). */
size_t fp8_linear_workspace_flag_bytes(fp8dit_linear h);

/*
 * Forward of one FP8 linear layer ("从 BF16 到 FP8", sections 三.1, 三.3, 三.5):
 *  - ordinary tensor: a_bf16 != NULL. A [M, K] bf16 (contiguous) is quantised
 *    per token into qa_scratch [M, K] and sa_scratch [M] (both caller-owned,
 *    written by this call), then multiplied. qa and sa must be NULL.
 *  - FP8 tensor: a_bf16 == NULL. qa [M, K] E4M3FN codes (contiguous) and
 *    sa [M] fp32 per-token scales are used as given; the scratch arguments
 *    are ignored.
 *   y [M, N] bf16 contiguous, 16-byte aligned:
 *     y[m, n] = bf16_rne((sum_k dec(qa[m,k]) dec(qw[n,k])) * sa[m] * sw[n] + bias[n])
 * M == 0 is a no-op. Must run on the handle's device.
 */
fp8dit_status fp8_scaled_linear(fp8dit_linear h, int64_t M, const uint16_t* a_bf16,
                                const uint8_t* qa, const float* sa, uint8_t* qa_scratch,
                                float* sa_scratch, uint16_t* y, fp8dit_stream_t stream);

/*
 * FP8 weight-only linear: the FP8 weight-only configuration with scales that
 * the longcat-avatar-compare page sets against NVFP4 W4A4 (section 速度总览). The
 * activation is not quantised; the layer's E4M3 weight is decoded to bf16 in
 * shared memory and multiplied on the BF16 tensor cores:
 *   y[m, n] = bf16_rne( (sum_k A[m,k] dec(qw[n,k])) * sw[n] + bias[n] ), fp32 accumulation.
 *   a_bf16 [M, K] bf16 contiguous, y [M, N] bf16 contiguous, both 16-byte aligned.
 * Uses the same handle (qw, sw, bias) as fp8_scaled_linear.
 */
fp8dit_status fp8_weight_only_linear(fp8dit_linear h, int64_t M, const uint16_t* a_bf16, uint16_t* y,
                                     fp8dit_stream_t stream);

/*
 * The FP8 linear from a bf16 activation in ONE launch (the fused variant of
 * "从 BF16 到 FP8", section 三.1: runtime per-token activation quantisation
 * feeding the FP8 GEMM; section 三.2 item 2: fewer extra reads and writes and
 * intermediate launches). The launch's CTAs first quantise A together: each
 * claims chunks of rows in row order, stages their bf16 values in shared
 * memory with bulk copies, and writes each row's E4M3 codes and scale with
 * the rowwise quantiser's arithmetic; every element is quantised exactly once.
 * Each CTA then runs the FP8 GEMM + epilogue of fp8_scaled_linear, a tile
 * starting as soon as its rows have been quantised. A chunk is only ever
 * claimed by a running CTA and that work waits for nothing, so no wait
 * depends on CTAs that have not started.
 * Result: qa_scratch and sa_scratch hold exactly what fp8_quantize_rowwise
 * writes, and y equals fp8_scaled_linear(h, M, a_bf16, ...) bit for bit where
 * both use 256 x 256 pair tiles (otherwise within the accumulation-order
 * difference of another tile plan).
 *   a_bf16     [M, K] bf16 contiguous, 16-byte aligned;
 *   qa_scratch [M, K] E4M3FN codes, 16-byte aligned, caller-owned: written;
 *   sa_scratch [M] fp32 per-token scales, 4-byte aligned, caller-owned: written;
 *   y          [M, N] bf16 contiguous, 16-byte aligned.
 * The layer must have a workspace attached (fp8_linear_set_workspace): its
 * counters, which every launch leaves at zero; calls that overlap on the GPU
 * must not share it. Requires K <= 8192 and M <= 1048576
 * (FP8DIT_ERR_UNSUPPORTED_SHAPE otherwise). M == 0 is a no-op. Must run on
 * the handle's device.
 */
fp8dit_status fp8_scaled_linear_fused(fp8dit_linear h, int64_t M, const uint16_t* a_bf16, uint8_t* qa_scratch,
                                      float* sa_scratch, uint16_t* y, fp8dit_stream_t stream);

/*
 * FP8 linear from HOST buffers, with the transfers pipelined around the
 * kernels (the library's runtime for callers whose activations live in host
 * memory; the pages have no counterpart). The result is fp8_scaled_linear's
 * from a bf16 activation, row for row (each row depends only on its own
 * activation row), computed chunk by chunk.
 *
 * fp8_linear_host_workspace_size: DEVICE bytes for `slots` slots of
 *   `chunk_rows` rows (per slot: bf16 activation, FP8 codes, scales, bf16
 *   output); 0 for invalid arguments (slots must be 2..8, chunk_rows > 0).
 * fp8_linear_set_host_pipeline: attach caller-owned DEVICE memory (256-byte
 *   aligned, at least that size) to the layer, creating two copy streams and
 *   the slot events on the layer's device; NULL workspace detaches (and frees
 *   the streams and events). Replacing or detaching a pipeline, and
 *   fp8_linear_destroy, first wait on the host for that pipeline's work in
 *   flight. The workspace belongs to this layer only and must stay allocated
 *   until the work of every call using it has completed.
 * fp8_scaled_linear_host: y_host [M, N] = the linear of a_host [M, K] (both
 *   bf16, contiguous, HOST memory; page-locked memory is needed for the
 *   copies to overlap anything). The M rows go in chunks: host-to-device copy
 *   (copy-in stream) -> quantise + GEMM (`stream`) -> device-to-host copy
 *   (copy-out stream), chunks and slots in a ring, so both copy directions and
 *   the kernels overlap, also with the previous call's copy-out.
 *   Ordering: `stream` passes the end of this call only once every output row
 *   is in y_host, so synchronising `stream` (or work queued on it later) sees
 *   the result. The input copies are ordered only after earlier calls' use of
 *   the same slots, NOT after other work queued on `stream`: a_host must hold
 *   the activation when the call is made and stay unchanged, and both host
 *   buffers stay allocated, until `stream` has passed this call. Calls on one
 *   handle are serialised by a lock. Errors as fp8_scaled_linear, plus
 *   FP8DIT_ERR_INVALID_ARG when no pipeline is attached.
 */
size_t fp8_linear_host_workspace_size(fp8dit_linear h, int64_t chunk_rows, int32_t slots);
fp8dit_status fp8_linear_set_host_pipeline(fp8dit_linear h, void* workspace, size_t bytes, int64_t chunk_rows,
                                           int32_t slots);
fp8dit_status fp8_scaled_linear_host(fp8dit_linear h, int64_t M, const uint16_t* a_host, uint16_t* y_host,
                                     fp8dit_stream_t stream);

/*
 * fp8_scaled_linear from a bf16 activation, for callers that cannot allocate
 * device memory. The pages have no counterpart: this entry exists for code
 * that has no way to hand the library qa / sa scratch, such as a plugin whose
 * host framework owns the device allocator, or code that must not call
 * cudaMalloc / cudaFree because they can synchronise the device and can fail
 * for lack of memory mid-step. The quantised activation is kept in a fixed
 * array that is part of the library's device image instead, so this call
 * allocates nothing.
 *   a_bf16 [M, K] bf16 contiguous, y [M, N] bf16 contiguous, both 16-byte
 *   aligned; results equal fp8_scaled_linear(h, M, a_bf16, NULL, NULL, ...).
 * Limits: M <= FP8DIT_NOALLOC_MAX_ROWS and M * K <= FP8DIT_NOALLOC_MAX_ACT_BYTES;
 * larger calls return FP8DIT_ERR_UNSUPPORTED_SHAPE and enqueue nothing.
 * Every GPU that loads the library holds the array (about 8.25 MiB) until the
 * process exits. All calls on a device share it and leave their data in it;
 * each call rewrites everything it reads, but calls whose work overlaps on the
 * GPU (e.g. on two streams) race. The first call on a device looks up the
 * array's device address; make that call before any stream capture.
 */
#define FP8DIT_NOALLOC_MAX_ACT_BYTES (8u << 20)
#define FP8DIT_NOALLOC_MAX_ROWS 65536
fp8dit_status fp8_scaled_linear_noalloc(fp8dit_linear h, int64_t M, const uint16_t* a_bf16, uint16_t* y,
                                        fp8dit_stream_t stream);

/*
 * n linear layers that read the same activation ("从 BF16 到 FP8", section
 * 三.4: quantise hidden_states once and feed the separate Q, K and V
 * projections). A [M, K] bf16 is quantised once into qa_scratch / sa_scratch,
 * then all n products run in one grouped launch.
 *   hs  HOST array of n handles (1 <= n <= 4), all with the same K and device.
 *   ys  HOST array of n device pointers, ys[i] is [M, N_i] bf16.
 * Results are bitwise identical to n fp8_scaled_linear calls whenever the
 * grouped launch and the single calls use the same tile plan and no split
 * (e.g. the 256 x 256 pair plan of the hidden_states projections); a split
 * schedule (workspace attached) may cut the grouped launch's K differently
 * from a single call's and round differently, within the same bound.
 */
fp8dit_status fp8_scaled_linear_multi(const fp8dit_linear* hs, int32_t n, int64_t M,
                                      const uint16_t* a_bf16, uint8_t* qa_scratch,
                                      float* sa_scratch, uint16_t* const* ys,
                                      fp8dit_stream_t stream);

/*
 * Tile plan that fp8_scaled_linear / _multi use for this handle at this M
 * (n_problems = 1 for a single layer): block_m x block_n output tiles,
 * `ctas` thread blocks. For reports and tests.
 */
fp8dit_status fp8_linear_plan(fp8dit_linear h, int64_t M, int32_t n_problems, int32_t* block_m,
                              int32_t* block_n, int32_t* ctas);

/* ------------------------------------------------------------ attention
 * What follows the Q, K and V projections ("从 BF16 到 FP8", section 三.4)
 * in a block: positions turned into q and k, k and v put into an 8-bit cache,
 * and attention over that cache. The pages describe the projections only;
 * these operators are defined here.
 */

#define FP8DIT_ROTARY_MAX_AXES 4
#define FP8DIT_ROTARY_MAX_DIM 256

typedef enum { FP8DIT_POS_I32 = 0, FP8DIT_POS_F32 = 1 } fp8dit_pos_dtype;

/* One bf16 tensor [tokens, heads, dim] seen through its strides (in elements;
 * the dim elements of a head are contiguous). Strides are multiples of 8 and
 * at least dim, the pointer is 16-byte aligned. A view into a merged
 * projection's output is one such tensor. */
typedef struct {
    uint16_t* ptr;
    int64_t token_stride;
    int64_t head_stride;
    int32_t heads; /* 0: absent (ptr is not looked at) */
    int32_t reserved;
} fp8dit_heads;

/*
 * Rotary positions with several axes (time, height, width, ...) for q and k in
 * one launch. The first R = sum(axis_dims) elements of every head are R / 2
 * pairs; the pairs are dealt to the axes in order, axis_dims[a] / 2 to axis a.
 * Pair i of token m turns by the angle positions[m, axis(i)] * freqs[i]:
 *     (x, y) -> (x cos - y sin, x sin + y cos)
 * with the pair at elements (2i, 2i + 1) (interleaved != 0) or (i, i + R / 2).
 * Elements from R on are copied. The angle is taken in turns in double
 * precision and reduced before its sine and cosine (fp32), so far positions
 * lose nothing; the rotation is fp32, rounded once to bf16.
 *   q, k            inputs [M, heads, dim]; k.heads may be 0.
 *   q_out, k_out    outputs, same heads as their inputs. An output may be its
 *                   own input (in place); any other overlap is an error of the caller.
 *   positions       [M, n_axes] int32 or fp32 (pos_dtype), row-major, 4-byte aligned.
 *   freqs           HOST array of R / 2 doubles, radians per unit of position.
 *   axis_dims       HOST array of n_axes even positive numbers.
 * Requires dim % 8 == 0, dim <= FP8DIT_ROTARY_MAX_DIM, n_axes <= FP8DIT_ROTARY_MAX_AXES, R <= dim, and for
 * split halves R % 8 == 0. M == 0 is a no-op.
 */
fp8dit_status fp8_rotary_axes(const fp8dit_heads* q, const fp8dit_heads* k, const fp8dit_heads* q_out,
                              const fp8dit_heads* k_out, int64_t M, int32_t dim, const void* positions,
                              fp8dit_pos_dtype pos_dtype, const double* freqs, const int32_t* axis_dims,
                              int32_t n_axes, int32_t interleaved, fp8dit_stream_t stream);

/*
 * A key / value cache in E4M3FN with one scale for each block of tokens and
 * head. A block holds block_tokens consecutive tokens of one request.
 *   k, v              codes [n_blocks, kv_heads, block_tokens, head_dim], contiguous, 16-byte aligned.
 *   k_scale, v_scale  fp32 [n_blocks, kv_heads], contiguous; written before they are read.
 * A scale is a power of two: S = 2^n with the smallest n >= -120 for which
 * 448 S >= |x| for every x put into the block. E4M3 keeps its relative
 * precision under any scale, and a power of two makes the quotient x / S, the
 * change of scale when a later token of the block is larger, and code * S
 * exact, but for codes that the change of scale makes subnormal, which are
 * rounded once more. (The largest bf16 becomes 256 * 2^120, which is infinite
 * in bf16 and fp32.)
 * head_dim is 64 or 128, block_tokens 16, 32, 64 or 128.
 */
typedef struct {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int32_t n_blocks;
    int32_t kv_heads;
    int32_t block_tokens;
    int32_t head_dim;
} fp8dit_kv_cache;

/*
 * The requests of one call. Their new tokens lie one behind the other: those
 * of request b are rows offsets[b] .. offsets[b + 1] of q, k, v and out, and
 * are the last tokens of its kv_lens[b] tokens in the cache. Token t of
 * request b is in block block_table[b, t / block_tokens] at t % block_tokens.
 * All pointers are DEVICE pointers, so a captured graph reads the lengths of
 * each replay.
 *   block_table  int32 [n_requests, table_width], contiguous; entries past a request's length are not read.
 *   kv_lens      int32 [n_requests]: tokens in the cache, the new ones included.
 *   offsets      int32 [n_requests + 1], not decreasing, 0 <= offsets[b] <= total_tokens.
 *                Rows from offsets[n_requests] on are neither read nor written.
 *   max_new      bound of offsets[b + 1] - offsets[b]; it sets the launch's size.
 *   max_kv       bound of kv_lens[b], at most table_width * block_tokens.
 * A request whose numbers break these bounds is left out, and so is a token
 * whose block index is not in 0 .. n_blocks - 1 (attention sees it as masked);
 * both raise FP8DIT_ERR_INDEX in fp8dit_device_error(). A call with n_requests,
 * total_tokens or max_new 0 returns FP8DIT_OK and does nothing: the device
 * arrays are not read, so nothing is reported either.
 */
typedef struct {
    const int32_t* block_table;
    const int32_t* kv_lens;
    const int32_t* offsets;
    int64_t total_tokens;
    int32_t n_requests;
    int32_t table_width;
    int32_t max_new;
    int32_t max_kv;
} fp8dit_kv_batch;

/*
 * Put the new tokens' keys and values into the cache: request b's new tokens
 * go to positions kv_lens[b] - (offsets[b + 1] - offsets[b]) .. kv_lens[b].
 * For every block they reach, and head: the scale grows to what the new
 * tokens need (a block with no older token of the request starts anew), when
 * it grows the block's other codes, older tokens' and unused rows', are
 * brought to the new scale, and the new codes are RNEsat(x / S). Blocks that
 * are not reached keep every bit.
 *   k, v  bf16 [total_tokens, kv_heads, head_dim]; finite values.
 * A block may be written by one request only (several may read it) and stands
 * once in its table.
 */
fp8dit_status fp8_kv_cache_append(const fp8dit_kv_cache* cache, const fp8dit_heads* k, const fp8dit_heads* v,
                                  const fp8dit_kv_batch* batch, fp8dit_stream_t stream);

/*
 * Attention of the new tokens' queries over their requests' cached tokens:
 *     out[r, h] = sum_t p_t V_t,  p = softmax_t(scale q[r, h] . K_t),  t < limit(r)
 * K_t, V_t = code * S of the head h / (q.heads / kv_heads). limit(r) is
 * kv_lens[b], or with causal = g > 0 (frames of g tokens; g = 1 is the usual
 * causal mask) min(kv_lens[b], (pos / g + 1) g) with pos the query's position
 * in its request: every query sees the frames up to its own whole. A row that
 * sees nothing is 0 (its lse -infinity). Scores, softmax sums and output are
 * held in fp32. Both products run in fp16, in which the codes are exact: q is
 * scaled by a power of two per row (what lies 2^-38 below the row's largest
 * |q| is lost), the block scales are applied outside, p is rounded to fp16
 * (what lies 2^-32 below the row's largest counts in the softmax's sum only).
 * Blocks whose |v| are all at most 448 2^-120 (their scale is the smallest)
 * lose bits beside blocks whose scale is above 2^-106, and count as zeros above
 * 2^-96. The output is rounded once to bf16.
 *   cache      no NaN codes or scales among a request's kv_lens[b] tokens; what lies behind them does not matter.
 *   q, out     bf16 [total_tokens, q heads, head_dim]; q.heads % kv_heads == 0; q finite;
 *              out must not overlap the inputs.
 *   lse        fp32 [total_tokens, q heads], contiguous: natural log of the sum of exp(scale q . K_t); or NULL.
 *   scale      > 0, and finite times log2(e); scores scale q . K_t have to be within fp32's range.
 *   workspace  DEVICE scratch of at least fp8_kv_cache_attention_workspace_size(...) bytes, 16-byte aligned
 *              (may be NULL when that is 0); its contents do not matter, calls that overlap must not share it.
 * Few queries over many tokens: the tokens are split over CTAs and their
 * partial results joined by a second launch. Results do not depend on timing;
 * the sizes decide on kernel and ranges, which differ by rounding only.
 */
size_t fp8_kv_cache_attention_workspace_size(const fp8dit_kv_cache* cache, const fp8dit_kv_batch* batch,
                                             int32_t q_heads);

/*
 * How fp8_kv_cache_attention cuts a call of these sizes (they alone decide, the
 * batch's device arrays are not read): rows_per_tile rows (new tokens x query
 * heads per kv head) per thread block, 256 on the tcgen05 kernel, 8 or 16 on
 * the one for few rows; key_ranges ranges of keys, joined by a second launch
 * if more than 1. Both 0 for a call without rows. For reports and tests.
 */
fp8dit_status fp8_kv_cache_attention_plan(const fp8dit_kv_cache* cache, const fp8dit_kv_batch* batch, int32_t q_heads,
                                          int32_t* rows_per_tile, int32_t* key_ranges);

fp8dit_status fp8_kv_cache_attention(const fp8dit_kv_cache* cache, const fp8dit_heads* q, const fp8dit_kv_batch* batch,
                                     const fp8dit_heads* out, float* lse, float scale, int32_t causal,
                                     void* workspace, size_t ws_bytes, fp8dit_stream_t stream);

/*
 * Synchronise `stream`, then read and clear the current device's error word.
 * Returns FP8DIT_ERR_TIMEOUT if a bounded device wait expired since the last
 * read, else FP8DIT_ERR_INDEX if a kernel met an index outside its range,
 * FP8DIT_ERR_CUDA if the synchronisation failed, else FP8DIT_OK.
 */
fp8dit_status fp8dit_device_error(fp8dit_stream_t stream);

/*
 * Launch one block whose single thread waits, with the library's bounded
 * wait, on an mbarrier that nothing arrives at, for at most limit_ns
 * nanoseconds (1e3 .. 1e10). The wait expires and sets the error word, so
 * the next fp8dit_device_error() reports FP8DIT_ERR_TIMEOUT. Exercises the
 * failure path without faulting the GPU.
 */
fp8dit_status fp8dit_selftest_expired_wait(int64_t limit_ns, fp8dit_stream_t stream);

/*
 * Exhaustive check of the quantisers' quotient arithmetic: for every finite
 * positive bf16 amax and every bf16 x with |x| <= amax, the FP8 code the
 * quantisers produce for x / S (S = amax / fmax) is compared with the code of
 * the IEEE fp32 division x / S, for E4M3FN and E5M2. Adds the number of
 * differing codes to mismatch[0] (E4M3FN) and mismatch[1] (E5M2), a DEVICE
 * array of two uint64 the caller zeroes. Asynchronous on `stream`.
 */
fp8dit_status fp8dit_selftest_quotient(unsigned long long* mismatch, fp8dit_stream_t stream);

/* Description of the last failure on this thread ("" if none). */
const char* fp8dit_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8DIT_H */
