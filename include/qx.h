/*
 * qx.h -- C ABI of the GB300 (sm_103a) block-quantised GEMV / GEMM library.
 *
 * The library computes the decode-time matrix-vector product of GGUF-style
 * block-quantised weight rows (Q4_K, Q6_K, Q8_0) with one activation vector,
 * in two methods (llamay docs, "Backends and hardware", section "Accelerate is
 * not bit-identical": dequantising the weights to float and quantising the
 * activation to int8 are two methods, not one method and its rounding error):
 *
 *   QX_MODE_F32  -- the weights are dequantised on the fly and dotted with an
 *                   f32 activation (llambda.lisp README, "Features &
 *                   Architecture": the f32 FMA GEMV over Q4_K_M / Q6_K).
 *   QX_MODE_W4A8 -- the activation is quantised to int8 once per matmul and
 *                   the weight rows are never materialised; per-block integer
 *                   dot products are scaled per block (llamay, "Backends and
 *                   hardware", section "CPU": the W4A8 fused dot product; and
 *                   section "CUDA": an integer dot for the W4A8 inner product).
 *
 * It also runs the same contraction at prefill batch sizes on the tensor
 * cores (llamay, section "CUDA": a tensor-core prefill kernel, whose missing
 * piece was staging the next weight tile behind the current multiply).
 *
 * And it runs what stands between those products in a decoder layer: rotated
 * keys and values appended to a paged cache (qx_rope_append), attention over
 * it (qx_attn_paged, qx_attn_shared) and the norms around a block
 * (qx_block_norm).  Their activations are f32, f16 or bf16, their caches f16 or
 * bf16; the pages have no counterpart of them.  A cache may also be held in 8
 * bits: keys and values quantised as they are appended (qx_rope_append_q8), read
 * by the attention as they are (qx_attn_paged_q8), and read back (qx_kv_read_q8).
 *
 * Conventions shared by every entry point:
 *   - Weights are a row-major array of blocks; row r starts at byte
 *     r * qx_row_bytes(fmt, cols).  Block layouts are the GGUF ones:
 *       Q4_K 256 weights / 144 B: d f16, dmin f16, 12 B of packed 6-bit
 *            scales and mins, 128 B of 4-bit quants; w = d*sc*q - dmin*m.
 *       Q6_K 256 weights / 210 B: ql[128] (low 4 bits), qh[64] (high 2 bits),
 *            scales[16] int8 (one per 16 weights), d f16 last;
 *            w = d*sc*(q - 32).
 *       Q8_0 32 weights / 34 B: d f16, 32 int8 quants; w = d*q.
 *   - Every pointer named "device" is device memory owned by the caller.  The
 *     library keeps no per-call state.  Per device it holds: one cached
 *     device-property query, the device error word (below), and the
 *     QX_CHAIN_MAX_JOBS + 1 arrival counters of qx_gemv_chain_noalloc (file-
 *     scope device arrays, present on every GPU that loads the library).  No
 *     entry point of this header allocates device memory; the one allocation
 *     in the library is the short-lived buffer of the measurement hook
 *     qx_debug_mma_rate (qx_debug.h).
 *   - Calls are asynchronous on stream `s` (NULL = the legacy default stream)
 *     and run on the current device.  Argument, shape and alignment errors
 *     return before anything is launched or written; a failed launch returns
 *     QX_ERR_CUDA.
 *   - Alignment: W, the f32 activation x and the qx_act_q8 buffers must be
 *     16-byte aligned; the outputs y, Y and P 4-byte aligned.  q, k, v, the
 *     cache, cos, sin and the outputs of the rotation and attention calls must
 *     be 16-byte aligned with strides that are multiples of 8 elements (an
 *     8-bit cache's: of 16 codes and 4 scales); the operands of qx_block_norm
 *     need only their elements' alignment.
 *   - Only compute capability 10.3 (GB300) is served.  Any other device is
 *     declined with QX_ERR_UNSUPPORTED_DEVICE rather than run through another
 *     kernel (llamay, section "CUDA": below its minimum capability the
 *     backend declines at open with a message naming the reason).
 *   - Kernels bound every wait.  A wait that runs out sets a device error
 *     word and the kernel returns; qx_device_check() reports it, and pages,
 *     lengths and positions out of range too.
 */
#ifndef QX_H
#define QX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* qx_stream_t;

/* Format tags (the GGML type ids, a naming convention only), and
 * QX_Q6_K_SOA: Q6_K repacked at load time by qx_repack (see there). */
typedef enum { QX_Q8_0 = 8, QX_Q4_K = 12, QX_Q6_K = 14, QX_Q6_K_SOA = 142 } qx_fmt;

typedef enum { QX_MODE_F32 = 0, QX_MODE_W4A8 = 1, QX_MODE_W4A8_FUSED = 2 } qx_mode;

/*
 * Launch flag, OR'd into the mode argument of qx_gemv and qx_gemv_multi.
 * QX_FLAG_PDL: programmatic dependent launch.  The launch may start while the
 * previous kernel in the stream is still running: it begins streaming its
 * weights at once and reads x (and writes y) only after that kernel has
 * completed and its memory is visible.  The caller guarantees that the
 * previous kernel in the stream does not write W.
 */
#define QX_FLAG_PDL 0x100

/* Status codes.  0 is success; every error is negative. */
typedef int qx_status;
#define QX_OK 0
#define QX_ERR_ARG (-1)                /* null pointer, bad count, bad path       */
#define QX_ERR_FMT (-2)                /* unknown format                          */
#define QX_ERR_SHAPE (-3)              /* cols not whole blocks, size out of range */
#define QX_ERR_ALIGN (-4)              /* a pointer is not 16-byte aligned        */
#define QX_ERR_MODE (-5)               /* unknown mode, or mode/format mismatch   */
#define QX_ERR_CUDA (-6)               /* a CUDA runtime call or launch failed    */
#define QX_ERR_DEVICE_TIMEOUT (-7)     /* a kernel's bounded wait ran out         */
#define QX_ERR_UNSUPPORTED_DEVICE (-8) /* current device is not compute 10.3      */
#define QX_ERR_RANGE (-9)              /* a kernel met a page, length or position out of range */

/* Largest activation width served (columns per row). */
#define QX_MAX_COLS 32768
/* Largest number of matrices in one qx_gemv_multi call. */
#define QX_MAX_MULTI 8

/*
 * An int8-quantised activation, m rows of `cols` values, in caller-owned
 * device buffers (llamay, "Backends and hardware", section "CPU": the
 * activation is quantised to int8 once per matmul):
 *   q   [m, cols]      int8, row-major
 *   d   [m, cols/32]   f32 scale of each block of 32
 *   sum [m, cols/32]   int32 sum of the 32 quants of each block
 * The struct itself lives in host memory.
 */
typedef struct {
    int8_t* q;
    float* d;
    int32_t* sum;
    int64_t m;
    int64_t cols;
} qx_act_q8;

/*
 * Quantise x (device, f32 [m, cols] row-major) per block of 32:
 *   d = amax / 127 (f32, correctly rounded), q = round-half-even(x / d)
 *   (correctly rounded f32 quotient) clamped to [-127, 127], q = 0 when
 *   d == 0, sum = sum of q.
 * Writes out->q, out->d, out->sum (device buffers sized for m x cols) and
 * sets out->m = m, out->cols = cols.  cols must be a positive multiple of 32
 * (QX_ERR_SHAPE), m >= 1.  Non-finite inputs are not checked; their outputs
 * are unspecified.  The launch uses programmatic dependent launch: it may
 * start while the previous kernel in the stream drains, but reads x and
 * writes the outputs only after that kernel has completed (plain stream
 * order), so a following qx_gemv with QX_FLAG_PDL streams its weights early.
 */
qx_status qx_quantize_act_q8(const float* x, int64_t m, int64_t cols, qx_act_q8* out, qx_stream_t s);

/*
 * y[r] = sum_i w[r, i] * x[i] for r in [0, rows)  (device y, f32 [rows]).
 *   mode QX_MODE_F32 : x is `const float*`, device, f32 [cols]; y is within
 *                      1e-4 * sum_i |w[r, i] * x[i]| of the exact sum.  Q6_K
 *                      and QX_Q6_K_SOA rows of 2048 or 4096 columns, and
 *                      Q4_K rows of 256 to 4096 columns (except launches of
 *                      at most 192 KB per SM with QX_FLAG_PDL), run the
 *                      products on the tensor pipe: the quants exact in
 *                      bf16, x scaled per 256 columns by a power of two and
 *                      split into bf16 hi + lo, so each product carries at
 *                      most 2^-17 of its magnitude for every x within 2^-100
 *                      of its 256-column block's largest (Q4_K's min term
 *                      d_min m sum(x) is taken per 32 columns in f32); both
 *                      Q6_K layouts give bit-identical y.  The others
 *                      dequantise each quant to f32 and use one FMA per
 *                      weight.
 *   mode QX_MODE_W4A8: x is `const qx_act_q8*` (host struct) with m == 1 and
 *                      cols == cols, produced by qx_quantize_act_q8; y is the
 *                      per-block-scaled sum of exact integer partial sums.
 *   mode QX_MODE_W4A8_FUSED: x is `const float*`, device, f32 [cols]; the
 *                      launch quantises it itself with the arithmetic of
 *                      qx_quantize_act_q8 (identical int8 codes) and then
 *                      computes exactly what QX_MODE_W4A8 computes.
 * mode may carry QX_FLAG_PDL.
 * cols must be a positive multiple of the block width (256 for Q4_K/Q6_K,
 * 32 for Q8_0) and at most QX_MAX_COLS; rows >= 1.  The lanes cover rows of
 * up to 32768 columns for Q4_K / Q6_K in W4A8 mode, 24576 for Q4_K / Q6_K in
 * f32 mode, and 8192 for Q8_0; wider rows return QX_ERR_SHAPE.
 */
qx_status qx_gemv(qx_fmt fmt, const void* W, int64_t rows, int64_t cols, const void* x, float* y,
                  qx_mode mode, qx_stream_t s);

/*
 * n independent GEMVs over one activation in a single launch, e.g. the Q, K
 * and V projections, or gate and up: y[k] = W[k] . x for k in [0, n).  The
 * activation is read (and in QX_MODE_W4A8_FUSED quantised) once for all n
 * matrices: the pages quantise it to int8 once per matmul (llamay docs,
 * "Backends and hardware", section "CPU"), and matrices that share one input
 * are one matmul over their stacked rows, whose rows are independent
 * (llambda.lisp README, "Features & Architecture": the GEMV's outer loop runs
 * in parallel with isolated writes).
 * fmt, W, rows and y are host arrays of n entries; W[k] and y[k] are device
 * pointers.  All entries share cols, x and mode; 1 <= n <= QX_MAX_MULTI.
 * Entries of different formats are run as one launch per format.
 */
qx_status qx_gemv_multi(int n, const qx_fmt* fmt, const void* const* W, const int64_t* rows, int64_t cols,
                        const void* x, float* const* y, qx_mode mode, qx_stream_t s);

/*
 * Prefill: Y[m, r] = sum_i w[r, i] * x'[m, i] for every row m of the
 * quantised activation X (X->m rows, X->cols == cols), with Y device f32
 * [X->m, rows] row-major.  The rows of X are independent W4A8 GEMVs (colibri
 * GPU_BACKENDS.md, XDNA lane: C = A x B is row-independent, so padding the
 * batch to a tile is legitimate and padded rows are never written).
 */
qx_status qx_gemm_prefill(qx_fmt fmt, const void* W, int64_t rows, int64_t cols, const qx_act_q8* X, float* Y,
                          qx_stream_t s);

/*
 * qx_gemm_prefill with a forced path:
 *   0 = automatic (by measured time): path 1 for one row of X, path 4 for
 *       2 to 16 rows, path 3 above;
 *   1 = one W4A8 GEMV launch per row of X (bit-for-bit the qx_gemv result);
 *   2 = mma.sync tensor-core GEMM, Q4_K only (integer-valued f16 operands,
 *       exact per-sub-block integer sums, scales applied per sub-block);
 *   3 = tcgen05 tensor-core GEMM, every format: the W4A8 product is the dot
 *       product of the dequantised activation dx*q_x with the dequantised
 *       weight (llamay docs, "Backends and hardware", sections "CPU" and
 *       "CUDA"); both are formed inside the kernel, in shared memory, from
 *       the int8 codes and the raw weight blocks, each as two bf16 terms (hi
 *       + lo, 16 significant bits), and Y = Xh Wh^T + Xh Wl^T + Xl Wh^T is
 *       accumulated in f32 in tensor memory.  Each product's error is about
 *       2^-15 of its magnitude.  When the tiles (256 rows of X x 128 weight
 *       rows) leave a last wave over the SMs at most half full, that wave's
 *       tiles are split in two along K (a second launch, started beside the
 *       first by programmatic dependent launch; Y = the first half's sum plus
 *       the second's); when all the tiles fill at most half a wave, every
 *       tile is, and when they fill at most a quarter (K of 1024 columns or
 *       more; 512 for Q8_0) every tile is split in four (Y = (a0 + a1) +
 *       (a2 + a3)); so results depend on the shape and the GPU's SM count but
 *       not on the run.  No workspace: the call allocates nothing, may
 *       be captured in a CUDA graph on its first use and may run concurrently
 *       on several streams.  Shapes whose weights span 2 GiB or more (the
 *       copy engine's 32-bit coordinates) or more than 2^29 - 1 tiles
 *       return QX_ERR_SHAPE; path 0 takes path 1 for them.
 *   4 = small-batch GEMV (decode of several tokens at once: speculative or
 *       batched decode), every format, the weights streamed once per group
 *       of rows of X: groups of eight while five or more rows remain, then
 *       one of up to four.  Groups of five to eight rows against rows of up
 *       to 4096 columns in whole 256-column units whose bytes are a 16-byte
 *       multiple (Q4_K, Q8_0; Q6_K at 2048 and 4096 columns) run on the
 *       integer tensor path (mma.sync, the rows of X as the MMA's eight
 *       columns: exact integer partials per 32-column block, or per 16 for
 *       Q6_K, scaled in registers); the others on dp4a lanes, each holding
 *       its column slice of the group's codes and dotting every weight word
 *       with each row's (rows of up to 14336 columns, or 28672 for Q4_K /
 *       Q6_K when at most four rows of X remain; path 0 takes path 1 for
 *       wider rows).  Both: the same per-block integer dot products and
 *       scales as qx_gemv's W4A8 path, in a different f32 summation order
 *       (within the same tolerance, not bit-for-bit path 1).
 * A path that cannot serve the call returns QX_ERR_FMT rather than falling
 * back.
 */
qx_status qx_gemm_prefill_ex(qx_fmt fmt, const void* W, int64_t rows, int64_t cols, const qx_act_q8* X,
                             float* Y, int path, qx_stream_t s);

/*
 * The exact integer partial sums of the W4A8 product, written instead of y:
 * P[r, g] = sum over group g of q_w * q_x, with groups of 32 weights for Q4_K
 * (q_w the unsigned 4-bit quant) and Q8_0 (q_w the int8 quant), and groups of
 * 16 for Q6_K and QX_Q6_K_SOA (q_w = q - 32).  P is device int32
 * [rows, cols/32] or [rows, cols/16].  Computed by the same kernel code as qx_gemv's W4A8 path
 * (colibri GPU_BACKENDS.md: a numerics-matched integer GPU kernel).
 */
qx_status qx_gemv_partials(qx_fmt fmt, const void* W, int64_t rows, int64_t cols, const qx_act_q8* x,
                           int32_t* P, qx_stream_t s);

/*
 * A chain of dependent GEMVs in one launch.  Decode runs its GEMVs one after
 * another, each reading what an earlier one wrote (llamay docs, "Backends and
 * hardware": decode streams every weight once per token; VKNN wiki, "Running
 * an LLM on VKNN", section "Performance": the decode step is
 * weight-bandwidth-bound).  Separate launches pay a launch, a prologue and a
 * tail each; a chain streams the weights of job j + 1 while job j finishes.
 *
 * Job j computes y[k] = W[k] . x for its n entries (one format, shared cols
 * and x, like qx_gemv_multi) in W4A8 mode with the activation quantised
 * inside the launch (QX_MODE_W4A8_FUSED).  Job j + 1 reads its x only after
 * every write of job j has completed, so its x may be (part of) job j's y.
 */
#define QX_CHAIN_MAX_JOBS 128
#define QX_CHAIN_MAX_ENTRIES 4
typedef struct {
    qx_fmt fmt;
    int n;                                  /* entries, 1..QX_CHAIN_MAX_ENTRIES */
    const void* W[QX_CHAIN_MAX_ENTRIES];    /* device, 16-byte aligned          */
    int64_t rows[QX_CHAIN_MAX_ENTRIES];
    float* y[QX_CHAIN_MAX_ENTRIES];         /* device, f32 [rows], 4-byte aligned */
    int64_t cols;
    const float* x;                         /* device, f32 [cols], 16-byte aligned */
} qx_gemv_job;

/* Device scratch bytes a chain of n_jobs needs (arrival counters). */
size_t qx_gemv_chain_scratch_bytes(int n_jobs);

/*
 * Run jobs[0 .. n_jobs) in order as one cooperative launch (all CTAs
 * resident).  `scratch` is caller-owned device memory of at least
 * qx_gemv_chain_scratch_bytes(n_jobs) bytes, zero-filled before the first
 * call; a call that completes leaves it zero-filled again.  Calls that may
 * overlap on the GPU need separate scratch.  After QX_ERR_DEVICE_TIMEOUT the
 * scratch must be zero-filled again.  1 <= n_jobs <= QX_CHAIN_MAX_JOBS.
 */
qx_status qx_gemv_chain(int n_jobs, const qx_gemv_job* jobs, void* scratch, qx_stream_t s);

/*
 * qx_gemv_chain without caller scratch: for callers that cannot allocate
 * device memory where they run a chain -- code running during CUDA graph
 * capture, where cudaMalloc is not allowed; runtimes that only hand out
 * memory from a pool fixed at start-up; plug-ins that must not use the
 * process's allocator.  (The pages have no counterpart: this is a library
 * convenience, not part of the method.)
 *
 * Same jobs and results as qx_gemv_chain.  The arrival counters live in a
 * fixed array inside the library (QX_CHAIN_MAX_JOBS + 1 words on every GPU
 * that loads the library, held until the process exits); the call allocates
 * nothing, and clears the counters on stream s before each launch.
 *   - n_jobs above QX_CHAIN_MAX_JOBS (the array's capacity) returns
 *     QX_ERR_ARG before anything is launched.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current); make that first call before any
 *     stream capture on the device.
 *   - Every call on a device shares the one array: calls that may overlap on
 *     the GPU (different streams without ordering) race and give wrong
 *     results.  Order them, or use qx_gemv_chain with separate scratch.
 */
qx_status qx_gemv_chain_noalloc(int n_jobs, const qx_gemv_job* jobs, qx_stream_t s);

/* Bytes of one row of `cols` weights, or 0 if fmt is unknown or cols is not
 * a positive multiple of the block width. */
size_t qx_row_bytes(qx_fmt fmt, int64_t cols);

/*
 * Load-time repack between the GGUF Q6_K layout and QX_Q6_K_SOA (llamay
 * docs, "Backends and hardware", section "Repacking is a per-device decision
 * now": block layouts are rewritten once, at load, for the device that runs
 * them).  A QX_Q6_K_SOA row of cols weights (nsb = cols / 256 super-blocks)
 * holds, for each super-block j, the 208 bytes ql[128], qh[64], scales[16]
 * of the GGUF block at bytes [208 j, 208 j + 208), then the nsb f16 d values
 * at byte 208 nsb, padded with zero bytes to a 16-byte multiple:
 * qx_row_bytes(QX_Q6_K_SOA, cols) = 208 nsb + 16 * ceil(2 nsb / 16) (the
 * GGUF row size when nsb is a multiple of 8).  Every field of every
 * super-block is then 16-byte aligned, which the GEMV lanes read with
 * vector loads; the values and the arithmetic are those of Q6_K, so
 * qx_gemv and qx_gemv_partials give the same bits on either layout.
 *   from, to: QX_Q6_K -> QX_Q6_K_SOA, or QX_Q6_K_SOA -> QX_Q6_K (the exact
 *             inverse: a round trip restores every byte).
 *   src, dst: device, rows * qx_row_bytes(from / to, cols) bytes, 16-byte
 *             aligned, not overlapping.
 * QX_Q6_K_SOA is served by qx_gemv, qx_gemv_multi, qx_gemv_partials and
 * prefill path 1 (and path 0, which then takes path 1); the other prefill
 * paths and qx_gemv_chain return QX_ERR_FMT for it.
 */
qx_status qx_repack(qx_fmt from, qx_fmt to, const void* src, int64_t rows, int64_t cols, void* dst,
                    qx_stream_t s);

/*
 * Between the weight products of a decoder layer: keys and values appended to
 * a paged cache with the position rotation applied on the way, attention over
 * that cache, and the norms around a block.
 *
 * Element types (the GGML type ids).
 */
typedef enum { QX_F32 = 0, QX_F16 = 1, QX_BF16 = 30 } qx_dtype;

/*
 * A paged key/value cache and the batch that a call runs on (host struct; its
 * pointers are device memory).  Key j of sequence b lies in page
 * table[b * table_stride + j / page_size], slot j % page_size: element d of
 * head h is k[page * page_stride + h * head_stride + slot * slot_stride + d]
 * (strides in elements, the same for v), so both a [page, head, slot, d] and a
 * [page, slot, head, d] cache can be described.  Sequence b brings the tokens
 * q_start[b] .. q_start[b + 1] - 1 of the call, and kv_len[b] keys with those
 * counted: token t of it stands at position
 *     pos = kv_len[b] - (q_start[b + 1] - q_start[b]) + (t - q_start[b]).
 * A token at a negative position is padding.  q_start is ascending from 0;
 * tokens from q_start[n_seqs] on belong to no sequence and are left alone.
 * table, kv_len and q_start are read when the kernels run, so a captured graph
 * can be replayed with their contents changed.  A page number outside
 * [0, n_pages), a key beyond table_stride * page_size or a position beyond
 * the rotation's table is neither read nor written; qx_device_check() then
 * returns QX_ERR_RANGE.
 */
typedef struct {
    void* k;
    void* v;
    qx_dtype dtype;       /* QX_F16 or QX_BF16                                  */
    int n_heads;          /* key/value heads                                    */
    int head_dim;         /* a multiple of 8, at most QX_MAX_HEAD_DIM           */
    int page_size;        /* a power of two, 16 .. 65536                        */
    int64_t n_pages;
    int64_t page_stride;  /* elements, multiples of 8, at least head_dim        */
    int64_t head_stride;
    int64_t slot_stride;
    const int32_t* table;
    int64_t table_stride; /* entries between the rows of table                  */
    const int32_t* kv_len;
    const int32_t* q_start;
    int n_seqs;
} qx_kv;
#define QX_MAX_HEAD_DIM 256
/* Most query heads that share a key head in the attention calls. */
#define QX_MAX_GROUP 128

/* The rows of a Q/K/V product (host struct, device pointers): token t's heads
 * of head_dim elements lie one after another from t * stride elements on, so
 * q, k and v may be parts of one buffer.  q may be NULL (n_q_heads 0). */
typedef struct {
    int64_t n_tokens;
    int n_q_heads;
    qx_dtype dtype;  /* QX_F32, QX_F16 or QX_BF16 */
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride; /* elements, multiples of 8; pointers 16-byte aligned */
    int64_t k_stride;
    int64_t v_stride;
} qx_qkv;

/*
 * Rotate the queries and keys of the call's tokens by their position, write
 * the keys and values to the cache and the queries to q_out (cache type,
 * [n_tokens, n_q_heads, head_dim]).  With c = cos[pos, i], s = sin[pos, i]
 * (device, f32 [n_pos, rot / 2]), i < rot / 2, and (a, b) the elements
 * (i, i + rot / 2) of a head, or (2 i, 2 i + 1) where `interleaved` is set
 * (GGUF's two conventions):  a' = a c - b s,  b' = b c + a s.  Elements from
 * rot on pass.  The arithmetic is in f32, rounded once to the cache's type.
 * rot is a multiple of 8, at most head_dim; 0 (cos and sin may be NULL)
 * rotates nothing.  Padding tokens append nothing and get zeros in q_out; a
 * token whose position has no row in cos and sin appends nothing, and its rows
 * of q_out are left as they are (QX_ERR_RANGE from qx_device_check).
 * Two tokens of a call that share a slot race; a page may belong to several
 * sequences as long as none of the call's tokens falls into it.
 */
qx_status qx_rope_append(const qx_kv* kv, const qx_qkv* in, const float* cos, const float* sin, int64_t n_pos,
                         int rot, int interleaved, void* q_out, qx_stream_t s);

/*
 * Attention of the call's tokens over the cache (which holds their own keys
 * already).  Query head h reads key head h / (n_q_heads / n_heads); row (t, h)
 *     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q . k_j),
 * over the keys j <= pos that the window leaves: all of them for window 0,
 * else j > pos - window or j < sinks (the first `sinks` keys stay visible).
 * q: device, cache type, token stride q_stride elements (a multiple of 8; heads
 * one after another); out: [n_tokens, n_q_heads, head_dim], the cache's type
 * or QX_F32; lse (may be NULL): f32 [n_tokens, n_q_heads], the natural log of
 * sum_j p_j.  A row that sees no key (a padding token) gets zeros and -inf.
 * Scores, maxima, sums and outputs are held in f32.  At head sizes 64 and 128
 * the probabilities are rounded to the cache's type before they meet v, so an
 * f32 out carries that much too: relative 2^-8 for bf16 and 2^-11 for f16, at
 * most; f16 holds those below 2^-26 of the row's largest to 2^-37 of it.  At
 * other head sizes they stay in f32.
 * A key that a row does not see has no effect on it, whatever its slot holds
 * (NaN and infinities, too; pages outside the window may be given back).
 * scratch: device, qx_attn_scratch_bytes() of the same sizes, 256-byte
 * aligned, its first QX_ATTN_COUNTER_BYTES bytes zero-filled before its first
 * use; a completed call leaves it fit for the next.  After a bounded wait that
 * ran out (QX_ERR_DEVICE_TIMEOUT from qx_device_check) they have to be
 * zero-filled again.  Calls that may overlap need separate scratch, and so do
 * the calls of a captured graph, whose replays use it for as long as the graph
 * lives.
 */
#define QX_ATTN_COUNTER_BYTES 2304
qx_status qx_attn_paged(const qx_kv* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride,
                        float scale, int64_t window, int64_t sinks, void* out, qx_dtype out_dtype, float* lse,
                        void* scratch, qx_stream_t s);

/*
 * qx_attn_paged without a window for sequences whose first shared_len keys and
 * values are the same: those keys are read through the first sequence's row of
 * the table, once for the whole batch, and each sequence's own keys after
 * them.  The caller guarantees that every sequence's keys below shared_len
 * hold what the first one's do (usually they are the same pages).
 * 0 <= shared_len <= kv_len[b] for every sequence.
 */
qx_status qx_attn_shared(const qx_kv* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride,
                         float scale, int64_t shared_len, void* out, qx_dtype out_dtype, float* lse, void* scratch,
                         qx_stream_t s);

/* Device scratch bytes that qx_attn_paged and qx_attn_shared need on the
 * current device for at most these sizes; 0 for invalid ones. */
size_t qx_attn_scratch_bytes(int64_t n_tokens, int n_q_heads, int n_heads, int head_dim, int n_seqs);

/*
 * A paged cache in 8 bits.  Each key and value head is held as int8 codes and
 * one f32 scale d and stands for d * code:
 *     d = amax / 127 (f32, correctly rounded), code = round-half-even(x / d)
 *     (correctly rounded f32 quotient) clamped to [-127, 127], 0 when d == 0,
 * the rule of qx_quantize_act_q8 with a head for a block (an element is off by
 * at most d / 2, 1 / 254 of its head's largest).  A head with an element that is
 * infinite or no number has a scale that is no number, and so stands for none.
 * Codes lie as qx_kv's elements do; the scales of key j of sequence b, head h,
 * at k_scale[page * scale_page_stride + h * scale_head_stride + slot] (the same
 * for v).  table, kv_len, q_start, positions, padding and what is out of range:
 * as for qx_kv.  A cache may be filled by other means than qx_rope_append_q8:
 * every code, -128 too, and every finite scale are served (the attention's bounds:
 * for those of values up to 2^100).
 */
typedef struct {
    int8_t* k;
    int8_t* v;
    float* k_scale;
    float* v_scale;
    qx_dtype dtype;       /* of queries and outputs: QX_F16 or QX_BF16           */
    int n_heads;          /* key/value heads                                     */
    int head_dim;         /* a multiple of 16, at most QX_MAX_HEAD_DIM           */
    int page_size;        /* a power of two, 16 .. 65536                         */
    int64_t n_pages;
    int64_t page_stride;  /* codes, multiples of 16, at least head_dim           */
    int64_t head_stride;
    int64_t slot_stride;
    int64_t scale_page_stride; /* scales, multiples of 4, at least page_size     */
    int64_t scale_head_stride;
    const int32_t* table;
    int64_t table_stride; /* entries between the rows of table                   */
    const int32_t* kv_len;
    const int32_t* q_start;
    int n_seqs;
} qx_kv_q8;

/* qx_rope_append into an 8-bit cache: queries rotated to q_out (kv->dtype), keys
 * rotated and quantised, values quantised.  The rotation's products and sums are
 * each rounded to f32, so codes and scales can be found again bit for bit. */
qx_status qx_rope_append_q8(const qx_kv_q8* kv, const qx_qkv* in, const float* cos, const float* sin, int64_t n_pos,
                            int rot, int interleaved, void* q_out, qx_stream_t s);

/* What the cache holds at the positions of the call's tokens: d * code, rounded
 * to f32 and from there to out_dtype (QX_F32, QX_F16 or QX_BF16), to k_out and v_out
 * (device, [n_tokens, n_heads, head_dim]; one of them may be NULL).  With q_start the sums
 * of kv_len, whole sequences.  Padding tokens get zeros; tokens of no sequence,
 * and those whose page is out of range, are left as they are. */
qx_status qx_kv_read_q8(const qx_kv_q8* kv, int64_t n_tokens, void* k_out, void* v_out, qx_dtype out_dtype, qx_stream_t s);

/*
 * qx_attn_paged over an 8-bit cache: q and out of kv->dtype (out also QX_F32),
 * the same scratch (qx_attn_scratch_bytes).  Row (t, h)
 *     out = sum_j p_j d^v_j c^v_j / sum_j p_j,   p_j = exp(scale d^k_j q . c^k_j).
 * over the keys that qx_attn_paged lets it see.  Codes are taken as they are, and so
 * are queries, but that a bf16 row's elements below 2^-28 of its largest may be held
 * to 2^-39 of that (head sizes 64 and 128, few rows a sequence); scores, maxima, sums
 * and outputs are held in f32.  q . c^k_j is summed up first; where that sum and the
 * score are in f32's range, the factors between them are of any size (a sum of zero
 * is a score of zero).  At head sizes 64 and 128 p_j d^v_j is rounded to f16
 * (relative 2^-11 at most) before it meets the codes; products below 2^-21 of D, the row's largest p_j times its largest d^v_j (or 2^-80,
 * where all of them are smaller), are held to 2^-32 of D, and the sum of the p_j holds
 * all of them down to 2^-38 of the largest: for value scales up to 2^100, however far
 * apart.  (Scales that are all below 2^-80 so lose bits, below 2^-112 all of them.)
 * At other head sizes the products stay in f32.
 * A key that a row does not see does not enter it, whatever its slot holds (NaN and
 * infinities, too), and the bounds above are of the keys that it sees; in which
 * power of two its products are rounded may go by other rows and keys, so a row's
 * last bits may.  One that it sees, and whose scale or whose value's scale is infinite
 * or no number, makes the row no numbers.
 */
qx_status qx_attn_paged_q8(const qx_kv_q8* kv, const void* q, int64_t n_tokens, int n_q_heads, int64_t q_stride,
                           float scale, int64_t window, int64_t sinks, void* out, qx_dtype out_dtype, float* lse,
                           void* scratch, qx_stream_t s);

/* The number of the capture that stream s takes part in, another one for each
 * capture of the process; 0 outside of captures.  A program that keeps scratch
 * for its streams learns by it when a call's has to be a graph's own. */
uint64_t qx_stream_capture_id(qx_stream_t s);

/*
 * The step from one block of a layer to the next, a row at a time:
 *     u  = y * w_post / sqrt(mean(y^2) + eps)     (w_post NULL: u = y)
 *     r' = r + alpha * gate * u                   (gate NULL: 1)
 *     x  = r' * w_pre / sqrt(mean(r'^2) + eps)    (w_pre NULL: no x)
 * y, gate and x: dtype; r and r_out: res_dtype (each QX_F32, QX_F16 or
 * QX_BF16); w_post and w_pre: f32 [cols].  Rows lie y_stride, gate_stride, ...
 * elements apart (gate_stride 0: one gate for all rows).  y NULL: u = 0, so x
 * is the norm of r.  r_out NULL: r' is not written.  The arithmetic is in f32;
 * x comes from r' before it is rounded.  r_out may be r and x may be y, with
 * the same stride; rows of r_out and of x may not overlap (strides of cols at
 * least, where there are several rows).
 * 1 <= cols <= QX_MAX_COLS.
 */
typedef struct {
    int64_t rows;
    int64_t cols;
    qx_dtype dtype;
    qx_dtype res_dtype;
    const void* y;
    const void* r;
    const void* gate;
    const float* w_post;
    const float* w_pre;
    float alpha;
    float eps;
    void* r_out;
    void* x;
    int64_t y_stride;
    int64_t r_stride;
    int64_t gate_stride;
    int64_t r_out_stride;
    int64_t x_stride;
} qx_norm_args;
qx_status qx_block_norm(const qx_norm_args* a, qx_stream_t s);

/* Synchronise stream s, then read and clear the device error word of the
 * current device: QX_OK, QX_ERR_DEVICE_TIMEOUT if a kernel's bounded wait ran
 * out since the last check, QX_ERR_RANGE if a kernel met a page, length or
 * position out of range, or QX_ERR_CUDA if the synchronisation failed. */
qx_status qx_device_check(qx_stream_t s);

/* Static, NUL-terminated strings. */
const char* qx_status_string(qx_status st);
/* The CUDA call and error text behind the most recent QX_ERR_CUDA returned
 * on the calling thread ("" if none); valid until the next call on it. */
const char* qx_last_error(void);
const char* qx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QX_H */
