/*
 * mxq.h -- C ABI of libmxq, GB300 (sm_103a) block-scaled quantization.
 *
 * The library turns a bf16 matrix into OCP-MX MXFP8 (E4M3 codes, one E8M0
 * scale per 32-element block) rowwise and colwise from a single HBM read,
 * optionally fused with a dbias column sum, a tanh-GELU or a SwiGLU gate, and
 * into NVFP4 (E2M1 codes, one E4M3 scale per 16 elements, one fp32 tensor
 * scale) rowwise and transposed; it multiplies what it quantized: MXFP8
 * products grouped by expert, their weight gradients, and NVFP4 weights times
 * a few rows; and it has what stands around those products in a feed-forward
 * block: RMSNorm into MXFP8, routing of tokens to experts and sorting of their
 * rows, and the gated activation with an 8-bit copy of its input.
 *
 * Kernel families this covers (TransformerEngine PR #3291 "Fix pointer
 * arithmatic to generate correct LDS/STS instructions", results tables
 * "MXFP8 generic quantize kernel", "MXFP8 specialized cast-only kernel
 * (bidimensional)", "MXFP8 gated (swiglu / geglu) kernel" and "NVFP4 2D
 * quantize-transpose kernel"; the colwise-only cast is the "dim1" cast of
 * torchao PR #12 "Multiply with inverse scale in loop instead of dividing",
 * section "Performance").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  * All pointers are DEVICE pointers unless stated otherwise; the caller
 *    owns every buffer.  The library never allocates, frees or synchronises:
 *    all work is enqueued on `stream` (NULL = the legacy default stream), and
 *    every buffer must stay valid until the stream has passed this call.
 *  * Matrices are row-major.  `x` is bf16 (raw 16-bit patterns) with a row
 *    stride of `ldx` elements; outputs are dense (row stride = width).
 *  * Host-checkable problems return a status synchronously and enqueue
 *    nothing.  A launch failure returns MXQ_ECUDA.
 *  * `dev_err` (optional, device, 4 bytes): every wait inside the kernels is
 *    bounded; if one runs out, the kernel ORs MXQ_DEVERR_TIMEOUT into
 *    *dev_err, waits (bounded) for its own copies in flight and exits
 *    without writing the remaining tiles.  The library never clears
 *    *dev_err; the caller zeroes it and reads it back after the stream.
 *    When *dev_err is nonzero after a call, every output of that call
 *    (codes, scales, dbias, the global scale) is undefined.
 *  * Alignment: `x`, every output and the workspace 16-byte aligned, `ldx`
 *    a multiple of 8.  Violations return MXQ_EALIGN.
 *  * A workspace serves one call at a time: calls that may overlap on the GPU
 *    (on two streams, or in two graphs that are replayed) take one each.
 *  * The device must be compute capability 10.3 (GB300): else MXQ_EARCH.
 *  * NaN or infinite inputs are outside the contract.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MXQ_API __attribute__((visibility("default")))
#else
#define MXQ_API
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st* mxq_stream_t;

typedef enum {
    MXQ_OK = 0,
    MXQ_EINVAL = 1,      /* NULL pointer, bad flag combination            */
    MXQ_ESHAPE = 2,      /* negative size or size not a block multiple    */
    MXQ_EALIGN = 3,      /* pointer or stride misaligned                  */
    MXQ_EARCH = 4,       /* current device is not sm_103                  */
    MXQ_EWORKSPACE = 5,  /* workspace missing or too small                */
    MXQ_ECUDA = 6        /* CUDA runtime error while launching            */
} mxq_status;

/* flags */
enum {
    MXQ_ROWWISE = 1,        /* 1x32 (MX) / 1x16 (NVFP4) blocks along K     */
    MXQ_COLWISE = 2,        /* 32x1 (MX) / 16x1 (NVFP4) blocks along M,    */
                            /* stored transposed: [K][M]                   */
    MXQ_DBIAS = 4,          /* fp32 column sums of x (mx_quantize_rowcol)  */
    MXQ_ACT_GELU_TANH = 8,  /* gelu_tanh: of x (mx_quantize_rowcol), of the */
                            /* gate (mx_quantize_gated: GeGLU), its         */
                            /* derivative (mx_quantize_dact / _dgated)     */
    MXQ_NVFP4_2D = 16,      /* 16x16 blocks (nvfp4_quantize_transpose)     */
    MXQ_ACT_SILU = 32,      /* silu: SwiGLU gate (the default of the gated */
                            /* calls), its derivative (mx_quantize_dact)   */
    MXQ_SCALE_RCEIL = 64,   /* MXFP8 calls: ceil-style E8M0 rule, below    */
    MXQ_SCALE_SWIZZLED = 128,/* MXFP8 calls: scales in 128x4 tiles, below   */
    MXQ_OUT_F32 = 256,      /* products: fp32 output instead of bf16       */
    MXQ_OUT_BF16 = 512,     /* mx_rmsnorm: y in bf16 too                   */
    MXQ_IN_F32 = 1024,      /* norm's weight, router's logits: fp32        */
    MXQ_ROUTE_SIGMOID = 2048, /* scores: sigmoid instead of softmax        */
    MXQ_ROUTE_RENORM = 4096,  /* weights divided by the chosen scores' sum */
    MXQ_ROUTE_GROUP_MAX = 8192 /* a group's score: its best expert's,      */
                            /* instead of the sum of its best two          */
};

/* bits of *dev_err */
enum {
    MXQ_DEVERR_TIMEOUT = 1,
    MXQ_DEVERR_OFFSETS = 2  /* grouped products: bad group offsets, below  */
};

/* operation ids for mxq_workspace_bytes */
enum { MXQ_OP_ROWCOL = 0, MXQ_OP_NVFP4 = 1, MXQ_OP_DACT = 2, MXQ_OP_ROWCOL_HOST = 3 };

/* operation id for mxq_workspace_bytes: mx_rmsnorm_backward */
enum { MXQ_OP_RMSNORM_BACKWARD = 7 };

/* operation ids for mxq_product_plan */
enum { MXQ_OP_GROUPED_GEMM = 4, MXQ_OP_GROUPED_WGRAD = 5, MXQ_OP_NVFP4_GEMV = 6 };

/* Human-readable name of a status code (static string, never NULL). */
MXQ_API const char* mxq_status_string(int status);

/* Workspace bytes `op` needs for an M x K input with `flags` on the current
 * device (0 when none is needed).  MXQ_OP_ROWCOL needs one only with
 * MXQ_DBIAS; MXQ_OP_NVFP4 needs 4 bytes when no amax_in is given;
 * MXQ_OP_RMSNORM_BACKWARD's depends on the device's SMs (0 without a GB300). */
MXQ_API size_t mxq_workspace_bytes(int op, int64_t M, int64_t K, uint32_t flags);

/*
 * mx_quantize_rowcol -- bf16 -> MXFP8 rowwise and/or colwise, one HBM read.
 *
 * Operation (per 32-value block B of y, y = x, or y = gelu_tanh(x) in fp32
 * with MXQ_ACT_GELU_TANH, gelu_tanh(x) = 0.5 x (1 + tanh(sqrt(2/pi)
 * (x + 0.044715 x^3)))):  a = max|y| over B;  e = floor(log2 a) - 8 clamped
 * to [-127, 127] (a = 0 -> scale code 0);  scale code = e + 127 (E8M0);
 * codes = E4M3(y * 2^-e), round-to-nearest-even, saturating to +-448.
 * With MXQ_SCALE_RCEIL (any MXFP8 call) e = ceil(log2(a / 448)) instead,
 * clamped the same way: the smallest power of two for which no element
 * exceeds 448, so nothing saturates.
 * With MXQ_SCALE_SWIZZLED (any MXFP8 call) each scale matrix [R][C] (R = M,
 * C = K/32 rowwise; R = K, C = M/32 colwise) is written in the tiled layout
 * block-scaled GEMMs read instead of row-major: padded to R' =
 * ceil(R/128)*128 rows and C' = ceil(C/4)*4 columns (padding bytes 0), cut
 * into 128x4 tiles stored one after another in row-major tile order (tile
 * (i, j) at byte (i * C'/4 + j) * 512); inside a tile, entry (r, c) is at
 * byte (r % 32) * 16 + (r / 32) * 4 + c.  The buffers must hold R' * C'
 * bytes.  (mx_quantize_dgated additionally needs N % 128 == 0.)  The
 * multiply by the exact power of two 2^-e replaces a per-element division
 * (torchao PR #12, rationale section).  Rowwise blocks are 1x32 along K,
 * colwise blocks 32x1 along M (TE PR #3291 tables, dir "row"/"col"/"both").
 * MXQ_DBIAS adds dbias[k] = sum_m x[m][k] in fp32 (TE PR #3291 fusion
 * "dbias"; not combinable with MXQ_ACT_GELU_TANH).
 *
 *   x       [M][ldx] bf16, M % 32 == 0, K % 32 == 0, ldx >= K.
 *   flags   MXQ_ROWWISE | MXQ_COLWISE (at least one), optional MXQ_DBIAS or
 *           MXQ_ACT_GELU_TANH.
 *   q_row   [M][K] E4M3 codes, s_row [M][K/32] E8M0 (needed with ROWWISE,
 *           else ignored).
 *   q_col   [K][M] E4M3 codes (row k holds column k of the blocks),
 *           s_col [K][M/32] E8M0 (needed with COLWISE, else ignored).
 *   dbias   [K] fp32 (needed with MXQ_DBIAS).
 *   workspace / workspace_bytes: device scratch of at least
 *           mxq_workspace_bytes(MXQ_OP_ROWCOL, M, K, flags) bytes, 16-byte
 *           aligned (dbias partial sums); may be NULL when that is 0.
 *   M == 0 or K == 0 is a valid empty call (dbias is zero-filled).
 */
MXQ_API mxq_status mx_quantize_rowcol(const void* x, int64_t M, int64_t K, int64_t ldx, uint32_t flags,
                              uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                              float* dbias, void* workspace, size_t workspace_bytes,
                              uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_quantize_rowcol_dbias_noalloc -- mx_quantize_rowcol with MXQ_DBIAS for
 * callers that cannot allocate device memory.  The pages have no
 * counterpart to this entry point.
 *
 * Some callers cannot provide the dbias workspace: code inside a framework
 * that owns all device memory through its own pool (an extra cudaMalloc
 * would bypass the pool and synchronise the device), loops that forbid
 * allocation after start-up, and plugin hosts that pass this library only
 * the tensors it reads and writes.  This entry point takes the same
 * arguments as mx_quantize_rowcol minus the workspace, always computes
 * dbias (MXQ_DBIAS is implied; MXQ_ACT_GELU_TANH is refused with
 * MXQ_EINVAL), and keeps its scratch in a device array the library owns:
 * 8 MiB, held on every GPU that loads the library until the process exits.
 *   - Limit: shapes needing more than 8 MiB of band sums
 *     (mxq_workspace_bytes(MXQ_OP_ROWCOL, M, K, MXQ_DBIAS) > 8 MiB, e.g.
 *     more than 16384 x 16384) return MXQ_EWORKSPACE; nothing is enqueued.
 *   - Every call looks up the array's device address in the current
 *     context; the first call with a device current also loads the
 *     library's device code there, so make that first call before any
 *     stream capture begins.
 *   - All calls share the array.  Nothing in it needs clearing (every value
 *     read is written earlier in the same call), but calls that overlap on
 *     the GPU race on it: order them, e.g. on one stream.  Calls queued one
 *     after another on one stream do not overlap.
 *   - As for every entry point, the outputs are undefined when the call
 *     reports a timeout through *dev_err.
 *   - It never calls cudaMalloc, cudaFree or any allocating routine.
 */
MXQ_API mxq_status mx_quantize_rowcol_dbias_noalloc(const void* x, int64_t M, int64_t K,
                                                    int64_t ldx, uint32_t flags, uint8_t* q_row,
                                                    uint8_t* s_row, uint8_t* q_col,
                                                    uint8_t* s_col, float* dbias,
                                                    uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_quantize_rowcol_host -- mx_quantize_rowcol on a matrix in host memory.
 * The pages have no counterpart: it is the path for callers whose data is
 * on the host, and what the benchmark's end-to-end figure measures.
 *
 * The same cast (plain, no dbias or activation) of x in row panels of up to
 * 2048 rows: each panel is copied to the device, quantized, and its outputs
 * copied back (colwise codes as 2-D copies into the [K][M] host layout;
 * row-major colwise scales gathered on the device for the whole matrix and
 * copied back once, after the last panel); two sets of device buffers
 * alternate and the copies run on two library-owned streams, so copies in,
 * casts and copies out of consecutive panels overlap.
 *
 *   x, q_row, s_row, q_col, s_col  host memory with the layouts of
 *           mx_quantize_rowcol; page-locked memory lets the copies run
 *           asynchronously (pageable memory works, without overlap).
 *   flags   MXQ_ROWWISE and/or MXQ_COLWISE.
 *   workspace  device memory, 256-byte aligned, at least
 *           mxq_workspace_bytes(MXQ_OP_ROWCOL_HOST, M, K, flags) bytes.
 *   stream  the call starts after the work already on `stream`, and work
 *           enqueued on `stream` afterwards starts after the outputs are on
 *           the host (synchronise the stream before reading them).
 * Calls from several host threads are serialised inside the library (they
 * share the per-device streams).
 */
MXQ_API mxq_status mx_quantize_rowcol_host(const void* x, int64_t M, int64_t K, int64_t ldx,
                                           uint32_t flags, uint8_t* q_row, uint8_t* s_row,
                                           uint8_t* q_col, uint8_t* s_col, void* workspace,
                                           size_t workspace_bytes, mxq_stream_t stream);

/*
 * mx_quantize_gated -- SwiGLU or GeGLU gate fused with MXFP8 quantization.
 *
 * Operation: y[m][n] = act(x[m][n]) * x[m][N + n] for n < N, computed in
 * fp32 (no intermediate bf16 rounding), then quantized exactly as
 * mx_quantize_rowcol quantizes y (TE PR #3291 table "MXFP8 gated (swiglu /
 * geglu) kernel", fusions "swiglu" and "geglu").  act is silu(g) =
 * g / (1 + e^-g) (SwiGLU; the default, or MXQ_ACT_SILU) or gelu_tanh
 * (GeGLU, MXQ_ACT_GELU_TANH).
 *
 *   x       [M][ldx] bf16 holding [gate | up], each N wide; ldx >= 2N.
 *   flags   MXQ_ROWWISE and/or MXQ_COLWISE, at most one activation flag.
 *   M % 32 == 0, N % 32 == 0.
 *   q_row [M][N], s_row [M][N/32], q_col [N][M], s_col [N][M/32] as above.
 */
MXQ_API mxq_status mx_quantize_gated(const void* x, int64_t M, int64_t N, int64_t ldx, uint32_t flags,
                             uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                             uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_quantize_dact -- backward activation fused with MXFP8 quantization.
 *
 * Operation (TE PR #3291 table "MXFP8 generic quantize kernel", fusions
 * "dgelu", "dsilu" and "dbias_dgelu"): y[m][k] = grad[m][k] * act'(x[m][k])
 * in fp32, with act' the derivative of gelu_tanh (MXQ_ACT_GELU_TANH) or of
 * silu (MXQ_ACT_SILU) -- exactly one of the two; y is quantized exactly as
 * mx_quantize_rowcol quantizes its input, and MXQ_DBIAS writes
 * dbias[k] = sum_m y[m][k].
 *
 *   grad    [M][ldg] bf16, the incoming gradient; x [M][ldx] bf16, the
 *           activation's input; M % 32 == 0, K % 32 == 0, ldg, ldx >= K,
 *           multiples of 8, both 16-byte aligned.
 *   outputs, dbias, workspace (mxq_workspace_bytes(MXQ_OP_DACT, M, K,
 *           flags) bytes with MXQ_DBIAS), dev_err, stream: as for
 *           mx_quantize_rowcol.
 */
MXQ_API mxq_status mx_quantize_dact(const void* grad, const void* x, int64_t M, int64_t K,
                                    int64_t ldg, int64_t ldx, uint32_t flags, uint8_t* q_row,
                                    uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, float* dbias,
                                    void* workspace, size_t workspace_bytes, uint32_t* dev_err,
                                    mxq_stream_t stream);

/*
 * mx_quantize_dgated -- backward of the gated activation fused with MXFP8
 * quantization (TE PR #3291 table "MXFP8 gated (swiglu / geglu) kernel",
 * fusion "dswiglu", and its GeGLU counterpart).
 *
 * Operation: with gate = x[m][n], up = x[m][N + n] and g = grad[m][n],
 * y[m][n] = g * up * act'(gate) (the gradient of the gate) and
 * y[m][N + n] = g * act(gate) (the gradient of up), n < N, in fp32; act is
 * silu (the default, or MXQ_ACT_SILU) or gelu_tanh (MXQ_ACT_GELU_TANH).  y
 * ([M][2N]) is quantized exactly as mx_quantize_rowcol quantizes its input.
 *
 *   grad    [M][ldg] bf16, ldg >= N; x [M][ldx] bf16 holding [gate | up],
 *           ldx >= 2N; M % 32 == 0, N % 32 == 0.
 *   q_row [M][2N], s_row [M][2N/32], q_col [2N][M], s_col [2N][M/32].
 */
MXQ_API mxq_status mx_quantize_dgated(const void* grad, const void* x, int64_t M, int64_t N,
                                      int64_t ldg, int64_t ldx, uint32_t flags, uint8_t* q_row,
                                      uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                                      uint32_t* dev_err, mxq_stream_t stream);

/*
 * bf16_amax -- largest |x| of a bf16 matrix, written as fp32 to *amax_out
 * (device).  The exact maximum, so the result does not depend on the order
 * of the reduction.  Needed for the NVFP4 tensor scale.
 *   x [M][ldx], K % 8 == 0.  M == 0 or K == 0 writes 0.
 */
MXQ_API mxq_status bf16_amax(const void* x, int64_t M, int64_t K, int64_t ldx, float* amax_out,
                     mxq_stream_t stream);

/*
 * nvfp4_quantize_transpose -- bf16 -> NVFP4, rowwise and transposed.
 *
 * Operation (TE PR #3291, "NVFP4 quantize-transpose" family: the 1D kernel
 * named in "Patched but not measurable" and the results table "NVFP4 2D
 * quantize-transpose kernel"; every step one fp32 IEEE operation in this
 * order):
 *   A = tensor amax (from amax_in, else from an internal bf16_amax pass);
 *   G = A / 2688 (2688 = 448 * 6), written to *global_scale;
 *   per block of 16 values (1x16 along K rowwise; 16x1 along M for the
 *   transposed output): b = block amax; s = E4M3((b / 6) / G) (RNE,
 *   saturating); d = value(s) * G; inv = 1 / d (0 when s == 0 or d == 0,
 *   the largest finite float if 1 / d overflows);
 *   codes = E2M1(x * inv), round-to-nearest-even, saturating to +-6,
 *   packed two per byte, element 2i in the low nibble.  A == 0 gives
 *   G = 0 and all-zero scales.
 *   With MXQ_NVFP4_2D the block is 16x16 (rows 16i.., columns 16j..): b is
 *   its amax and every element of it is quantized with its one scale in
 *   both outputs; the scale arrays keep the shapes below, each block's
 *   scale repeated in its 16 rows (s_row) or 16 columns (s_t), so q_t is
 *   exactly the transpose of q_row.
 *
 *   x       [M][ldx] bf16, M % 32 == 0, K % 32 == 0 (so that every packed
 *           code row is a multiple of 16 bytes, as the bulk-copy engine
 *           that writes them needs).
 *   flags   MXQ_ROWWISE and/or MXQ_COLWISE (= the transposed output),
 *           optional MXQ_NVFP4_2D.
 *   amax_in device fp32 tensor amax, or NULL to compute it here (then the
 *           workspace must hold 4 bytes).
 *   global_scale  device fp32, receives G (required).
 *   q_row [M][K/2], s_row [M][K/16] (E4M3); q_t [K][M/2], s_t [K][M/16].
 */
MXQ_API mxq_status nvfp4_quantize_transpose(const void* x, int64_t M, int64_t K, int64_t ldx,
                                    uint32_t flags, const float* amax_in, float* global_scale,
                                    uint8_t* q_row, uint8_t* s_row, uint8_t* q_t, uint8_t* s_t,
                                    void* workspace, size_t workspace_bytes, uint32_t* dev_err,
                                    mxq_stream_t stream);

/*
 * mx_grouped_gemm -- rows sorted by expert times their experts' weights.
 *
 * Operation: for every group e < E and row offsets[e] <= m < offsets[e + 1],
 * out[m][n] = sum_k X[m][k] * W[e][n][k], with X[m][k] = E4M3(x_q[m][k]) *
 * 2^(x_s[m][k / 32] - 127) and W alike: the operands mx_quantize_rowcol
 * writes with MXQ_ROWWISE (row-major scales), products exact, sums in the
 * tensor cores' fp32 accumulators, which cut off towards zero (below), one
 * rounding to bf16 (none with MXQ_OUT_F32).  The input gradient dX = dY W
 * is the same call: dY rowwise as x, and as w each expert's weight [N][K]
 * quantized MXQ_COLWISE (its q_col [K][N], s_col [K][N/32]).  E = 1 with
 * offsets {0, M} is a plain product.
 *
 *   x_q [M][K], x_s [M][K/32]; w_q [E][N][K], w_s [E][N][K/32]; K % 32 == 0;
 *           M and N are any.  A scale code of 255 is NaN.
 *   offsets [E + 1] int32 on the device, not decreasing, within [0, M]; a
 *           group may be empty, and rows in no group are not written.
 *           Offsets that break this set MXQ_DEVERR_OFFSETS in *dev_err and
 *           nothing is written.  E <= 512.
 *   out     [M][ldo] bf16 or fp32, aligned to its element (16-byte aligned
 *           rows are written with wider stores); ldo >= N.
 *   K == 0 writes zeros; M, N or E == 0 is a valid empty call.
 * The inputs are 16-byte aligned.
 * Errors: cut off sums lose more than rounded ones, and to one side.  The errors
 * of an fp32 output of random operands stay below 2^-20 of its norm (2^-23.7 at
 * K = 1056, 2^-21.7 at 4096, 2^-20.5 from 8192 on, since longer sums are taken
 * apart and added in fp32; of rounded additions 2^-24.4, 2^-23.3 and 2^-22.7).  A
 * bf16 output's sums are not taken apart; its rounding is larger.
 * Order: an element is the sum of 1, 2 or 4 ranges of k, each summed in the order
 * of k and added in order.  How many follows from M, N, K, E, the output's type
 * and the GPU's SMs (plan[3] of mxq_product_plan: few tiles share their
 * contraction), and with K it alone decides the bits: where the rows lie, which
 * kernel takes them and what else a call holds do not.  So the same call gives the
 * same bits, but a row in a batch of 8 may differ from itself in a batch of 4096
 * by the errors above.
 */
MXQ_API mxq_status mx_grouped_gemm(const uint8_t* x_q, const uint8_t* x_s, const uint8_t* w_q,
                                   const uint8_t* w_s, const int32_t* offsets, int64_t M,
                                   int64_t N, int64_t K, int64_t E, uint32_t flags, void* out,
                                   int64_t ldo, uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_grouped_wgrad -- the weights' gradients of mx_grouped_gemm.
 *
 * Operation: dw[e][n][k] = sum over offsets[e] <= m < offsets[e + 1] of
 * G[m][n] * X[m][k], with G and X quantized along m: the operands that
 * mx_quantize_rowcol writes with MXQ_COLWISE for dY [M][N] and x [M][K].
 * Sums as in mx_grouped_gemm, along m; dw bf16, or fp32 with MXQ_OUT_F32.
 *
 *   g_q [N][M], g_s [N][M/32]; x_q [K][M], x_s [K][M/32]; M % 32 == 0; N and
 *           K are any.
 *   offsets as for mx_grouped_gemm, and multiples of 32 (a block of 32 rows
 *           has one scale, so no group may start or end inside one: pad
 *           groups with zero rows).
 *   dw      [E][N][K], every element written (zeros for an empty group).
 * Order: as in mx_grouped_gemm.  Ranges end on multiples of 128 of the buffer's
 * rows, so that a group's bits also depend on where it starts, modulo 128.
 */
MXQ_API mxq_status mx_grouped_wgrad(const uint8_t* g_q, const uint8_t* g_s, const uint8_t* x_q,
                                    const uint8_t* x_s, const int32_t* offsets, int64_t M,
                                    int64_t N, int64_t K, int64_t E, uint32_t flags, void* dw,
                                    uint32_t* dev_err, mxq_stream_t stream);

/*
 * nvfp4_gemv -- few rows of bf16 times NVFP4 weights.
 *
 * Operation: out[r][n] = G[e] * sum_k x[r / share][k] * E4M3(w_s[e][n][k/16])
 * * E2M1(w_q[e][n][k]) for r < T * share, with e = experts[r], or 0 when
 * experts is NULL: the operands that nvfp4_quantize_transpose writes with
 * MXQ_ROWWISE for each expert's weight [N][K].  Sums in fp32 (the tensor
 * cores' cut off sums are of 512 terms at most, added in fp32); out bf16, or
 * fp32 with MXQ_OUT_F32.
 *
 *   x       [T][ldx] bf16, ldx % 8 == 0; K % 32 == 0; N is any.
 *   share   output rows that read one row of x (a token's experts), >= 1.
 *   w_q [E][N][K/2], w_s [E][N][K/16], w_global [E] fp32 on the device;
 *           E <= 4096.
 *   experts [T * share] int32 on the device: a row whose expert is negative
 *           or >= E is zero (it belongs to another rank, or to no token).
 *           NULL: one weight (E == 1, share == 1).
 *   out     [T * share][ldo].
 * Meant for up to 16 rows of each expert; more are right.  The weights are read
 * once for every 16 rows; with experts, an expert's once for every 12 of its rows
 * at least, or every 6 where T * share is at most 4 times the smaller of E and
 * T * share.
 * Order: fixed, so that the same call gives the same bits.  How a sum is grouped
 * follows from the sizes, the GPU's SMs and how many rows an expert has.
 */
MXQ_API mxq_status nvfp4_gemv(const void* x, int64_t ldx, const uint8_t* w_q, const uint8_t* w_s,
                              const float* w_global, const int32_t* experts, int64_t T,
                              int64_t share, int64_t N, int64_t K, int64_t E, uint32_t flags,
                              void* out, int64_t ldo, uint32_t* dev_err, mxq_stream_t stream);

/*
 * mxq_product_plan -- how a product's call is cut on a GPU of num_sms SMs.  Host
 * code only: it needs no device, so that tests can name the kernel that a call
 * takes.
 *
 *   MXQ_OP_GROUPED_GEMM, MXQ_OP_GROUPED_WGRAD: the call's M, N, K, E, flags.
 *   MXQ_OP_NVFP4_GEMV: M = T * share; E = 0 stands for a call without experts.
 *   plan [7], grouped: CTAs that work on a tile; a tile's columns; 1 where few
 *           rows a group make the weight the 128-row operand; CTAs that share a
 *           tile's contraction; tiles at most; CTAs launched; 0.
 *   plan [7], nvfp4_gemv: rows of the kernel (8 or 16); blocks of 16 columns an
 *           item; CTAs that share an item's K; rows of x at a time; items at
 *           most; CTAs launched; 1 where how much of K is staged follows each
 *           expert's rows.
 * MXQ_ESHAPE for sizes that the call refuses or that make it empty.
 */
MXQ_API mxq_status mxq_product_plan(int op, int64_t M, int64_t N, int64_t K, int64_t E,
                                    uint32_t flags, int num_sms, int32_t* plan);

/*
 * mx_rmsnorm -- residual addition, RMSNorm and MXFP8 quantization in one.
 *
 * Operation, for every row m:  h = bf16(x + residual) (one fp32 addition,
 * rounded to the residual stream's type, which the backward pass reads; h = x
 * without a residual);  rstd = 1 / sqrt(mean_k h^2 + eps), the mean in fp32;
 * y = (h * rstd) * weight in fp32.  y is rounded to bf16 with MXQ_OUT_BF16, and
 * quantized, from its fp32 values, as mx_quantize_rowcol quantizes its input
 * (MXQ_ROWWISE, MXQ_COLWISE, MXQ_SCALE_RCEIL, MXQ_SCALE_SWIZZLED as there).
 *
 *   x, residual  bf16 [M][ldx], [M][ldr]; residual may be NULL.
 *   weight  [K] bf16, or fp32 with MXQ_IN_F32; 16-byte aligned.
 *   M       any, a multiple of 32 with MXQ_COLWISE; K % 32 == 0, K <= 32768.
 *   eps     > 0 and finite.
 *   flags   at least one of MXQ_ROWWISE, MXQ_COLWISE, MXQ_OUT_BF16.
 *   h       bf16 [M][ldh], NULL without a residual; may be NULL with one unless
 *           MXQ_COLWISE.  It may be x or residual itself (same pointer and
 *           stride); otherwise outputs and inputs do not overlap.
 *   rstd    [M] fp32, 16-byte aligned.
 *   y       bf16 [M][ldy] with MXQ_OUT_BF16, else ignored.
 *   q_row, s_row, q_col, s_col, dev_err, stream  as for mx_quantize_rowcol.
 * Strides are multiples of 8 elements.  Values above 2^55 overflow the sum of
 * squares (rstd and y are then 0).  M == 0 or K == 0 is a valid empty call.
 * Order: a row's results depend on the row, the weight and K alone, not on the other
 * rows nor on what else the call computes.
 */
MXQ_API mxq_status mx_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* weight, int64_t M, int64_t K, float eps, uint32_t flags,
                              void* h, int64_t ldh, float* rstd, void* y, int64_t ldy,
                              uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                              uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_rmsnorm_backward -- gradients of mx_rmsnorm (of y; the quantization is
 * passed straight through).
 *
 * Operation: with n = h * rstd and g = dy * weight,
 *   dx = dh + rstd * (g - n * mean_k(g * n)),  dweight[k] = sum_m dy * n,
 * sums in fp32, dx rounded once to bf16.  dx is the gradient of x and of the
 * residual alike; dh is the gradient that reaches h past the norm (NULL: none).
 *
 *   dy [M][lddy], h [M][ldh], dh [M][lddh], dx [M][lddx]  bf16; dx may be dy or
 *           dh itself (same pointer and stride).
 *   rstd    [M] fp32, as mx_rmsnorm wrote it.
 *   weight  [K] bf16, or fp32 with MXQ_IN_F32 (the one flag).
 *   dweight [K] fp32, 16-byte aligned, or NULL.
 *   workspace  with dweight: device memory, 16-byte aligned, at least
 *           mxq_workspace_bytes(MXQ_OP_RMSNORM_BACKWARD, M, K, 0) bytes.
 *   dev_err, stream  as for mx_quantize_rowcol.
 * M is any; K as for mx_rmsnorm.  M == 0 writes zeros to dweight.
 * Order: fixed by M, K and the GPU's SMs, so that the same call gives the same
 * bits.
 */
MXQ_API mxq_status mx_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                                       const float* rstd, const void* weight, const void* dh,
                                       int64_t lddh, int64_t M, int64_t K, uint32_t flags, void* dx,
                                       int64_t lddx, float* dweight, void* workspace,
                                       size_t workspace_bytes, uint32_t* dev_err,
                                       mxq_stream_t stream);

/*
 * mx_quantize_gated_save -- mx_quantize_gated that also writes an 8-bit
 * checkpoint of its input for the backward pass.
 *
 * Operation: q_row .. s_col as mx_quantize_gated writes them, and x_q [M][2N],
 * x_s [M][2N/32]: x = [gate | up] as mx_quantize_rowcol writes it with
 * MXQ_ROWWISE under the same scale rule (row-major scales whatever the flags).
 * The activation is that of x itself, not of the checkpoint.  Arguments as for
 * mx_quantize_gated; x_q and x_s 16-byte aligned.
 */
MXQ_API mxq_status mx_quantize_gated_save(const void* x, int64_t M, int64_t N, int64_t ldx,
                                          uint32_t flags, uint8_t* q_row, uint8_t* s_row,
                                          uint8_t* q_col, uint8_t* s_col, uint8_t* x_q,
                                          uint8_t* x_s, uint32_t* dev_err, mxq_stream_t stream);

/*
 * mx_quantize_dgated_saved -- mx_quantize_dgated with its input read from the
 * 8-bit checkpoint.
 *
 * Operation: as mx_quantize_dgated, with x[m][k] = E4M3(x_q[m][k]) *
 * 2^(x_s[m][k / 32] - 127) in fp32 (exact; a scale code of 255 is NaN).  The
 * activation and its slope come from one sigmoid s, the slope as s plus a multiple of
 * x - x s, which cancels where s is near 1: the slope (of at most 1.13) is off by up to
 * 2^-17, where mx_quantize_dgated's is by a few fp32 ulps.  A code at a rounding's
 * border may so differ from mx_quantize_dgated's.
 * x_q and x_s are those of mx_quantize_gated_save, or of mx_quantize_rowcol with
 * MXQ_ROWWISE and row-major scales.  MXQ_SCALE_SWIZZLED needs N % 128 == 0.
 */
MXQ_API mxq_status mx_quantize_dgated_saved(const void* grad, int64_t ldg, const uint8_t* x_q,
                                            const uint8_t* x_s, int64_t M, int64_t N,
                                            uint32_t flags, uint8_t* q_row, uint8_t* s_row,
                                            uint8_t* q_col, uint8_t* s_col, uint32_t* dev_err,
                                            mxq_stream_t stream);

/*
 * moe_route -- which experts take a token, and with which weights.
 *
 * Operation, for every token t: scores s_e = softmax_e(logits[t]), or
 * sigmoid(logits[t][e]) with MXQ_ROUTE_SIGMOID.  Keys are s_e + bias[e].  Of
 * `groups` groups of E / groups consecutive experts the `kept` with the largest
 * sum of their two largest keys (the one key of groups of one expert; the largest
 * key with MXQ_ROUTE_GROUP_MAX) are kept; the key of an expert that is not
 * available is -inf, so that groups with fewer than two available come last.  The
 * k experts with the largest keys of those (without a bias: with the largest
 * logits) are chosen, in that order; ties go to the lower expert or group.
 * weights[t][i] = scale * s of the i-th, divided by the sum of the k chosen scores
 * with MXQ_ROUTE_RENORM.
 * The choice is that of exact scores, as far as 64 bits tell them apart: keys are
 * computed in fp32, and again in 64 bits where fp32 does not decide.  Weights are
 * fp32; renormalised ones are ratios that hold however small the scores are.
 *
 *   logits  [T][ldl] bf16, or fp32 with MXQ_IN_F32, aligned to the element; any
 *           stride ldl >= E.  A logit of -inf (not the type's lowest value) is an
 *           expert that is not available.  A token with a NaN or +inf logit gets
 *           no experts, and NaN weights.
 *   bias    [E] fp32 or NULL; -inf makes an expert unavailable; NaN or +inf are
 *           outside the contract.
 *   E <= 512, groups <= 32, E % groups == 0, 1 <= kept <= groups,
 *   1 <= k <= 32, k <= E / groups * kept.
 *   experts [T][k] int32, what mx_grouped_gemm's offsets come from (moe_sort) and
 *           nvfp4_gemv reads; -1 with weight 0 in the slots that are left where
 *           fewer than k experts are available.
 *   weights [T][k] fp32.
 */
MXQ_API mxq_status moe_route(const void* logits, int64_t ldl, const float* bias, int64_t T,
                             int64_t E, int64_t k, int64_t groups, int64_t kept, float scale,
                             uint32_t flags, int32_t* experts, float* weights, mxq_stream_t stream);

/*
 * moe_route_backward -- the logits' gradient from the weights' (the choice itself
 * has none, nor has the bias).
 *
 *   dweights [T][k] fp32; logits, experts, k, scale and flags as for moe_route.
 *           Entries of experts outside [0, E) are skipped; an expert that has
 *           several slots of a token gets the sum of their parts.
 *   dlogits [T][ldd] in the logits' type, every element of a row's E written:
 *           zero where no gradient reaches it.
 */
MXQ_API mxq_status moe_route_backward(const float* dweights, const void* logits, int64_t ldl,
                                      const int32_t* experts, int64_t T, int64_t E, int64_t k,
                                      float scale, uint32_t flags, void* dlogits, int64_t ldd,
                                      mxq_stream_t stream);

/*
 * moe_sort -- the rows of the grouped products from the router's choice.
 *
 * Operation: pair i goes to row rows[i] of the buffer sorted by expert, pairs of
 * one expert in the order of i, every expert's first row offsets[e] a multiple of
 * `align` (32 for mx_grouped_wgrad).  A pair whose expert is not in [0, E) has row
 * -1.
 *
 *   experts [n] int32 on the device; E <= 512; 1 <= align <= 65536.
 *   rows    [n] int32.
 *   offsets [E + 1] int32: offsets[E] ends the last expert's padded rows.
 *   sizes   [E] int32 or NULL: pairs of each expert, without padding.
 *   source  [source_rows] int32 or NULL: the pair in each row, -1 in rows of none;
 *           source_rows >= n + min(n, E) * (align - 1).
 */
MXQ_API mxq_status moe_sort(const int32_t* experts, int64_t n, int64_t E, int64_t align,
                            int32_t* rows, int32_t* offsets, int32_t* sizes, int32_t* source,
                            int64_t source_rows, mxq_stream_t stream);

/*
 * mxq_selftest_bounded_wait -- launches one warp that waits on a barrier
 * nothing will ever complete, through the same bounded-wait routine the
 * quantization kernels use, with a limit of `timeout_ns` nanoseconds
 * (1e3..5e9).  The kernel ORs MXQ_DEVERR_TIMEOUT into *dev_err (required)
 * and returns, leaving the context usable.  Lets a test check the timeout
 * path without faulting or hanging a GPU.
 */
MXQ_API mxq_status mxq_selftest_bounded_wait(uint64_t timeout_ns, uint32_t* dev_err, mxq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MXQ_H */
