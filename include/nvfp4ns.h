/*
 * nvfp4ns.h — C ABI of the NVFP4 Newton–Schulz library for MI355X (gfx950).
 *
 * The operations follow "Full-Stack FP4: Stable LLM Pretraining with
 * Quantized Projections, Optimizers, and Attention" (arXiv 2607.04422):
 *   - the NVFP4 format of §2 "Preliminaries", paragraph "NVFP4 format":
 *     E2M1 element codes, one FP8 E4M3 scale s per 16-element block, one
 *     FP32 scale s_g per tensor, value = x_E2M1 * s * s_g;
 *   - the Root optimizer's Newton–Schulz iteration of §2 ("Root optimizer")
 *     in the NVFP4 form of §3.4 ("NVFP4 Root Optimizer", the three-line
 *     NVFP4 NS iteration), every quantization round-to-nearest.
 *
 * Conventions shared by every entry point
 *   - Pointers named x, codes, scales, G, out, ws, global_scale and the
 *     per-matrix arrays' elements are DEVICE pointers; coeffs, m, n, clip
 *     and the pointer arrays themselves are HOST memory.
 *   - Matrices are dense row-major with no padding.
 *   - Device arrays must be 16-byte aligned, and single device floats or
 *     words (global_scale, sg_p, sg_q, amax_out, ns_abs_quantile's out)
 *     4-byte aligned; hipMalloc and torch allocations are.  What a call
 *     writes (outputs and workspace) must not overlap what it reads or
 *     another of its outputs, except that nvfp4_gemm's addend may be out
 *     itself.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Every call
 *     only enqueues work on it and returns; nothing synchronises.  The
 *     caller owns all memory; the library allocates no device memory and
 *     keeps no data between calls (ns_orthogonalize_grouped and _ex keep
 *     only their streams; ns_orthogonalize_grouped_on keeps nothing).
 *   - Arguments are validated before anything is enqueued; a negative
 *     status means nothing was launched.  NS_ERR_HIP means a launch failed.
 *   - Data-dependent cases are defined, never errors: a NaN or infinity in
 *     a tensor makes its s_g NaN, all its scale bytes 0x7F and all its
 *     magnitude codes 0, and NaN propagates to every result; an all-zero
 *     tensor gives s_g = 0, zero scales and codes carrying only sign bits.
 *
 * NVFP4 storage (readings of the format paragraph, which prints the decode
 * rule only): s_g = RN_f32(amax / 2688); s = RNE_E4M3FN(amax_block /
 * (6 s_g)) of the exact quotient, saturating at 448 (0 if it rounds to 0);
 * code = sign | RNE_E2M1(|x| / (s s_g)) of the exact quotient, ties to the
 * even code, saturating at 6, magnitude 0 when s or s_g is 0.  Codes are
 * packed two per byte, element 2i in the low nibble; scales are E4M3FN
 * bytes, row-major [rows][cols/16].
 */
#ifndef NVFP4NS_H
#define NVFP4NS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NS_OK = 0,
  NS_ERR_ARG = -1,        /* null pointer, bad enum, k <= 0, clip NaN or <= 0, a
                             misaligned pointer, overlapping arrays */
  NS_ERR_SHAPE = -2,      /* a dimension <= 0 or not a multiple of 16, or a matrix of
                             2^31 or more elements in ns_orthogonalize / nvfp4_gemm */
  NS_ERR_WORKSPACE = -3,  /* ws is NULL or ws_bytes is below the required size */
  NS_ERR_HIP = -4         /* a kernel launch failed */
} ns_status;

typedef enum { NS_F32 = 0, NS_BF16 = 1 } ns_dtype;

/* NVFP4_ROWS: Q_1x16, blocks of 16 consecutive elements along each row.
 * NVFP4_COLS: Q_16x1, blocks of 16 down each column, stored as the Q_1x16
 * layout of the transpose (cols rows of rows/2 code bytes and rows/16
 * scale bytes). */
typedef enum { NVFP4_ROWS = 0, NVFP4_COLS = 1 } nvfp4_axis;

/* Workspace of nvfp4_quantize, nvfp4_quantize_rht and nvfp4_quantize_46, in
 * bytes (the partial tensor maxima: 2 KiB, independent of the shape). */
size_t nvfp4_quantize_workspace_bytes(int64_t rows, int64_t cols);

/*
 * nvfp4_quantize — Q_1x16 or Q_16x1 of a rows x cols matrix
 * (§2 "NVFP4 format"; the quantizers Q_1x16 / Q_16x1 of §3.4).
 *   x            [rows][cols] FP32 or BF16 (xt), read only.
 *   codes        out, rows*cols/2 bytes.
 *   scales       out, rows*cols/16 bytes.
 *   global_scale out, one float (s_g).
 *   ws           scratch of nvfp4_quantize_workspace_bytes(); contents on
 *                entry are ignored.
 * rows and cols must be positive multiples of 16.
 */
ns_status nvfp4_quantize(const void* x, ns_dtype xt, int64_t rows, int64_t cols,
                         nvfp4_axis axis, uint8_t* codes, uint8_t* scales,
                         float* global_scale, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * nvfp4_quantize_noalloc — nvfp4_quantize without a workspace argument, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  Its scratch, the
 * nvfp4_quantize_workspace_bytes() (2 KiB) of partial tensor maxima, lives in
 * a static device array of 2 KiB that each GPU the library runs on holds
 * until the process ends; the call allocates nothing.  Every call on one GPU
 * shares that array: calls that overlap on one GPU (concurrent streams)
 * race and must be ordered by the caller.  The array is cleared by a kernel
 * of each call.  Arguments, layouts, results and errors as nvfp4_quantize;
 * NS_ERR_WORKSPACE if a shape ever needed more scratch than the array holds
 * (none does: the scratch does not grow with the tensor); NS_ERR_HIP if the
 * array's device address cannot be obtained.
 */
ns_status nvfp4_quantize_noalloc(const void* x, ns_dtype xt, int64_t rows, int64_t cols,
                                 nvfp4_axis axis, uint8_t* codes, uint8_t* scales,
                                 float* global_scale, void* stream);

/*
 * nvfp4_quantize_rht — the quantizers of the §3.4 NS iteration with the
 * random Hadamard transform: Q_1x16(x H) (NVFP4_ROWS) or Q_16x1(H^T x)
 * (NVFP4_COLS, stored as the Q_1x16 layout of the transpose), where
 * H = H_16^r acts on every 16-block along the blocked axis.
 *   mask  H_16^r = diag(s) H_16 / 4 with H_16 the Sylvester Hadamard matrix,
 *         s_j = -1 where bit j of mask is set, else +1.
 *   The transformed values are computed in FP32 by the radix-2 butterfly:
 *   signs applied, then half-widths 1, 2, 4, 8, each pair (a, b) becoming
 *   (a + b, a - b) rounded to nearest even, then times 1/4.  The tensor
 *   scale s_g is that of the transformed tensor.
 * Other arguments, layout and errors as nvfp4_quantize.  nvfp4_dequantize
 * of the result returns the transformed tensor's approximation (the
 * transform is not undone).
 */
ns_status nvfp4_quantize_rht(const void* x, ns_dtype xt, int64_t rows, int64_t cols,
                             nvfp4_axis axis, uint16_t mask, uint8_t* codes, uint8_t* scales,
                             float* global_scale, void* ws, size_t ws_bytes, void* stream);

/*
 * nvfp4_quantize_46 — nvfp4_quantize with adaptive 4/6 block scaling, the
 * quantization the Root iteration uses (Full-Stack FP4 §3.4: RTN with
 * adaptive 4/6 scaling; §5: adaptive M = 4 / M = 6 block scaling of Four
 * Over Six).  Each block is encoded twice, with its maximum mapped to 6
 * (s = RNE_E4M3FN(amax_b / (6 s_g)), as nvfp4_quantize) and to 4
 * (s = RNE_E4M3FN(amax_b / (4 s_g)), saturating at 448), and keeps the
 * encoding whose squared error sum (x - q s s_g)^2 -- each operation rounded
 * in double, elements in order -- is smaller; M = 6 on ties.  s_g, the
 * layouts, the decode rule and the errors are those of nvfp4_quantize.
 */
ns_status nvfp4_quantize_46(const void* x, ns_dtype xt, int64_t rows, int64_t cols,
                            nvfp4_axis axis, uint8_t* codes, uint8_t* scales,
                            float* global_scale, void* ws, size_t ws_bytes, void* stream);

/*
 * nvfp4_dequantize — x_hat = x_E2M1 * s * s_g (§2 "NVFP4 format").
 * Inputs as written by nvfp4_quantize for the same rows, cols and axis;
 * out is [rows][cols] in the ORIGINAL orientation (an NVFP4_COLS tensor is
 * transposed back), FP32 or BF16 (ot), each value rounded once (RNE) from
 * the exact product.
 */
ns_status nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales,
                           const float* global_scale, int64_t rows, int64_t cols,
                           nvfp4_axis axis, void* out, ns_dtype ot, void* stream);

/*
 * nvfp4_gemm — one NVFP4 product of the §3.4 iteration, C = P * Q^T with
 * both operands in the Q_1x16 layout along the contraction axis K:
 *   P: codes_p [M][K/2], scales_p [M][K/16], s_g at sg_p (device float)
 *   Q: codes_q [N][K/2], scales_q [N][K/16], s_g at sg_q
 * and the epilogue
 *   out[i][j] = beta * addend[i][j] + alpha * s_gP * s_gQ * sum_k P_ik Q_jk
 * with products of dequantized values exact and FP32 accumulation.
 *   symmetric != 0: P and Q must be the same tensor (M == N); only the
 *     upper triangle is computed and mirrored, so out is exactly symmetric
 *     (the Gram products A = qX qX^T and qA qA^T).
 *   addend may be NULL when beta == 0, and may equal out.
 *   amax_out (device uint32, may be NULL): atomically maxed with the bit
 *     pattern of |out| (non-finite values count as NaN); the caller zeroes it.
 *   ws: device scratch of nvfp4_gemm_workspace_bytes(); it lets the tiles
 *     left over after an equal number per CU be split along K across
 *     workgroups (FP32 partials summed in a fixed order, so results do not
 *     depend on timing).  ws = NULL, ws_bytes = 0 runs every tile whole.
 *     Calls sharing one ws must not overlap.  ws must be ordinary device
 *     memory of the GPU that runs the call (hipMalloc, a torch tensor):
 *     within one launch the K-parts of a tile hand their partials to the
 *     part that sums them through ws, with stores and loads coherent at
 *     device scope and a device-scope counter, which relies on ws being
 *     device-local memory.
 * M, N, K must be positive multiples of 16.
 */
size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int symmetric);
ns_status nvfp4_gemm(const uint8_t* codes_p, const uint8_t* scales_p, const float* sg_p,
                     const uint8_t* codes_q, const uint8_t* scales_q, const float* sg_q,
                     int64_t M, int64_t N, int64_t K, int symmetric,
                     float alpha, float beta, const float* addend,
                     float* out, uint32_t* amax_out, void* ws, size_t ws_bytes,
                     void* stream);

/* Workspace of ns_orthogonalize for one m x n matrix, in bytes. */
size_t ns_workspace_bytes(int64_t m, int64_t n);

/*
 * ns_workspace_map — where ns_orthogonalize (and its _rht / _ex variants)
 * keeps the iteration's operands inside its workspace, as byte offsets from
 * ws.  An inspection aid (tests, debugging); the kernels need nothing from
 * the caller beyond ns_workspace_bytes().  The iterate is xm x xn with
 * xm = min(m, n), xn = max(m, n) (G^T when m > n).
 *   x                  FP32 X [xm][xn]
 *   a, b               FP32 A and B [xm][xm]; only the elements with
 *                      row <= col are written (A and B are symmetric)
 *   qx_codes/_scales   Q_1x16(X [H]): [xm][xn/2] codes, [xm][xn/16] scales
 *   qt_codes/_scales   Q_16x1([H^T] X) stored as rows of X^T: [xn][xm/2], [xn][xm/16]
 *   qa_codes/_scales   Q_1x16(A [H]): [xm][xm/2], [xm][xm/16]
 *   qb_codes/_scales   Q_1x16(B [H]): likewise
 *   global_scales      4 floats: s_g of qX, qA, qB, and of qX16 under the
 *                      transform (without it qX16 uses s_g of qX)
 * After a call of k steps these hold the last step's values: its input
 * iterate X_{k-1} in x when the call is untransposed with FP32 output (the
 * last product writes `out` directly), else X_k; the last step's A, B and
 * every quantized operand of that step.
 * Returns NS_ERR_SHAPE for shapes ns_orthogonalize rejects, NS_ERR_ARG for
 * map == NULL.
 */
typedef struct {
  int64_t xm, xn;
  size_t x, a, b;
  size_t qx_codes, qx_scales, qt_codes, qt_scales;
  size_t qa_codes, qa_scales, qb_codes, qb_scales;
  size_t global_scales;
  size_t total;             /* == ns_workspace_bytes(m, n) */
} ns_workspace_map;
ns_status ns_workspace_layout(int64_t m, int64_t n, ns_workspace_map* map);

/*
 * ns_orthogonalize — k NVFP4 Newton–Schulz steps (§2 "Root optimizer",
 * §3.4 NVFP4 NS iteration) on one matrix:
 *   X_0 = clamp(G, -clip, clip) / (||clamp(G)||_F + 1e-7)     (on G^T if m > n)
 *   for i < k:  A = qX qX^T;  B = b_i A + c_i qA qA^T;  X = a_i X + qB qX16
 *   out = X (transposed back if m > n)
 *   G      [m][n] FP32 or BF16 (gt), read only.
 *   coeffs HOST array of k triples (a_i, b_i, c_i).
 *   clip   > 0; +inf disables clipping.  NaN passes through the clamp.
 *   out    [m][n] FP32 or BF16 (ot); must not overlap G or ws.
 *   ws     device scratch of ns_workspace_bytes(m, n).
 */
ns_status ns_orthogonalize(const void* G, ns_dtype gt, int64_t m, int64_t n,
                           const float* coeffs, int k, float clip,
                           void* out, ns_dtype ot, void* ws, size_t ws_bytes,
                           void* stream);

/*
 * ns_orthogonalize_rht — ns_orthogonalize with the random Hadamard transform
 * of the §3.4 iteration on every quantized operand:
 *   qX = Q_1x16(X H), qX16 = Q_16x1(H^T X), A = qX qX^T
 *   qA = Q_1x16(A H), qA16 = Q_16x1(H^T A), B = b A + c qA qA16
 *   qB = Q_1x16(B H), X' = a X + qB qX16
 * with H = H_16^r of step i built from masks[i] as in nvfp4_quantize_rht
 * (H H^T = I, so each product still approximates the untransformed one).
 *   masks  HOST array of k 16-bit sign masks, one per step (not NULL).
 * X H and H^T X each take their own s_g.  Other arguments, workspace
 * (ns_workspace_bytes) and errors as ns_orthogonalize.
 */
ns_status ns_orthogonalize_rht(const void* G, ns_dtype gt, int64_t m, int64_t n,
                               const float* coeffs, int k, float clip, const uint16_t* masks,
                               void* out, ns_dtype ot, void* ws, size_t ws_bytes, void* stream);

/*
 * ns_abs_quantile — the q-quantile of |x| over `count` elements, the clip
 * threshold of the NVFP4 Root path (§3.4 "p99 outlier clipping"; App. F
 * Table 8 "Root quantile ratio 0.99"), read as an order statistic: the k-th
 * smallest magnitude, k = ceil(q * count) computed in double and clamped to
 * [1, count].  Magnitudes are ordered by their FP32 bit patterns with the
 * sign cleared (BF16 widened exactly); NaN and infinity count as NaN, above
 * every finite value, so a result that reaches them is NaN.
 *   x      device, `count` FP32 or BF16 (xt) values, read only.
 *   q      in (0, 1].
 *   out    device, one float (written when the enqueued work runs).
 *   ws     device scratch of ns_abs_quantile_workspace_bytes() (256 KiB).
 * count must be a positive multiple of 16 below 2^31.
 */
size_t ns_abs_quantile_workspace_bytes(void);
ns_status ns_abs_quantile(const void* x, ns_dtype xt, int64_t count, double q, float* out,
                          void* ws, size_t ws_bytes, void* stream);

/* Options of ns_orthogonalize_ex. */
typedef struct {
  float clip;               /* as in ns_orthogonalize; ignored when clip_quantile > 0 */
  double clip_quantile;     /* 0: use clip.  In (0, 1]: clip = the clip_quantile-quantile
                               of |G| (as ns_abs_quantile), found on the device */
  const uint16_t* rht_masks;/* NULL, or a HOST array of k masks (as ns_orthogonalize_rht) */
  int adaptive46;           /* nonzero: every quantization of the iteration uses adaptive
                               4/6 block scaling (as nvfp4_quantize_46) */
} ns_options;

/*
 * ns_orthogonalize_ex — ns_orthogonalize with the clip threshold taken on
 * the device as a quantile of |G|, the random Hadamard transform and/or
 * adaptive 4/6 block scaling, as set in `opt` (HOST pointer, not NULL).
 * NS_ERR_ARG for a clip_quantile outside {0} U (0, 1].  Workspace
 * ns_workspace_bytes(m, n); other arguments and errors as ns_orthogonalize.
 */
ns_status ns_orthogonalize_ex(const void* G, ns_dtype gt, int64_t m, int64_t n,
                              const float* coeffs, int k, const ns_options* opt, void* out,
                              ns_dtype ot, void* ws, size_t ws_bytes, void* stream);

/* Workspace of ns_orthogonalize_grouped for `count` matrices (host arrays m, n). */
size_t ns_grouped_workspace_bytes(int count, const int64_t* m, const int64_t* n);

/*
 * ns_orthogonalize_grouped — ns_orthogonalize on `count` independent
 * matrices with one coefficient schedule, as one batch of launches.
 *   G, out  HOST arrays of `count` device pointers.
 *   m, n    HOST arrays of shapes.   clip  HOST array of per-matrix clips.
 *   ws      device scratch of ns_grouped_workspace_bytes() (one part per
 *           matrix).
 * Matrices that share an iterate shape (min(m, n) x max(m, n), either
 * orientation) run in batches: each pass of a step is one launch for
 * several of them, each matrix on its single call's kernels and tile
 * schedule.  The batches run concurrently on up to four library-owned
 * streams of the current device (default priority, created on the first
 * grouped call and kept until the process ends), forked from `stream`
 * through an event and
 * joined back into it: the call is ordered on `stream` like any other and
 * can be captured into a graph.  Each result equals its single call's bit
 * for bit.  Calls that overlap on one device share the streams.
 */
ns_status ns_orthogonalize_grouped(int count, const void* const* G, const int64_t* m,
                                   const int64_t* n, ns_dtype gt, const float* coeffs,
                                   int k, const float* clip, void* const* out,
                                   ns_dtype ot, void* ws, size_t ws_bytes, void* stream);

/*
 * ns_orthogonalize_grouped_ex — ns_orthogonalize_grouped with the options of
 * ns_orthogonalize_ex shared by every matrix: with opt->clip_quantile > 0
 * each matrix is clipped at that quantile of its own |G| (clip may then be
 * NULL), else at clip[i]; opt->rht_masks (k masks) and opt->adaptive46
 * apply to every matrix.
 * Workspace ns_grouped_workspace_bytes(); concurrency and ordering as for
 * ns_orthogonalize_grouped.
 */
ns_status ns_orthogonalize_grouped_ex(int count, const void* const* G, const int64_t* m,
                                      const int64_t* n, ns_dtype gt, const float* coeffs, int k,
                                      const float* clip, const ns_options* opt, void* const* out,
                                      ns_dtype ot, void* ws, size_t ws_bytes, void* stream);

/*
 * ns_orthogonalize_grouped_on — ns_orthogonalize_grouped_ex on streams the
 * caller owns: the matrices run on streams[0 .. nstreams-1] (hipStream_t
 * values, 1 <= nstreams <= 16, none NULL), forked from `stream` through an
 * event and joined back into it, so the call is ordered on `stream` (work
 * already queued on the given streams runs before their share) and can be
 * captured into a graph.  The library keeps nothing between calls.  opt may
 * be NULL: clip[i] per matrix, no transform, no 4/6.  Results equal
 * ns_orthogonalize_grouped_ex's bit for bit.  NS_ERR_ARG for a bad stream
 * list; other arguments and errors as ns_orthogonalize_grouped_ex.
 */
ns_status ns_orthogonalize_grouped_on(int count, const void* const* G, const int64_t* m,
                                      const int64_t* n, ns_dtype gt, const float* coeffs, int k,
                                      const float* clip, const ns_options* opt, void* const* out,
                                      ns_dtype ot, void* ws, size_t ws_bytes,
                                      void* const* streams, int nstreams, void* stream);

/* ======================================================================
 * MXFP4: 4-bit values with power-of-two block scales, the 4-bit format
 * that gfx950's matrix instructions multiply themselves.
 *
 * A block is 32 consecutive elements along the blocked axis: E2M1 codes and
 * one E8M0 byte b, value = x_E2M1 * 2^(b - 127); b = 255 makes the block
 * NaN.  There is no tensor scale, so a block's encoding depends on the block
 * alone (one pass; the same bytes whatever surrounds it):
 *   b = max(floor(log2 max|x|) - 2 + 127, 0) (0 for an all-zero block),
 *   code = sign | RNE_E2M1(|x| / 2^(b - 127)), ties to the even code, values
 *   of 5 and more (up to 8 occur) becoming 6;
 *   a block with a NaN or an infinity: b = 255, codes 0.
 *
 * Storage ("panels"): rows are cut along the blocked axis into panels of 256
 * elements; codes are [panels][rows][128] bytes, two codes a byte, element
 * 2i in the low nibble, scales [panels][rows][8] bytes, with
 * panels = ceil(length / 256).  Behind a row's end a panel holds all-zero
 * blocks (codes 0; b = 0 for blocks without elements).  NVFP4_COLS stores the
 * transpose: its rows are the matrix's columns.
 *
 * Dimensions are 1 .. 2^24, of any parity, a matrix up to 2^36 elements.
 * ====================================================================== */
size_t mxfp4_codes_bytes(int64_t rows, int64_t cols, nvfp4_axis axis);
size_t mxfp4_scales_bytes(int64_t rows, int64_t cols, nvfp4_axis axis);

/*
 * mxfp4_quantize — a rows x cols matrix to MXFP4, blocked along its rows
 * (NVFP4_ROWS) or down its columns (NVFP4_COLS).
 *   x       [rows][cols] FP32 or BF16 (xt), read only.
 *   codes   out, mxfp4_codes_bytes();  scales  out, mxfp4_scales_bytes().
 */
ns_status mxfp4_quantize(const void* x, ns_dtype xt, int64_t rows, int64_t cols, nvfp4_axis axis,
                         uint8_t* codes, uint8_t* scales, void* stream);

/*
 * mxfp4_quantize_both — both of the above in one pass over x: what training
 * needs of activations, gradients and weights, which are contracted along one
 * axis forward and along the other backward.  Same bytes as two calls.
 */
ns_status mxfp4_quantize_both(const void* x, ns_dtype xt, int64_t rows, int64_t cols,
                              uint8_t* codes_rows, uint8_t* scales_rows, uint8_t* codes_cols,
                              uint8_t* scales_cols, void* stream);

/*
 * mxfp4_dequantize — the values, [rows][cols] in the original orientation,
 * FP32 or BF16 (ot); both hold every MXFP4 value exactly.
 */
ns_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                           nvfp4_axis axis, void* out, ns_dtype ot, void* stream);

/*
 * mxfp4_gemm — out = beta * addend + alpha * P Q^T, P [M][K] and Q [N][K] in
 * MXFP4 blocked along K, products exact and accumulated in FP32.
 *   addend  [M][N] FP32; NULL when beta == 0; may be out itself when ot is
 *           NS_F32.
 *   out     [M][N] FP32 or BF16 (ot), rounded once.
 *   ws      device scratch of mxfp4_gemm_workspace_bytes(), through which
 *           tiles split along K pass FP32 partials, summed in a fixed order;
 *           NULL with ws_bytes 0 runs every tile whole.  Calls sharing one ws
 *           must not overlap.
 * A NaN block makes the rows (columns) of out that it meets NaN.
 */
size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
ns_status mxfp4_gemm(const uint8_t* codes_p, const uint8_t* scales_p, const uint8_t* codes_q,
                     const uint8_t* scales_q, int64_t M, int64_t N, int64_t K, float alpha,
                     float beta, const float* addend, void* out, ns_dtype ot, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * mxfp4_linear — y = Q(x) w^T for T tokens: x [T][K] FP32 or BF16, quantized
 * along K by the call, w [N][K] in MXFP4 (NVFP4_ROWS), y [T][N] FP32 or BF16.
 *   kept_codes, kept_scales  both NULL, or out: x quantized along the tokens
 *           (NVFP4_COLS), which mxfp4_linear_backward takes for the weights'
 *           gradient.
 *   ws      device scratch of mxfp4_linear_workspace_bytes().
 */
size_t mxfp4_linear_workspace_bytes(int64_t T, int64_t N, int64_t K);
ns_status mxfp4_linear(const void* x, ns_dtype xt, int64_t T, int64_t K, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t N, void* y, ns_dtype yt,
                       uint8_t* kept_codes, uint8_t* kept_scales, void* ws, size_t ws_bytes,
                       void* stream);

/*
 * mxfp4_linear_backward — the gradients of mxfp4_linear with the quantizers'
 * own derivative taken as 1 (straight through):
 *   dx [T][K] = Q_N(dy) w         Q_N: along N, w along N (wt)
 *   dw [N][K] = beta dw + Q_T(dy)^T Q_T(x)   Q_T: along the tokens
 *   dy      [T][N] FP32 or BF16.
 *   wt      the weights quantized down their columns (NVFP4_COLS of [N][K]);
 *           may be NULL when dx is.
 *   kept    as written by mxfp4_linear; may be NULL when dw is.
 *   dx, dw  FP32 or BF16; either may be NULL.  beta != 0 adds to what dw
 *           holds and needs FP32.
 *   ws      device scratch of mxfp4_linear_backward_workspace_bytes().
 */
size_t mxfp4_linear_backward_workspace_bytes(int64_t T, int64_t N, int64_t K);
ns_status mxfp4_linear_backward(const void* dy, ns_dtype dyt, int64_t T, int64_t N, int64_t K,
                                const uint8_t* wt_codes, const uint8_t* wt_scales,
                                const uint8_t* kept_codes, const uint8_t* kept_scales, void* dx,
                                ns_dtype dxt, void* dw, ns_dtype dwt, float beta, void* ws,
                                size_t ws_bytes, void* stream);

/* ======================================================================
 * Newton–Schulz without quantization: f16 operands, FP32 accumulation.
 *   X_0 = clamp(G, -clip, clip) / (||clamp(G)||_F + 1e-7)    (on G^T if m > n)
 *   A = X X^T;  B = a I + b A + c A A;  X <- B X
 * X (times 256), A and B are rounded to f16 once per step, and what that
 * takes from A's and B's diagonals is put back in FP32; BF16 sources enter
 * without rounding.  The rounding of X leaves an error of 2e-4 of its norm,
 * spread evenly over all directions, and the steps amplify it there as they
 * amplify X: small directions by up to the product of the a's (485 for five
 * quintic steps).  What five quintic steps are off by (relative Frobenius norm,
 * before the output's own rounding) therefore goes by the spectrum of G:
 *   singular values alike                     0.4e-3 to 2e-3
 *   spread evenly (log scale) over a decade   1e-3
 *   over two decades                          2e-3 to 4e-3
 *   over three decades                        3e-3 (2048 rows) to 1.5e-2 (16)
 *   up to 32 above a floor of 1/100 of them   0.5e-3 (2048 rows) to 1.5e-2
 *   the same, a floor of 1/1000               0.5e-2 to 6e-2
 * and it is at most 2e-3 + 0.2 / ||X_k||_F.  BF16 sources, without the rounding
 * of X_0, are off by up to 40% less.  |X| beyond 255 (divergent coefficients)
 * overflows to infinities and NaN.  NaN or infinity in a matrix makes
 * its result NaN; a zero matrix gives zero.  Dimensions are 1 .. 2^24, of any
 * parity, m * n < 2^31.
 * ====================================================================== */

/* Workspace of the calls below for `count` matrices, in bytes (matrices of one
 * shape run as a batch; different shapes share it one after another). */
size_t ns_f16_workspace_bytes(int count, const int64_t* m, const int64_t* n);

/* ns_orthogonalize_f16 — one matrix; arguments as ns_orthogonalize, workspace
 * ns_f16_workspace_bytes(1, &m, &n). */
ns_status ns_orthogonalize_f16(const void* G, ns_dtype gt, int64_t m, int64_t n, const float* coeffs,
                               int k, float clip, void* out, ns_dtype ot, void* ws, size_t ws_bytes,
                               void* stream);

/* ns_orthogonalize_f16_grouped — `count` matrices, arguments as
 * ns_orthogonalize_grouped (clip may be NULL: no clipping), everything on
 * `stream`.  A matrix's result may differ from its single call's in the last
 * bits: products are split along K by the batch's size. */
ns_status ns_orthogonalize_f16_grouped(int count, const void* const* G, const int64_t* m,
                                       const int64_t* n, ns_dtype gt, const float* coeffs, int k,
                                       const float* clip, void* const* out, ns_dtype ot, void* ws,
                                       size_t ws_bytes, void* stream);

/* Options of ns_muon_step. */
typedef struct {
  float lr, momentum, weight_decay;
  int nesterov;             /* nonzero: U = G + momentum M, else U = M */
} ns_muon_options;

/*
 * ns_muon_step — one Muon step on `count` weight matrices:
 *   M <- momentum M + G                      (stored in M's type)
 *   U = G + momentum M  or  M                (M as stored)
 *   W <- (1 - lr weight_decay) W - lr scale_i NS(U)
 * with NS the k steps above (no clipping): f16 operands, off by what the list
 * above says for U's spectrum.  U itself is FP32.
 *   W, M    HOST arrays of device pointers, updated in place, FP32 or BF16
 *           (wt, mt); G likewise (gt), read only.  m, n  HOST arrays.
 *   scale   HOST array of one factor per matrix (such as
 *           0.2 sqrt(max(m, n))), or NULL: 1.
 *   ws      device scratch of ns_f16_workspace_bytes().
 * No array may overlap another.  A NaN or infinity in U makes W NaN.
 */
ns_status ns_muon_step(int count, void* const* W, ns_dtype wt, void* const* M, ns_dtype mt,
                       const void* const* G, ns_dtype gt, const int64_t* m, const int64_t* n,
                       const float* coeffs, int k, const ns_muon_options* opt, const float* scale,
                       void* ws, size_t ws_bytes, void* stream);

/* ======================================================================
 * Between two 4-bit linear layers: the root-mean-square norm with the
 * residual's addition and dropout in front, activations in 8 bits, and
 * products with 4-bit weights.
 *
 * MXFP8: a block is 32 consecutive elements along a row, E4M3FN codes and one
 * E8M0 byte b, value = x_E4M3 * 2^(b - 127); b = 255 makes the block NaN.
 *   b = max(floor(log2 max|x|) - 8 + 127, 0) (0 for an all-zero block),
 *   code = RNE_E4M3(x / 2^(b - 127)), ties to the even code, magnitudes beyond
 *   448 (up to 512 occur) becoming 448;
 *   a block with a NaN or an infinity: b = 255, codes 0.
 * Storage as MXFP4's, in panels of 256 elements: codes [panels][rows][256]
 * bytes, scales [panels][rows][8]; all-zero blocks behind a row's end.
 *
 * Dropout: random bits come from Philox4x32-10 with `rng`, a DEVICE array of
 * two 64-bit words, as seed and offset, read when the call runs (a captured
 * call draws anew after the words change).  Element (t, c) takes half c % 2 of
 * word c / 2 % 4 (low half first) of the counter (c / 8, t, offset low, offset
 * high) under the key (seed low, seed high); it is kept where these 16 bits are
 * at least P = floor(65536 p + 1/2), and what is kept is multiplied by
 * 65536 / (65536 - P) (in FP32), so that means are kept exactly.  The mask is
 * never stored: a backward pass draws the same bits again.  0 <= p < 1 with
 * P < 65536; p = 0 keeps everything.
 *
 * Dimensions are 1 .. 2^24, of any parity, a matrix up to 2^36 elements.
 * ====================================================================== */

/*
 * mx_dropout — out = k x / (1 - p), [rows][cols] FP32 or BF16; also its own
 * gradient (of dy, with the same p and rng).  out may be x itself.
 */
ns_status mx_dropout(const void* x, ns_dtype xt, int64_t rows, int64_t cols, double p, const void* rng,
                     void* out, void* stream);

/*
 * mx_rms_norm — h = residual + k x / (1 - p);  y = h / sqrt(mean(h^2) + eps) weight
 * row by row.  h is rounded to its type first and normed as stored; the sum
 * runs in FP64 and r = 1 / sqrt(..) is rounded to FP32 once, y is the FP32
 * product (h r) weight, so that codes do not depend on how a row was split.
 *   x        [T][C] FP32 or BF16 (xt).
 *   residual [T][C] of type ht, or NULL: none.
 *   weight   [C] FP32 or BF16 (wt).
 *   h        out [T][C] FP32 or BF16 (ht), the new residual stream; may be
 *            residual itself.  NULL without residual and dropout (then h is x,
 *            and ht has to be xt).
 *   rstd     out [T] FP32, r of each row for the backward pass; or NULL.
 *   y        out [T][C] FP32 or BF16 (yt); or NULL.
 *   codes8, scales8          out, y in MXFP8 (mxfp8_codes_bytes(T, C)); or NULL.
 *   codes4, scales4          out, y in MXFP4 along the rows; or NULL.
 *   kept_codes, kept_scales  out, y in MXFP4 along the tokens (NVFP4_COLS), as
 *            mxfp4_linear_backward takes it for the weights' gradient; or NULL.
 *            Needs rstd.
 *   eps      at least 2^-254 (so that r is finite), finite.  drop, rng: as above;
 *            rng may be NULL when drop is 0.
 * C is at most 32768, T below 2^22 where C is more than 1024.  At least one
 * output is needed.  A NaN in h makes NaN of its whole row of y; an infinity
 * becomes NaN and its row's finite values 0; a block that holds a NaN is NaN.
 */
typedef struct {
  const void* x;
  const void* residual;
  const void* weight;
  const void* rng;
  void* h;
  float* rstd;
  void* y;
  uint8_t *codes8, *scales8, *codes4, *scales4, *kept_codes, *kept_scales;
  int64_t T, C;
  double eps, drop;
  ns_dtype xt, ht, wt, yt;
} mx_norm_args;
ns_status mx_rms_norm(const mx_norm_args* args, void* stream);

/*
 * mx_rms_norm_backward — the gradients of mx_rms_norm (a quantizer's derivative
 * taken as 1), with u = h r as stored by the forward call:
 *   dh = dh_in + r (weight dy - u mean(weight dy u))
 *   dx = k dh / (1 - p), of dh before its rounding
 *   dweight = beta dweight + sum over the rows of dy u
 *   dy       [T][C] FP32 or BF16 (dyt), the gradient of y.
 *   h        as written by the forward call (x where that had no h).
 *   dh_in    [T][C] of ht, what reaches h by other ways (the residual stream);
 *            or NULL: nothing.
 *   dh       out [T][C] of ht, the gradient of h and of residual; may be dh_in.
 *   dx       out [T][C] FP32 or BF16 (xt), the gradient of x; or NULL (without
 *            dropout it is dh).
 *   dweight  out [C] FP32; or NULL.  The sum's order is fixed.
 *   ws       device scratch of mx_rms_norm_backward_workspace_bytes(); not
 *            needed without dweight.
 */
typedef struct {
  const void* dy;
  const void* h;
  const float* rstd;
  const void* weight;
  const void* dh_in;
  const void* rng;
  void* dh;
  void* dx;
  float* dweight;
  int64_t T, C;
  double drop;
  float beta;
  ns_dtype dyt, ht, wt, xt;
} mx_norm_backward_args;
size_t mx_rms_norm_backward_workspace_bytes(int64_t T, int64_t C);
ns_status mx_rms_norm_backward(const mx_norm_backward_args* args, void* ws, size_t ws_bytes, void* stream);

/* mxfp8_quantize — a rows x cols matrix, FP32 or BF16 (xt), to MXFP8 along its
 * rows; mxfp8_dequantize — the values, FP32 (exact) or BF16 (exact but for
 * subnormals; ot). */
size_t mxfp8_codes_bytes(int64_t rows, int64_t cols);
size_t mxfp8_scales_bytes(int64_t rows, int64_t cols);
ns_status mxfp8_quantize(const void* x, ns_dtype xt, int64_t rows, int64_t cols, uint8_t* codes,
                         uint8_t* scales, void* stream);
ns_status mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                           void* out, ns_dtype ot, void* stream);

/*
 * mxfp8_gemm — out = beta * addend + alpha * P Q^T, P [M][K] in MXFP8
 * (activations) and Q [N][K] in MXFP4 (weights), both along K; arguments as
 * mxfp4_gemm.  FP32 outputs, and all of up to 16 rows: products are exact and
 * accumulated in FP32.  BF16 outputs of more rows: the matrix instruction adds
 * the products of eight neighbours of K in a window that ends 2^13 below the
 * largest one's leading bit, so that each of the others loses up to 2^-13 of
 * that; sums of these are FP32.
 *   ws       device scratch of mxfp8_gemm_workspace_bytes(), or NULL with
 *            ws_bytes 0 (slower where a long K feeds few outputs).
 */
size_t mxfp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
ns_status mxfp8_gemm(const uint8_t* codes_p, const uint8_t* scales_p, const uint8_t* codes_q,
                     const uint8_t* scales_q, int64_t M, int64_t N, int64_t K, float alpha, float beta,
                     const float* addend, void* out, ns_dtype ot, void* ws, size_t ws_bytes, void* stream);

/*
 * nvfp4_linear — y = x W^T for T tokens, W [N][K] in NVFP4 along its rows
 * (codes, scales and global scale as nvfp4_quantize writes them for
 * NVFP4_ROWS), x [T][K] FP32 or BF16 as it is: the layer of a program that
 * serves from NVFP4 weights, built for few tokens (the weights are read once
 * for every 32, or 16 in FP32).  K is a multiple of 16, N of any size, T * N at
 * most 2^30.  Products are exact for BF16 x and within FP32's own rounding
 * otherwise (of an FP32 x, what lies below 2^-133 is cut off), sums in FP32 and
 * of s_g's magnitude: they leave FP32 where sums of x W do.
 */
ns_status nvfp4_linear(const void* x, ns_dtype xt, int64_t T, int64_t K, const uint8_t* w_codes,
                       const uint8_t* w_scales, const float* w_global_scale, int64_t N, void* y,
                       ns_dtype yt, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4NS_H */
