/*
 * mxfp8moe.h -- C ABI of the MXFP8 MoE expert grouped-GEMM library (gfx950).
 *
 * The hot path of an MoE expert linear layer on MXFP8 data, as described on
 * the NVIDIA TransformerEngine pull-request pages
 *   [P3244] "[Pytorch] Add support for row-wise quanted input for grouped gemm"
 *   [P3545] "[PyTorch] Fix distributed BF16 weights and trim NVFP4 saved state
 *            in the fused grouped MLP"
 *   [P3224] "Improve device-init grouped linear module with single grouped
 *            weight support"
 * with the MXFP8 arithmetic of the OCP Microscaling Formats (MX) v1.0
 * specification (sections 5 and 6.3), which the pages leave unstated.
 *
 * Formats and conventions used by every entry point
 * -------------------------------------------------
 *  - bf16 tensors are passed as their 16-bit patterns (uint16_t).
 *  - MXFP8 data bytes are E4M3 ("FN": max 448, no infinity) and scale bytes
 *    are E8M0 (value 2^(u-127)).  A block of 32 values shares one scale:
 *      X = floor(log2(max|v|)) - 8, clamped to [-127, 127] (0 for an all-zero
 *      block, i.e. byte 0); each element is the E4M3 value nearest to v/2^X,
 *      ties to the even code, saturating at +-448; the sign of zero is kept.
 *  - Row-wise data of a [R, C] tensor: bytes [R, C] row-major, scales
 *    [R, C/32] row-major, blocks of 1 x 32 along C ([P3244] Description).
 *  - Column-wise data of a [R, C] tensor (blocks of 32 x 1 along R) is stored
 *    transposed: bytes [C, R] and scales [C, R/32], both row-major.  It is the
 *    copy the wgrad GEMM reads ([P3244] Greptile Summary flowchart;
 *    [P3545] Description: every wgrad path takes the column-wise tiles).
 *  - bf16 inputs must be finite.  Neither the pages nor the OCP rule give a
 *    scale for a block that holds Inf or NaN; the bytes written for such a
 *    block are unspecified (they are not NaN-propagating), and there the
 *    fused mxfp8_group_quantize_requant may differ from the separate
 *    quantize and requantize calls.  No entry point checks for this.
 *  - Scale arrays have exactly the shape (T, K/32): the page's padded shape
 *    (round_up(T,128), round_up(K/32,4)) ([P3244] review thread on
 *    scale_shape) has no padding under the alignment contract below.
 *  - Alignment contract ([P3244] review thread on scale_shape: per-expert
 *    128-token alignment from the dispatch, hidden % 512 == 0, assert rather
 *    than pad): T % 128 == 0, every m_splits[g] % 128 == 0 and >= 0,
 *    sum(m_splits) == T, K % 512 == 0, N % 512 == 0.  Host-checkable parts
 *    are checked (MXFP8_EINVAL); the device-resident splits are checked only
 *    by mxfp8_validate_splits.  Under this contract column-wise blocks never
 *    straddle an expert boundary, so the quantize/requant bytes do not depend
 *    on the split.
 *  - m_splits is a DEVICE array of int64 ([P3224] review: the native grouped
 *    path requires CUDA int64 m_splits and errors on host splits).  A host
 *    pointer is rejected with MXFP8_EINVAL.
 *  - Every buffer is caller-owned device memory.  Outputs are fully
 *    overwritten in place (the output= reuse of [P3224] Greptile Summary).
 *    No entry point allocates, frees or synchronizes; all work is enqueued on
 *    `stream` (a hipStream_t; NULL = the default stream), so the calls can
 *    be captured in a HIP graph.  Kernels never fill memory with a memset
 *    node.
 *  - T = 0 (no token routed to any expert) is valid everywhere: the buffers
 *    whose size is a multiple of T are empty and may be NULL; outputs that
 *    do not depend on T (the wgrad's [G, N, K], dbias [G, N]) must still be
 *    given and are written as for experts without tokens (zeros), and an
 *    accumulated main_grad is left as it is.
 *  - Errors: the return value is a status code; mxfp8_last_error() gives a
 *    message for the last failing call on this thread.  MXFP8_EINVAL mirrors
 *    the pages' ValueError (bad shapes, NULL pointers, host m_splits),
 *    MXFP8_ENOTSUP their NotImplementedError (unsupported format requests),
 *    MXFP8_EHIP their RuntimeError (a HIP launch failure).
 */
#ifndef MXFP8MOE_H
#define MXFP8MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mxfp8_status {
  MXFP8_OK = 0,
  MXFP8_EINVAL = 1,
  MXFP8_ENOTSUP = 2,
  MXFP8_EHIP = 3
} mxfp8_status;

/* GEMM layouts, row-major letters: NT: C = A B^T, NN: C = A B, TN: C = A^T B. */
typedef enum mxfp8_layout {
  MXFP8_LAYOUT_NT = 0, /* forward  */
  MXFP8_LAYOUT_NN = 1, /* dgrad    */
  MXFP8_LAYOUT_TN = 2  /* wgrad    */
} mxfp8_layout;

typedef enum mxfp8_out_dtype {
  MXFP8_OUT_F32 = 0,
  MXFP8_OUT_BF16 = 1
} mxfp8_out_dtype;

#define MXFP8_ROWWISE 1u
#define MXFP8_COLWISE 2u

/* Message for the last failing call on this thread ("" if none). */
const char* mxfp8_last_error(void);

/* ABI version of this header (incremented on any signature change). */
int32_t mxfp8_abi_version(void);

/*
 * mxfp8_group_quantize -- bf16 grouped token tensor -> MXFP8.
 * Row-wise ([P3244] Description: the grouped GEMM takes input already
 * quantized row-wise) and/or column-wise ([P3244] review: the column-wise
 * scales come from the group quantize kernel) in one pass over x.
 *
 *   x      [T, K] bf16, row-major (device)
 *   usage  MXFP8_ROWWISE | MXFP8_COLWISE (at least one)
 *   q_row  [T, K] u8,  s_row [T, K/32] u8        (required iff ROWWISE)
 *   q_col  [K, T] u8,  s_col [K, T/32] u8        (required iff COLWISE)
 *   noop_flag  NULL, or a device int32 read when the kernels run: non-zero
 *          makes the call write nothing, so the outputs keep their previous
 *          contents ([P3224] Greptile Summary and its test list: the group
 *          quantize's noop flag, replayed in a CUDA graph).  A captured
 *          graph can thereby skip re-quantizing weights that did not change;
 *          the flag is set or cleared by the caller's own kernels.
 * The same call quantizes a grouped weight [G, N, K] viewed as [G*N, K]
 * (T = G*N); its column-wise copy is then [K, G*N], expert g being columns
 * [g*N, (g+1)*N).
 * Errors: EINVAL for NULL required pointers, T % 128, K % 512, usage == 0.
 */
mxfp8_status mxfp8_group_quantize(const uint16_t* x, int64_t T, int64_t K, uint32_t usage,
                                  uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                  uint8_t* s_col, const int32_t* noop_flag, void* stream);

/*
 * Bytes of device workspace that mxfp8_requant_colwise (with dbias) and
 * mxfp8_grouped_dbias need for a [T, N] operand: one fp32 partial sum per
 * 128-row tile and column, i.e. (T/128) * N * 4.
 */
size_t mxfp8_dbias_workspace_bytes(int64_t T, int64_t N);

/*
 * mxfp8_requant_colwise -- row-wise MXFP8 -> exact dequantize -> column-wise
 * MXFP8, optionally with the fused grouped bias gradient
 * ([P3244] Description: dequant + requant with col-wise to save for
 * backward / for wgrad; Greptile Summary: dbias reduced directly from the
 * dequantized gradient).
 *
 *   q_row [T, K] u8, s_row [T, K/32] u8     (device)
 *   q_col [K, T] u8, s_col [K, T/32] u8     (device, written)
 *   dbias NULL, or [G, K] fp32 (device, written): dbias[g, k] = sum over the
 *         rows r of expert g of dequant(q_row)[r, k]; 0 for an empty expert.
 *         Needs m_splits (device int64 [G]) and a workspace of
 *         mxfp8_dbias_workspace_bytes(T, K) bytes; the sum order is fixed, so
 *         results are bitwise reproducible.
 * Errors: EINVAL for NULL pointers, T % 128, K % 512, G < 1, host m_splits,
 * a workspace smaller than required.
 */
mxfp8_status mxfp8_requant_colwise(const uint8_t* q_row, const uint8_t* s_row, int64_t T,
                                   int64_t K, uint8_t* q_col, uint8_t* s_col,
                                   const int64_t* m_splits, int32_t G, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp8_group_quantize_requant -- mxfp8_group_quantize(ROWWISE) followed by
 * mxfp8_requant_colwise (with its optional dbias) in one pass over x: the
 * backward's gradient is quantized row-wise for dgrad, and its column-wise
 * copy for wgrad is requantized from those row-wise values, not quantized
 * from bf16 ([P3244] Description and Greptile flowchart: dequantize, then
 * column-wise requantize, with the bias reductions from the dequantized
 * grad).  x is read once instead of the row-wise codes being read back.
 *  x: bf16 [T, K]; q_row/s_row: [T, K] + [T, K/32]; q_col/s_col: the
 *  transposed column-wise copy [K, T] + [K, T/32]; dbias, m_splits, G,
 *  workspace as for mxfp8_requant_colwise.
 *  For finite x every output byte (and dbias, bit for bit) equals what the
 *  two calls give.
 * Errors: EINVAL for NULL pointers (T > 0), T % 128, K % 512, and as
 * mxfp8_requant_colwise for dbias.
 */
mxfp8_status mxfp8_group_quantize_requant(const uint16_t* x, int64_t T, int64_t K,
                                          uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                          uint8_t* s_col, const int64_t* m_splits, int32_t G,
                                          float* dbias, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * mxfp8_group_quantize_requant_noalloc -- mxfp8_group_quantize_requant for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation): the same work and
 * the same bytes, with no workspace argument.  The dbias partial sums live in
 * a static device array of MXFP8_NOALLOC_SCRATCH_BYTES bytes inside the
 * library (one per GPU, held until the process ends; its address is looked
 * up on the first call on each device).  The call allocates and frees
 * nothing.
 *  Arguments as mxfp8_group_quantize_requant, without workspace.
 *  Limit: with dbias, (T/128) * K * 4 bytes of partials must fit the array,
 *  i.e. mxfp8_dbias_workspace_bytes(T, K) <= MXFP8_NOALLOC_SCRATCH_BYTES
 *  (32 MiB: for K = 14336, T up to 74880; for K = 7168, up to 149760);
 *  without dbias there is no limit.
 *  Every call on one GPU shares that GPU's array, and the array keeps the
 *  last call's partials: calls with dbias that may overlap on one GPU (on
 *  different streams, or from different threads) race on it and give wrong
 *  dbias.  Stream-ordered calls, graph replays included, are safe.  Nothing
 *  needs clearing: each call writes every partial its finalize reads.
 * Errors: as mxfp8_group_quantize_requant, and EINVAL when the partials of
 * the requested dbias exceed the static array.
 */
#define MXFP8_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
mxfp8_status mxfp8_group_quantize_requant_noalloc(const uint16_t* x, int64_t T, int64_t K,
                                                  uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                                  uint8_t* s_col, const int64_t* m_splits,
                                                  int32_t G, float* dbias, void* stream);

/*
 * mxfp8_grouped_dbias -- grouped bias gradient from row-wise MXFP8 dY with no
 * column-wise copy (the frozen-weight case: [P3244] Greptile Summary, dbias
 * reduced without a wgrad stage).
 *   q_row [T, N] u8, s_row [T, N/32] u8; dbias [G, N] fp32 (written).
 * Same workspace and errors as mxfp8_requant_colwise.
 */
mxfp8_status mxfp8_grouped_dbias(const uint8_t* q_row, const uint8_t* s_row, int64_t T,
                                 int64_t N, const int64_t* m_splits, int32_t G, float* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp8_grouped_scaled_bias_grad -- gradients of a bias scaled by each
 * token's routing scale, from row-wise MXFP8 dY ([P3244] Greptile Summary:
 * scaled-bias gradient reductions; its flowchart takes the bias and
 * routing-scale reductions from the dequantized gradient).  With the forward
 * out_r = x_r W_g^T + s_r b_g for row r of expert g:
 *   dbias[g, n] = sum over rows r of expert g of s_r * dY[r, n]
 *   dscales[r]  = sum over n of dY[r, n] * b[g, n]
 * dY is dequantized exactly; sums in fp32 in a fixed order (bitwise
 * reproducible).  An expert with no rows gets dbias[g] = 0.
 *   q_row [T, N] + s_row [T, N/32]: row-wise dY; m_splits: device int64 [G];
 *   scales: device fp32 [T] (needed for dbias); bias: device fp32 [G, N]
 *   (needed for dscales); dbias: fp32 [G, N] or NULL; dscales: fp32 [T] or
 *   NULL (at least one); workspace: device, at least
 *   mxfp8_scaled_bias_workspace_bytes(T, N) bytes.
 * Errors: EINVAL for NULL inputs, neither output requested, an output without
 * its input, T % 128, N % 512, host m_splits, a small workspace.
 */
size_t mxfp8_scaled_bias_workspace_bytes(int64_t T, int64_t N);
mxfp8_status mxfp8_grouped_scaled_bias_grad(const uint8_t* q_row, const uint8_t* s_row,
                                            int64_t T, int64_t N, const int64_t* m_splits,
                                            int32_t G, const float* scales, const float* bias,
                                            float* dbias, float* dscales, void* workspace,
                                            size_t workspace_bytes, void* stream);

/*
 * mxfp8_grouped_gemm -- the three grouped GEMMs of an expert linear
 * y = x W^T (in_features K, out_features N, grouped weight [G, N, K],
 * [P3224] Greptile Summary) on MXFP8 operands, fp32 accumulation.
 * Expert g owns token rows [o_g, o_g + m_splits[g]), o_g = sum of the
 * previous splits.
 *
 *  NT (forward, [P3244] Description: row-wise data goes straight to the
 *      forward grouped GEMM):
 *      a = X row-wise  [T, K] + [T, K/32]
 *      b = W row-wise  [G, N, K] + [G, N, K/32]
 *      c [T, N]:  c[r] = X[r] W_g^T for r in expert g
 *  NN (dgrad, [P3244] Description backward paragraph; [P3545] last commit
 *      message: the column-wise weight copy exists for dgrad):
 *      a = dY row-wise [T, N] + [T, N/32]
 *      b = W column-wise copy [K, G*N] + [K, G*N/32]
 *      c [T, K]:  c[r] = dY[r] W_g
 *  TN (wgrad, [P3244] flowchart: column-wise requantize feeds the wgrad
 *      grouped GEMM):
 *      a = dY column-wise copy [N, T] + [N, T/32]
 *      b = X column-wise copy  [K, T] + [K, T/32]
 *      c [G, N, K]: c[g] = sum over r in expert g of dY[r]^T X[r];
 *      an expert with no rows gets c[g] = 0.
 *  c_dtype: MXFP8_OUT_F32 or MXFP8_OUT_BF16 (round to nearest even).
 *  Rows of c that belong to no expert (none under the contract) are not
 *  written by NT/NN.
 *  With fp32 output, an NT/NN call may split the few long tiles of its
 *  grid's last round into two contraction halves: it then enqueues a small
 *  kernel that zeroes those tiles' rows of c, and the two halves add into
 *  them.  The result is deterministic (two fp32 adds onto zero commute) and
 *  the launches stay stream-ordered and graph-capturable; their rounding
 *  differs from the unsplit sum only by the order of the fp32 additions.
 * Errors: EINVAL for NULL pointers, bad layout, T % 128, N % 512, K % 512,
 * G < 1, host m_splits; ENOTSUP for another c_dtype.
 */
mxfp8_status mxfp8_grouped_gemm(int32_t layout, const uint8_t* a_data, const uint8_t* a_scale,
                                const uint8_t* b_data, const uint8_t* b_scale, void* c,
                                int32_t c_dtype, int64_t T, int64_t N, int64_t K,
                                const int64_t* m_splits, int32_t G, void* stream);

/*
 * mxfp8_grouped_gemm_swiglu_quantize -- the forward (NT) grouped GEMM of the
 * fused expert MLP's first linear, FC1, with its activation and the MXFP8
 * quantize of the activation in the GEMM's epilogue ([P3545] Description:
 * the fused grouped MLP runs FC1 -> activation -> FC2 as one op; its
 * saved-state commit: the FC2 forward reads the row-wise tiles of the
 * activation and the FC2 wgrad the column-wise ones).  The activation is
 * SwiGLU (not defined on the pages): gate = columns [0, F) of h, up =
 * columns [F, 2F).
 *      h[r] = X[r] W1_g^T  (bf16, round to nearest even), r in expert g
 *      a    = silu(gate) * up from the bf16 h, fp32 math, bf16 rounding
 *      a quantized row-wise and/or column-wise
 *  The outputs are byte-identical to mxfp8_grouped_gemm (NT, bf16 output)
 *  followed by mxfp8_swiglu_quantize on its h; a itself is never written.
 *   a_data/a_scale  X row-wise [T, K] + [T, K/32]
 *   b_data/b_scale  W1 row-wise [G, 2F, K] + [G, 2F, K/32]
 *   h               [T, 2F] bf16, written (the SwiGLU backward reads it)
 *   usage           MXFP8_ROWWISE | MXFP8_COLWISE (at least one)
 *   q_row [T, F] u8, s_row [T, F/32] u8     (required iff ROWWISE)
 *   q_col [F, T] u8, s_col [F, T/32] u8     (required iff COLWISE)
 * Errors: EINVAL for NULL required pointers, T % 128, F % 512, K % 512,
 * G < 1 or G > 1024, host m_splits, usage == 0.
 */
mxfp8_status mxfp8_grouped_gemm_swiglu_quantize(const uint8_t* a_data, const uint8_t* a_scale,
                                                const uint8_t* b_data, const uint8_t* b_scale,
                                                uint16_t* h, int64_t T, int64_t F, int64_t K,
                                                const int64_t* m_splits, int32_t G,
                                                uint32_t usage, uint8_t* q_row, uint8_t* s_row,
                                                uint8_t* q_col, uint8_t* s_col, void* stream);

/*
 * mxfp8_grouped_gemm_wgrad_accumulate -- the TN (wgrad) product of
 * mxfp8_grouped_gemm added into an existing fp32 weight-gradient buffer
 * instead of overwriting it, the form a training step uses when the weight
 * gradient accumulates into an fp32 main_grad ([P3545] last commit message:
 * the fused grouped MLP's weight gradients are checked in main_grad):
 *      main_grad[g] += sum over r in expert g of dY[r]^T X[r]
 *  a, b, T, N, K, m_splits, G as for the TN layout of mxfp8_grouped_gemm;
 *  main_grad: caller-owned device fp32 [G, N, K], read and written.  The sum
 *  of an expert's product is formed in fp32 as for mxfp8_grouped_gemm and
 *  added to main_grad once (one fp32 rounding).  An expert with no rows
 *  leaves its main_grad[g] untouched (bit for bit).
 * Errors: EINVAL for NULL pointers, T % 128, N % 512, K % 512, G < 1 or
 * G > 1024, host m_splits.
 */
mxfp8_status mxfp8_grouped_gemm_wgrad_accumulate(const uint8_t* a_data, const uint8_t* a_scale,
                                                 const uint8_t* b_data, const uint8_t* b_scale,
                                                 float* main_grad, int64_t T, int64_t N, int64_t K,
                                                 const int64_t* m_splits, int32_t G,
                                                 void* stream);

/*
 * mxfp8_grouped_gemm_ws, mxfp8_grouped_gemm_wgrad_accumulate_ws -- the same
 * calls with a caller-owned device workspace holding a tile counter, through
 * which the TN (wgrad) tiles are handed out in order as workgroups finish
 * theirs: greedy longest-first placement of the experts' tiles, instead of a
 * fixed assignment that, under skewed routing, lets a few workgroups with the
 * largest experts' tiles run long after the rest (the routing skew of the
 * [P3224] m_splits use case; [P3545]'s fused grouped MLP).  The outputs are
 * bit-identical to those of the calls without a workspace (each tile is
 * computed the same way, by whichever workgroup takes it).  NT/NN ignore the
 * workspace.
 *  The kernel keeps the fixed order when 1 expert in 8 or more has no token:
 *  those experts' tiles store zeros only, and the fixed order runs them
 *  beside the contraction instead of last.
 *  workspace: device memory of at least mxfp8_grouped_gemm_workspace_bytes()
 *  bytes, owned by the caller; its contents need no initialisation (the call
 *  enqueues a one-thread kernel that sets the counter before the GEMM) and
 *  are meaningless afterwards.  Calls that may run at the same time (other
 *  streams) need workspaces of their own; stream-ordered calls, graph replays
 *  included, can share one.
 * Errors: as the calls without a workspace, and EINVAL for a NULL or too
 * small workspace.
 */
size_t mxfp8_grouped_gemm_workspace_bytes(void);
mxfp8_status mxfp8_grouped_gemm_ws(int32_t layout, const uint8_t* a_data, const uint8_t* a_scale,
                                   const uint8_t* b_data, const uint8_t* b_scale, void* c,
                                   int32_t c_dtype, int64_t T, int64_t N, int64_t K,
                                   const int64_t* m_splits, int32_t G, void* workspace,
                                   size_t workspace_bytes, void* stream);
mxfp8_status mxfp8_grouped_gemm_wgrad_accumulate_ws(const uint8_t* a_data,
                                                    const uint8_t* a_scale, const uint8_t* b_data,
                                                    const uint8_t* b_scale, float* main_grad,
                                                    int64_t T, int64_t N, int64_t K,
                                                    const int64_t* m_splits, int32_t G,
                                                    void* workspace, size_t workspace_bytes,
                                                    void* stream);

/*
 * mxfp8_validate_splits -- device-side check of the alignment contract on the
 * device splits ([P3224] review: an alignment check must accompany device
 * m_splits).  Writes *flag (device int32) = bitmask: 1 = a negative split,
 * 2 = a split not a multiple of 128, 4 = sum != T.  0 means valid.  The host
 * reads the flag only when it wants to (no synchronization here).
 */
mxfp8_status mxfp8_validate_splits(const int64_t* m_splits, int32_t G, int64_t T, int32_t* flag,
                                   void* stream);

/*
 * SwiGLU between the two linears of the fused expert MLP ([P3545]
 * Description: FC1 -> activation -> FC2; the activation is not defined on
 * the pages).  Gate = columns [0, F), up = columns [F, 2F) of h:
 *   a = silu(gate) * up;  fp32 math, bf16 in and out (round to nearest even).
 *   h [T, 2F] bf16, a [T, F] bf16.  Errors: EINVAL for NULL, T < 0, F % 8.
 */
mxfp8_status mxfp8_swiglu_fwd(const uint16_t* h, int64_t T, int64_t F, uint16_t* a,
                              void* stream);

/*
 * mxfp8_swiglu_quantize -- SwiGLU fused with the MXFP8 quantize of its output,
 * the FC2 input of the fused expert MLP ([P3545] Description: FC1 ->
 * activation -> FC2 as one op; its saved-state commit: the FC2 wgrad reads
 * the column-wise tiles of that input, the FC2 forward the row-wise ones).
 * The bf16 activation a = silu(h[:, :F]) * h[:, F:] is formed in registers
 * (exactly the bf16 values mxfp8_swiglu_fwd writes) and quantized as
 * mxfp8_group_quantize quantizes a [T, F] tensor, without writing a:
 * the outputs are byte-identical to mxfp8_swiglu_fwd followed by
 * mxfp8_group_quantize.
 *
 *   h      [T, 2F] bf16 (device)
 *   usage  MXFP8_ROWWISE | MXFP8_COLWISE (at least one)
 *   q_row  [T, F] u8,  s_row [T, F/32] u8        (required iff ROWWISE)
 *   q_col  [F, T] u8,  s_col [F, T/32] u8        (required iff COLWISE)
 * Errors: EINVAL for NULL required pointers, T % 128, F % 512, usage == 0.
 */
mxfp8_status mxfp8_swiglu_quantize(const uint16_t* h, int64_t T, int64_t F, uint32_t usage,
                                   uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                   uint8_t* s_col, void* stream);

/*
 * Backward of mxfp8_swiglu_fwd: given h [T, 2F] and da [T, F] (bf16), writes
 * dh [T, 2F] bf16: d gate = da * up * s * (1 + gate * (1 - s)), s = sigmoid(gate);
 * d up = da * silu(gate).  Errors as mxfp8_swiglu_fwd.
 */
mxfp8_status mxfp8_swiglu_bwd(const uint16_t* h, const uint16_t* da, int64_t T, int64_t F,
                              uint16_t* dh, void* stream);

/*
 * mxfp8_swiglu_bwd_quantize -- the SwiGLU backward fused with the quantize of
 * its output for the FC1 backward of the fused expert MLP ([P3545]
 * Description: FC1 -> activation -> FC2 as one op; the FC1 dgrad reads the
 * row-wise and its wgrad the column-wise copy of dh, and [P3244] Description
 * and Greptile flowchart: the column-wise copy requantized from the
 * dequantized row-wise values, the bias gradient reduced from them).  dh =
 * mxfp8_swiglu_bwd(h, da) is formed in registers and handled exactly as
 * mxfp8_group_quantize_requant handles a [T, 2F] tensor, without writing dh:
 * every output byte, and dbias bit for bit, equals mxfp8_swiglu_bwd followed
 * by mxfp8_group_quantize_requant.
 *   h      [T, 2F] bf16 (gate | up, device);  da [T, F] bf16 (device)
 *   q_row  [T, 2F] u8,  s_row [T, 2F/32] u8
 *   q_col  [2F, T] u8,  s_col [2F, T/32] u8
 *   m_splits, G, dbias [G, 2F] fp32, workspace: as mxfp8_group_quantize_requant
 *   with K = 2F (dbias optional: NULL skips it and needs no workspace).
 * Errors: EINVAL for NULL pointers (T > 0), T % 128, F % 256, and as
 * mxfp8_requant_colwise for dbias.
 */
mxfp8_status mxfp8_swiglu_bwd_quantize(const uint16_t* h, const uint16_t* da, int64_t T,
                                       int64_t F, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                       uint8_t* s_col, const int64_t* m_splits, int32_t G,
                                       float* dbias, void* workspace, size_t workspace_bytes,
                                       void* stream);

/*
 * mxfp8_convert_sweep -- diagnostic: runs the device's E4M3 / E8M0 conversion
 * helpers (the ones every quantize kernel encodes and decodes with) over
 * every (value, scale byte) pair, so that a test can compare them with an
 * independent encoder (OCP Microscaling Formats v1.0, sections 5.3-5.4 and
 * 6.3: E4M3 round to nearest even, saturated to 448; value = code * 2^X).
 * Not a step of the hot path.
 *   mode 0: out holds 2^24 u16; entry 65536 * s + h = the codes of the bf16
 *           values (h, h ^ 0x8000) encoded with scale byte s (byte 0 is h).
 *   mode 1: out holds 2^24 u8; entry 65536 * x + 256 * s + c = code c decoded
 *           with scale byte s and encoded again with scale byte x.
 *   mode 2: out holds 2^16 pairs of fp32 bit patterns; entry 256 * s + c =
 *           the codes (c, c ^ 0x80) decoded with scale byte s.
 * out: device buffer of at least mxfp8_convert_sweep_bytes(mode) bytes,
 * written asynchronously on `stream`.  Errors: EINVAL for an unknown mode, a
 * NULL or too small buffer.
 */
size_t mxfp8_convert_sweep_bytes(int32_t mode);
mxfp8_status mxfp8_convert_sweep(int32_t mode, void* out, size_t out_bytes, void* stream);

/*
 * Experts with any number of rows, in 16-bit floating point and in 8-bit
 * integers, and the routing around them.  These calls share none of the
 * multiples-of-128 contract above: every size from 1 up is taken, splits may
 * be any numbers.  Element types:
 */
typedef enum mxfp8_type {
  MXFP8_TYPE_F32 = 0,
  MXFP8_TYPE_BF16 = 1,
  MXFP8_TYPE_F16 = 2
} mxfp8_type;

/*
 * mxfp8_ragged_gemm -- one product of an expert linear over ragged experts.
 * Expert g owns m_splits[g] consecutive rows of the R rows of the product, in
 * order; i(r) = row_index[r], or r where row_index is NULL (then S = R):
 *   NT  C[r, n]    = sum_k X[i(r), k] W[g, n, k]       forward
 *   NN  C[r, k]    = sum_n dY[r, n] W[g, n, k]         gradient of the input
 *   TN  C[g, n, k] = sum over r of g of dY[r, n] X[i(r), k]   of the weight
 * Sums are fp32, rounded once (nearest even) to the output's type.  Results are
 * the same from run to run.
 *   type    MXFP8_TYPE_BF16 or MXFP8_TYPE_F16: X, dY, W
 *   a       NT: X [S, K]; NN, TN: dY [R, N].  Row stride lda >= the row length
 *   b       NT, NN: W [G, N, K] contiguous (ldb ignored); TN: X [S, K], row
 *           stride ldb
 *   c       NT [R, N], NN [R, K], row stride ldc; TN [G, N, K] contiguous (ldc
 *           ignored).  c_type: MXFP8_TYPE_F32 or `type`
 *   m_splits  device int64 [G], 1 <= G <= 1024.  A negative split counts as 0.
 *           Rows of C past the last expert's are not written, and rows past R
 *           not read, whatever the splits sum to
 *   row_index  NULL or device int32 [R] (NT, TN).  Entries outside [0, S) stand
 *           for a row of zeros (of scale 0 in 8-bit integers): results are those
 *           of an X that has such a row, NaN where it meets an infinity or NaN of
 *           W, dY or w_scale.  Entries past the last expert's row are not read
 * TN writes zeros for an expert without rows.  Row values of experts that own
 * other rows never reach a result (infinities and NaN included).
 * Strides are in elements.  Faster where pointers, strides and the contraction
 * length are multiples of 16 bytes; right for all.
 *   workspace  NULL, or device memory, 16-byte aligned, that no other call running
 *           at the same time uses; needs no initialisation.  With
 *           mxfp8_ragged_gemm_workspace_bytes() bytes of it, tiles that do not fill
 *           the GPU are split along the contraction and joined in a fixed order,
 *           and operands whose rows do not start on 16 bytes are laid out anew
 *           where that pays.  Results do not depend on it but for the order of
 *           sums.
 * mxfp8_ragged_gemm_workspace_bytes: for operands of elem_bytes (2, or 1 for
 * mxfp8_ragged_gemm_int8) that are contiguous and on 16 bytes; 0 where none is used,
 * and for sizes that are refused.  Strided or shifted operands whose rows start off
 * 16 bytes find no room in it to be laid out anew, and a gathered X of 4 GiB or more
 * is never: those take a form that is two to eight times slower on large products.
 * Errors: EINVAL for NULL pointers, sizes < 1 (R, S >= 0), strides shorter than
 * a row, G out of range, host m_splits, row_index with NN, S != R without
 * row_index, over 2^31 - 1 rows, columns or tiles; ENOTSUP for other types.
 */
mxfp8_status mxfp8_ragged_gemm(int32_t layout, int32_t type, const void* a, int64_t lda,
                               const void* b, int64_t ldb, void* c, int64_t ldc, int32_t c_type,
                               int64_t R, int64_t S, int64_t N, int64_t K,
                               const int64_t* m_splits, int32_t G, const int32_t* row_index,
                               void* workspace, size_t workspace_bytes, void* stream);
size_t mxfp8_ragged_gemm_workspace_bytes(int32_t layout, int32_t elem_bytes, int64_t R, int64_t S,
                                         int64_t N, int64_t K, int32_t G);

/*
 * mxfp8_quantize_int8 -- a tensor's rows as 8-bit integers with a scale each:
 *   scale[t] = max|x[t]| / 127 in fp32 (nearest); q[t] = the integers nearest
 *   to x[t] / scale[t], ties to even, in [-127, 127].
 * A row of zeros: scale 0, codes 0.  A row with an infinity or NaN: scale NaN,
 * codes 0, so that products with it are NaN.  For weights, rows are output
 * channels.
 *   x [T, K] bf16 / fp16 (type), row stride ldx; q int8 [T, K]; scale fp32 [T]
 * Errors: EINVAL for NULL, K < 1, T < 0, ldx < K; ENOTSUP for other types.
 */
mxfp8_status mxfp8_quantize_int8(const void* x, int32_t type, int64_t T, int64_t K, int64_t ldx,
                                 int8_t* q, float* scale, void* stream);

/*
 * mxfp8_ragged_gemm_int8 -- the forward product in 8-bit integers:
 *   C[r, n] = (sum_k q[i(r), k] w[g, n, k]) * scale[i(r)] * w_scale[g, n]
 * The integer sum is exact; it is then rounded to fp32, multiplied by the two
 * scales in that order and rounded to the output's type.
 *   q [S, K] int8, row stride ldq; scale [S]; w [G, N, K] int8; w_scale [G, N];
 *   c [R, N], row stride ldc, c_type any mxfp8_type; the rest as
 *   mxfp8_ragged_gemm (NT).
 * Errors: as mxfp8_ragged_gemm; EINVAL for K > 131071 (sums past 32 bits).
 */
mxfp8_status mxfp8_ragged_gemm_int8(const int8_t* q, int64_t ldq, const float* scale,
                                    const int8_t* w, const float* w_scale, void* c, int64_t ldc,
                                    int32_t c_type, int64_t R, int64_t S, int64_t N, int64_t K,
                                    const int64_t* m_splits, int32_t G, const int32_t* row_index,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp8_moe_route -- the top_k experts of each token, their weights, and the
 * order of the rows that the products above take.
 * Choice: the top_k largest logits, equal ones by lowest expert.  Logits of
 * -inf or NaN are never chosen; a token whose mask is 0 chooses none and its
 * logits are not looked at.  Logits must not be +inf.
 * Weights: exp(logit) over its sum over the chosen experts (renormalize != 0)
 * or over all experts.
 *   logits [T, E] (type: any mxfp8_type), 1 <= E <= 1024, top_k <= min(E, 16)
 *   token_mask  NULL or uint8 [T]
 *   ids int32 [T, top_k]      by falling logit; -1 where there is none
 *   weights fp32 [T, top_k]   0 where there is none
 *   m_splits int64 [E]        rows of each expert
 *   row_token int32 [T top_k] token of each row, rows ordered by expert, then
 *                             token; -1 past the last row
 *   row_pos int32 [T, top_k]  row of each choice, -1 where there is none
 *   workspace   of mxfp8_moe_route_workspace_bytes(T, E) bytes; needs no
 *               initialisation (NULL where that is 0, as for sizes that are refused)
 * Time grows with T, past some 10^6 tokens faster (128 experts: 0.5 ms for 2^20,
 * 2.8 ms for 2^22).
 * Errors: EINVAL for NULL, sizes out of range, T top_k >= 2^31, a small
 * workspace; ENOTSUP for other types.  T = 0 writes m_splits only.
 */
size_t mxfp8_moe_route_workspace_bytes(int64_t T, int32_t E);
mxfp8_status mxfp8_moe_route(const void* logits, int32_t type, int64_t T, int32_t E,
                             int32_t top_k, int32_t renormalize, const uint8_t* token_mask,
                             int32_t* ids, float* weights, int64_t* m_splits, int32_t* row_token,
                             int32_t* row_pos, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * mxfp8_moe_route_bwd -- gradient of the logits from that of the weights:
 * dlogits [T, E] of the logits' type, every value written (0 for masked tokens and,
 * when renormalized, for experts that were not chosen).  ids and weights as
 * mxfp8_moe_route gave them; dweights fp32 [T, top_k], ignored where ids is -1.
 */
mxfp8_status mxfp8_moe_route_bwd(const void* logits, int32_t type, int64_t T, int32_t E,
                                 int32_t top_k, int32_t renormalize, const int32_t* ids,
                                 const float* weights, const float* dweights, void* dlogits,
                                 void* stream);

/*
 * mxfp8_moe_combine -- out[t] = sum_j weights[t, j] y[row_pos[t, j]], fp32 sums in
 * the order of j, rounded once.  A row_pos outside [0, R) adds nothing.
 *   y [R, H], out [T, H] bf16 / fp16 (type); row_pos int32 [T, top_k];
 *   weights fp32 [T, top_k] or NULL (all 1: the gradient of the gather that
 *   row_token does); 1 <= top_k <= 16
 */
mxfp8_status mxfp8_moe_combine(const void* y, int32_t type, int64_t T, int64_t R, int64_t H,
                               int32_t top_k, const int32_t* row_pos, const float* weights,
                               void* out, void* stream);

/*
 * mxfp8_moe_combine_bwd -- dy[row_pos[t, j]] = weights[t, j] dout[t] and
 * dweights[t, j] = <y[row_pos[t, j]], dout[t]> (fp32; 0 where row_pos is
 * outside [0, R)).  dy or dweights may be NULL (not wanted; y may be NULL
 * without dweights).  No row is named twice; rows of dy that none names are
 * not written.
 */
mxfp8_status mxfp8_moe_combine_bwd(const void* dout, const void* y, int32_t type, int64_t T,
                                   int64_t R, int64_t H, int32_t top_k, const int32_t* row_pos,
                                   const float* weights, void* dy, float* dweights,
                                   void* stream);

/*
 * mxfp8_ragged_gemm_swiglu -- the gated feed-forward block of ragged experts up to its
 * activation, in one kernel: both projections of mxfp8_ragged_gemm (NT), the activation
 * and the product (the rows of W are the gate's, then the up projection's):
 *   z[r, n] = sum_k X[i(r), k] W[g, n, k],  n in [0, 2F)
 *   a[r, f] = silu(z[r, f]) * z[r, F + f],  h = z
 * Sums and the activation are fp32; a and h are each rounded once from them (a does not go
 * through the rounded h, as mxfp8_swiglu_fwd of h would).  A sigmoid below 2^-126 counts as 0.
 *   type    MXFP8_TYPE_BF16 or MXFP8_TYPE_F16: X, W, a, h
 *   x       [S, K], row stride ldx;  w [G, 2F, K]
 *   a       [R, F], row stride lda;  h [R, 2F] (gate | up) or NULL: not kept
 *   m_splits, G, row_index, workspace: as mxfp8_ragged_gemm, rows of a and h past the last
 *   expert's are not written.  No output may overlap an input or the other output.
 * Faster where pointers and ldx, lda, K and F are multiples of 16 bytes; right for all.
 * Errors: as mxfp8_ragged_gemm with N = 2F.
 */
mxfp8_status mxfp8_ragged_gemm_swiglu(int32_t type, const void* x, int64_t ldx, const void* w, void* a,
                                      int64_t lda, void* h, int64_t R, int64_t S, int64_t F, int64_t K,
                                      const int64_t* m_splits, int32_t G, const int32_t* row_index,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp8_ragged_gemm_swiglu_bwd -- the backward pass of that activation inside the down
 * projection's input gradient (mxfp8_ragged_gemm NN), whose result da is never written:
 *   da[r, f] = sum_n dY[r, n] W[g, n, f],  n in [0, N)
 *   s = sigmoid(h[r, f]):  dh[r, f] = da * h[r, F + f] * s * (1 + h[r, f] * (1 - s))
 *                          dh[r, F + f] = da * silu(h[r, f])
 *   a[r, f] = silu(h[r, f]) * h[r, F + f]      anew, for the down projection's weight gradient
 * Sums and derivatives are fp32, results are rounded once.
 *   dy  [R, N], row stride lddy;  w [G, N, F];  h, dh [R, 2F] (gate | up);
 *   a   [R, F] or NULL: not wanted
 *   type, m_splits, G, workspace: as mxfp8_ragged_gemm.  dh and a may not overlap h, dy or w.
 * The gradients of the weights and of X follow with mxfp8_ragged_gemm: TN of dy and a, TN of
 * dh and X, NN of dh and the first weights.
 * Errors: as mxfp8_ragged_gemm (NN) with K = F.
 */
mxfp8_status mxfp8_ragged_gemm_swiglu_bwd(int32_t type, const void* dy, int64_t lddy, const void* w,
                                          const void* h, void* dh, void* a, int64_t R, int64_t N,
                                          int64_t F, const int64_t* m_splits, int32_t G, void* workspace,
                                          size_t workspace_bytes, void* stream);
/* Workspace of the two calls (backward: 0 or 1) for contiguous operands on 16 bytes; C is K of the
 * first, N of the second.  0 where none is used, and for sizes that are refused. */
size_t mxfp8_ragged_gemm_swiglu_workspace_bytes(int32_t backward, int64_t R, int64_t F, int64_t C, int32_t G);

/*
 * mxfp8_quantize_fp8 -- a tensor's rows in 8-bit floating point (E4M3, as above) with an fp32
 * scale for each block of 128 values:
 *   scale[t, b] = max|x[t, 128 b ..]| / 448 in fp32 (nearest); q[t, k] = the E4M3 value
 *   nearest to x[t, k] / scale[t, k / 128], ties to even, at most 448 in size.
 * A block of zeros: scale 0, codes 0.  A block with an infinity or NaN: scale NaN, codes 0, so
 * that products with it are NaN.
 *   x [T, K] bf16 / fp16 (type), row stride ldx;  q u8 [T, K];  scale fp32 [T, ceil(K / 128)]
 * Errors: EINVAL for NULL, K < 1, T < 0, ldx < K; ENOTSUP for other types.
 */
mxfp8_status mxfp8_quantize_fp8(const void* x, int32_t type, int64_t T, int64_t K, int64_t ldx, uint8_t* q,
                                float* scale, void* stream);

/*
 * mxfp8_quantize_fp8_weight -- the same for the weights of G experts, w [G, N, K], with a
 * scale for each block of 128 x 128 of an expert's matrix: q u8 [G, N, K], scale fp32
 * [G, ceil(N / 128), ceil(K / 128)].
 * Errors: EINVAL for NULL (G > 0), N < 1, K < 1, G < 0, over 2^31 - 1 blocks; ENOTSUP for
 * other types.
 */
mxfp8_status mxfp8_quantize_fp8_weight(const void* w, int32_t type, int64_t G, int64_t N, int64_t K,
                                       uint8_t* q, float* scale, void* stream);

/*
 * mxfp8_ragged_gemm_fp8 -- the forward product of ragged experts on such data:
 *   C[r, n] = sum_b scale[i(r), b] w_scale[g, n / 128, b] sum_{k in block b} q[i(r), k] w[g, n, k]
 * The two scales are multiplied first (one fp32 rounding), blocks are formed and added in fp32,
 * the result is rounded once to its type.
 *   q [S, K], row stride ldq;  scale [S, ceil(K / 128)];  w [G, N, K];
 *   w_scale [G, ceil(N / 128), ceil(K / 128)];  c [R, N], row stride ldc, c_type any
 *   mxfp8_type;  the rest as mxfp8_ragged_gemm (NT).  Rows of zeros have scale 0.  For the
 *   input's gradient, w holds the transposed weights [G, K, N], w_scale the transposed scales.
 * mxfp8_ragged_gemm_fp8_workspace_bytes: for results of 16 bits; 0 where none is used, and for
 * sizes that are refused.  fp32 results use none.
 * Errors: as mxfp8_ragged_gemm.
 */
mxfp8_status mxfp8_ragged_gemm_fp8(const uint8_t* q, int64_t ldq, const float* scale, const uint8_t* w,
                                   const float* w_scale, void* c, int64_t ldc, int32_t c_type, int64_t R,
                                   int64_t S, int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                                   const int32_t* row_index, void* workspace, size_t workspace_bytes,
                                   void* stream);
size_t mxfp8_ragged_gemm_fp8_workspace_bytes(int64_t R, int64_t S, int64_t N, int64_t K, int32_t G);

/*
 * mxfp8_ragged_gemm_fp8_fast -- the same with fewer bits in the sums, where speed counts for more: a
 * block's sum may be formed by 8-bit matrix instructions, which keep 13 bits below the largest
 * of 8 consecutive products (an error of about 1.5e-5 of the sum on normal values; at most 2^-9
 * of the sum of the largest 8 consecutive products' sizes).  Sizes and alignment decide whether it is, so
 * that a row's result may differ with the rows beside it.  Arguments and workspace as there.
 * Errors: as there, and ENOTSUP for fp32 results.
 */
mxfp8_status mxfp8_ragged_gemm_fp8_fast(const uint8_t* q, int64_t ldq, const float* scale, const uint8_t* w,
                                        const float* w_scale, void* c, int64_t ldc, int32_t c_type, int64_t R,
                                        int64_t S, int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                                        const int32_t* row_index, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * mxfp8_residual_norm -- what follows a block whose output is f (for an expert layer, the
 * join's): f normalized, gated and added to the scaled residual stream, and the sum
 * normalized for the next block, in one pass.  For each row t, n(v) = v / sqrt(mean(v^2) + eps):
 *   b[t] = n(f[t]) post_weight     f[t] where post_weight is NULL
 *   r[t] = residual_scale x[t] + gate[t] b[t]     gate 1 where it is NULL
 *   y[t] = n(r[t]) pre_weight
 * n(r) is of r as it is stored (rounded to x's type), which is what the backward pass and
 * every later reader see.  Statistics are fp32: the squares' sum must not pass 2^127, nor
 * mean(v^2) + eps fall under 2^-126 (a row of zeros with eps 0 is NaN, as the formula says).
 *   x, r   [T, H], x_type: MXFP8_TYPE_F32 or `type`.  r may be x itself
 *   f, y   [T, H], type: MXFP8_TYPE_BF16 or MXFP8_TYPE_F16
 *   gate   fp32 [T] or NULL;  post_weight, pre_weight [H] or NULL, w_type: MXFP8_TYPE_F32 or `type`
 *   f NULL: the norm before the first block, y[t] = n(x[t]) pre_weight; r, gate and
 *          post_weight must be NULL, residual_scale is not used.
 *   pre_weight NULL: y is not wanted and must be NULL (with f given).
 *   H      1 to 16384
 * Errors: EINVAL for NULL, sizes out of range, neither output, a negative or non-finite eps;
 * ENOTSUP for other types.
 */
mxfp8_status mxfp8_residual_norm(const void* x, int32_t x_type, const void* f, int32_t type, int64_t T,
                                 int64_t H, float residual_scale, const float* gate,
                                 const void* post_weight, const void* pre_weight, int32_t w_type, float eps,
                                 void* r, void* y, void* stream);

/*
 * mxfp8_residual_norm_bwd -- its gradients.  dy is that of y, dr the one that reaches r past
 * this norm (from the blocks after it):
 *   total  = dr + gradient of r through y
 *   dx     = residual_scale total                  [T, H], x_type
 *   df     = gradient of f for gate total          [T, H], type
 *   dgate  [t] = <total[t], b[t]>                  fp32 [T]
 *   dpost_weight, dpre_weight                      fp32 [H], sums over the rows in a fixed order
 * Every output may be NULL (not wanted), not all of them.
 *   dy  [T, H] type, NULL without pre_weight;  dr [T, H] x_type, or NULL (zeros); not both NULL
 *   r   [T, H] x_type, as mxfp8_residual_norm stored it (x where f is NULL);  f as given there
 *   the rest as there; dx may be dr, df may be dy or f.  f NULL: dx = total, df, dgate and
 *   dpost_weight must be NULL.
 *   workspace of mxfp8_residual_norm_bwd_workspace_bytes(T, H) bytes, 4-byte aligned, for the two
 *   weights' gradients (NULL without both); needs no initialisation.
 * T = 0 writes zeros to the weights' gradients.
 * Errors: as mxfp8_residual_norm, and EINVAL for an output without what it is the gradient of,
 * a small workspace.
 */
size_t mxfp8_residual_norm_bwd_workspace_bytes(int64_t T, int64_t H);
mxfp8_status mxfp8_residual_norm_bwd(const void* dy, const void* dr, const void* r, int32_t x_type,
                                     const void* f, int32_t type, int64_t T, int64_t H,
                                     float residual_scale, const float* gate, const void* post_weight,
                                     const void* pre_weight, int32_t w_type, float eps, void* dx, void* df,
                                     float* dgate, float* dpost_weight, float* dpre_weight,
                                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8MOE_H */
