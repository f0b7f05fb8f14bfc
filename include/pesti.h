/*
 * pesti.h - C ABI of the MI355X (gfx950) quantized mat-vec library.
 *
 * What is computed
 *   The decode-step linear layer y = W x (+ b) with block-quantized W, as the
 *   row-major matrix-vector product that dominates a decode step and the
 *   fused dequantize + mat-vec that never expands W to float32 ("Project
 *   scaffold: modules, CLI, and correctness harness", file summaries of
 *   tensor.rs and quant.rs), over the GGUF K-family formats that "PESTI -
 *   Portable Execution Substrate for Transformer Inference" dequantizes
 *   byte-exactly ("What This Is").  The same boundary carries the small-M
 *   prompt-width linear layer x @ w + b ("inferno" README, "Design notes"
 *   and "Benchmarks": c_attn / c_proj / mlp_fc at 32 prompt tokens).
 *
 * Block formats (the pages name them; the byte layouts are the GGUF ones):
 *   Q8_0   34 B / 32 weights : binary16 d, int8 q[32].          w = d*q
 *   Q4_K  144 B / 256 weights: binary16 d, binary16 dmin, 12 B of packed
 *          6-bit scales sc[8] and mins m[8], 128 B of 4-bit codes.
 *                                                  w = d*sc[j]*q - dmin*m[j]
 *   Q2_K   84 B / 256 weights: 16 bytes of (4-bit scale, 4-bit min) per
 *          16-weight sub-block, 64 B of 2-bit codes, binary16 d, dmin.
 *          Weight 128h+32j+16c+l: bits 2j of code byte 32h+16c+l, sub-block
 *          8h+2j+c.                                w = d*sc[s]*q - dmin*m[s]
 *   Q3_K  110 B / 256 weights: 32 B of high bits, 64 B of 2-bit codes (as
 *          Q2_K), 12 B of sixteen 6-bit scales, binary16 d.  The code is
 *          the low bits minus 4 where its high bit (bit 4h+j of byte 16c+l)
 *          is clear.                               w = d*(scale[s]-32)*q
 *   Q5_K  176 B / 256 weights: d, dmin, the 12 scale/min bytes of Q4_K,
 *          32 B of fifth bits, 128 B of low 4-bit codes (Q4_K's runs).
 *                                                  w = d*sc[j]*q - dmin*m[j]
 *   Q6_K  210 B / 256 weights: 128 B low 4-bit parts, 64 B high 2-bit parts,
 *          int8 sc[16], binary16 d.                w = d*sc[i/16]*(q - 32)
 *   i8row int8 codes [out][in] plus one float32 scale per row. w = s[o]*q
 *   i4row 4-bit two's complement codes (-8..7), two per byte: weight 2k in
 *          the low nibble of byte k, 2k+1 in the high nibble; a row is
 *          32 B per 64 weights (padded with codes that are never read into
 *          the result), plus one float32 scale per row.      w = s[o]*q
 *
 * Layouts and conventions (every entry point)
 *   - W has out_features rows.  A packed row is ceil(in/QK) whole blocks
 *     (QK = 32 for Q8_0, 256 for the K family); rows follow each other with
 *     stride pesti_row_bytes(format, in_features) bytes.  When in_features
 *     is not a multiple of 256, the columns in_features..end of the last
 *     super-block are padding: they are never read into the result and
 *     their bytes may hold anything.
 *   - x is float32 [batch][in_features], y is float32 [batch][out_features],
 *     bias is float32 [out_features] or NULL.  y is overwritten:
 *     y[b][o] = sum_i w[o][i] * x[b][i] + bias[o].
 *   - Accumulation is float32; dequantized weights are never written out.
 *     Result bound: |y - exact| <= 1e-4 * sum_i |w_i x_i| + 1e-6 for the
 *     mat-vec (2e-3 for the f16 GEMM).
 *   - Pointers are device pointers owned by the caller, on the calling
 *     thread's current HIP device, and must be 16-byte aligned (blocks, x,
 *     y, w, codes; bias and row_scales 4-byte aligned).  x and y must not
 *     overlap.  `stream` is a hipStream_t (NULL = the legacy default
 *     stream).
 *   - Calls only enqueue work on `stream` and return; they never allocate,
 *     free or synchronize, and keep no state between calls, so they may be
 *     issued concurrently on any number of streams.
 *
 * Errors
 *   Return 0 on success or a negative PESTI_ERR_* code.  On any non-zero
 *   return nothing was enqueued and y is untouched.  An empty output
 *   (out_features == 0 or batch == 0, or rows == 0 for dequant) returns 0
 *   without touching any pointer.  in_features == 0 is a valid shape:
 *   y = bias (or 0).  Faults inside a kernel surface at the caller's next
 *   synchronization, as with any HIP kernel.  Nothing falls back to the CPU.
 */
#ifndef PESTI_H
#define PESTI_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PESTI_ABI_VERSION 3

#define PESTI_OK 0
#define PESTI_ERR_NULL (-1)   /* a required pointer is NULL                 */
#define PESTI_ERR_SHAPE (-2)  /* negative size, in_features % 32 != 0,     */
                              /* in_features above PESTI_MAX_IN_FEATURES,   */
                              /* another limit that a call states, or an    */
                              /* unknown format                             */
#define PESTI_ERR_BATCH (-3)  /* batch outside [0, 8]; GEMM m outside [0,  */
                              /* PESTI_MAX_GEMM_M]; rows of X or Y of the   */
                              /* 8-bit and expert GEMMs outside [0,         */
                              /* PESTI_MAX_TOKENS]; rows or lists of the    */
                              /* key-value cache outside their limits       */
#define PESTI_ERR_ALIGN (-4)  /* a pointer breaks the alignment rule above  */
#define PESTI_ERR_LAUNCH (-5) /* the HIP launch reported an error           */
#define PESTI_ERR_DEVICE (-6) /* current device is not gfx950, or no device */
#define PESTI_ERR_WORKSPACE (-7) /* workspace missing or too small          */

#define PESTI_FMT_Q8_0 0
#define PESTI_FMT_Q4_K 1
#define PESTI_FMT_Q6_K 2
#define PESTI_FMT_I8ROW 3
#define PESTI_FMT_Q5_K 4
#define PESTI_FMT_Q2_K 5
#define PESTI_FMT_Q3_K 6
#define PESTI_FMT_I4ROW 7
#define PESTI_FMT_Q4_K_STREAM 8
/* binary16 weights [out][in]: for the small-M GEMM calls that take a format */
#define PESTI_FMT_F16 16
/* float32 values: for the calls that take the format of X or Y */
#define PESTI_FMT_F32 17

#define PESTI_MAX_BATCH 8
#define PESTI_MAX_IN_FEATURES 32768
#define PESTI_MAX_GEMM_M 4096
#define PESTI_MAX_TOKENS (1 << 20)  /* rows of X or Y: 8-bit and expert GEMMs */
#define PESTI_MAX_EXPERTS 1024

/* --- quantized mat-vec, y = W x + b ------------------------------------ */

/* Q8_0 (34-byte blocks of 32 weights).  blocks: out_features rows of
 * in_features/32 blocks.  batch in [0, 8].  Matrices of at least 16384 rows
 * with rows of an even block count and at most 1024 weights, at batch 4..8,
 * run on the matrix cores with x split as described for pesti_gemv_q4_k
 * (same bound). */
int pesti_gemv_q8_0(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);

/* Q4_K (144-byte super-blocks of 256 weights, rows padded to whole
 * super-blocks).  Same arguments as pesti_gemv_q8_0.  Matrices of at least
 * 16384 rows with rows of at most 1024 weights, at batch 3..8, run on the
 * matrix cores: each 32-weight block of x is scaled by a power of two and
 * split into binary16 high and low parts (products with the exact codes
 * are exact), which adds at most 2^-22 |x_i| + 2^-39 max|x_block| per
 * element of x to the float32 error; the result meets the same
 * 1e-4 * sum|w x| + 1e-6 bound. */
int pesti_gemv_q4_k(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);

/* Q4_K in the stream layout: the byte-minimal layout of rows that are not a
 * whole number of super-blocks (the 896-weight rows of "PESTI ..." README,
 * "Conformance": hidden size 896 is 3.5 super-blocks).  The matrix's
 * weights in row-major order, weight (r, c) at position r * in + c of one
 * stream, are cut into 144-byte Q4_K super-blocks in stream order; only the
 * last super-block holds padding.  `blocks` is pesti_matrix_bytes(
 * PESTI_FMT_Q4_K_STREAM, out_features, in_features) bytes: a 896-weight row
 * takes 504 bytes instead of 576, and rows start at weight 0 or 128 of a
 * super-block.  in_features must be a multiple of 64 (rows of whole 64-weight
 * runs), else PESTI_ERR_SHAPE; for multiples of 256 the layout is the row
 * layout of pesti_gemv_q4_k byte for byte.  Same arguments and bound as
 * pesti_gemv_q4_k; every batch runs on the vector ALUs. */
int pesti_gemv_q4_k_stream(int64_t out_features, int64_t in_features, const void* blocks,
                           const float* x, float* y, const float* bias, int32_t batch,
                           void* stream);

/* Q2_K (84-byte) and Q3_K (110-byte) super-blocks of 256 weights, rows
 * padded to whole super-blocks ("PESTI ..." README, "What This Is": all
 * K-family quantizations, Q2_K to Q8_0).  Same arguments as
 * pesti_gemv_q8_0.  Matrices of at least 16384 rows with rows of at most
 * 1024 weights, at batch 3..8, run on the matrix cores with x split as
 * described for pesti_gemv_q4_k (same bound). */
int pesti_gemv_q2_k(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);
int pesti_gemv_q3_k(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);

/* Q5_K (176-byte super-blocks of 256 weights, rows padded to whole
 * super-blocks; "PESTI ..." README, "What This Is": all K-family
 * quantizations).  Same arguments as pesti_gemv_q8_0.  Matrices of at least
 * 16384 rows with rows of at most 1024 weights, at batch 3..8, run on the
 * matrix cores with x split as described for pesti_gemv_q4_k (same
 * bound). */
int pesti_gemv_q5_k(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);

/* Q6_K (210-byte super-blocks of 256 weights, rows padded to whole
 * super-blocks).  Same arguments as pesti_gemv_q8_0.  Matrices of at least
 * 16384 rows with rows of at most 1024 weights, at batch 5..8, run on the
 * matrix cores with x split as described for pesti_gemv_q4_k (same
 * bound). */
int pesti_gemv_q6_k(int64_t out_features, int64_t in_features, const void* blocks,
                    const float* x, float* y, const float* bias, int32_t batch,
                    void* stream);

/* Per-row symmetric int8 ("Project scaffold ...", quant.rs): codes int8
 * [out][in] row-major, row_scales float32 [out]. */
int pesti_gemv_i8row(int64_t out_features, int64_t in_features, const int8_t* codes,
                     const float* row_scales, const float* x, float* y,
                     const float* bias, int32_t batch, void* stream);

/* Per-row symmetric int4 ("Project scaffold ...", quant.rs lists INT4 beside
 * INT8): packed int4 rows of pesti_row_bytes(PESTI_FMT_I4ROW, in) bytes,
 * row_scales float32 [out].  Matrices of at least 16384 rows with rows of at
 * most 1024 weights, at batch 2..8, run on the matrix cores with x split as
 * described for pesti_gemv_q4_k.  Both kernels take every code exactly
 * (the vector-ALU kernel as the signed byte 16 q, the sum then scaled by
 * 2^-4 exactly), so the mat-vec bound above holds unchanged. */
int pesti_gemv_i4row(int64_t out_features, int64_t in_features, const void* packed,
                     const float* row_scales, const float* x, float* y,
                     const float* bias, int32_t batch, void* stream);

/* --- grouped mat-vec: several independent products in one launch ---------
 * One mat-vec of a group: y = W x + b with the layouts above (w is the
 * packed rows, or the int8 codes for i8row; row_scales only for i8row and
 * i4row). */
typedef struct pesti_gemv_op {
  int64_t out_features;
  int64_t in_features;
  const void* w;
  const float* row_scales;
  const float* x;
  float* y;
  const float* bias;
} pesti_gemv_op;

#define PESTI_MAX_GROUP 8

/* Up to PESTI_MAX_GROUP independent mat-vecs of one PESTI_FMT_* format and
 * one batch size, computed by one kernel launch (two or three when the ops
 * need different kernels: each op takes the kernel its own single call
 * would take - Q8_0 rows of an odd or even block count, tall K-quant, Q8_0
 * and int4 matrices on the matrix cores - so every op's y has the bits of its single
 * call).  This is the decode-step
 * case of projections that read the same activations (Q, K and V; gate and
 * up: "PESTI ..." README, "Conformance", per-head GQA and SwiGLU), where
 * one launch replaces several dependent ones.  ops is a host array read
 * during the call; each op follows the conventions and checks of the
 * single-matrix entry points (an op with out_features == 0 is skipped);
 * the y buffers of different ops must not overlap.  Returns the first
 * failing op's error, before anything is enqueued. */
int pesti_gemv_group(int32_t format, int32_t n_ops, const pesti_gemv_op* ops, int32_t batch,
                     void* stream);

/* --- fused SwiGLU feed-forward input, h = silu(W_gate x) * (W_up x) ------
 * The gate and up projections of a decode step's feed-forward block and
 * the SwiGLU that joins them ("PESTI ..." README, "Conformance": SwiGLU =
 * silu(gate) * up with the sigmoid-based SiLU, silu(g) = g / (1 + e^-g)),
 * in one launch: each lane group computes row o of both matrices and writes
 * only h[b][o].  w_gate and w_up are two matrices of one PESTI_FMT_* format
 * and the same shape, laid out as for the single mat-vecs (no bias);
 * gate_scales / up_scales are their row scales for PESTI_FMT_I8ROW and
 * PESTI_FMT_I4ROW and are ignored otherwise.  x float32 [batch][in], h float32 [batch][out].  Rows
 * must fit one load round: in_features up to 4096 (K family, i8row, i4row, Q8_0
 * with in % 64 == 0) or 2048 (other Q8_0), else PESTI_ERR_SHAPE.
 * Bound: |h - exact| <= 1.1 * eg * |u| + |silu(g)| * eu + 2 * eg * eu
 * + 1e-6 * |h| + 1e-6, with eg, eu the mat-vec bounds of g and u. */
int pesti_gemv_swiglu(int32_t format, int64_t out_features, int64_t in_features,
                      const void* w_gate, const void* w_up, const float* gate_scales,
                      const float* up_scales, const float* x, float* h, int32_t batch,
                      void* stream);

/* --- small-M binary16 linear layer, Y = X W^T + b ------------------------
 * X binary16 [m][in], W binary16 [out][in] (the same row orientation as the
 * mat-vec; a GPT-2 c_attn "768x2304" has in = 768, out = 2304), Y float32
 * [m][out], bias float32 [out] or NULL.  m in [0, PESTI_MAX_GEMM_M]; float32
 * accumulation; matrix cores for m >= 16, vector ALUs below. */
int pesti_gemm_f16_smallm(int64_t m, int64_t out_features, int64_t in_features,
                          const uint16_t* w, const uint16_t* x, float* y,
                          const float* bias, void* stream);

/* --- small-M linear layer on quantized weights, Y = X W^T + b -------------
 * The prompt-width product of the same layer ("inferno" README,
 * "Benchmarks": x @ w + b at prompt width) with W kept in the block format
 * of the mat-vec ("Project scaffold ...", quant.rs: dequantize fused into
 * the product, W never expanded).  blocks: out_features packed rows exactly
 * as for pesti_gemv_q8_0 / pesti_gemv_q4_k / pesti_gemv_q6_k; X binary16 [m][in] (16-byte
 * aligned), Y float32 [m][out], bias float32 [out] or NULL; m in [0,
 * PESTI_MAX_GEMM_M].  The matrix cores multiply the exact integer codes by
 * X (every product exact in float32) one 32-weight block or sub-block at a
 * time, and the block scales are applied to each partial sum in float32.
 * Any m >= 1 works; for m <= 8 the batched mat-vec on float32 X is the
 * faster call.  Errors as for pesti_gemm_f16_smallm. */
int pesti_gemm_q8_0_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);
int pesti_gemm_q4_k_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);
/* Q2_K, Q3_K and Q5_K rows as for their mat-vecs.  Their codes times the
 * code's own sub-block scale are small binary16 integers (q * sc <= 45,
 * |q * (sc - 32)| <= 128, q * sc <= 1953), so the operand carries the scale
 * and each lane its own sub-block's; mins (Q2_K, Q5_K) are products of X
 * sums or of X against the mins. */
int pesti_gemm_q2_k_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);
int pesti_gemm_q3_k_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);
int pesti_gemm_q5_k_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);
/* Q6_K rows as for pesti_gemv_q6_k.  Its codes are exact too (q - 32), but
 * each 32-weight k-step spans two 16-weight sub-blocks, so a step is two
 * products (each on half the operand) scaled apart. */
int pesti_gemm_q6_k_smallm(int64_t m, int64_t out_features, int64_t in_features,
                           const void* blocks, const uint16_t* x, float* y,
                           const float* bias, void* stream);

/* --- the same GEMMs with a caller's workspace (split K) -------------------
 * Narrow layers (fewer than 96 16-column tiles, e.g. the 896-wide down
 * projection) with long rows (in_features over 4096) run one workgroup per
 * output tile and leave most compute units idle.  With a workspace, K is
 * split over 2..4 workgroups per tile (more workgroups for fewer row tiles
 * of X; binary16 only at m 16; Q8_0, Q3_K and Q6_K take two row tiles of X
 * per workgroup), each writing its partial tile to the
 * workspace, and a second launch on the same stream sums the partials in a
 * fixed order and adds the bias: results do not depend on timing, but the
 * summation order differs from the call without workspace (same bound).
 *
 * pesti_gemm_workspace_bytes returns the bytes the split needs for this
 * format (PESTI_FMT_F16 or one of the six block formats) and shape: 0 when
 * the shape does not split, at most PESTI_GEMM_SCRATCH_BYTES (512 KiB);
 * negative PESTI_ERR_* for an unknown format or a bad shape.  Host-only,
 * no device needed.
 *
 * pesti_gemm_smallm_ws: arguments as for pesti_gemm_<format>_smallm (w is
 * the binary16 W or the packed blocks), plus `workspace`, device memory of
 * at least that many bytes, 16-byte aligned, owned by the caller and used
 * only by the work this call enqueues (calls that run concurrently need
 * their own); ignored when the shape needs none.  Errors as for the
 * format's call, PESTI_ERR_SHAPE for an unknown format, and
 * PESTI_ERR_WORKSPACE if a needed workspace is NULL or smaller. */
int64_t pesti_gemm_workspace_bytes(int32_t format, int64_t m, int64_t out_features, int64_t in_features);
int pesti_gemm_smallm_ws(int32_t format, int64_t m, int64_t out_features, int64_t in_features,
                         const void* w, const uint16_t* x, float* y, const float* bias,
                         void* workspace, int64_t workspace_bytes, void* stream);

/* --- allocation-free form of pesti_gemm_smallm_ws --------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * GEMM with the split partials in the library's own scratch, a static device
 * array of PESTI_GEMM_SCRATCH_BYTES on each GPU the library runs on, held
 * until the process ends.  Nothing is allocated; every shape's workspace
 * fits.  All calls on one GPU share that GPU's array: calls that overlap in
 * time on one GPU (on different streams, or graphs replayed concurrently)
 * race and may return wrong results; calls ordered on one stream are safe.
 * Nothing in the array needs to start at zero.  Results equal
 * pesti_gemm_smallm_ws bit for bit.  Errors as for pesti_gemm_smallm_ws;
 * PESTI_ERR_WORKSPACE if a shape ever needed more than the array. */
#define PESTI_GEMM_SCRATCH_BYTES (512 * 1024)
int pesti_gemm_smallm_noalloc(int32_t format, int64_t m, int64_t out_features, int64_t in_features,
                              const void* w, const uint16_t* x, float* y, const float* bias,
                              void* stream);

/* --- linear layer on 8-bit integers, a scale per token and per channel ----
 * The prompt-width product of the per-row int8 weights (pesti_gemv_i8row)
 * with X in 8 bits too: Y[t][o] = x_scales[t] * row_scales[o] *
 * sum_i x_codes[t][i] * codes[o][i] + bias[o], the sum taken exactly in
 * 32-bit integers on the matrix cores.  X is quantized once and serves every
 * layer that reads it (Q, K and V; gate and up).
 *
 * For 1..8 rows of float32 X pesti_gemv_i8row does the same layer in one
 * launch and does not round X.  It is also the faster one for one or two
 * rows, and for four of short layers (us a layer, mat-vec against the two
 * calls here: 896x896 at 1 / 4 / 8 rows 2.9 / 3.9 / 5.1 against 4.9 / 5.4 / 5.5,
 * 4864x896 4.0 / 5.1 / 6.8 against 6.1 / 6.6 / 6.9, 4096x4096 7.1 / 14 / 31 against
 * 9.6 / 10 / 10, 151936x896 25 / 35 / 50 against 29 / 30 / 31).  These calls are
 * for more rows, for large layers from four rows on, and for X that is in
 * 8 bits already or that several layers share (the quantizer is 2.3-2.9 of it).
 *
 * pesti_quant_i8token: x [m][in] in x_format (PESTI_FMT_F32 or
 * PESTI_FMT_F16) to codes int8 [m][in] and scales float32 [m], the rule of
 * the per-row weights: scale = max|x| / 127 (one float32 rounding), code =
 * the exact x / scale rounded half away from zero, -127..127.  A row of
 * zeros (or one whose scale rounds to zero) gets scale 0 and codes 0; a row
 * that holds an infinity or NaN gets scale NaN and codes 0, so that its
 * outputs are NaN.  With in_features == 0 the scales are 0.
 *
 * pesti_gemm_i8row_i8token: codes int8 [out][in] and row_scales float32
 * [out] as for pesti_gemv_i8row, x_codes int8 [m][in] and x_scales float32
 * [m] (any codes -128..127), Y [m][out] in y_format (PESTI_FMT_F32, or
 * PESTI_FMT_F16 rounded once from float32).  The float32 value is
 * fma(float(sum) * x_scale, row_scale, bias): three roundings.
 *
 * m in [0, PESTI_MAX_TOKENS], else PESTI_ERR_BATCH; out_features below 2^31
 * and fewer than 2^31 tiles of Y, else PESTI_ERR_SHAPE, as is an unknown
 * format; codes, x and Y 16-byte aligned, scales and bias 4. */
int pesti_quant_i8token(int32_t x_format, int64_t m, int64_t in_features, const void* x,
                        int8_t* codes, float* scales, void* stream);
int pesti_gemm_i8row_i8token(int64_t m, int64_t out_features, int64_t in_features,
                             const int8_t* codes, const float* row_scales,
                             const int8_t* x_codes, const float* x_scales, int32_t y_format,
                             void* y, const float* bias, void* stream);

/* --- linear layers grouped by expert ---------------------------------------
 * Y's rows are sorted by expert: rows offsets[e] .. offsets[e+1]-1 belong to
 * expert e and are Y[r] = X[x_rows[r]] W_e^T + b_e, any number of them per
 * expert, none included, in one launch (the grouped mat-vec's case with one
 * matrix per expert and row counts that only the device knows).
 *
 * format: PESTI_FMT_F16 (W and X binary16, the scale arguments ignored) or
 * PESTI_FMT_I8ROW (W and X int8 with w_scales float32 [experts][out] and
 * x_scales float32 [x_tokens], as for pesti_gemm_i8row_i8token).
 *   offsets  int32 [experts + 1] in device memory, non-decreasing within
 *            0..rows.  Rows of Y outside every expert's range (before
 *            offsets[0], from offsets[experts] on) are left as they were.
 *            Values outside 0..rows count as the nearer end, and an expert
 *            whose end lies before its start has no rows; what rows of Y
 *            hold after a call with decreasing offsets is not specified.
 *   w        [experts][out][in]; bias float32 [experts][out] or NULL
 *   x        [x_tokens][in]
 *   x_rows   int32 [rows] in device memory, the row of X for each row of Y
 *            (the same one any number of times), or NULL for row r itself,
 *            which needs x_tokens >= rows (else PESTI_ERR_BATCH).  An index
 *            outside 0..x_tokens-1 stands for a row of zeros: in binary16 its
 *            sums are 0 whatever W holds, in 8 bits codes and scale are 0.
 *            Rows that are picked are addressed in 32 bits: X of 4 GiB or
 *            more with x_rows is PESTI_ERR_SHAPE.
 *   y        [rows][out] in y_format (PESTI_FMT_F32 or PESTI_FMT_F16)
 *
 * pesti_gemm_experts_swiglu joins the gate and up products of the same rows
 * (h = silu(X W_gate^T) * (X W_up^T), as pesti_gemv_swiglu): w_gate and w_up
 * [experts][out][in] of one format, gate_scales and up_scales their scales,
 * h [rows][out] in h_format; no bias.
 *
 * rows and x_tokens in [0, PESTI_MAX_TOKENS] (PESTI_ERR_BATCH), experts in
 * [0, PESTI_MAX_EXPERTS] and out_features below 2^31 (PESTI_ERR_SHAPE); sums
 * in float32 (binary16) or exactly in 32-bit integers.  rows, out_features or
 * experts of 0 return 0 without touching a pointer. */
int pesti_gemm_experts(int32_t format, int64_t rows, int64_t experts, int64_t out_features,
                       int64_t in_features, const int32_t* offsets, const void* w,
                       const float* w_scales, int64_t x_tokens, const void* x,
                       const float* x_scales, const int32_t* x_rows, int32_t y_format, void* y,
                       const float* bias, void* stream);
int pesti_gemm_experts_swiglu(int32_t format, int64_t rows, int64_t experts,
                              int64_t out_features, int64_t in_features, const int32_t* offsets,
                              const void* w_gate, const void* w_up, const float* gate_scales,
                              const float* up_scales, int64_t x_tokens, const void* x,
                              const float* x_scales, const int32_t* x_rows, int32_t h_format,
                              void* h, void* stream);

/* --- 4-bit weights with a scale and a zero point per group ----------------
 * The mat-vec of the formats above for 4-bit matrices whose scales lie in an
 * array of their own, one per group of consecutive weights of a row:
 *
 *   w[o][i] = scales[o][i / group] * (q[o][i] - zeros[o][i / group])
 *
 *   packed  4-bit codes 0..15, two per byte (weight 2k in the low nibble of
 *           byte k, 2k + 1 in the high one); rows of in_features / 2 bytes
 *   scales  binary16 [out][groups], groups = ceil(in_features / group)
 *   zeros   uint8 [out][groups] (any value), or NULL: 8 for every group
 *   group   weights per scale: a power of two, 32..PESTI_MAX_IN_FEATURES (the
 *           last group of a row may be short), else PESTI_ERR_SHAPE
 *
 * x, y, bias, batch, stream and errors as for pesti_gemv_q8_0; packed 16-byte
 * aligned, scales 2.  The codes less their zero points are exact integers.  Ops
 * of few products (a single column, or a small matrix; by sizes and batch
 * alone) multiply them with float32 x on the vector ALUs, the others on the
 * matrix cores with x in two binary16 parts: each run of 128 weights of a column
 * is scaled by a power of two that brings its largest finite |x| to [2^14,
 * 2^15), and what the first part leaves is held 2^11 times as large in the
 * second, which adds at most 2^-22 |x_i| + 2^-50 max|x| (of the run) per element
 * to the float32 error.  Group sums are float32 and take their scale once; an
 * infinite or NaN scale makes infinities or NaN of its own row alone.
 *
 * pesti_gemv_group_i4group: up to PESTI_MAX_GROUP such mat-vecs of one group
 * size and batch in one launch, as pesti_gemv_group; every op's y has the bits
 * of its single call.
 * pesti_gemv_i4group_swiglu: h = silu(W_gate x) * (W_up x) of two matrices of
 * one shape and group size in one launch, rows of any length (no bias).
 * pesti_dequant_i4group: the weights in float32, bit-exact (each product of a
 * binary16 scale and q - z has a float32 value). */
typedef struct pesti_gemv_i4group_op {
  int64_t out_features;
  int64_t in_features;
  const void* packed;
  const uint16_t* scales;
  const uint8_t* zeros;
  const float* x;
  float* y;
  const float* bias;
} pesti_gemv_i4group_op;

int pesti_gemv_i4group(int64_t out_features, int64_t in_features, int64_t group, const void* packed,
                       const uint16_t* scales, const uint8_t* zeros, const float* x, float* y,
                       const float* bias, int32_t batch, void* stream);
int pesti_gemv_group_i4group(int32_t n_ops, const pesti_gemv_i4group_op* ops, int64_t group,
                             int32_t batch, void* stream);
int pesti_gemv_i4group_swiglu(int64_t out_features, int64_t in_features, int64_t group,
                              const void* gate_packed, const uint16_t* gate_scales,
                              const uint8_t* gate_zeros, const void* up_packed,
                              const uint16_t* up_scales, const uint8_t* up_zeros, const float* x,
                              float* h, int32_t batch, void* stream);
int pesti_dequant_i4group(int64_t rows, int64_t in_features, int64_t group, const void* packed,
                          const uint16_t* scales, const uint8_t* zeros, float* w_out, void* stream);

/* --- paged key-value cache --------------------------------------------------
 * What stands between a decode step's Q/K/V and O projections ("PESTI ..."
 * README, "Conformance": grouped-query attention, 14 query and 2 KV heads of
 * 64; "Current Status": paged attention and KV updates during generation).
 * K and V of all layers lie in pools of pages of page_size tokens; a page
 * number stands for the same page of every layer, of K and of V.  The caller
 * owns every array; the library keeps nothing between calls.
 *
 *   format     PESTI_FMT_F16, or PESTI_FMT_I8ROW: int8 codes with a float32
 *              scale per token and head, by the rule of pesti_quant_i8token
 *   layers     1..PESTI_MAX_LAYERS;  pages 0..PESTI_MAX_PAGES
 *   page_size  a power of two, 8..1024
 *   kv_heads   1..PESTI_MAX_HEADS;  head_dim a multiple of 32, 32..256
 *   k, v       [layers][pages][kv_heads][page_size][head_dim], 16-byte aligned
 *   k_scales, v_scales  (I8ROW) [layers][pages][kv_heads][page_size], 16-byte
 *
 * pesti_kv_table holds which pages the sequences have:
 *   seqs       sequence slots, 0..PESTI_MAX_SEQS
 *   width      page numbers per slot; width * page_size <= 2^30
 *   table      int32 [seqs][width]: token t of a sequence is token t %
 *              page_size of page table[seq][t / page_size]
 *   lengths    int32 [seqs]: tokens of each sequence (below 0 counts as 0,
 *              above width * page_size as that)
 *   refs       int32 [pages]: how many sequences hold the page; 0: it is free
 * Only entries of a sequence's ceil(length / page_size) pages count.  A page
 * number outside 0..pages-1 names no page: attention leaves its tokens out,
 * rows for it are not written, and page upkeep passes over it.
 *
 * The structs are host data, read during the call; a field outside its limits
 * is PESTI_ERR_SHAPE, a missing array PESTI_ERR_NULL (table and lengths always,
 * refs where pages are taken or given back, k, v and the scales where pages are
 * touched), an unaligned one PESTI_ERR_ALIGN (int32 arrays 4 bytes).  Lists
 * (seq_ids, positions, parents, ...) are int32 in device memory; a list entry
 * outside 0..seqs-1 names no sequence and is passed over (attention: a row of
 * zeros).  rows and n are 0..PESTI_MAX_SEQS (pesti_cache_append: 0..
 * PESTI_MAX_TOKENS, pesti_cache_copy_pages: 0..PESTI_MAX_PAGES), else
 * PESTI_ERR_BATCH; 0 returns 0 without touching a pointer.  Calls that change
 * one table or pool have to be ordered with the others that use it, as on one
 * stream. */
#define PESTI_MAX_LAYERS 1024
#define PESTI_MAX_PAGES (1 << 22)
#define PESTI_MAX_HEADS 1024
#define PESTI_MAX_SEQS 4096

typedef struct pesti_kv_cache {
  int64_t format;
  int64_t layers;
  int64_t pages;
  int64_t page_size;
  int64_t kv_heads;
  int64_t head_dim;
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
} pesti_kv_cache;

typedef struct pesti_kv_table {
  int64_t seqs;
  int64_t width;
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
} pesti_kv_table;

/* Pages for more tokens: lengths[seq] += counts[i] (NULL: 1; below 0 counts as
 * 0) for every listed sequence seq_ids[i] (NULL: i), and the pages that this
 * needs are taken, the lowest free ones in list order.  A sequence listed
 * again is passed over.  *status (int32 in device memory): 0, or the number of
 * free pages that are missing, or -1 where a sequence would outgrow its row of
 * the table; nothing has changed then. */
int pesti_cache_extend(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n,
                       const int32_t* seq_ids, const int32_t* counts, int32_t* status, void* stream);

/* K and V of new tokens into their places in one layer's pages: row r is token
 * positions[r] (NULL: the last one) of sequence seq_ids[r] (NULL: r), all KV
 * heads, k and v [rows][stride] in x_format (PESTI_FMT_F32 or PESTI_FMT_F16)
 * with kv_heads * head_dim values a row (so parts of a fused projection's
 * output do as they are).  Rows of positions outside the sequence are not
 * written.  Into binary16 values are rounded to nearest even.  k and v 16-byte
 * aligned, stride * value size a multiple of 16 (else PESTI_ERR_ALIGN) and
 * stride >= kv_heads * head_dim (PESTI_ERR_SHAPE).  Two rows for one place: it
 * holds one of them, which is not specified (in 8 bits perhaps the scale of the
 * other). */
int pesti_cache_append(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t layer,
                       int64_t rows, int32_t x_format, const void* k, const void* v, int64_t stride,
                       const int32_t* seq_ids, const int32_t* positions, void* stream);

/* Attention of one new token per row over its sequence's cache:
 *   y[r][h] = sum_t softmax_t(scale * q[r][h] . k[t][h / g]) v[t][h / g]
 * over the lengths[seq_ids[r]] tokens of the sequence (NULL: sequence r), g =
 * heads / kv_heads query heads to a KV head (heads a multiple, up to
 * PESTI_MAX_HEADS).  The new token's own K and V are in the cache already
 * (pesti_cache_extend, pesti_cache_append).  q [rows][q_stride] in q_format, y
 * [rows][heads][head_dim] in y_format (PESTI_FMT_F32 or PESTI_FMT_F16); q and
 * y 16-byte aligned, q_stride >= heads * head_dim and its bytes a multiple of
 * 16.  A row without tokens (length 0, or no valid page) is zeros, as is one
 * whose every score is -infinity.  An infinity of K makes a score infinite (NaN
 * where q's value is 0, or 2^-39 of the head's largest and less), a NaN of q or K
 * makes NaN of the heads that it enters, a NaN or infinity of V NaN or infinities
 * of its dimension (in 8 bits, where a row's scale holds it, of all), whatever its
 * token weighs.
 *
 * Scores, maximum, sum and result are float32.  q times scale and the softmax's
 * weights enter the matrix cores in two binary16 parts each (22 bits), K and V
 * as they are (the int8 codes exactly, scales applied in float32).
 *
 * The cache's length is split over workgroups where rows and KV heads do not
 * fill the GPU, and the parts are joined in a fixed order.  max_length, 1..
 * 2^30, is the caller's bound of the rows' lengths, which chooses the split; a
 * longer sequence is attended whole all the same.  workspace: device memory of
 * pesti_attn_paged_workspace_bytes(cache, rows, heads, max_length) bytes (0:
 * none needed), 16-byte aligned, for one call at a time.  It serves every call
 * on that cache with as many rows and as long a bound or fewer: the size of the
 * largest call is enough for a program's others.  PESTI_ERR_WORKSPACE if NULL or
 * smaller than the call's own parts.  Nothing in it needs to start at zero.  The
 * function is host-only and gives a negative PESTI_ERR_* for bad arguments. */
int64_t pesti_attn_paged_workspace_bytes(const pesti_kv_cache* cache, int64_t rows, int64_t heads,
                                         int64_t max_length);
int pesti_attn_paged(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t layer,
                     int64_t rows, int64_t heads, const int32_t* seq_ids, int32_t q_format,
                     const void* q, int64_t q_stride, int32_t y_format, void* y, float scale,
                     int64_t max_length, void* workspace, int64_t workspace_bytes, void* stream);

/* pesti_cache_fork: sequence children[i] becomes a copy of parents[i]: it
 * shares the parent's whole pages (refs + 1), and a last page that is not full
 * is copied, in every layer, to the lowest free page, in list order.  A child
 * has to be empty (length 0) and to be listed once: other pairs, and a child
 * listed again, are passed over.  Parents are taken as they were before the
 * call.  *status: 0, or the number of free pages that are missing; nothing has
 * changed then.  n up to seqs (else PESTI_ERR_BATCH).
 *
 * pesti_cache_free: the listed sequences (seq_ids; NULL: 0..n-1; each any
 * number of times) become empty: refs - 1 for each of their pages, their table entries -1.
 *
 * pesti_cache_compact: live pages (refs > 0) move to 0..live-1: the i-th live
 * page from live on to the i-th free page below it, with its contents in every
 * layer; refs and the sequences' table entries follow.  *live (int32 in device
 * memory) is their number.
 *
 * pesti_cache_copy_pages: page src[i] to page dst[i], K, V and scales of every
 * layer.  A dst that is also another pair's src or dst holds a mixture that is
 * not specified.  Table and refs are not looked at.
 *
 * fork and compact need a workspace of pesti_cache_workspace_bytes(cache,
 * table) bytes, 16-byte aligned, for one call at a time (host-only function,
 * negative PESTI_ERR_* for bad arguments); PESTI_ERR_WORKSPACE if NULL or
 * smaller. */
int64_t pesti_cache_workspace_bytes(const pesti_kv_cache* cache, const pesti_kv_table* table);
int pesti_cache_fork(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n,
                     const int32_t* parents, const int32_t* children, int32_t* status,
                     void* workspace, int64_t workspace_bytes, void* stream);
int pesti_cache_free(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n,
                     const int32_t* seq_ids, void* stream);
int pesti_cache_compact(const pesti_kv_cache* cache, const pesti_kv_table* table, int32_t* live,
                        void* workspace, int64_t workspace_bytes, void* stream);
int pesti_cache_copy_pages(const pesti_kv_cache* cache, int64_t n, const int32_t* src,
                           const int32_t* dst, void* stream);

/* --- dequantization to float32 (bit-exact; checks the unpacking) --------
 * w_out float32 [rows][in_features]: each weight rounded once from its
 * exact value (all formats here dequantize exactly in float32 except the
 * final subtraction of Q2_K / Q4_K / Q5_K and the scale product of
 * i8row and i4row). */
int pesti_dequant_q8_0(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_q4_k(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_q4_k_stream(int64_t rows, int64_t in_features, const void* blocks,
                              float* w_out, void* stream);
int pesti_dequant_q2_k(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_q3_k(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_q5_k(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_q6_k(int64_t rows, int64_t in_features, const void* blocks,
                       float* w_out, void* stream);
int pesti_dequant_i8row(int64_t rows, int64_t in_features, const int8_t* codes,
                        const float* row_scales, float* w_out, void* stream);
int pesti_dequant_i4row(int64_t rows, int64_t in_features, const void* packed,
                        const float* row_scales, float* w_out, void* stream);

/* --- measurement hook ----------------------------------------------------
 * A plain streaming read of `bytes` bytes (a multiple of 16) at `buf`
 * (16-byte aligned): the streaming-read ceiling that a mat-vec reading the
 * same number of bytes is measured against.  PESTI_READ_GROUPS workgroups
 * each write the XOR of the dwords they read to partial[group] (the XOR of
 * all entries is the XOR of the whole buffer); `partial` is a device array
 * of PESTI_READ_GROUPS uint32 owned by the caller. */
#define PESTI_READ_GROUPS 4096
int pesti_stream_read(const void* buf, int64_t bytes, uint32_t* partial, void* stream);

/* --- host-only helpers (no device work) --------------------------------- */

/* Packed bytes per row for a PESTI_FMT_* format (code bytes only for
 * i8row); -1 for an unknown format, a negative / non-multiple-of-32
 * in_features, or PESTI_FMT_Q4_K_STREAM (whose rows have no fixed size:
 * see pesti_matrix_bytes). */
int64_t pesti_row_bytes(int32_t format, int64_t in_features);

/* Packed bytes of a whole matrix of `rows` rows: rows * pesti_row_bytes for
 * the row layouts, the super-blocks holding rows * in_features weights for
 * PESTI_FMT_Q4_K_STREAM (in_features a multiple of 64); -1 for an unknown
 * format or an invalid size. */
int64_t pesti_matrix_bytes(int32_t format, int64_t rows, int64_t in_features);

/* Static text for a status code. */
const char* pesti_strerror(int status);

/* PESTI_ABI_VERSION of the built library. */
int32_t pesti_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PESTI_H */
