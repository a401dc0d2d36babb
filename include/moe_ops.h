/*
 * moe_ops.h -- C ABI of the operators around the expert layer of moe.h: layer
 * norm, rows sorted by expert and back, and the experts' product in
 * microscaled 4-bit floating point (MXFP4), for GB300 (sm_103a).
 *
 * They are what a program needs that runs the layer's steps itself: the norm
 * in front of the layer, rows moved to an expert function of the program's own
 * and back with their gradients, and experts whose frozen weights are held in
 * 4 bits.
 *
 * Conventions (those of moe.h, with two differences):
 *  - The caller owns every buffer; no call allocates or synchronises.  Every
 *    call runs on `stream` alone.
 *  - Device pointers need the alignment of their element type only; 16-byte
 *    aligned rows take the fast path.  (Exceptions are named at the call: the
 *    4-bit operands and workspaces are 128-byte aligned.)
 *  - Row strides (ld...) are in elements and at least the row's length.
 *  - Sizes of zero are calls that write what an empty sum leaves and return
 *    MOE_OK; the pointers of empty arrays may be NULL.
 *  - Outputs must not overlap inputs or each other unless the call says so.
 *  - No floating-point atomics: outputs are bitwise the same from run to run.
 */
#ifndef MOE_OPS_GB300_H
#define MOE_OPS_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1, MOE_DT_F16 = 2 } moe_dtype;

/* ------------------------------------------------------------- layer norm
 * y = (x - mean) * rstd * weight + bias for each row of d elements, with
 * mean = sum(x) / d and rstd = 1 / sqrt(sum((x - mean)^2) / d + eps).
 *   dtype: of x and y (and dy, dx, dadd); wdtype: of weight and bias (and
 *   their gradients), either dtype or MOE_DT_F32.
 *   weight, bias: [d], either may be NULL (1 and 0).
 *   mean, rstd: [rows] fp32 outputs for the backward; both NULL or neither.
 *   Statistics and arithmetic in fp32, y rounded once.  y may be x (the same
 *   pointer and stride).  rows >= 0, 1 <= d <= 65536, eps >= 0 and finite. */
moe_status moe_layernorm_forward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d,
                                 const void* x, int64_t ldx, const void* weight, const void* bias,
                                 float eps, void* y, int64_t ldy, float* mean, float* rstd,
                                 moe_stream_t stream);

/* Bytes of device workspace moe_layernorm_backward needs (host arithmetic; 0
 * for sizes that the call refuses). */
size_t moe_layernorm_workspace_bytes(int64_t rows, int32_t d);

/* Backward of moe_layernorm_forward.  With g = dy * weight and
 * xh = (x - mean) * rstd:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dadd
 *   dweight = sum over rows of dy * xh, dbias = sum over rows of dy
 *   mean, rstd: as the forward wrote them for these rows.
 *   dadd: NULL, or a gradient [rows, d] added to dx in fp32 before its one
 *   rounding (the residual branch of a pre-norm block).
 *   dweight, dbias: [d] of wdtype, either may be NULL; summed in fp32 in an
 *   order that depends on the sizes alone; zeros for rows = 0.
 *   dx may be dy or dadd (the same pointer and stride).
 *   ws: 128-byte aligned, needed when dweight or dbias is given. */
moe_status moe_layernorm_backward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d,
                                  const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                  const void* weight, const float* mean, const float* rstd,
                                  const void* dadd, int64_t ldadd, void* dx, int64_t lddx,
                                  void* dweight, void* dbias, void* ws, size_t ws_bytes,
                                  moe_stream_t stream);

/* --------------------------------------------- rows by expert and back
 * The order moe_schedule gives the layer's own rows, for expert ids chosen
 * elsewhere.  Routed row r = t*k + j is slot j of token t.  An id outside
 * [0, E) leaves its row without an expert ("dropped": over an expert's
 * capacity, or another GPU's expert).
 *   ids     [R]   int32 in
 *   counts  [E]   int32   rows of each expert
 *   offsets [E+1] int32   exclusive prefix sum; offsets[E] = rows kept
 *   perm    [R]   int32   perm[p] = r: by expert, ascending r within one;
 *                         the dropped rows behind all others, ascending
 *   inv     [R]   int32   its inverse; inv[r] >= offsets[E] marks a dropped row
 * 0 <= R <= 2^28, 1 <= E <= 1024.  ws: 128-byte aligned, of
 * moe_sort_workspace_bytes(R, E) bytes, whose contents need not be kept. */
size_t moe_sort_workspace_bytes(int64_t R, int32_t E);
moe_status moe_sort_rows(const int32_t* ids, int64_t R, int32_t E, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

/* Rows to expert order: xp[inv[t*k+j]] = x[t] for every slot j; rows of xp
 * from offsets[E] on (dropped rows) are zeros.
 *   x [T, d] with row stride ldx; xp [T*k, d] contiguous; inv, offsets as
 *   moe_sort_rows (or moe_schedule) wrote them; T*k <= 2^28, 1 <= k <= 32.
 * Its backward is moe_unpermute without weights. */
moe_status moe_permute(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* x,
                       int64_t ldx, const int32_t* inv, const int32_t* offsets, void* xp,
                       moe_stream_t stream);

/* Rows back to token order with the routing weights applied:
 *   out[t] = base[t] + sum_j w[t*k+j] * y[inv[t*k+j]]
 * over the slots that were not dropped, in slot order in fp32 from base,
 * rounded once.  Rows of y from offsets[E] on are not read.
 *   y [T*k, d] contiguous; w [T*k] fp32 or NULL (all 1); base [T, d] or NULL
 *   (zeros); out [T, d].  out may be base (the same pointer and stride). */
moe_status moe_unpermute(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* y,
                         const float* w, const int32_t* inv, const int32_t* offsets,
                         const void* base, int64_t ldbase, void* out, int64_t ldout,
                         moe_stream_t stream);

/* Backward of moe_unpermute for an upstream gradient dout [T, d] (also the
 * gradient of base):
 *   dy[inv[t*k+j]] = w[t*k+j] * dout[t]   (zeros for dropped rows)
 *   dw[t*k+j] = <dout[t], y[inv[t*k+j]]>  (fp32; 0 for dropped rows)
 *   w NULL: all 1.  dw may be NULL, and y with it. */
moe_status moe_unpermute_backward(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E,
                                  const void* dout, int64_t lddout, const void* y, const float* w,
                                  const int32_t* inv, const int32_t* offsets, void* dy, float* dw,
                                  moe_stream_t stream);

/* ---------------------------------------------------------------- MXFP4
 * OCP MX blocks: 32 consecutive elements along K share a UE8M0 scale 2^s and
 * are E2M1 codes of 4 bits (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
 * s is the smallest exponent with max |v| <= 6 * 2^s (as moe_quantize_mxfp8
 * chooses it: no element saturates), at least -127; elements are rounded to
 * the nearest value, ties to the even code.  A block with a NaN or an infinity
 * gets the scale byte 255 (NaN), so whatever it enters becomes NaN.
 * Two codes a byte, the element of lower index in the low bits.  K is a
 * multiple of 32.  Scale bytes (s + 127) lie in 512-byte tiles of up to 128
 * rows x 4 blocks, ceil(K / 128) tiles side by side along K (a run): row r of
 * the tile, block kb at byte 16*(r%32) + 4*(r/32) + kb%4.
 *   Weights [batch, N, K]: ceil(N / 128) runs an expert, expert by expert.
 *   Rows [rows, K] in expert order, offsets [G+1] as above: rows
 *   [128 i, 128 i + 128) of expert g are run offsets[g] / 128 + g + i.
 * The bytes of blocks past K in a row's last tile are read: any but 255 (the
 * quantisers write 127).  Codes and scales are 128-byte aligned. */
enum { MOE_ACT_NONE = 0, MOE_ACT_SWIGLU = 1 };

size_t moe_mxfp4_weight_scale_bytes(int64_t batch, int32_t K, int32_t N);
size_t moe_mxfp4_row_scale_bytes(int64_t rows, int32_t K, int32_t G);

/* Weights w [batch, K, N] (the layer's W1 and W2 layouts) -> q [batch, N, K/2]
 * and scales of moe_mxfp4_weight_scale_bytes bytes.  paired != 0 (N even):
 * row 2i of an expert's codes is column i (gate) and row 2i + 1 column
 * N/2 + i (up), the order MOE_ACT_SWIGLU works on. */
moe_status moe_quantize_mxfp4(int32_t dtype, const void* w, int64_t batch, int32_t K, int32_t N,
                              int32_t paired, uint8_t* q, uint8_t* scales, moe_stream_t stream);
/* The values of quantised weights, w [batch, K, N]. */
moe_status moe_dequantize_mxfp4(int32_t dtype, const uint8_t* q, const uint8_t* scales,
                                int64_t batch, int32_t K, int32_t N, int32_t paired, void* w,
                                moe_stream_t stream);

/* Rows x (row stride ldx) -> q [rows, K/2] and scales of
 * moe_mxfp4_row_scale_bytes(rows, K, G) bytes.
 *   G, offsets: the experts' segments; offsets NULL: one segment (G = 1).
 *   perm: NULL, or [rows] int32: row p is x row perm[p] / k (rows gathered
 *   into expert order on the way; moe_sort_rows' perm).  k >= 1.
 *   Rows from offsets[G] on are not written, nor are those before offsets[0]
 *   (the offsets of some of the experts, with all rows). */
moe_status moe_quantize_mxfp4_rows(int32_t dtype, int64_t rows, int32_t K, const void* x,
                                   int64_t ldx, int32_t G, const int32_t* offsets,
                                   const int32_t* perm, int32_t k, uint8_t* q, uint8_t* scales,
                                   moe_stream_t stream);
/* The values of quantised rows, y [rows, K] with row stride ldy; rows outside
 * [offsets[0], offsets[G]) are not written. */
moe_status moe_dequantize_mxfp4_rows(int32_t dtype, int64_t rows, int32_t K, const uint8_t* q,
                                     const uint8_t* scales, int32_t G, const int32_t* offsets,
                                     void* y, int64_t ldy, moe_stream_t stream);

/* Every expert's rows times its weights: out[p] = xq[p] * wq[g]^T for p in
 * [offsets[g], offsets[g+1]), products and sums in fp32, rounded once.
 *   xq, xscales: moe_quantize_mxfp4_rows with the same rows, G and offsets
 *   (offsets NULL: G = 1, all rows).  wq, wscales: moe_quantize_mxfp4.
 *   act MOE_ACT_NONE: out [rows, N].  MOE_ACT_SWIGLU (paired weights): out
 *   [rows, N/2], out[p, i] = silu(h[2i]) * h[2i+1] of the fp32 products h.
 *   (silu to fp32 accuracy for fp32 results; for 16-bit ones to 2^-18, and 0
 *   for gates below -87, where it is below 1e-36.)
 *   dtype: of out (row stride ldo).  Rows outside [offsets[0], offsets[G]) are
 *   not written.
 *   0 <= rows <= 2^28, 1 <= G <= 1024, N >= 1, K a multiple of 32, K >= 32.
 *   ws: 128-byte aligned; moe_read_status(ws, stream) reports a wait that ran
 *   out in the last call that was given ws (each call, one without rows too,
 *   clears what the one before left). */
size_t moe_mxfp4_product_workspace_bytes(int64_t rows, int32_t N, int32_t K, int32_t G);
moe_status moe_mxfp4_product(int32_t dtype, int64_t rows, int32_t N, int32_t K, int32_t G,
                             const int32_t* offsets, const uint8_t* xq, const uint8_t* xscales,
                             const uint8_t* wq, const uint8_t* wscales, int32_t act, void* out,
                             int64_t ldo, void* ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPS_GB300_H */
