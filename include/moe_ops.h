/*
 * moe_ops.h -- C ABI of the operators around the expert layer of moe.h: layer
 * norm, rows sorted by expert and back, the experts' products with their
 * gradients, SwiGLU and activation checkpoints in 8 bits (MXINT8), and the
 * experts' product in microscaled 4-bit floating point (MXFP4), for GB300
 * (sm_103a).
 *
 * They are what a program needs that runs the layer's steps itself: the norm
 * in front of the layer, rows moved to an expert function of the program's own
 * and back with their gradients, that function's products and activation in
 * training, and experts whose frozen weights are held in 4 bits.
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

/* ------------------------------------------------- products by expert
 * Every expert's rows times its weights, on rows as moe_permute lays them:
 * expert g's are [offsets[g], offsets[g+1]), any number of them, none included.
 *   out[p] = x[p] * w[g]     w [G, K, N]  (the layer's W1 and W2 layouts)
 *   out[p] = x[p] * w[g]^T   w [G, N, K]  (transposed != 0)
 * With w [G, K, N] the gradient of the rows of the first form is the second
 * form on dy [rows, N] with K and N changed places; that of the weights is
 * moe_grouped_product_dw.
 *   dtype: of x and w; odtype: of out, dtype or MOE_DT_F32.  Products and sums
 *   in fp32, each result rounded once.  (All run on the tensor cores, which add 16
 *   terms at a time and truncate.  A sum there takes 512 terms, 1024 for 16-bit
 *   results; longer ones are added up from several, rounded to nearest.  So the sums
 *   are off by less than 2^-16 of their n terms' magnitudes and n 2^-32 of them, and
 *   in practice by 5e-7 of a result whatever n (operands of 16 bits; of fp32 3e-7;
 *   for 16-bit results 1e-6 before their rounding).  fp32 values are split into three
 *   parts of 8 bits: below 2^-102 they are held to 2^-126, and a sum with an infinity
 *   in it may be NaN instead.)
 *   x [rows, K], out [rows, N] with row strides ldx, ldo; w contiguous.  A
 *   result overlaps no operand.
 *   offsets [G+1], not decreasing; NULL: G = 1, all rows.  Rows outside
 *   [offsets[0], offsets[G]) are neither used nor written.
 *   0 <= rows <= 2^28, 1 <= G <= 1024, 1 <= K, N <= 2^22, no array of more than
 *   2^40 elements.
 *   16-byte aligned x, w and row strides are the fast path.
 *   ws: 128-byte aligned, of moe_grouped_product_workspace_bytes(rows, K, N, G)
 *   bytes, which serve both calls and either form, of these or fewer rows (at most
 *   about 20 MB); calls that may overlap need one each.  moe_read_status(ws, stream) reports a wait that ran out in the
 *   last call that was given ws. */
size_t moe_grouped_product_workspace_bytes(int64_t rows, int32_t K, int32_t N, int32_t G);
moe_status moe_grouped_product(int32_t dtype, int32_t odtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                               const int32_t* offsets, const void* x, int64_t ldx, const void* w,
                               int32_t transposed, void* out, int64_t ldo, void* ws, size_t ws_bytes,
                               moe_stream_t stream);
/* Gradient of the weights: dw[g] = sum over g's rows p of x[p]^T * dy[p], [G, K, N]
 * contiguous; an expert without rows gets zeros.
 *   wdtype: of dw, dtype or MOE_DT_F32.  accumulate != 0: added to dw (in fp32,
 *   rounded once), which an expert without rows then keeps. */
moe_status moe_grouped_product_dw(int32_t dtype, int32_t wdtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                                  const int32_t* offsets, const void* x, int64_t ldx, const void* dy,
                                  int64_t lddy, void* dw, int32_t accumulate, void* ws, size_t ws_bytes,
                                  moe_stream_t stream);

/* ---------------------------------------------------------------- MXINT8
 * Rows kept in 8 bits between a forward and its backward.  32 consecutive
 * elements of a row (its last block may be shorter) share a UE8M0 scale 2^s and
 * are whole numbers c in [-127, 127]; their values are c * 2^s.
 * s is the smallest exponent with max |v| <= 127 * 2^s, at least -127; elements
 * are rounded to the nearest, ties to even, so a value is off by at most
 * 2^(s-1) <= max |v| / 127.  (A block that ends in the last 2^122 of fp32's
 * range is cut to 63 * 2^122: finite values stay finite.)  A block with a NaN
 * or an infinity gets the scale byte 255 (NaN) and comes back as NaN.
 * (The OCP MX format of this name counts its elements in 64ths, c / 64 * 2^s: the
 * same codes have a scale byte that is 6 higher there.  What leaves the program for
 * a reader of that format needs 6 added to each byte below 249.)
 *   codes [rows, n] contiguous, scale bytes (s + 127) [rows, ceil(n / 32)]
 *   contiguous.  Codes in 8-byte aligned rows take the fast path. */
size_t moe_mxint8_scale_bytes(int64_t rows, int32_t n);
moe_status moe_quantize_mxint8_rows(int32_t dtype, int64_t rows, int32_t n, const void* x, int64_t ldx,
                                    int8_t* q, uint8_t* scales, moe_stream_t stream);
/* The values, y [rows, n] with row stride ldy (in fp16 at most 65504). */
moe_status moe_dequantize_mxint8_rows(int32_t dtype, int64_t rows, int32_t n, const int8_t* q,
                                      const uint8_t* scales, void* y, int64_t ldy, moe_stream_t stream);

/* ---------------------------------------------------------------- SwiGLU
 * a = silu(g) * u of rows h = [g | u] of 2f elements, silu(g) = g / (1 + exp(-g)),
 * in fp32, rounded once.  (silu is within 2^-20 of itself in fp32; for 16-bit types
 * within 2^-18 for gates from -20 on, 2^-16 down to -87, and 0 below, where it is
 * below 1e-36.)
 *   q, scales: NULL, or a checkpoint of h for the backward: MXINT8 of the two
 *   halves of each row, codes [rows, 2f] and scales [rows, 2 * ceil(f / 32)]
 *   (moe_quantize_mxint8_rows of 2 * rows rows of f).
 *   h [rows, 2f], a [rows, f] with row strides ldh, lda.
 *   0 <= rows <= 2^30, 1 <= f <= 2^22 (n of the calls above too). */
moe_status moe_swiglu_forward(int32_t dtype, int64_t rows, int32_t f, const void* h, int64_t ldh, void* a,
                              int64_t lda, int8_t* q, uint8_t* scales, moe_stream_t stream);
/* Backward for the gradient da [rows, f] of a: with s = 1 / (1 + exp(-g)),
 *   dh = [da * u * s * (1 + g * (1 - s)) | da * g * s]
 *   a  = g * s * u again (NULL: not wanted), the rows of the next weights'
 *        gradient, which then need not be kept.
 *   g, u: of h, or where h is NULL of the checkpoint q, scales.
 *   dh may be h and a may be da (the same pointer and stride). */
moe_status moe_swiglu_backward(int32_t dtype, int64_t rows, int32_t f, const void* da, int64_t ldda,
                               const void* h, int64_t ldh, const int8_t* q, const uint8_t* scales, void* dh,
                               int64_t lddh, void* a, int64_t lda, moe_stream_t stream);

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
 *   (silu to fp32 accuracy for fp32 results; for 16-bit ones to 2^-18 for gates
 *   from -20 on, 2^-16 down to -87, and 0 below, where it is below 1e-36.)
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
