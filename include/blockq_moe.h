/*
 * blockq_moe.h -- C ABI of libblockq, the expert layer: products with 4-bit weights (I4), the
 * codec of those weights, and tokens sorted by expert and back, with gradients.
 *
 * The entry points are exported by the same library as blockq.h's and follow its conventions
 * on streams, errors (bq_status), ownership, aliasing, the 2^48 byte limit on an operand's
 * span, and device and host pointers.  In place calls are not allowed: every output is apart
 * from every input.  Where a size makes the result empty, OK is returned, nothing is launched
 * and no pointer is read, unless an entry says otherwise.  Unlike blockq.h's codecs these
 * entries take non-finite values: the moved and summed rows follow IEEE arithmetic, the 4-bit
 * codec and products as stated there, and no value reaches the results of another row.
 */
#ifndef BLOCKQ_MOE_H
#define BLOCKQ_MOE_H

#include "blockq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ==== I4: 4-bit weights with group scales ============================================
 *
 * A matrix W of N rows and K columns as three row-major arrays:
 *   c     u8[N][ldc]: column 2j of a row in the low nibble of byte j, column 2j+1 in the
 *         high nibble, codes 0..15;
 *   scale bf16[N][lds] (binary16 in the _f16 calls): entry g of a row scales columns
 *         [g*group, (g+1)*group);
 *   zero  u8[N][ldz], or NULL: entry g is the zero point of the same columns, 0..15
 *         (bits 4..7 are ignored); NULL means 8 everywhere.
 * W[n][k] = (code - zero) * scale.  group is 32, 64 or 128 and K a multiple of it.
 * Layout rules: c 16-byte aligned, ldc >= K/2, ldc % 16 == 0; scale 8-byte aligned, lds >=
 * K/group, lds % 4 == 0; zero 4-byte aligned, ldz >= K/group, ldz % 4 == 0.  Scale and zero
 * rows are read in whole fours of entries, so the entries after the last group, up to the
 * next multiple of 4, must be readable (they are not used). */

/* bf16 rows -> I4 codes and scales, symmetric (zero point 8).  Per group: amax = max |x|;
 * scale = bf16_rne(fl32(amax / 7)); code = 8 + q, q = round-half-even(fl32(x / scale))
 * clamped to [-7, 7]; q = 0 where the scale is +0.  A NaN in a group makes its scale NaN and
 * its codes 8; without one, an infinity makes the scale +inf, infinities q = 7 and -7 and
 * finite values q = 0 (so that they come back as themselves and as NaN).  x: bf16[rows][ldx], 16-byte aligned,
 * ldx >= cols, ldx % 8 == 0.  Entries of c and scale beyond a row's columns and groups are
 * not written.  rows * cols / 8 < 2^32.  _f16: x and scale are IEEE binary16 (scale =
 * f16_rne(fl32(amax / 7))). */
bq_status bq_quant_i4(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int group,
                      uint8_t* c, int64_t ldc, uint16_t* scale, int64_t lds, void* stream);
bq_status bq_quant_i4_f16(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int group,
                          uint8_t* c, int64_t ldc, uint16_t* scale, int64_t lds, void* stream);

/* I4 -> bf16: y = bf16_rne((code - zero) * scale), the product exact in binary32.
 * y: bf16[rows][ldy], 16-byte aligned, ldy >= cols, ldy % 8 == 0.  _f16: binary16. */
bq_status bq_dequant_i4(const uint8_t* c, int64_t ldc, const uint16_t* scale, int64_t lds,
                        const uint8_t* zero, int64_t ldz, int64_t rows, int64_t cols, int group,
                        uint16_t* y, int64_t ldy, void* stream);
bq_status bq_dequant_i4_f16(const uint8_t* c, int64_t ldc, const uint16_t* scale, int64_t lds,
                            const uint8_t* zero, int64_t ldz, int64_t rows, int64_t cols,
                            int group, uint16_t* y, int64_t ldy, void* stream);

/* Y[m][n] = bf16_rne( sum over k of X[m][k] * W[n][k] ): X bf16[M][ldx] (16-byte aligned,
 * ldx >= K, ldx % 8 == 0), W the I4 matrix of N rows; y bf16[M][ldy], ldy >= N.  The sums over
 * a group are taken in binary32 by the matrix cores from exact products (of x and code -
 * zero, or of x and 16 + code and of x alone, subtracted afterwards), the group's scale is
 * applied to them in binary32, and y is rounded once.  The same call gives the same bits;
 * the order of the sums depends on the sizes.  No finite x overflows a group's sums (bf16 takes
 * them at 2^-12 of their size), so y is finite where the sum over the groups is; bf16 results
 * below about 2^-100 hold an absolute error of up to 2^-138 a group.  A NaN or an infinity in a
 * row of x makes every value of that row of y NaN or infinite, one among a row's scales every
 * value of that column.  M == 0 or N == 0
 * launches nothing; K must be positive, M and K at most 2^30 and N at most 2^26 (else
 * BQ_ERR_SIZE).  y must not overlap an input.  _f16: X, scale and
 * Y are binary16. */
bq_status bq_mm_i4(const uint16_t* x, int64_t ldx, const uint8_t* c, int64_t ldc,
                   const uint16_t* scale, int64_t lds, const uint8_t* zero, int64_t ldz,
                   int64_t M, int64_t N, int64_t K, int group, uint16_t* y, int64_t ldy,
                   void* stream);
bq_status bq_mm_i4_f16(const uint16_t* x, int64_t ldx, const uint8_t* c, int64_t ldc,
                       const uint16_t* scale, int64_t lds, const uint8_t* zero, int64_t ldz,
                       int64_t M, int64_t N, int64_t K, int group, uint16_t* y, int64_t ldy,
                       void* stream);

/* ==== The expert layer: tokens sorted by expert, expert products, and back ============
 *
 * A router gives every token topk experts; slot t*topk + j is token t's choice j.  Sorted
 * rows are the slots ordered by expert, equal experts in slot order; slots whose id is
 * outside [0, experts) are dropped: they come last, and nothing of their rows is used.
 * Three int32 arrays describe the order, and every call below reads it from them:
 *   off[experts + 1]: rows [off[e], off[e+1]) belong to expert e; off[experts] rows are kept;
 *   src[tokens*topk]: the slot in each row;   pos[tokens*topk]: the row of each slot.
 * 1 <= topk <= BQ_MAX_TOPK, 1 <= experts <= BQ_MAX_EXPERTS (else BQ_ERR_NSRC); tokens * topk
 * < 2^30 and at most 2^22 columns in a row that is moved (else BQ_ERR_SIZE).  Entries of the arrays that are out of range (arrays not made
 * by bq_moe_sort) are never used as addresses: rows past the arrays' ends are skipped.
 * int32 and float arrays are 4-byte aligned. */
#define BQ_MAX_TOPK 64
#define BQ_MAX_EXPERTS 1024

/* Scratch bytes of bq_moe_sort: 0 up to 4096 slots, else 1024 * (experts + 1).  Returns -1
 * for sizes outside the limits. */
int64_t bq_moe_sort_ws_bytes(int64_t tokens, int topk, int experts);

/* The stable sort: expert int32[tokens*topk] -> off, src, pos.  ws: caller-owned scratch of
 * ws_bytes >= bq_moe_sort_ws_bytes (else BQ_ERR_SCRATCH), 4-byte aligned, may be NULL where
 * that is 0; its contents before and after do not matter.  tokens == 0 writes off = 0. */
bq_status bq_moe_sort(const int32_t* expert, int64_t tokens, int topk, int experts, int32_t* off,
                      int32_t* src, int32_t* pos, void* ws, int64_t ws_bytes, void* stream);

/* out[pos[t*topk + j]] = x[t] for every kept slot, and zeros in the rows of dropped slots:
 * x [tokens][ldx], out [tokens*topk][ldo], cols values of esize bytes (2 or 4) in a row; any
 * cols, ldx >= cols, ldo >= cols, pointers aligned to esize.  Its gradient is
 * bq_moe_combine without weights. */
bq_status bq_moe_gather(const void* x, int64_t ldx, const int32_t* pos, const int32_t* off,
                        int64_t tokens, int topk, int experts, int64_t cols, int esize, void* out,
                        int64_t ldo, void* stream);

/* y[t] = rne( sum over kept slots j of weight[t*topk + j] * rows[pos[t*topk + j]] ), j
 * ascending, products and sums rounded separately in binary32, +0 for a token without kept
 * slots.  weight: float[tokens*topk], or NULL for weights of 1.  rows: [tokens*topk][ldr],
 * y: [tokens][ldy], cols values in a row, any cols; bf16, binary16 (_f16) or binary32
 * (_f32), naturally aligned.  What the rows of dropped slots hold (NaN too) has no effect. */
bq_status bq_moe_combine(const uint16_t* rows, int64_t ldr, const int32_t* pos, const int32_t* off,
                         const float* weight, int64_t tokens, int topk, int experts, int64_t cols,
                         uint16_t* y, int64_t ldy, void* stream);
bq_status bq_moe_combine_f16(const uint16_t* rows, int64_t ldr, const int32_t* pos,
                             const int32_t* off, const float* weight, int64_t tokens, int topk,
                             int experts, int64_t cols, uint16_t* y, int64_t ldy, void* stream);
bq_status bq_moe_combine_f32(const float* rows, int64_t ldr, const int32_t* pos,
                             const int32_t* off, const float* weight, int64_t tokens, int topk,
                             int experts, int64_t cols, float* y, int64_t ldy, void* stream);

/* The gradient of bq_moe_combine.  For every kept slot s = t*topk + j: drows[pos[s]] =
 * rne(weight[s] * dy[t]) and dweight[s] = sum over columns of rows[pos[s]] * dy[t] in
 * binary32 (a fixed order for given cols); for a dropped slot both are 0.  dy: [tokens][lddy],
 * rows and drows: [tokens*topk][ldr], [tokens*topk][lddr]; weight, dweight:
 * float[tokens*topk]. */
bq_status bq_moe_combine_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* rows, int64_t ldr,
                             const int32_t* pos, const int32_t* off, const float* weight,
                             int64_t tokens, int topk, int experts, int64_t cols, uint16_t* drows,
                             int64_t lddr, float* dweight, void* stream);
bq_status bq_moe_combine_bwd_f16(const uint16_t* dy, int64_t lddy, const uint16_t* rows,
                                 int64_t ldr, const int32_t* pos, const int32_t* off,
                                 const float* weight, int64_t tokens, int topk, int experts,
                                 int64_t cols, uint16_t* drows, int64_t lddr, float* dweight,
                                 void* stream);
bq_status bq_moe_combine_bwd_f32(const float* dy, int64_t lddy, const float* rows, int64_t ldr,
                                 const int32_t* pos, const int32_t* off, const float* weight,
                                 int64_t tokens, int topk, int experts, int64_t cols, float* drows,
                                 int64_t lddr, float* dweight, void* stream);

/* The expert products on sorted rows: for every expert e and row p in [off[e], off[e+1]),
 * y[p] = rne( X_p W_e^T ) with bq_mm_i4's arithmetic, X_p = x[p], or x[src[p] / topk] where
 * src is not NULL (the tokens unsorted; x_rows rows of x).  W_e is the I4 matrix of N rows
 * and K columns at c + e*stride_c, scale + e*stride_s, zero + e*stride_z (strides in
 * elements: at least N rows, stride_c % 16 == 0, the others % 4 == 0).  rows is the number of
 * rows of y (tokens*topk); rows outside every expert are not written, and a row whose source
 * names no row of x (src negative, or too large) becomes 0.  topk is ignored
 * where src is NULL; x must then hold `rows` rows (x_rows >= rows). */
bq_status bq_moe_mm_i4(const uint16_t* x, int64_t ldx, int64_t x_rows, const int32_t* src, int topk,
                       const int32_t* off, int experts, int64_t rows, const uint8_t* c,
                       int64_t ldc, int64_t stride_c, const uint16_t* scale, int64_t lds,
                       int64_t stride_s, const uint8_t* zero, int64_t ldz, int64_t stride_z,
                       int64_t N, int64_t K, int group, uint16_t* y, int64_t ldy, void* stream);
bq_status bq_moe_mm_i4_f16(const uint16_t* x, int64_t ldx, int64_t x_rows, const int32_t* src,
                           int topk, const int32_t* off, int experts, int64_t rows,
                           const uint8_t* c, int64_t ldc, int64_t stride_c, const uint16_t* scale,
                           int64_t lds, int64_t stride_s, const uint8_t* zero, int64_t ldz,
                           int64_t stride_z, int64_t N, int64_t K, int group, uint16_t* y,
                           int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* BLOCKQ_MOE_H */
