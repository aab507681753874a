/*
 * blockq_kv.h -- C ABI of libblockq, the 4-bit cache of keys and values (KV-I4): rows quantised
 * into it and read back, and attention over it.
 *
 * The entry points are exported by the same library as blockq.h's and follow its conventions
 * on streams, errors (bq_status), ownership, aliasing, the 2^48 byte limit on an operand's
 * span, and device and host pointers.  Where a size makes the result empty, OK is returned,
 * nothing is launched and no pointer is read.  Non-finite values are taken as stated at each
 * entry.  _f16 entries: every bf16 below is IEEE binary16.
 */
#ifndef BLOCKQ_KV_H
#define BLOCKQ_KV_H

#include "blockq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A pool of pages, each with room for page_size tokens of every key-value head.  Slot
 * page * page_size + i is place i of a page.  A token's keys (values) of one head are dim
 * numbers; number d is code * scale + least, with a 4-bit code for each number and a bf16 scale
 * and least value for each group of `group` numbers.
 *
 * Codes of k: dim/2 bytes a token.  The 32-bit word g * (dim/32) + i of a token's row holds
 * numbers 32i + 8g .. 32i + 8g + 7, the first in the lowest nibble (g < 4, i < dim/32).
 * Codes of v: blocks of 8 tokens, 4 * dim bytes each.  Number 16j + r of token t of a block is
 * nibble j % 4 of half-word t % 2 of the block's 32-bit word (r*4 + t/2) * (dim/64) + j/4.
 * ks, vs: [dim/group][page_size] pairs of 16-bit numbers, scale and least.
 *
 * Page p of head h: codes at p * page_stride + h * head_stride bytes, scales at
 * p * spage_stride + h * shead_stride 16-bit entries; the same strides serve k and v, and pages
 * and heads may be nested either way.  dim is 64, 128 or 256; group 32, 64 or 128, at most dim;
 * page_size a multiple of 8, pages * page_size < 2^31, 1 <= heads <= 1024 (else BQ_ERR_SIZE).
 * Pointers are 16-byte aligned, code strides multiples of 16, scale strides of 8 entries (else
 * BQ_ERR_ALIGN); pages and heads must not overlap (else BQ_ERR_BOUNDS).  The struct is read
 * during a call only. */
typedef struct bq_kv_i4 {
    uint8_t* k;
    uint8_t* v;
    uint16_t* ks;
    uint16_t* vs;
    int64_t page_stride, head_stride;
    int64_t spage_stride, shead_stride;
    int32_t pages, page_size, heads, dim, group;
} bq_kv_i4;

/* Rows of keys and values -> the cache, asymmetric.  Per group: lo and hi are the least and the
 * largest number; scale = bf16_rne(fl32((hi - lo) / 15)), least = lo; code = round-half-even(
 * fl32((x - lo) / scale)) clamped to [0, 15], 0 where the scale is 0.  A group with a NaN or
 * an infinity gets a scale and a least value of NaN.
 * k, v: bf16, head h of token t at t * ldk + h * hsk (t * ldv + h * hsv) entries, any strides
 * >= 0 that are multiples of 8, 16-byte aligned pointers.  slot: int32[tokens]; tokens whose
 * slot is outside [0, pages * page_size) are left out.  Slots of one call must differ: one that is
 * named twice holds a mix of its tokens' codes.  tokens < 2^31 / heads. */
bq_status bq_kv_write_i4(const uint16_t* k, int64_t ldk, int64_t hsk, const uint16_t* v, int64_t ldv,
                         int64_t hsv, const int32_t* slot, int64_t tokens, const bq_kv_i4* cache,
                         void* stream);
bq_status bq_kv_write_i4_f16(const uint16_t* k, int64_t ldk, int64_t hsk, const uint16_t* v,
                             int64_t ldv, int64_t hsv, const int32_t* slot, int64_t tokens,
                             const bq_kv_i4* cache, void* stream);

/* The cache -> rows: bf16_rne(fl32(code * scale + least)), one rounding to binary32.  A scale that
 * was rounded up can take a group's largest number past the type's range; it comes back infinite then.
 * Rows of slots outside the cache become 0; a slot may be named any number of times.  k and v as above,
 * apart from each other, heads and tokens that do not overlap. */
bq_status bq_kv_read_i4(const bq_kv_i4* cache, const int32_t* slot, int64_t tokens, uint16_t* k,
                        int64_t ldk, int64_t hsk, uint16_t* v, int64_t ldv, int64_t hsv,
                        void* stream);
bq_status bq_kv_read_i4_f16(const bq_kv_i4* cache, const int32_t* slot, int64_t tokens, uint16_t* k,
                            int64_t ldk, int64_t hsk, uint16_t* v, int64_t ldv, int64_t hsv,
                            void* stream);

/* Attention over the cache.  Sequence b has lens[b] tokens in the cache, token t in place
 * t % page_size of page table[b * ldt + t / page_size], and rows [starts[b], starts[b+1]) of q
 * (starts NULL: row b alone), n_b of them, which are its last tokens: row i stands at place
 * lens[b] - n_b + i.  q: `heads` heads of dim numbers, head j reads the cache's head
 * j / (heads / cache->heads).  For every row and head, over the tokens t that the row sees:
 *   score_t = scale * sum over d of q_d * k_td;   lse = ln(sum over t of exp(score_t));
 *   out_d = bf16_rne( sum over t of exp(score_t - lse) * v_td ).
 * A row at place p sees tokens [0, lens[b]); with causal != 0 those up to p; with window > 0
 * those after p - window.  A row that sees nothing becomes 0, its lse -inf.  Rows of no
 * sequence are not written.  |scale| is at most 2^126 (else BQ_ERR_SIZE); where |scale| times a number of
 * q passes 2^117, that row and head may become NaN.  Tokens that a row does not see have no effect on it, whatever their
 * codes and scales hold (but for the bits that much larger scales of v cost, see below).
 *
 * Scores, softmax and sums are in binary32; q is exact but for numbers 2^-24 below the largest of
 * their row, and in rows below 2^-100.  Before the product with the values, exp(score_t - lse) is
 * held to half a step of binary16 (2^-11 relative; in the _f16 calls 2^-21), and so is v_t where a
 * call has many rows.  In the _f16 calls v_t may be beyond binary16's range; it is read back as an
 * infinity, but counts as what it is here.  Values of v that are 2^-16 of the largest of their
 * sequence and head or less lose further bits, the smaller the more; weights and lse do not go by
 * the values.  Scales and least values, of keys too, are at most 2^100.  A NaN or an infinity in a
 * row of q makes every value of that row and head NaN, one in the scales of a token does not reach
 * rows that do not see it.  The same call gives the same bits.
 *
 * q, out: row stride ldq, ldo, head stride hsq, hso entries, multiples of 8, 16-byte aligned;
 * rows and heads of out must not overlap.  table: int32, `table_cols` <= ldt entries a sequence;
 * lens: int32[seqs]; starts: int32[seqs + 1], ascending, or NULL
 * (max_q is then taken as 1).  lse: float[rows][heads] or NULL.
 * max_q, max_len: at least every n_b and lens[b]; 0 <= lens[b].  What the arrays hold beyond
 * that is brought inside: lens to [0, min(max_len, table_cols * page_size)], rows of a sequence
 * beyond max_q are not computed (the others stay in their places), and the tokens of a page outside [0, pages) are seen by no row.
 * heads is a multiple of cache->heads, at most 64 times as many; seqs, max_q <= 2^20, rows *
 * heads < 2^31, max_len < 2^30 (else BQ_ERR_SIZE).  With n = max_q * heads / cache->heads rows to a
 * sequence and head of the cache, seqs * cache->heads * ceil(n / 16) is below 2^24 for n <= 64, and
 * seqs * cache->heads * ceil(n / 128) below 2^23 else; where ws is used, seqs * max_q * heads
 * is below 2^24 (else BQ_ERR_SIZE).
 * ws: scratch of at least bq_attn_i4_ws_bytes bytes, 16-byte aligned, never more than 64 MiB,
 * NULL where that is 0; its contents do not matter, and calls that may run at the same time
 * (two streams, two graphs) need one each. */
bq_status bq_attn_i4(const uint16_t* q, int64_t ldq, int64_t hsq, const bq_kv_i4* cache,
                     const int32_t* table, int64_t ldt, int64_t table_cols, const int32_t* lens,
                     const int32_t* starts, int64_t seqs, int64_t rows, int64_t max_q,
                     int64_t max_len, int heads, int causal, int64_t window, float scale,
                     uint16_t* out, int64_t ldo, int64_t hso, float* lse, void* ws,
                     int64_t ws_bytes, void* stream);
bq_status bq_attn_i4_f16(const uint16_t* q, int64_t ldq, int64_t hsq, const bq_kv_i4* cache,
                         const int32_t* table, int64_t ldt, int64_t table_cols, const int32_t* lens,
                         const int32_t* starts, int64_t seqs, int64_t rows, int64_t max_q,
                         int64_t max_len, int heads, int causal, int64_t window, float scale,
                         uint16_t* out, int64_t ldo, int64_t hso, float* lse, void* ws,
                         int64_t ws_bytes, void* stream);

/* Scratch bytes of bq_attn_i4 for these sizes; -1 for sizes outside the limits. */
int64_t bq_attn_i4_ws_bytes(int64_t seqs, int64_t rows, int64_t max_q, int64_t max_len, int heads,
                            int kv_heads, int dim);

#ifdef __cplusplus
}
#endif
#endif /* BLOCKQ_KV_H */
