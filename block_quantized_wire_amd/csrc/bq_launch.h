// bq_launch.h -- internal launchers of the libblockq kernels (host side).
//
// Arguments are assumed valid: the public entry points in bq_abi.cpp validate every
// pointer, size, alignment and overlap before calling these.  Each launcher enqueues
// one kernel on `stream` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "blockq_kv.h"

namespace bq {

// Launch `kernel` with its one by-value argument struct on `stream` and return the
// status of this launch itself (not the thread's sticky last error, which may hold
// an earlier failure of some unrelated runtime call).
template <typename Arg>
hipError_t launch1(void (*kernel)(Arg), dim3 grid, dim3 block, hipStream_t stream, Arg arg) {
    void* args[] = {&arg};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, args, 0, stream);
}

// Flat block formats on the wire, one overload per codec (selected by the payload and
// scale pointer types): block INT8 (int8_t payload, one float scale per 128 values)
// and flat MXFP8 (uint8_t E4M3 payload, one uint8_t E8M0 byte per 32 values).  Both
// are 132 bytes per 128 values.  Segment i of a batch is (x[i] -> q[i], s[i]), n values.
hipError_t launch_quant(int count, const uint16_t* const* x, int8_t* const* q, float* const* s,
                        int64_t n, hipStream_t stream);
hipError_t launch_quant(int count, const uint16_t* const* x, uint8_t* const* v,
                        uint8_t* const* e, int64_t n, hipStream_t stream);
// skip_shard_n > 0: segment i leaves values [i*skip_shard_n, (i+1)*skip_shard_n) of
// its output untouched (the shard an all-to-all owner has already materialized).
hipError_t launch_dequant(int count, const int8_t* const* q, const float* const* s,
                          uint16_t* const* y, int64_t n, hipStream_t stream,
                          int64_t skip_shard_n = 0);
hipError_t launch_dequant(int count, const uint8_t* const* v, const uint8_t* const* e,
                          uint16_t* const* y, int64_t n, hipStream_t stream,
                          int64_t skip_shard_n = 0);
hipError_t launch_ring_hop(int count, const int8_t* const* q_in, const float* const* s_in,
                           const uint16_t* const* local, int8_t* const* q_out,
                           float* const* s_out, int64_t n, hipStream_t stream);
hipError_t launch_ring_hop(int count, const uint8_t* const* v_in, const uint8_t* const* e_in,
                           const uint16_t* const* local, uint8_t* const* v_out,
                           uint8_t* const* e_out, int64_t n, hipStream_t stream);
// nseg segments of seg_n values: segment j reads q[k] + j*seg_n (scales likewise) for
// every source k in order and writes y + j*seg_n.
hipError_t launch_accum(int nsrc, const int8_t* const* q, const float* const* s, uint16_t* y,
                        int nseg, int64_t seg_n, hipStream_t stream);
hipError_t launch_accum(int nsrc, const uint8_t* const* v, const uint8_t* const* e, uint16_t* y,
                        int nseg, int64_t seg_n, hipStream_t stream);
// The fused all-to-all owner step: accumulate as above, requantize each owner's bf16
// sum into q_out/s_out (segment j at j*seg_n), materialize it into y[j] (y or y[j] may
// be null) and store the bf16 sums into red (may be null).
hipError_t launch_a2a_reduce(int nsrc, const int8_t* const* q, const float* const* s, int nseg,
                             int64_t seg_n, int8_t* q_out, float* s_out, uint16_t* const* y,
                             uint16_t* red, hipStream_t stream);
hipError_t launch_a2a_reduce(int nsrc, const uint8_t* const* v, const uint8_t* const* e,
                             int nseg, int64_t seg_n, uint8_t* v_out, uint8_t* e_out,
                             uint16_t* const* y, uint16_t* red, hipStream_t stream);

// MXFP8 (row-major with leading dimensions; cols a multiple of 128).
// f16: x holds IEEE binary16 values instead of bf16.
hipError_t launch_quant_mx(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx,
                           uint8_t* v, int64_t ldv, uint8_t* e8m0, int64_t lds,
                           hipStream_t stream, bool f16 = false);
hipError_t launch_dequant_mx(const uint8_t* v, int64_t ldv, const uint8_t* e8m0, int64_t lds,
                             int64_t rows, int64_t cols, uint16_t* y, int64_t ldy,
                             hipStream_t stream);

// The same with the scales in the scaled-MFMA layout of `rb` 16-row blocks (base e_layout);
// the matrix's column 0 is K step `step0` of the layout.
hipError_t launch_quant_mx_mfma(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx,
                                uint8_t* v, int64_t ldv, uint8_t* e_layout, int64_t rb,
                                int64_t step0, hipStream_t stream, bool f16 = false);
hipError_t launch_dequant_mx_mfma(const uint8_t* v, int64_t ldv, const uint8_t* e_layout,
                                  int64_t rb, int64_t rows, int64_t cols, uint16_t* y,
                                  int64_t ldy, hipStream_t stream);

// The dense MXFP8 GEMM Y = bf16(X W^T) (M, N >= 1; K a positive multiple of 128).
hipError_t launch_mm_mx(const uint8_t* xv, int64_t ldxv, const uint8_t* xe, int64_t ldxe,
                        const uint8_t* wv, int64_t ldwv, const uint8_t* we, int64_t ldwe,
                        int64_t M, int64_t N, int64_t K, uint16_t* y, int64_t ldy,
                        hipStream_t stream);
// The same GEMM with both operands' scales in the scaled-MFMA layout, of xrb and wrb
// 16-row blocks.
// The column count (256 or 224) of the GEMM's workgroup tiles for an M x N product on `cus`
// compute units.
int mm_tile_cols(int64_t M, int64_t N, int cus);
hipError_t launch_mm_mx_mfma(const uint8_t* xv, int64_t ldxv, const uint8_t* xe, int64_t xrb,
                             const uint8_t* wv, int64_t ldwv, const uint8_t* we, int64_t wrb,
                             int64_t M, int64_t N, int64_t K, uint16_t* y, int64_t ldy,
                             hipStream_t stream);

// E4M3 128-block codec.
hipError_t launch_quant_e4m3_b128(const uint16_t* x, uint8_t* v, float* s, int64_t n,
                                  hipStream_t stream);
hipError_t launch_dequant_e4m3_b128(const uint8_t* v, const float* s, uint16_t* y, int64_t n,
                                    hipStream_t stream);

// The I4 codec.  f16: x, scale and y hold IEEE binary16 values instead of bf16.
// rows * (cols / 8) < 2^32.
hipError_t launch_quant_i4(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int group,
                           uint8_t* c, int64_t ldc, uint16_t* scale, int64_t lds, bool f16,
                           hipStream_t stream);
hipError_t launch_dequant_i4(const uint8_t* c, int64_t ldc, const uint16_t* scale, int64_t lds,
                             const uint8_t* zero, int64_t ldz, int64_t rows, int64_t cols,
                             int group, uint16_t* y, int64_t ldy, bool f16, hipStream_t stream);

// Products with I4 weights: y = x W^T.  Dense: off is null, `rows` rows of x and y.  Experts:
// row p in [off[e], off[e+1]) of y is x's row p, or src[p] / topk where src is not null.
struct I4Mm {
    const uint16_t* x;
    const int32_t* src;
    const int32_t* off;
    const uint8_t* c;
    const uint16_t* s;
    const uint8_t* z;
    uint16_t* y;
    int64_t ldx, ldc, lds, ldz, ldy;
    int64_t stride_c, stride_s, stride_z;
    int32_t rows, x_rows, N, K;
    int32_t topk, experts;
};
hipError_t launch_mm_i4(const I4Mm& a, int group, bool f16, hipStream_t stream);

// Tokens sorted by expert.  Sorts of up to kMoeSortOneBlock slots take one workgroup and no
// scratch, larger ones at most kMoeSortBlocks workgroups and one count per bucket and
// workgroup.
constexpr int64_t kMoeSortOneBlock = 4096;
constexpr int64_t kMoeSortBlocks = 256;
hipError_t launch_moe_sort(const int32_t* expert, int64_t slots, int experts, int32_t* off,
                           int32_t* src, int32_t* pos, void* ws, hipStream_t stream);

// Rows out and back: the order and the shape every call shares.
struct MoeRows {
    const int32_t* pos;
    const int32_t* off;
    int64_t tokens;
    int topk, experts;
    int64_t cols;
};
enum class MoeType { kBf16, kF16, kF32 };
hipError_t launch_moe_gather(const MoeRows& r, const void* x, int64_t ldx, int esize, void* out,
                             int64_t ldo, hipStream_t stream);
hipError_t launch_moe_combine(const MoeRows& r, MoeType type, const void* rows, int64_t ldr,
                              const float* weight, void* y, int64_t ldy, hipStream_t stream);
hipError_t launch_moe_combine_bwd(const MoeRows& r, MoeType type, const void* dy, int64_t lddy,
                                  const void* rows, int64_t ldr, const float* weight, void* drows,
                                  int64_t lddr, float* dweight, hipStream_t stream);

// The 4-bit cache of keys and values (see include/blockq_kv.h for the layouts).
struct KvRows {
    const uint16_t *k, *v;     // rows read by a write
    uint16_t *ko, *vo;         // rows written by a read
    int64_t ldk, hsk, ldv, hsv;
    const int32_t* slot;
    int64_t tokens;
};
hipError_t launch_kv_write(const KvRows& r, const bq_kv_i4& c, bool f16, hipStream_t stream);
hipError_t launch_kv_read(const KvRows& r, const bq_kv_i4& c, bool f16, hipStream_t stream);

struct AttnI4 {
    const uint16_t* q;
    bq_kv_i4 c;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    uint16_t* out;
    float* lse;
    void* ws;
    int64_t ldq, hsq, ldo, hso, ldt;
    int32_t table_cols, seqs, rows, max_q, max_len, heads;
    int32_t causal, window;
    float scale;
};
// How a call is cut.  The rows of one cache head (tokens times the heads that share it) go into
// tiles; few rows: all sequences' tokens are dealt out to `dealt` workgroups, many rows: the tokens of
// a sequence to `splits` of them.  The workspace holds their partial results.
struct AttnPlan {
    bool by_rows;      // waves of a workgroup take rows of their own, not tokens
    int cols;          // blocks of 16 rows to a wave
    int tiles, splits, dealt;
    int64_t ws_bytes;
};
// The workspace goes by the group too: 32 is dealt out sooner, 64 to more workgroups.
AttnPlan attn_plan(int64_t seqs, int64_t rows, int64_t max_q, int64_t max_len, int heads,
                   int kv_heads, int dim, int group);
hipError_t launch_attn_i4(const AttnI4& a, const AttnPlan& p, bool f16, hipStream_t stream);

}  // namespace bq
