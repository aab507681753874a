// bq_mmi4.hip -- products with 4-bit weights and group scales (I4), dense and by expert.
//
// Definition: Y[m][n] = rne( sum over k of X[m][k] * (code[n][k] - zero[n][g]) * scale[n][g] ),
// g = k / G the group of G = 32, 64 or 128 columns.  For one group
//   sum x (code - zero) = sum x (16 + code) - (16 + zero) * sum x,
// and 16 + code is a bf16 (binary16) number whose significand holds the code's four bits as
// they are: a pair of codes becomes a pair of matrix operands with one shift and one
// and-or.  Both sums run on the matrix cores in binary32 (sum x as a product with ones), and
// the group's scale multiplies their difference once, in binary32.  The offset of 16 costs
// at most a factor of 16 + zero over |code - zero| in the rounding of binary32 sums.  (bf16
// has no packed subtraction; binary16 has, and k_mm_i4 subtracts the zero point there.)
//
// Range.  A group's sums reach 128 * 31 |x|, which bf16's larger values would take out of
// binary32 although the product itself is finite.  So bf16's operands are (16 + code) / 4096 and,
// for sum x, 1 / 4096: no finite x overflows, and nothing is lost below, since x is a multiple
// of 2^-133 and the products one of 2^-145, where binary32 ends at 2^-149 (the matrix cores
// keep subnormals).  The factor comes back once, on a finished result: a power of two changes no
// rounding of the sums, but results below about 2^-100 hold up to 2^-138 a group of error, and
// the scales stay as they are, so that the largest ones do not overflow either.  Binary16 sums
// stay below 2^28 as they are.
//
// Three kernels, chosen by the row counts (launch_shape): k_ms_i4 for up to 16 rows, bound by the
// bytes of the weights; k_mv_i4 for more in products that keep few workgroups busy, bound by
// the making of operands; and k_mm_i4, bound by the matrix cores and the vector
// instructions that feed them.  Rates at a stated size stand at each.
#include "bq_device.h"
#include "bq_launch.h"
#include "bq_ranges.h"

namespace bq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

constexpr int kUnit = 256;       // columns of a unit: 128 bytes of codes of a row

// What the sums of x are made with (two to a word): 1, or bf16's 2^-12.
template <bool F16>
constexpr uint32_t kOnes = F16 ? 0x3C003C00u : 0x39803980u;

template <bool F16>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h16x8, a),
                                                      __builtin_bit_cast(h16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ float to_f32(uint32_t h) {   // the low half of h
    if constexpr (F16)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    else
        return __uint_as_float(h << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float f) {
    if constexpr (F16)
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    else
        return (uint16_t)pack_bf16x2(f, 0.0f);
}

// A finished sum, back at its size and rounded.
template <bool F16>
__device__ __forceinline__ uint16_t result(float sum) {
    return from_f32<F16>(F16 ? sum : sum * 4096.0f);
}

// The 8 codes of a word as operands 16 + code (bf16: over 4096), in the order 0,4, 1,5, 2,6, 3,7
// (codes i and i+4 are 16 bits apart).  The code's bits go to the top of the significand: bits
// 3..6 of a bf16 2^-8 (0x3B80), bits 6..9 of a binary16 16.0 (0x4C00).  The mask and the base are held
// in registers, so that the two steps are one shift and one and-or (an instruction takes no
// two literals).
template <bool F16>
struct Codes {
    uint32_t mask, base;
    __device__ __forceinline__ Codes()
        : mask(F16 ? 0x03C003C0u : 0x00780078u), base(F16 ? 0x4C004C00u : 0x3B803B80u) {
        asm("" : "+s"(mask));
        asm("" : "+v"(base));
    }
    __device__ __forceinline__ u32x4 operands(uint32_t w) const {
        constexpr int up = F16 ? 6 : 3;
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = 4 * i < up ? w << (up - 4 * i) : w >> (4 * i - up);
            r[i] = (v & mask) | base;
        }
        return r;
    }
};

// 8 values of x (16 bytes) in the operands' order.
__device__ __forceinline__ u32x4 in_order(u32x4 x) {
    return u32x4{__builtin_amdgcn_perm(x.z, x.x, 0x05040100u),
                 __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                 __builtin_amdgcn_perm(x.w, x.y, 0x05040100u),
                 __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

// A lane loads 32 consecutive columns of its row of W: lane quarter g has columns [32g, 32g+32)
// of 128, 8 to a word.  The four words of the four quarters are exchanged (halves of the wave
// first, then odd and even quarters), so that word j holds columns [32j + 8g, 32j + 8g + 8):
// one matrix instruction then takes 32 adjacent columns, which lie in one group, and its
// operand of x is 64 adjacent bytes of each row.
__device__ __forceinline__ u32x4 exchange(u32x4 q) {
    const auto a = __builtin_amdgcn_permlane32_swap(q.x, q.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(q.y, q.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

struct Args : I4Mm {
    int32_t units;      // ceil(K / 256)
    int32_t block0;     // first row block of a launch of many
};

// The row of x that row m of y is made from, and whether a source names one that is there (a
// row whose source is out of range gives zeros, and reads row 0 meanwhile).
__device__ __forceinline__ bool x_row_ok(const Args& p, int m) {
    return !p.src || source_row(p.src[m], p.topk, p.x_rows) >= 0;
}
__device__ __forceinline__ int64_t x_row(const Args& p, int m) {
    return p.src ? max(source_row(p.src[m], p.topk, p.x_rows), 0) : m;
}

// One unit's data of one block of 16 rows of W: 256 columns are one 128-byte line of codes of
// each row, and the scales and zero points of a row's 256 / G groups.
template <int G, bool Z>
struct Weights {
    u32x4 q[2];
    uint32_t s[kUnit / G / 2];            // two scales to a word
    uint32_t z[G == 32 ? 2 : 1];          // four zero points to a word
};

template <int G, bool Z, bool Tail>
__device__ __forceinline__ void load_unit(Weights<G, Z>& w, const uint8_t* c, const uint16_t* s,
                                          const uint8_t* z, int unit, int g, int K) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = unit * kUnit + h * 128 + 32 * g;
        w.q[h] = ld16(c + (Tail ? min(k, K - 32) : k) / 2);
    }
    if constexpr (G == 128) {
        w.s[0] = *reinterpret_cast<const uint32_t*>(s + unit * 2);
        if constexpr (Z)
            w.z[0] = *reinterpret_cast<const uint16_t*>(z + unit * 2);
    } else if constexpr (G == 64) {
        const u32x2 v = ld8(s + unit * 4);
        w.s[0] = v.x;
        w.s[1] = v.y;
        if constexpr (Z)
            w.z[0] = *reinterpret_cast<const uint32_t*>(z + unit * 4);
    } else {
        // rows of scales are whole fours of groups, which a unit may have one or two of
        const int second = Tail ? min(unit * 8 + 4, (K / 32 - 1) & ~3) : unit * 8 + 4;
        const u32x2 u = ld8(s + unit * 8), v = ld8(s + second);
        w.s[0] = u.x;
        w.s[1] = u.y;
        w.s[2] = v.x;
        w.s[3] = v.y;
        if constexpr (Z) {
            w.z[0] = *reinterpret_cast<const uint32_t*>(z + unit * 8);
            w.z[1] = *reinterpret_cast<const uint32_t*>(z + second);
        }
    }
}

// Everything a wave reads for a unit: R blocks of 16 weight rows, and the 8 operands of x of
// MT blocks of 16 tokens.
template <int G, bool Z, int MT, int R>
struct Buf {
    Weights<G, Z> w[R];
    u32x4 x[MT][8];
};

// Global-to-LDS load of 16 (4) bytes per lane: lane i's land at lds + 16 i (4 i).
__device__ __forceinline__ void lds_load16(const void* p, void* lds) {
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}
__device__ __forceinline__ void lds_load4(const void* p, void* lds) {
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
}
// Until at most N of this wave's loads are outstanding, and then for the other waves.
template <int N>
__device__ __forceinline__ void wait_and_join() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Few rows of x, by expert or more than 16 of them: the weights go straight into registers, one
// unit of 256 columns at a time; what covers a unit's loads are the other waves of the compute
// unit.  A workgroup takes R blocks of 16 weight rows and KW waves that take the units in turn;
// their sums meet in LDS in wave order.  A wave's products take MT blocks of 16 rows of x; dense
// rows beyond them are other workgroups', an expert's are this one's next.  Operand row n16 of a
// block is token n16 / 4 + 4 (n16 % 4), so that lane quarter g holds the results of tokens g + 4i.
// Tail: K is not a multiple of 256.  The columns that the last unit lacks are whole groups:
// their loads are moved to columns that are there, and the groups are left out.
template <bool F16, int G, bool Z, bool Tail, int MT, int R, int KW>
__global__ __launch_bounds__(64 * KW) __attribute__((amdgpu_waves_per_eu(2))) void k_mv_i4(Args p) {
    constexpr int kGroups = kUnit / G, kPer = 8 / kGroups;
    constexpr int kTokens = 16 * MT;
    __shared__ float red[KW][R * MT * 4][64];
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * R;
    const uint8_t* c = p.c;
    const uint16_t* s = p.s;
    const uint8_t* z = p.z;
    int lo = blockIdx.y * kTokens, hi = min(p.rows, lo + kTokens);
    if (p.off) {
        const int e = blockIdx.y;
        const RowRange r = expert_rows(p.off[e], p.off[e + 1], p.rows);
        lo = r.lo;
        hi = r.hi;
        c += e * p.stride_c;
        s += e * p.stride_s;
        z += e * p.stride_z;
    }
    if (lo >= hi)
        return;
    const uint8_t* cr[R];
    const uint16_t* sr[R];
    const uint8_t* zr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = min(n0 + 16 * r + n16, p.N - 1);   // rows past N: never stored
        cr[r] = c + n * p.ldc;
        sr[r] = s + n * p.lds;
        zr[r] = Z ? z + n * p.ldz : nullptr;
    }
    const u32x4 ones{kOnes<F16>, kOnes<F16>, kOnes<F16>, kOnes<F16>};
    const Codes<F16> codes;

    for (int m0 = lo; m0 < hi; m0 += kTokens) {
        // operand rows without a token repeat the last one's, and their results are never stored
        const uint16_t* xr[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + 16 * t + (n16 >> 2) + 4 * (n16 & 3);
            xr[t] = p.x + x_row(p, min(m, hi - 1)) * p.ldx;
        }
        const auto load = [&](Buf<G, Z, MT, R>& b, int unit) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                load_unit<G, Z, Tail>(b.w[r], cr[r], sr[r], zr[r], unit, g, p.K);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int col = unit * kUnit + 32 * j + 8 * g;
                    b.x[t][j] = ld16(xr[t] + (Tail ? min(col, p.K - 8) : col));
                }
            }
            // left alone, the compiler moves these loads among the products before them
            __builtin_amdgcn_sched_barrier(0);
        };
        float sum[R][MT][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[r][t][i] = 0.0f;

        const auto compute = [&](Buf<G, Z, MT, R>& b, int unit) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                b.w[r].q[0] = exchange(b.w[r].q[0]);
                b.w[r].q[1] = exchange(b.w[r].q[1]);
            }
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                if (Tail && gr > 0 && unit * kUnit + gr * G >= p.K)
                    break;
                f32x4 xs[MT], acc[R][MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    xs[t] = f32x4{};
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[r][t] = f32x4{};
                }
#pragma unroll
                for (int j = gr * kPer; j < (gr + 1) * kPer; ++j) {
                    u32x4 w[R];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        w[r] = codes.operands(b.w[r].q[j >> 2][j & 3]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const u32x4 x = in_order(b.x[t][j]);
                        xs[t] = mma<F16>(x, ones, xs[t]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            acc[r][t] = mma<F16>(x, w[r], acc[r][t]);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float scale = to_f32<F16>(b.w[r].s[gr / 2] >> (16 * (gr & 1)));
                    float zero = 24.0f;
                    if constexpr (Z)
                        zero = 16.0f + (float)((b.w[r].z[gr / 4] >> (8 * (gr & 3))) & 15u);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[r][t][i] = __builtin_fmaf(
                                scale, __builtin_fmaf(-zero, xs[t][i], acc[r][t][i]), sum[r][t][i]);
                }
            }
            // The sums are finished here, before the branch that follows.  Wrong sums were seen once
            // without this, in a form of the kernel that was not kept (binary16, group 128, one
            // unit a wave); the cause is not known.  It is no shortened wait in this file: with
            // it or without, the compiler leaves 8 wait states or more on every path from a matrix
            // instruction to a reader of its result.  It costs no time.
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        asm volatile("" : "+v"(sum[r][t][i]));
            __builtin_amdgcn_sched_barrier(0);
        };

        if (wave < p.units) {
            Buf<G, Z, MT, R> buf;
            load(buf, wave);
            int k = wave;
            for (; k + KW < p.units; k += KW) {
                compute(buf, k);
                load(buf, k + KW);
            }
            compute(buf, k);
        }

#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[wave][(r * MT + t) * 4 + i][lane] = sum[r][t][i];
        __syncthreads();
        for (int u = wave; u < R * MT * 4; u += KW) {
            float v = red[0][u][lane];
#pragma unroll
            for (int w = 1; w < KW; ++w)
                v += red[w][u][lane];
            const int i = u % 4, t = u / 4 % MT, r = u / (4 * MT);
            const int m = m0 + 16 * t + g + 4 * i, n = n0 + 16 * r + n16;
            if (m < hi && n < p.N)
                p.y[m * p.ldy + n] = result<F16>(x_row_ok(p, m) ? v : 0.0f);
        }
        __syncthreads();
    }
}

// ---- many rows ------------------------------------------------------------------------------
//
// With many rows of x the matrix cores bound the work.  A workgroup computes TM x TN results (TM
// rows of x, TN rows of W), each wave all TM rows by its share of the others.  Stages of 64 columns
// go through LDS, x and codes both, brought there by global-to-LDS loads in a ring of three: while
// a stage is computed, the next one has landed or is landing and the one after it is being
// fetched.  Scales and zero points come for several stages (a unit) at once.
// Per stage a wave turns its codes into operands once and uses them for all blocks of 16
// rows of x; each group's products start from zero and are multiplied by the scale into the
// running sums, in registers.
//
// 128 x 256, 4 waves, two workgroups to a compute unit.  Measured on MI355X (a large library
// product reaches 1400 TFLOP/s): 24594 sorted rows over 32 experts of 2048 x 7168, group 64 with
// zero points, 832 to 861 us in binary16 (839 to 868 TFLOP/s) and 1042 in bf16, whose zero points
// cost a second multiply-add for each result; group 128 without 776 (930 TFLOP/s) and 901.
// What bounds it are the instructions between the matrix instructions: 264 vector and 64 matrix
// instructions a stage and wave, of which 128 scale results and 88 make operands, with two
// waves to a SIMD.  By the counters the two kinds run one after the other: matrix cores busy 45% of
// the cycles and vector instructions 51% in binary16, 33% and 54% in bf16.  Scaling the operands instead of the results would save half of them and
// round every weight to 8 (11) bits, which it must not.  bf16's sums of x are made inside the
// stage, with a barrier of their own: made a stage ahead they need a stage more in flight
// (1146 against 917 us).  Registers are short: a spilled one is read back behind the stage's
// loads (531 against 689 TFLOP/s), so the scales' addresses are made anew and bf16 with zero
// points holds one block of x instead of two.  8 waves read x from LDS twice as often (929
// against 845 us).
//
// 64 x 256, 8 waves: fewer rows an expert, or fewer workgroups (256 x 7168 x 7168: 97 us, and
// 108 with 4 waves).
//
// 64 x 128, 4 waves in each of two parts, for products that leave compute units idle.  There a
// stage's chain (LDS to registers, sums of x, a barrier, operands, products) takes the time, 0.8 us
// whatever else runs.  So a stage's inputs are read from LDS a stage ahead, each wave makes the sums
// of x for itself (8 matrix instructions more on 16), the ring holds six stages, and the
// two parts of a workgroup take half of the columns each and add their sums at the end.
// 256 x 7168 x 7168: 97 us as 64 x 256, 84 as 64 x 128, 68 with inputs a stage ahead, 55 in two
// parts (19 at the rate of a large product).
constexpr int kStage = 64;
// Waves of a part of a workgroup, and its parts.
template <int TM, int TN>
constexpr int kTileWaves = TM == 128 ? 4 : TN / 32;
template <int TN>
constexpr int kTileParts = TN == 128 ? 2 : 1;
constexpr int64_t kMaxGridY = 65535, kComputeUnits = 256;

template <int TM, int TN>
struct alignas(16) TileStage {
    uint8_t x[TM * 128];     // rows of 8 chunks of 16 bytes; chunk c of row r in slot c ^ (r & 7)
    uint8_t w[TN * 32];     // rows of 32 bytes of codes
};

template <int G, bool Z, bool F16, int TM, int TN>
struct alignas(16) TileShared {
    static constexpr int kUnit = G == 32 ? 128 : 256;    // columns whose scales come together
    static constexpr int kS = kUnit / G / 2;             // words of scales of a row and unit
    static constexpr int kRing = TN == 128 ? 6 : 3;
    TileStage<TM, TN> stage[kRing];
    uint32_t s[2][TN * kS];
    uint32_t z[Z ? 2 : 1][Z ? TN : 1];                   // one word of zero points
    alignas(16) float xs[F16 ? 4 : 2 * TM];              // sums of x per row and half stage
};
// two workgroups of 128 rows fit a compute unit's 160 KB
static_assert(sizeof(TileShared<32, true, false, 128, 256>) <= 80 * 1024, "LDS of a workgroup");

// The 8 codes of a word as operands in column order, less the zero point where the type has
// a packed subtraction.  Codes 2i, 2i+1 are byte i of the even and of the odd nibbles.
//  bf16: (16 + code) / 4096.  The code's bits sit in the low byte under a set bit 7; the high
//        byte is 0x3B (2^-8 is 0x3B80).
//  binary16: (code - zero) / 512, exactly.  A byte by itself is the subnormal code * 2^-24; one
//        packed fused multiply-add by 2^15 makes it normal and subtracts the zero point.
template <bool F16>
struct TileCodes {
    uint32_t mask, set, high;
    __device__ __forceinline__ TileCodes()
        : mask(F16 ? 0x0F0F0F0Fu : 0x78787878u), set(0x80808080u), high(0x3B3B3B3Bu) {
        asm("" : "+s"(mask));
        asm("" : "+v"(set));
        asm("" : "+s"(high));
    }
    __device__ __forceinline__ u32x4 operands(uint32_t w, h16x2 less) const {
        u32x4 r;
        if constexpr (F16) {
            const uint32_t e = w & mask, o = (w >> 4) & mask;
            const h16x2 up{(_Float16)32768.0f, (_Float16)32768.0f};
            constexpr uint32_t sel[4] = {0x0C040C00u, 0x0C050C01u, 0x0C060C02u, 0x0C070C03u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const h16x2 c = __builtin_bit_cast(h16x2, __builtin_amdgcn_perm(o, e, sel[i]));
                r[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, up, less));
            }
        } else {
            const uint32_t e = ((w << 3) & mask) | set, o = ((w >> 1) & mask) | set;
            const uint32_t lo = __builtin_amdgcn_perm(o, e, 0x05010400u);   // codes 0 1 2 3
            const uint32_t hi = __builtin_amdgcn_perm(o, e, 0x07030602u);   // codes 4 5 6 7
            r[0] = __builtin_amdgcn_perm(high, lo, 0x04010400u);
            r[1] = __builtin_amdgcn_perm(high, lo, 0x04030402u);
            r[2] = __builtin_amdgcn_perm(high, hi, 0x04010400u);
            r[3] = __builtin_amdgcn_perm(high, hi, 0x04030402u);
        }
        return r;
    }
};

// The expert and the first row of row block `block`, blocks counted expert by expert; -1 for one
// past the last.
template <int TM>
__device__ __forceinline__ int find_block(const Args& p, int block, int& lo, int& hi) {
    if (!p.off) {
        lo = block * TM;
        hi = p.rows;
        return lo < hi ? 0 : -1;
    }
    const int lane = threadIdx.x & 63;
    int seen = 0;
    for (int base = 0; base < p.experts; base += 64) {
        const int e = base + lane;
        RowRange r{0, 0};
        if (e < p.experts)
            r = expert_rows(p.off[e], p.off[e + 1], p.rows);
        const int mine = (r.hi - r.lo + TM - 1) / TM;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            inc += lane >= d ? o : 0;
        }
        const uint64_t past = __ballot(seen + inc > block);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            lo = __shfl(r.lo, l) + (block - seen - __shfl(inc - mine, l)) * TM;
            hi = __shfl(r.hi, l);
            return base + l;
        }
        seen += __shfl(inc, 63);
    }
    return -1;
}

template <bool F16, int G, bool Z, int TM, int TN>
__global__ __launch_bounds__((64 * kTileWaves<TM, TN> * kTileParts<TN>), TM == 128 || TN == 128 ? 2 : 4) void k_mm_i4(Args p) {
    using Shared = TileShared<G, Z, F16, TM, TN>;
    using Stage = TileStage<TM, TN>;
    constexpr int kRing = Shared::kRing;
    constexpr int kWaves = kTileWaves<TM, TN>, kWaveN = TN / kWaves, kNB = kWaveN / 16, kMB = TM / 16;
    constexpr int kXLoads = TM / (8 * kWaves), kWLoads = TN / (32 * kWaves);
    __shared__ Shared parts[kTileParts<TN>];
    constexpr bool kOne = kTileParts<TN> == 1;
    const int tid = kOne ? threadIdx.x : threadIdx.x & (64 * kWaves - 1);
    const int lane = tid & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int part = kOne ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kWaves));
    Shared& sm = parts[part];
    int lo, hi;
    const int expert =
        __builtin_amdgcn_readfirstlane(find_block<TM>(p, p.block0 + blockIdx.y, lo, hi));
    if (expert < 0)
        return;
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(min(hi, lo + TM));
    const int n0 = blockIdx.x * TN;
    const uint8_t* c = p.c + expert * p.stride_c;
    const uint16_t* s = p.s + expert * p.stride_s;
    const uint8_t* z = Z ? p.z + expert * p.stride_z : nullptr;

    // what this thread brings: x rows tid / 8 + 8 kWaves i, chunk tid % 8 (of the slot's row);
    // codes of rows tid / 2 + 32 kWaves i, half tid % 2
    const uint16_t* xp[kXLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
        const int r = (tid >> 3) + 8 * kWaves * i;
        xp[i] = p.x + x_row(p, min(lo + r, hi - 1)) * p.ldx;
    }
    const int xc = 8 * ((tid & 7) ^ ((tid >> 3) & 7));
    const uint8_t* cp[kWLoads];
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
        cp[i] = c + min(n0 + (tid >> 1) + 32 * kWaves * i, p.N - 1) * p.ldc;
    const int stages = (p.K + kStage - 1) / kStage;
    const auto issue = [&](int stage, int slot) {
        Stage& t = sm.stage[slot];
        const int k = stage * kStage;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            lds_load16(xp[i] + min(k + xc, p.K - 8), t.x + (wave + i * kWaves) * 1024);
        const int kc = min(k + 32 * (tid & 1), p.K - 32) / 2;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)
            lds_load16(cp[i] + kc, t.w + (wave + i * kWaves) * 1024);
    };
    // a wave's own rows of scales and zero points, word by word
    constexpr int kS = Shared::kS, kUnitGroups = Shared::kUnit / G;
    constexpr int kSLoads = (kWaveN * kS + 63) / 64;
    const int groups = p.K / G;
    const auto issue_scales = [&](int unit) {
        int l = lane;
        asm volatile("" : "+v"(l));     // addresses are made anew: registers are short
#pragma unroll
        for (int i = 0; i < kSLoads; ++i)
            if (kWaveN * kS % 64 == 0 || 64 * i + l < kWaveN * kS) {
                const int row = min(n0 + wave * kWaveN + i * (64 / kS) + l / kS, p.N - 1);
                const int at = min(unit * kUnitGroups + 2 * (l % kS), (groups - 1) & ~1);
                lds_load4(s + row * p.lds + at, &sm.s[unit & 1][(wave * kWaveN + i * (64 / kS)) * kS]);
            }
        if (Z && (kWaveN == 64 || l < kWaveN)) {
            const int row = min(n0 + wave * kWaveN + l, p.N - 1);
            const int at = min(unit * kUnitGroups, groups - 1) & ~3;
            lds_load4(z + row * p.ldz + at, &sm.z[unit & 1][wave * kWaveN]);
        }
    };
    constexpr int kStageLoads = kXLoads + kWLoads, kScaleLoads = kSLoads + (Z ? 1 : 0);

    f32x4 sum[kMB][kNB];
#pragma unroll
    for (int t = 0; t < kMB; ++t)
#pragma unroll
        for (int b = 0; b < kNB; ++b)
            sum[t][b] = f32x4{};
    const TileCodes<F16> codes;
    constexpr int kHalves = G == 32 ? 2 : 1;    // groups of a stage

    // the chunk of a row of x that feeds matrix instruction j: a lane quarter's 16 codes are
    // columns [16 g, 16 g + 16), traded between the halves of the wave where a group has 32
    const auto chunk = [&](int j) {
        return G == 32 ? 4 * j + ((g & 1) << 1 | g >> 1) : 2 * g + j;
    };
    const auto x_at = [&](const Stage& t, int block, int j) {
        const int r = 16 * block + n16;
        return *reinterpret_cast<const u32x4*>(t.x + r * 128 + 16 * (chunk(j) ^ (r & 7)));
    };
    // bf16: the sums of x per row and group of a stage, each wave its share of the blocks of rows
    // (negative, and times the 24 of the constant zero point, where the products start from them)
    const auto sums_of_x = [&](const Stage& t) {
        const u32x4 ones{kOnes<F16>, kOnes<F16>, kOnes<F16>, kOnes<F16>};
        for (int block = wave; block < kMB; block += kWaves) {
            f32x4 a = mma<F16>(x_at(t, block, 0), ones, f32x4{});
            f32x4 b = mma<F16>(x_at(t, block, 1), ones, kHalves == 2 ? f32x4{} : a);
            a *= Z ? -1.0f : -24.0f;
            b *= Z ? -1.0f : -24.0f;
            asm volatile("" : "+v"(a), "+v"(b));    // before the branch (see k_mv_i4)
            if (n16 == 0) {
                float* xs = sm.xs + 16 * block + 4 * g;
                *reinterpret_cast<f32x4*>(xs) = kHalves == 2 ? a : b;
                if (kHalves == 2)
                    *reinterpret_cast<f32x4*>(xs + TM) = b;
            }
        }
    };
    // What a stage's operands are made of, and the operands with their scales and zero points.
    struct Raw {
        u32x2 c[kNB];
        uint32_t s[kNB], z[kNB];
    };
    struct Operands {
        u32x4 w[kNB][2];
        float scale[kNB][kHalves], zero[kNB][kHalves];
    };
    const auto read_raw = [&](Raw& raw, int q, int slot, int unit) {
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            const int row = wave * kWaveN + 16 * b + n16;
            raw.c[b] = *reinterpret_cast<const u32x2*>(sm.stage[slot].w + row * 32 + 8 * g);
            // the word with this stage's group (or its two)
            raw.s[b] = sm.s[unit & 1][row * kS + (G == 128 ? 0 : G == 64 ? q / 2 : q)];
            if constexpr (Z)
                raw.z[b] = sm.z[unit & 1][row];
        }
    };
    const auto make = [&](Operands& o, Raw& raw, int stage, int q, int unit) {
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            if constexpr (G == 32) {
                const auto v =
                    __builtin_amdgcn_permlane32_swap(raw.c[b].x, raw.c[b].y, false, false);
                raw.c[b] = u32x2{v[0], v[1]};
            }
            h16x2 less[kHalves];
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const int half = G == 128 ? q / 2 : G == 64 ? q & 1 : h;    // of the word
                float scale = to_f32<F16>(raw.s[b] >> (16 * half)), zero = 8.0f;
                if (h == 1 && stage * kStage + 32 >= p.K)   // half a last stage
                    scale = 0.0f;
                if constexpr (Z) {
                    const int byte = G == 128 ? 2 * (unit & 1) + q / 2 : G == 64 ? q : 2 * q + h;
                    zero = (float)((raw.z[b] >> (8 * byte)) & 15u);
                }
                if constexpr (F16) {
                    scale *= 512.0f;
                    const _Float16 l = (_Float16)(zero * (-1.0f / 512.0f));
                    less[h] = h16x2{l, l};
                } else {
                    less[h] = h16x2{};
                    zero += 16.0f;
                }
                o.scale[b][h] = scale;
                o.zero[b][h] = zero;
            }
            o.w[b][0] = codes.operands(raw.c[b].x, less[0]);
            o.w[b][1] = codes.operands(raw.c[b].y, less[kHalves - 1]);
        }
    };
    const auto compute = [&](int stage, int q, int slot, int unit) {
        const Stage& t = sm.stage[slot];
        // everything the operands are made of is read first, and block 0 of x
        Raw raw;
        read_raw(raw, q, slot, unit);
        if constexpr (!F16)
            sums_of_x(t);
        // bf16 with zero points has no registers for two blocks (a spill would wait for the loads
        // of later stages): its next operand is read when the last one has been used
        constexpr int kXBufs = !F16 && Z && TM == 128 ? 1 : 2;
        u32x4 x[kXBufs][2];
        x[0][0] = x_at(t, 0, 0);
        x[0][1] = x_at(t, 0, 1);
        Operands o;
        make(o, raw, stage, q, unit);
        if constexpr (!F16)     // the other waves' sums of x
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

        // A step is one block of rows of x, or one group of it where a stage has two.  Its products
        // run on the matrix cores while the vector units scale the step before and the next
        // block of x comes from LDS: slots of one matrix instruction and its share of the
        // scaling, held in this order.
        constexpr int kSlots = 2 * kNB / kHalves, kSteps = kMB * kHalves;
        f32x4 acc[2][kNB], xs[kXBufs];
        const auto fold = [&](int step, int part) {
            const int m = step / kHalves, h = step % kHalves;
#pragma unroll
            for (int e = part * 4 * kNB / kSlots; e < (part + 1) * 4 * kNB / kSlots; ++e) {
                const int b = e / 4, i = e % 4;
                float v = acc[step & 1][b][i];
                if constexpr (!F16 && Z)
                    v = __builtin_fmaf(o.zero[b][h], xs[step % kXBufs][i], v);
                sum[m][b][i] = __builtin_fmaf(o.scale[b][h], v, sum[m][b][i]);
            }
        };
        const auto read_xs = [&](int step) {
            if constexpr (!F16)
                xs[step % kXBufs] = *reinterpret_cast<const f32x4*>(sm.xs + (step % kHalves) * TM +
                                                               16 * (step / kHalves) + 4 * g);
        };
        if constexpr (kXBufs == 2)
            read_xs(0);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            const int m = step / kHalves, h = step % kHalves;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int b = i % kNB, j = kHalves == 2 ? h : i / kNB;
                f32x4 from{};
                if (i >= kNB)
                    from = acc[step & 1][b];
                else if (!F16 && !Z)
                    from = xs[step % kXBufs];
                acc[step & 1][b] = mma<F16>(x[m % kXBufs][j], o.w[b][j], from);
                if constexpr (kXBufs == 2) {
                    if (i == 0 && h == 0 && m + 1 < kMB) {
                        x[(m + 1) & 1][0] = x_at(t, m + 1, 0);
                        x[(m + 1) & 1][1] = x_at(t, m + 1, 1);
                    }
                } else {
                    if (b == kNB - 1 && m + 1 < kMB)
                        x[0][j] = x_at(t, m + 1, j);
                }
                if (step > 0)
                    fold(step - 1, i);
                // over those of the step before, whose last use this was; with one block of x for
                // the scaling of this step, in the next
                if (i == kSlots - 1 && kXBufs == 1)
                    read_xs(step);
                else if (i == kSlots - 1 && step + 1 < kSteps)
                    read_xs(step + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            fold(kSteps - 1, i);
        // finished before the next branch (see k_mv_i4)
#pragma unroll
        for (int m = 0; m < kMB; ++m)
#pragma unroll
            for (int b = 0; b < kNB; ++b)
                asm volatile("" : "+v"(sum[m][b]));
    };

    constexpr int kUnitStages = Shared::kUnit / kStage;
    if constexpr (TN == 128) {
        // A stage's inputs, read from LDS during the stage before it; a wave makes the sums of x
        // for itself, so the waves meet once a stage.
        struct Inputs {
            Raw raw;
            u32x4 x[kMB][2];
        };
        const auto read = [&](Inputs& in, int q, int slot, int unit) {
            read_raw(in.raw, q, slot, unit);
#pragma unroll
            for (int m = 0; m < kMB; ++m) {
                in.x[m][0] = x_at(sm.stage[slot], m, 0);
                in.x[m][1] = x_at(sm.stage[slot], m, 1);
            }
        };
        const auto compute_read = [&](Inputs& in, int stage, int q, int unit) {
            Operands o;
            make(o, in.raw, stage, q, unit);
            const u32x4 ones{kOnes<F16>, kOnes<F16>, kOnes<F16>, kOnes<F16>};
            f32x4 xs[kMB][kHalves], acc[kMB][kNB][kHalves];
#pragma unroll
            for (int m = 0; m < kMB; ++m)
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    xs[m][h] = f32x4{};
                    if constexpr (!F16) {
                        xs[m][h] = mma<F16>(in.x[m][h], ones, f32x4{});
                        if (kHalves == 1)
                            xs[m][h] = mma<F16>(in.x[m][1], ones, xs[m][h]);
                        xs[m][h] *= Z ? -1.0f : -24.0f;
                    }
                }
#pragma unroll
            for (int m = 0; m < kMB; ++m)
#pragma unroll
                for (int b = 0; b < kNB; ++b)
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        f32x4 from{};
                        if (!F16 && !Z)
                            from = xs[m][h];
                        acc[m][b][h] = mma<F16>(in.x[m][h], o.w[b][h], from);
                        if (kHalves == 1)
                            acc[m][b][h] = mma<F16>(in.x[m][1], o.w[b][1], acc[m][b][h]);
                    }
#pragma unroll
            for (int m = 0; m < kMB; ++m)
#pragma unroll
                for (int b = 0; b < kNB; ++b) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v = acc[m][b][h][i];
                            if constexpr (!F16 && Z)
                                v = __builtin_fmaf(o.zero[b][h], xs[m][h][i], v);
                            sum[m][b][i] = __builtin_fmaf(o.scale[b][h], v, sum[m][b][i]);
                        }
                    asm volatile("" : "+v"(sum[m][b]));     // (see k_mv_i4)
                }
        };
        // each part takes its units of the columns; what is past them is fetched and not used
        const int units = (stages + kUnitStages - 1) / kUnitStages, share = (units + 1) / 2;
        const int first = part * share;
        const auto fetch = [&](int stage, int slot) { issue(min(stage, stages - 1), slot); };
        issue_scales(first);
#pragma unroll
        for (int d = 0; d < kRing - 1; ++d)
            fetch(first * kUnitStages + d, d);
        wait_and_join<0>();
        Inputs in[2];
        read(in[0], 0, 0, first);
        int slot = 0;
        for (int unit = first; unit < first + share; ++unit) {
#pragma unroll
            for (int q = 0; q < kUnitStages; ++q) {
                constexpr int kLast = kUnitStages - 1;
                const int stage = unit * kUnitStages + q, next = slot == kRing - 1 ? 0 : slot + 1;
                if (q == 0)
                    issue_scales(unit + 1);
                // into the slot that was read two stages ago
                fetch(stage + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);
                read(in[(q + 1) & 1], q == kLast ? 0 : q + 1, next, q == kLast ? unit + 1 : unit);
                __builtin_amdgcn_sched_barrier(0);
                if (stage < stages)
                    compute_read(in[q & 1], stage, q, unit);
                // the stage after the next has landed, and before the unit's last stage the next
                // unit's scales, which kLast stages were asked for after
                if (q == kLast - 1)
                    wait_and_join<(kLast < kRing - 3 ? kLast : kRing - 3) * kStageLoads>();
                else
                    wait_and_join<(kRing - 3) * kStageLoads>();
                slot = next;
            }
        }
        // the second part's sums to the first, through LDS that nothing lands in any more
        wait_and_join<0>();
        f32x4* trade = reinterpret_cast<f32x4*>(&parts[0]) + wave * kMB * kNB * 64 + lane;
        static_assert(sizeof(Shared) >= TM * TN * sizeof(float), "room for the sums");
        if (part == 1) {
#pragma unroll
            for (int m = 0; m < kMB; ++m)
#pragma unroll
                for (int b = 0; b < kNB; ++b)
                    trade[(m * kNB + b) * 64] = sum[m][b];
        }
        wait_and_join<0>();
        if (part == 1)
            return;
#pragma unroll
        for (int m = 0; m < kMB; ++m)
#pragma unroll
            for (int b = 0; b < kNB; ++b)
                sum[m][b] += trade[(m * kNB + b) * 64];
    } else {
        issue_scales(0);
        issue(0, 0);
        issue(min(1, stages - 1), 1);
        wait_and_join<0>();
        int slot = 0;
        for (int unit = 0; unit * kUnitStages < stages; ++unit) {
#pragma unroll
            for (int q = 0; q < kUnitStages; ++q) {
                const int stage = unit * kUnitStages + q;
                const int next = slot == kRing - 1 ? 0 : slot + 1;
                issue(min(stage + 2, stages - 1), next == kRing - 1 ? 0 : next + 1);
                if (q == 0)
                    issue_scales(unit + 1);
                if (stage < stages)
                    compute(stage, q, slot, unit);
                // the next stage has landed when only what this one issued is outstanding
                if (q == 0)
                    wait_and_join<kStageLoads + kScaleLoads>();
                else
                    wait_and_join<kStageLoads>();
                slot = next;
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing lands in LDS after the end

#pragma unroll
    for (int m = 0; m < kMB; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = lo + 16 * m + 4 * g + i;
            if (row < hi) {
                const bool ok = x_row_ok(p, row);
#pragma unroll
                for (int b = 0; b < kNB; ++b) {
                    const int n = n0 + wave * kWaveN + 16 * b + n16;
                    if (n < p.N)
                        p.y[row * p.ldy + n] = result<F16>(ok ? sum[m][b][i] : 0.0f);
                }
            }
        }
    }
}

template <bool F16, int G, bool Z, int TM, int TN>
hipError_t launch_tile(const Args& a0, hipStream_t st) {
    Args a = a0;
    // experts: every expert's last block may be partial
    const int64_t blocks = a.off ? a.rows / TM + a.experts : (a.rows + TM - 1) / TM;
    hipError_t e = hipSuccess;
    for (int64_t b = 0; b < blocks && e == hipSuccess; b += kMaxGridY) {
        a.block0 = (int32_t)b;
        const int64_t n = blocks - b < kMaxGridY ? blocks - b : kMaxGridY;
        const dim3 grid((unsigned)((a.N + TN - 1) / TN), (unsigned)n);
        e = launch1(k_mm_i4<F16, G, Z, TM, TN>, grid, dim3(64 * kTileWaves<TM, TN> * kTileParts<TN>), st, a);
    }
    return e;
}

template <bool F16, int G, bool Z, bool Tail, int MT, int R, int KW>
hipError_t launch_mv(const Args& a, hipStream_t st) {
    const int chunks = (a.rows + 16 * MT - 1) / (16 * MT);
    const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)), a.off ? a.experts : chunks);
    return launch1(k_mv_i4<F16, G, Z, Tail, MT, R, KW>, grid, dim3(64 * KW), st, a);
}

// ---- few rows, staged through LDS -----------------------------------------------------------
//
// The same sums as k_mv_i4's for up to 16 rows, with every byte brought to LDS by global-to-LDS
// loads.  A matrix operand wants 16 different rows in 16 adjacent lanes, and a load in that
// order touches 16 lines of memory for every 256 bytes; through LDS each load instruction reads
// whole lines.  A wave keeps to itself: its own units of 256 columns, its own ring of D units,
// no barriers until the sums meet.  x has up to 4 NI rows (NI = 1, 2 or 4): a lane has NI results
// for each block of 16 rows of W, result i of lane quarter g that of token g + 4i.
// Measured at 16 x 7168 x 43008, group 64 with zero points (170 MB, 35 us at the rate of a large
// copy): 56 us, against 74 with loads to registers.  Units of 128 columns, which leave room
// for 8 waves, take 70 (runs of 64 bytes); pairs of waves that share a unit's x and meet at a
// barrier for each 65; 16 rows of W 71, 64 rows 98.  Bound by the loads of x, 8 KB for 4 KB of
// codes, with one wave to a SIMD: one row of x takes 41 to 44 us (3.9 to 4.1 TB/s).
template <int G, bool Z, int NI, int R>
struct alignas(16) Staged {
    static constexpr int kS = kUnit / G / 2;         // words of scales of a row and unit
    static constexpr int kZ = G == 32 ? 2 : 1;       // words of zero points
    static constexpr int kSLoads = (16 * R * kS + 63) / 64, kZLoads = Z ? (16 * R * kZ + 63) / 64 : 0;
    uint8_t w[16 * R * 128];         // rows of 8 chunks of 16 bytes, chunk c in slot c ^ (row & 7)
    uint8_t x[4 * NI * 512];         // rows of 32 chunks, chunk c in slot c ^ (row & 7)
    uint32_t s[64 * kSLoads];
    uint32_t z[Z ? 64 * kZLoads : 4];
};

// Waves on a SIMD that the rings leave room for: one where a workgroup of four waves takes more
// than half of a compute unit's LDS (9 to 16 rows of x).
template <int G, bool Z, int NI, int R, int KW, int D>
constexpr int kStagedWaves =
    160 * 1024 / (KW * D * (int)sizeof(Staged<G, Z, NI, R>)) * KW >= 8 ? 2 : 1;

template <bool F16, int G, bool Z, bool Tail, int NI, int R, int KW, int D>
__global__ __launch_bounds__(64 * KW)
__attribute__((amdgpu_waves_per_eu(kStagedWaves<G, Z, NI, R, KW, D>))) void k_ms_i4(Args p) {
    using St = Staged<G, Z, NI, R>;
    constexpr int kGroups = kUnit / G, kPer = 8 / kGroups;
    constexpr int kS = St::kS, kZ = St::kZ;
    __shared__ St ring[KW][D];
    static_assert(sizeof(St) * D >= R * NI * 64 * 4, "the sums fit a wave's ring");
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * R;
    const int groups = p.K / G;
    const u32x4 ones{kOnes<F16>, kOnes<F16>, kOnes<F16>, kOnes<F16>};
    const Codes<F16> codes;
    // Addresses are a uniform base that moves with the unit and a lane's 32-bit offset, which
    // the launch has checked to be enough.  First what this lane brings of the weights.
    uint32_t co[2 * R], so[St::kSLoads], zo[Z ? St::kZLoads : 1];
    const uint32_t wk = 16 * ((lane & 7) ^ (lane >> 3));     // bytes of this lane's chunk
    const int left_n = p.N - 1 - n0;
#pragma unroll
    for (int i = 0; i < 2 * R; ++i)
        co[i] = (uint32_t)(min(8 * i + (lane >> 3), left_n) * p.ldc);
#pragma unroll
    for (int i = 0; i < St::kSLoads; ++i)
        so[i] = (uint32_t)(min(min((64 * i + lane) / kS, 16 * R - 1), left_n) * p.lds);
#pragma unroll
    for (int i = 0; i < St::kZLoads; ++i)
        zo[i] = (uint32_t)(min(min((64 * i + lane) / kZ, 16 * R - 1), left_n) * p.ldz);
    const uint8_t* c0 = p.c + n0 * p.ldc;
    const uint16_t* s0 = p.s + n0 * p.lds;
    const uint8_t* z0 = Z ? p.z + n0 * p.ldz : nullptr;

    uint32_t xo[2 * NI], xk[2 * NI];       // values
#pragma unroll
    for (int i = 0; i < 2 * NI; ++i) {
        const int r = 2 * i + (lane >> 5);
        xo[i] = (uint32_t)(min(r, p.rows - 1) * p.ldx);
        xk[i] = 8 * ((lane & 31) ^ (r & 7));
    }
    const auto issue = [&](int unit, int slot) {
        St& t = ring[wave][slot];
        const uint32_t k = unit * kUnit, left = p.K - k;    // columns from here on
        const uint8_t* cu = c0 + k / 2;
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
            lds_load16(cu + (co[i] + (Tail ? min(wk, left / 2 - 16) : wk)), t.w + 1024 * i);
        const uint16_t* xu = p.x + k;
#pragma unroll
        for (int i = 0; i < 2 * NI; ++i)
            lds_load16(xu + (xo[i] + (Tail ? min(xk[i], left - 8) : xk[i])), t.x + 1024 * i);
        // scales two to a word, zero points four; a word past the last group repeats its word
        const uint32_t first = unit * kGroups, at4 = first & ~3u;
        const uint32_t end2 = ((groups - 1) & ~1u) - first, end4 = ((groups - 1) & ~3u) - at4;
        const uint16_t* su = s0 + first;
#pragma unroll
        for (int i = 0; i < St::kSLoads; ++i) {
            const uint32_t w = 2 * ((64 * i + lane) % kS);
            lds_load4(su + (so[i] + (Tail ? min(w, end2) : w)), t.s + 64 * i);
        }
        if constexpr (Z) {
            const uint8_t* zu = z0 + at4;
#pragma unroll
            for (int i = 0; i < St::kZLoads; ++i) {
                const uint32_t w = 4 * ((64 * i + lane) % kZ);
                lds_load4(zu + (zo[i] + (Tail ? min(w, end4) : w)), t.z + 64 * i);
            }
        }
    };
    constexpr int kLoads = 2 * R + 2 * NI + St::kSLoads + St::kZLoads;

    float sum[R][NI];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i)
            sum[r][i] = 0.0f;
    const auto compute = [&](int unit, int slot) {
        const St& t = ring[wave][slot];
        u32x4 q[R][2];
        uint32_t sw[R][kS], zw[R][kZ];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 16 * r + n16;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[r][h] = exchange(*reinterpret_cast<const u32x4*>(
                    t.w + row * 128 + 16 * ((4 * h + g) ^ (row & 7))));
#pragma unroll
            for (int i = 0; i < kS; ++i)
                sw[r][i] = t.s[row * kS + i];
#pragma unroll
            for (int i = 0; i < kZ; ++i)
                zw[r][i] = Z ? t.z[row * kZ + i] : 0;
        }
        const int xr = (n16 >> 2) + 4 * ((n16 & 3) % NI);   // the token of operand row n16
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
            if (Tail && gr > 0 && unit * kUnit + gr * G >= p.K)
                break;
            f32x4 xs{}, acc[R] = {};
#pragma unroll
            for (int j = gr * kPer; j < (gr + 1) * kPer; ++j) {
                const u32x4 x = in_order(*reinterpret_cast<const u32x4*>(
                    t.x + xr * 512 + 16 * ((4 * j + g) ^ (xr & 7))));
                xs = mma<F16>(x, ones, xs);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r] = mma<F16>(x, codes.operands(q[r][j >> 2][j & 3]), acc[r]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float scale = to_f32<F16>(sw[r][gr / 2] >> (16 * (gr & 1)));
                float zero = 24.0f;
                if constexpr (Z) {
                    const int byte = G == 128 ? 2 * (unit & 1) + gr : gr & 3;
                    zero = 16.0f + (float)((zw[r][G == 32 ? gr / 4 : 0] >> (8 * byte)) & 15u);
                }
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    sum[r][i] =
                        __builtin_fmaf(scale, __builtin_fmaf(-zero, xs[i], acc[r][i]), sum[r][i]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                asm volatile("" : "+v"(sum[r][i]));     // see k_mv_i4
    };

    if (wave < p.units) {
        const int last = p.units - 1;
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            issue(min(wave + d * KW, last), d);
        int slot = 0;
        for (int unit = wave; unit < p.units; unit += KW) {
            issue(min(unit + (D - 1) * KW, last), slot == 0 ? D - 1 : slot - 1);
            // this unit has landed when only the D - 1 after it are outstanding
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * kLoads) : "memory");
            compute(unit, slot);
            slot = slot == D - 1 ? 0 : slot + 1;
        }
    }
    // this wave's ring holds its sums once the last loads have landed
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    float* red = reinterpret_cast<float*>(ring[wave]);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i)
            red[(r * NI + i) * 64 + lane] = sum[r][i];
    __syncthreads();
    for (int u = wave; u < R * NI; u += KW) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
            v += reinterpret_cast<const float*>(ring[w])[u * 64 + lane];
        const int m = g + 4 * (u % NI), n = n0 + 16 * (u / NI) + n16;
        if (m < p.rows && n < p.N)
            p.y[m * p.ldy + n] = result<F16>(v);
    }
}

template <bool F16, int G, bool Z, bool Tail, int NI, int R, int KW, int D>
hipError_t launch_ms(const Args& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)));
    return launch1(k_ms_i4<F16, G, Z, Tail, NI, R, KW, D>, grid, dim3(64 * KW), st, a);
}

// The kernel for few rows.  Rules and measurements on MI355X (us):
//  - Dense, up to 16 rows: k_ms_i4, in forms for 4, 8 and 16 rows, with 32 rows of W for each
//    workgroup (1 x 7168 x 7168, group 128: 7.3), or 16 where 32 would leave more than half of the
//    compute units without one (1 x 1024 x 43008: 18.0 against 26; 16 x 1024 x 43008 27.6 against
//    37).
//    Its lanes' offsets have 32 bits; where rows are so far apart that they do not fit, k_mv_i4.
//  - Above 16 rows k_mv_i4 with blocks of 16 tokens, two up to 32 rows (32 x 7168 x 7168: 19.4
//    against 25.6 with four), else four; 16 rows of W to a workgroup of 8 waves instead of 32 to 4
//    where that still fits one round (64 x 1024 x 8192: 33 against 38, 24 rows 17 against 20).
//  - By expert k_mv_i4 with four blocks of 16 rows of W to share the operands of x (8 rows for
//    each of 64 experts of 4096 x 7168: 243 against 280 with two), or two where four leave
//    less than two workgroups to a compute unit.
template <bool F16, int G, bool Z, bool Tail>
hipError_t launch_few(const Args& a, int64_t m, hipStream_t st) {
    if (a.off) {
        if ((int64_t)a.experts * (a.N / 64) >= 512)
            return launch_mv<F16, G, Z, Tail, 1, 4, 4>(a, st);
        return launch_mv<F16, G, Z, Tail, 1, 2, 4>(a, st);
    }
    if (m <= 16) {
        const bool narrow = a.N < 4096;
        const auto near = [](int64_t rows, int64_t ld) { return ld < ((int64_t)1 << 31) / rows; };
        if (!near(32, a.ldc) || !near(32, a.lds) || !near(32, a.ldz) || !near(16, a.ldx))
            return launch_mv<F16, G, Z, Tail, 1, 2, 4>(a, st);
        if (m <= 4)
            return narrow ? launch_ms<F16, G, Z, Tail, 1, 1, 8, 3>(a, st)
                          : launch_ms<F16, G, Z, Tail, 1, 2, 8, 2>(a, st);
        if (m <= 8)
            return narrow ? launch_ms<F16, G, Z, Tail, 2, 1, 8, 2>(a, st)
                          : launch_ms<F16, G, Z, Tail, 2, 2, 4, 2>(a, st);
        return narrow ? launch_ms<F16, G, Z, Tail, 4, 1, 4, 2>(a, st)
                      : launch_ms<F16, G, Z, Tail, 4, 2, 4, 2>(a, st);
    }
    if (((int64_t)a.N + 15) / 16 * ((m + 63) / 64) <= kComputeUnits)
        return m <= 32 ? launch_mv<F16, G, Z, Tail, 2, 1, 8>(a, st)
                       : launch_mv<F16, G, Z, Tail, 4, 1, 8>(a, st);
    return m <= 32 ? launch_mv<F16, G, Z, Tail, 2, 2, 4>(a, st)
                   : launch_mv<F16, G, Z, Tail, 4, 2, 4>(a, st);
}

// The kernel and tile for many rows (us, bf16, group 128, 8192 columns where no others are given):
//  - k_mv_i4 while its workgroups, 64 rows of x by 32 of W, fit one round of a workgroup per
//    compute unit: 64 x 8192 40 against 57 in tiles of 64 x 128, 64 x 16384 72 against 58.  Up to 32
//    rows its rounds are shorter and three are taken (24 x 24576: 55 against 60), or six where such
//    tiles would not fit one round (24 x 40960: 89 against 119; 24 x 57344: 123 against 115).
//  - Tiles of 64 x 128, in two parts of the columns, while they fit one round: 256 x 7168 x 7168
//    55 against 95 in tiles of 64 x 256; 512 x 7168 x 7168, 448 of them, 103 against 96.
//  - Tiles of 128 x 256 where they make workgroups enough (7168 x 7168): 2048 rows 247 against
//    290 in tiles of 64, 1024 rows 168 against 149; by expert 96 rows 688 against 651, 160 rows
//    969 against 971.
//  - By expert the tiles win from 16 rows an expert (64 experts of 4096 x 7168: 346 against 346
//    there, 408 against 610 at 32).  The mean over the experts decides, since the host does not
//    know their rows: 1024 rows that all go to one of the 64 stay with k_mv_i4, whose workgroups
//    for that expert take them 16 at a time (1031; dealt evenly 337).
template <bool F16, int G, bool Z>
hipError_t launch_shape(const Args& a, hipStream_t st) {
    const int64_t m = a.off ? (a.rows + a.experts - 1) / a.experts : a.rows;
    // of 64 rows of x; experts: every expert's last one may be partial
    const int64_t blocks = a.off ? a.rows / 64 + a.experts : (m + 63) / 64;
    const bool one_round = blocks * ((a.N + 127) / 128) <= kComputeUnits;
    const int rounds = m > 32 ? 1 : one_round ? 3 : 6;
    if (m <= 16 || (!a.off && blocks * ((a.N + 31) / 32) <= rounds * kComputeUnits))
        return a.K % kUnit != 0 ? launch_few<F16, G, Z, true>(a, m, st)
                                : launch_few<F16, G, Z, false>(a, m, st);
    if (one_round)
        return launch_tile<F16, G, Z, 64, 128>(a, st);
    const bool tall = a.off ? m > 128 : (m + 127) / 128 * ((a.N + 255) / 256) >= 384;
    return tall ? launch_tile<F16, G, Z, 128, 256>(a, st) : launch_tile<F16, G, Z, 64, 256>(a, st);
}

template <bool F16, int G>
hipError_t launch_zero(const Args& a, hipStream_t st) {
    return a.z ? launch_shape<F16, G, true>(a, st) : launch_shape<F16, G, false>(a, st);
}

}  // namespace

hipError_t launch_mm_i4(const I4Mm& m, int group, bool f16, hipStream_t stream) {
    Args a{};
    static_cast<I4Mm&>(a) = m;
    a.units = (a.K + kUnit - 1) / kUnit;
    if (f16)
        return group == 32 ? launch_zero<true, 32>(a, stream)
             : group == 64 ? launch_zero<true, 64>(a, stream)
                           : launch_zero<true, 128>(a, stream);
    return group == 32 ? launch_zero<false, 32>(a, stream)
         : group == 64 ? launch_zero<false, 64>(a, stream)
                       : launch_zero<false, 128>(a, stream);
}

}  // namespace bq
