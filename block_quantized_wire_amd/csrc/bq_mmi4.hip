// bq_mmi4.hip -- products with 4-bit weights and group scales (I4), dense and by expert.
//
// Definition: Y[m][n] = rne( sum over k of X[m][k] * (code[n][k] - zero[n][g]) * scale[n][g] ),
// g = k / G the group of G = 32, 64 or 128 columns.  For one group
//   sum x (code - zero) = sum x (16 + code) - (16 + zero) * sum x,
// and 16 + code is a bf16 (binary16) number whose significand holds the code's four bits as
// they are: a pair of codes becomes a pair of matrix operands with one shift and one
// and-or.  Both sums run on the matrix cores in binary32 (sum x as a product with ones), and
// the group's scale multiplies their difference once, in binary32.  The offset of 16 costs
// at most a factor of 16 + zero over |code - zero| in the rounding of binary32 sums.
#include "bq_device.h"
#include "bq_launch.h"

namespace bq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

constexpr int kTK = 128;         // columns of a step: 16 bytes of codes per lane
constexpr int kWaves = 8, kThreads = 64 * kWaves;

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

// The 8 codes of a word as operands 16 + code, in the order 0,4, 1,5, 2,6, 3,7 (codes i and
// i+4 are 16 bits apart).  The code's bits go to the top of the significand: bits 3..6 of
// a bf16 16.0 (0x4180), bits 6..9 of a binary16 16.0 (0x4C00).
template <bool F16>
__device__ __forceinline__ u32x4 operands(uint32_t w) {
    constexpr uint32_t mask = F16 ? 0x03C003C0u : 0x00780078u;
    constexpr uint32_t base = F16 ? 0x4C004C00u : 0x41804180u;
    constexpr int up = F16 ? 6 : 3;
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = 4 * i < up ? w << (up - 4 * i) : w >> (4 * i - up);
        r[i] = (v & mask) | base;
    }
    return r;
}

// 8 values of x (16 bytes) in the operands' order.
__device__ __forceinline__ u32x4 in_order(u32x4 x) {
    return u32x4{__builtin_amdgcn_perm(x.z, x.x, 0x05040100u),
                 __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                 __builtin_amdgcn_perm(x.w, x.y, 0x05040100u),
                 __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

// A lane loads 32 consecutive columns of its row: lane quarter g has columns [32g, 32g+32) of
// the 128.  Word j of every quarter is one matrix instruction's 32 columns, which belong to
// one group only where G is 128.  For smaller groups the words trade places between the
// quarters: exchanging the halves of the wave puts the columns of each 64 together, and
// exchanging odd and even quarters then those of each 32.
template <int G>
__device__ __forceinline__ void regroup(u32x4& q) {
    if constexpr (G <= 64) {
        auto a = __builtin_amdgcn_permlane32_swap(q.x, q.z, false, false);
        auto b = __builtin_amdgcn_permlane32_swap(q.y, q.w, false, false);
        q = u32x4{a[0], b[0], a[1], b[1]};
    }
    if constexpr (G == 32) {
        auto a = __builtin_amdgcn_permlane16_swap(q.x, q.y, false, false);
        auto b = __builtin_amdgcn_permlane16_swap(q.z, q.w, false, false);
        q = u32x4{a[0], a[1], b[0], b[1]};
    }
}

// The first of the 8 columns that lane quarter g feeds into matrix instruction j of a step.
template <int G>
__device__ __forceinline__ int col_of(int j, int g) {
    if constexpr (G == 128)
        return 32 * g + 8 * j;
    else if constexpr (G == 64)
        return 64 * (j >> 1) + 32 * (g & 1) + 16 * (g >> 1) + 8 * (j & 1);
    else
        return 32 * j + 8 * g;
}

struct Args : I4Mm {
    int32_t steps;      // ceil(K / 128)
    int32_t chunk;      // row chunks between two of a workgroup's (dense)
};

// One step's data of one block of 16 rows of W: the lane's codes, and the scales and zero
// points of its row's 128 / G groups.
template <int G, bool Z>
struct Step {
    static constexpr int kGroups = kTK / G;
    u32x4 q;
    uint32_t s[kGroups];
    uint32_t z;
};

template <int G, bool Z>
__device__ __forceinline__ void load_step(Step<G, Z>& st, const uint8_t* c, const uint16_t* s,
                                          const uint8_t* z, int step, int g, int K) {
    constexpr int kGroups = kTK / G;
    const int k = step * kTK + 32 * g;
    st.q = k < K ? ld16(c + k / 2) : u32x4{};
    if constexpr (kGroups == 1) {
        st.s[0] = s[step];
    } else if constexpr (kGroups == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(s + step * 2);
        st.s[0] = v & 0xFFFFu;
        st.s[1] = v >> 16;
    } else {
        const u32x2 v = ld8(s + step * 4);
        st.s[0] = v.x & 0xFFFFu;
        st.s[1] = v.x >> 16;
        st.s[2] = v.y & 0xFFFFu;
        st.s[3] = v.y >> 16;
    }
    if constexpr (Z) {
        if constexpr (kGroups == 1)
            st.z = z[step];
        else if constexpr (kGroups == 2)
            st.z = *reinterpret_cast<const uint16_t*>(z + step * 2);
        else
            st.z = *reinterpret_cast<const uint32_t*>(z + step * 4);
    }
}

// NI results per lane and block of 16 tokens: the token of lane quarter g's result i is
// g + 4i, so a block of 4 tokens needs one result per lane.  MT blocks of tokens, R blocks of
// 16 weight rows per workgroup.  The 8 waves share the steps, and their sums meet in LDS.
template <bool F16, int G, bool Z, int NI, int MT, int R>
__global__ __launch_bounds__(kThreads) void k_mv_i4(Args p) {
    constexpr int kGroups = kTK / G, kPer = 4 / kGroups;
    constexpr int kTokens = MT == 1 ? 4 * NI : 16 * MT;
    __shared__ float red[kWaves][R * MT * NI][64];
    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * R;
    const uint8_t* c = p.c;
    const uint16_t* s = p.s;
    const uint8_t* z = p.z;
    int lo = blockIdx.y * kTokens, hi = p.rows, stride = p.chunk * kTokens;
    if (p.off) {
        const int e = blockIdx.y;
        lo = max(p.off[e], 0);
        hi = min(p.off[e + 1], p.rows);
        stride = kTokens;
        c += e * p.stride_c;
        s += e * p.stride_s;
        z += e * p.stride_z;
    }
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
    const int first = wave * p.steps / kWaves, last = (wave + 1) * p.steps / kWaves;
    constexpr uint32_t kOne = F16 ? 0x3C003C00u : 0x3F803F80u;
    const u32x4 ones{kOne, kOne, kOne, kOne};

    for (int m0 = lo; m0 < hi; m0 += stride) {
        // the row of x of operand row n16 of each block of tokens: token n16 / 4 + 4 (n16 % 4)
        const uint16_t* xr[MT];
        bool live[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int i = n16 & 3;
            const int m = m0 + 16 * t + (n16 >> 2) + 4 * i;
            live[t] = i < NI && m < hi;
            int64_t row = m;
            if (p.src && live[t])
                row = p.src[m] / p.topk;
            live[t] = live[t] && row >= 0 && row < p.x_rows;
            xr[t] = p.x + (live[t] ? row : 0) * p.ldx;
        }
        float sum[R][MT][NI];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    sum[r][t][i] = 0.0f;

        for (int k = first; k < last; ++k) {
            Step<G, Z> st[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_step<G, Z>(st[r], cr[r], sr[r], zr[r], k, g, p.K);
                regroup<G>(st[r].q);
            }
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                if (gr > 0 && k * kTK + gr * G >= p.K)   // a last step of fewer groups
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
                    const int col = k * kTK + col_of<G>(j, g);
                    u32x4 w[R];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        w[r] = operands<F16>(st[r].q[j]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        u32x4 x{};
                        if (live[t] && col < p.K)
                            x = in_order(ld16(xr[t] + col));
                        xs[t] = mma<F16>(x, ones, xs[t]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            acc[r][t] = mma<F16>(x, w[r], acc[r][t]);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float scale = to_f32<F16>(st[r].s[gr]);
                    float zero = 24.0f;
                    if constexpr (Z)
                        zero = 16.0f + (float)((st[r].z >> (8 * gr)) & 15u);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < NI; ++i)
                            sum[r][t][i] = __builtin_fmaf(
                                scale, __builtin_fmaf(-zero, xs[t][i], acc[r][t][i]), sum[r][t][i]);
                }
            }
        }

#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    red[wave][(r * MT + t) * NI + i][lane] = sum[r][t][i];
        __syncthreads();
        for (int u = wave; u < R * MT * NI; u += kWaves) {
            float v = red[0][u][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                v += red[w][u][lane];
            const int i = u % NI, t = u / NI % MT, r = u / (NI * MT);
            const int m = m0 + 16 * t + g + 4 * i, n = n0 + 16 * r + n16;
            if (m < hi && n < p.N)
                p.y[m * p.ldy + n] = from_f32<F16>(v);
        }
        __syncthreads();
    }
}

template <bool F16, int G, bool Z, int NI, int MT, int R>
hipError_t launch_mv(const Args& a0, hipStream_t st) {
    Args a = a0;
    constexpr int kTokens = MT == 1 ? 4 * NI : 16 * MT;
    const int64_t chunks = ((int64_t)a.rows + kTokens - 1) / kTokens;
    a.chunk = (int32_t)(chunks < 16384 ? chunks : 16384);
    const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)), a.off ? a.experts : a.chunk);
    return launch1(k_mv_i4<F16, G, Z, NI, MT, R>, grid, dim3(kThreads), st, a);
}

template <bool F16, int G, bool Z>
hipError_t launch_rows(const Args& a, hipStream_t st) {
    const int64_t m = a.off ? (a.rows + a.experts - 1) / a.experts : a.rows;
    if (m <= 4)
        return launch_mv<F16, G, Z, 1, 1, 1>(a, st);
    if (m <= 8)
        return launch_mv<F16, G, Z, 2, 1, 1>(a, st);
    if (m <= 16)
        return launch_mv<F16, G, Z, 4, 1, 2>(a, st);
    return launch_mv<F16, G, Z, 4, 4, 2>(a, st);
}

template <bool F16, int G>
hipError_t launch_zero(const Args& a, hipStream_t st) {
    return a.z ? launch_rows<F16, G, true>(a, st) : launch_rows<F16, G, false>(a, st);
}

}  // namespace

hipError_t launch_mm_i4(const I4Mm& m, int group, bool f16, hipStream_t stream) {
    Args a{};
    static_cast<I4Mm&>(a) = m;
    a.steps = (a.K + kTK - 1) / kTK;
    if (f16)
        return group == 32 ? launch_zero<true, 32>(a, stream)
             : group == 64 ? launch_zero<true, 64>(a, stream)
                           : launch_zero<true, 128>(a, stream);
    return group == 32 ? launch_zero<false, 32>(a, stream)
         : group == 64 ? launch_zero<false, 64>(a, stream)
                       : launch_zero<false, 128>(a, stream);
}

}  // namespace bq
