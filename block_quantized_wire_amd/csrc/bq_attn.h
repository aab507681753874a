// bq_attn.h -- attention over the 4-bit cache of keys and values: the kernels, for one head width.
//
// A cached number is c * s + m: a code 0..15, a scale and a least value of its group.  For a row q
// of the queries and a token t,
//     score = scale * sum over groups g of [ s_tg * (q_g . c_tg) + m_tg * sum(q_g) ],
//     out_d = ( sum_t (p_t s_tg) c_td + sum_t p_t m_tg ) / sum_t p_t,   p_t = exp(score - R),
// so both products are matrix products with the codes themselves, and scales and least values
// come in beside them, in binary32.
//
// Codes of keys are operands without a conversion: the bits of a code in the low bits of a binary16
// number are that number's subnormal c * 2^-24 (c * 2^-20 four bits higher), which the matrix
// cores take exactly.  A word of 8 codes becomes 4 registers of 2 operands with 4 ANDs and a
// shift.  q is scaled by a power of two to just below 2^14 (its numbers that meet the codes four
// bits higher by 2^-4 more), so binary16 holds it exactly but for numbers 2^-24 below the largest.
// Codes of values are centred to c - 8 first, an instruction more for two: over many tokens the
// result is small beside the sums of c s and of m, and would be lost in their binary32 rounding.
// p_t s_tg goes in as one binary16 number where the result is bf16, whose rounding is 8 times as
// large; for binary16 results as a sum of two (22 bits in all).
//
// Steps.  A wave takes 32 tokens a step, as the rows of two 16x16x32 products with 16 * NC rows of
// q (rows of one cache head: tokens times the heads that share it).  Row 4b + i of the two is
// token 8b + i and 8b + 4 + i, so that the four lanes of a quarter wave end up with 8 whole
// tokens of their row of q: exactly the operand of the second product, V^T P^T, without a
// move between lanes.  The cache's layouts (include/blockq_kv.h) give each lane its codes in
// one run of dim/8 and one of dim/4 bytes.
//
// Softmax: R, the reference of a row, is only raised when a score passes it by 8 (a
// factor of 2^8), which a wave tests once a step.  p is 2^k times as large as written above, with
// a k of the wave that brings the largest scale of values to just below 2^7: p s then fills the
// range of binary16.  2^k is in the row's sums of p too, and leaves with the division.
#pragma once

#include <type_traits>
#include <utility>

#include "bq_device.h"
#include "bq_launch.h"

namespace bq {
namespace attn {

typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStep = 32;           // tokens of a step
constexpr float kRaise = 8.0f;      // a score may pass R by this, in powers of two

struct Args {
    AttnI4 a;
    int32_t units;      // seqs * cache heads * splits
    int32_t tiles, splits, share, bpp;
    float scale2;       // scale * log2(e)
    float* part;        // partial results [splits][rows][heads][D], relative to their R
    float* ml;          // [splits][rows][heads][2]: R, sum of p
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// The value of lane `Lane` of each row of 16 lanes.
template <int Lane>
__device__ __forceinline__ float bcast(float v) {
    return __uint_as_float(dpp<0x150 + Lane>(__float_as_uint(v)));
}

template <bool F16>
__device__ __forceinline__ float lo16(uint32_t w) {
    if constexpr (F16)
        return (float)__builtin_bit_cast(h16x2, w).x;
    else
        return bf16_lo(w);
}
template <bool F16>
__device__ __forceinline__ float hi16(uint32_t w) {
    if constexpr (F16)
        return (float)__builtin_bit_cast(h16x2, w).y;
    else
        return bf16_hi(w);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, h16x2{(_Float16)a, (_Float16)b});
    else
        return pack_bf16x2(a, b);
}

// Sum, maximum over the four lanes that hold a row of q.
__device__ __forceinline__ float quarter_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float quarter_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16));
    return __builtin_fmaxf(v, __shfl_xor(v, 32));
}

// Which rows of q and which tokens a sequence has; brought inside the arrays.
struct Seq {
    int row0, n, len;
};
__device__ __forceinline__ Seq seq_of(const AttnI4& a, int b) {
    Seq s;
    if (a.starts) {
        s.row0 = clampi(a.starts[b], 0, a.rows);
        const int end = clampi(a.starts[b + 1], s.row0, a.rows);
        s.n = end - s.row0;
        if (s.n > a.max_q)
            s.n = a.max_q;
    } else {
        s.row0 = b;
        s.n = b < a.rows ? 1 : 0;
    }
    const int64_t room = (int64_t)a.table_cols * a.c.page_size;
    s.len = clampi(a.lens[b], 0, room < a.max_len ? (int)room : a.max_len);
    return s;
}

// 8 codes as 8 operands: pairs (0, 4), (1, 5) * 16, (2, 6), (3, 7) * 16.
__device__ __forceinline__ h16x8 codes8(uint32_t w) {
    const uint32_t h = w >> 8;
    return __builtin_bit_cast(
        h16x8, u32x4{w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u});
}

// Codes c of the low (high: of the next four) bits of both half-words as c - 8 (16 times that):
// 1024 + c is a binary16 number with c in its low bits.
__device__ __forceinline__ uint32_t centred(uint32_t w, bool high) {
    const uint32_t m = high ? 0x00F000F0u : 0x000F000Fu;
    const h16x2 off = high ? h16x2{(_Float16)-1152.0f, (_Float16)-1152.0f}
                           : h16x2{(_Float16)-1032.0f, (_Float16)-1032.0f};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h16x2, (w & m) | 0x64006400u) + off);
}

// N words of a lane, 4 N bytes that follow each other.
template <int N>
__device__ __forceinline__ void ld_words(const uint8_t* at, uint32_t* w) {
    if constexpr (N == 2) {
        const u32x2 x = ld8(at);
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 x = ld16(at + 4 * i);
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    }
}

template <bool F16>
__device__ __forceinline__ void put4(uint16_t* o, f32x4 y, float by) {
    *reinterpret_cast<u32x2*>(o) = u32x2{pack2<F16>(y[0] * by, y[1] * by), pack2<F16>(y[2] * by, y[3] * by)};
}

__device__ __forceinline__ float lse_of(float ref, float sum) {
    return sum == 0.0f ? -__builtin_inff()
                       : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945309f;
}

// What is kept for 16 * NC rows of q while the tokens pass, and a step.
template <int D, int G, bool F16, int NC>
struct State {
    static constexpr int W = D / 32;      // products over the head's width; words of k to a lane
    static constexpr int NJ = D / 16;     // blocks of 16 numbers of the result; words of v to a lane
    static constexpr int NG = D / G;      // groups

    const Args& p;
    const int lane, r, g;
    int head, lo, hi;         // the cache's head; tokens that some row sees

    h16x8 q[NC][W];
    float qs[NC][NG], fac[NC];
    int seen_lo[NC], seen_hi[NC];
    int full_lo, full_hi;     // tokens that every row sees
    f32x4 acc[NC][NJ];
    float R[NC], l[NC], mb[NC][NG];
    float k2, s_lim;          // the power of two of p, largest scale that it is meant for

    __device__ explicit State(const Args& args)
        : p(args), lane(threadIdx.x & 63), r(lane & 15), g(lane >> 4) {}

    // The tokens that rows [first, first + 16 NC) of a sequence see: [lo, hi).
    __device__ __forceinline__ void range(const Seq& sq, int first, int n, int rows, int& from,
                                          int& to) const {
        const int last = (first + n < rows ? first + n : rows) - 1, at0 = sq.len - sq.n;
        to = first >= rows ? 0 : p.a.causal ? clampi(at0 + last / p.share + 1, 0, sq.len) : sq.len;
        from = p.a.window > 0 ? clampi(at0 + first / p.share + 1 - p.a.window, 0, to) : 0;
    }

    // Rows of q of this wave: `first` is the first of them among the sequence's rows.
    __device__ __forceinline__ void load_q(const Seq& sq, int first, int rows) {
        range(sq, first, 16 * NC, rows, lo, hi);
        full_lo = 0;
        full_hi = 1 << 30;
        // a negative scale is that of -q
        const float sign = p.scale2 < 0.0f ? -1.0f : p.scale2 > 0.0f ? 1.0f : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int row = first + 16 * c + r;
            const bool in = row < rows;
            const int qi = in ? row / p.share : 0, hd = in ? row % p.share : 0;
            const uint16_t* x = p.a.q + (int64_t)(sq.row0 + qi) * p.a.ldq +
                                (int64_t)(head * p.share + hd) * p.a.hsq + 8 * g;
            float f[8 * W];
            float top = 0.0f;
            bool fine = true;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const u32x4 w = in ? ld16(x + 32 * k) : u32x4{};
                if constexpr (F16)
                    unpack_f16x8(w, f + 8 * k);
                else
                    unpack_bf16x8(w, f + 8 * k);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float m = __builtin_fabsf(f[8 * k + i]);
                    fine = fine && m < __builtin_inff();
                    top = __builtin_fmaxf(top, m);
                    f[8 * k + i] *= sign;
                }
            }
            top = quarter_max(top);
            const bool all_fine = quarter_sum(fine ? 0.0f : 1.0f) == 0.0f;
            const int e = all_fine ? __builtin_amdgcn_frexp_expf(top) : 0;
            fac[c] = sign == 0.0f ? 1.0f : __builtin_ldexpf(__builtin_fabsf(p.scale2), 10 + e);
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8 * W / NG; ++i)
                    sum += __builtin_ldexpf(f[k * (8 * W / NG) + i], -10 - e);
                qs[c][k] = all_fine ? quarter_sum(sum) : __builtin_nanf("");
            }
#pragma unroll
            for (int k = 0; k < W; ++k) {
                h16x8 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int sh = (i & 1 ? 10 : 14) - e;
                    o[2 * i] = (_Float16)__builtin_ldexpf(f[8 * k + i], sh);
                    o[2 * i + 1] = (_Float16)__builtin_ldexpf(f[8 * k + i + 4], sh);
                }
                q[c][k] = o;
            }
            const int at = sq.len - sq.n + qi;      // the row's place
            seen_hi[c] = p.a.causal && in ? (at + 1 < sq.len ? at + 1 : sq.len) : sq.len;
            seen_lo[c] = p.a.window > 0 && in && at + 1 - p.a.window > 0 ? at + 1 - p.a.window : 0;
            if (!in) {      // sees what its wave sees
                seen_lo[c] = 0;
                seen_hi[c] = 1 << 30;
            }
            full_lo = seen_lo[c] > full_lo ? seen_lo[c] : full_lo;
            full_hi = seen_hi[c] < full_hi ? seen_hi[c] : full_hi;
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const int a = __shfl_xor(full_lo, d), b = __shfl_xor(full_hi, d);
            full_lo = a > full_lo ? a : full_lo;
            full_hi = b < full_hi ? b : full_hi;
        }
        full_lo = __builtin_amdgcn_readfirstlane(full_lo);
        full_hi = __builtin_amdgcn_readfirstlane(full_hi);
        full_hi = full_hi < hi ? full_hi : hi;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            R[c] = -__builtin_inff();
            l[c] = 0.0f;
#pragma unroll
            for (int k = 0; k < NG; ++k)
                mb[c][k] = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        k2 = 0.0f;
        s_lim = 0.0f;
    }

    // 32 tokens from `tok` on.  What the source gives: k(h, w) and v(j), operands; k_scales<group>
    // and v_scales<group>, scale and least value of the 8 tokens of this quarter wave (of values
    // m + 8 s); s_max, the largest scale of values among this lane's.  ok: the 8 tokens' page is there.
    template <bool MASK, typename Src>
    __device__ __forceinline__ void step(const Src& src, int tok, bool ok) {
        float x[NC][8];
        unroll<NG>([&](auto gi) {
            constexpr int k = decltype(gi)::value;
            f32x4 a[NC][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    a[c][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = k * (W / NG); w < (k + 1) * (W / NG); ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const h16x8 op = src.k(h, w);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        a[c][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op, q[c][w], a[c][h], 0, 0, 0);
                }
            float s[8], m[8];
            src.template k_scales<k>(s, m);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float b = a[c][i / 4][i % 4];
                    x[c][i] = __builtin_fmaf(m[i], qs[c][k],
                                             k == 0 ? s[i] * b : __builtin_fmaf(s[i], b, x[c][i]));
                }
        });
        float top[NC];
        bool raise = src.s_max > s_lim;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (MASK) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = tok + 8 * g + i;
                    const bool in = ok && t >= seen_lo[c] && t < seen_hi[c] && t < hi;
                    x[c][i] = in ? x[c][i] : -__builtin_inff();
                }
            }
            top[c] = x[c][0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top[c] = __builtin_fmaxf(top[c], x[c][i]);
            top[c] *= fac[c];
            raise = raise || top[c] > R[c] + kRaise;
        }
        if (__any(raise))
            new_reference(top, src.s_max);
        float pr[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float ref = R[c] == -__builtin_inff() ? 0.0f : R[c] - k2;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[c][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[c][i], fac[c], -ref));
                sum += pr[c][i];
            }
            l[c] += sum;
        }
        unroll<NG>([&](auto gi) {
            constexpr int k = decltype(gi)::value;
            h16x8 ph[NC], pl[NC];
            float s[8], m[8];
            src.template v_scales<k>(s, m);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float ps[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ps[i] = pr[c][i] * s[i];
                    if constexpr (MASK) {
                        // what a row does not see has no effect on it, a scale of NaN neither
                        const bool in = !(x[c][i] == -__builtin_inff());
                        ps[i] = in ? ps[i] : 0.0f;
                        mb[c][k] += in ? pr[c][i] * m[i] : 0.0f;
                    } else {
                        mb[c][k] = __builtin_fmaf(pr[c][i], m[i], mb[c][k]);
                    }
                }
                u32x4 uh, ul;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x2 two{ps[2 * i], ps[2 * i + 1]};
                    const h16x2 h = __builtin_convertvector(two, h16x2);
                    uh[i] = __builtin_bit_cast(uint32_t, h);
                    if constexpr (F16) {
                        const f32x2 rest{two.x - (float)h.x, two.y - (float)h.y};
                        ul[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, h16x2));
                    }
                }
                ph[c] = __builtin_bit_cast(h16x8, uh);
                if constexpr (F16)
                    pl[c] = __builtin_bit_cast(h16x8, ul);
            }
#pragma unroll
            for (int j = k * (NJ / NG); j < (k + 1) * (NJ / NG); ++j) {
                const h16x8 o = src.v(j);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if constexpr (F16)
                        acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, pl[c], acc[c][j], 0, 0, 0);
                    acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, ph[c], acc[c][j], 0, 0, 0);
                }
            }
        });
    }

    // Raises the rows' references to their largest scores, and fits 2^k to the largest scale.
    __device__ __forceinline__ void new_reference(const float (&top)[NC], float s_max) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            s_max = __builtin_fmaxf(s_max, __shfl_xor(s_max, d));
        float up = 0.0f;
        if (s_max > s_lim) {
            const int e = clampi(__builtin_amdgcn_frexp_expf(s_max), -93, 107);
            up = (float)(7 - e) - k2;
            k2 = (float)(7 - e);
            s_lim = __builtin_ldexpf(1.0f, e);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float m = __builtin_fmaxf(R[c], quarter_max(top[c]));
            const float by = R[c] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(R[c] - m + up);
            R[c] = m;
            l[c] *= by;
#pragma unroll
            for (int k = 0; k < NG; ++k)
                mb[c][k] *= by;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][j][i] *= by;
        }
    }

    template <int N, typename F>
    static __device__ __forceinline__ void unroll(F&& f) {
        unroll_at(f, std::make_integer_sequence<int, N>{});
    }
    template <typename F, int... I>
    static __device__ __forceinline__ void unroll_at(F& f, std::integer_sequence<int, I...>) {
        (f(std::integral_constant<int, I>{}), ...);
    }

    // The row's result before the division, numbers 16j + 4g .. +3.
    __device__ __forceinline__ f32x4 result(int c, int j, const float (&least)[NG]) const {
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = __builtin_fmaf(acc[c][j][i], j & 1 ? 0x1p-4f : 1.0f, least[j / (NJ / NG)]);
        return o;
    }
    // The reference that the sums are relative to.
    __device__ __forceinline__ float reference(int c) const { return R[c] - k2; }

    __device__ __forceinline__ int64_t cell(const Seq& sq, int row) const {
        return (int64_t)(sq.row0 + row / p.share) * p.a.heads + head * p.share + row % p.share;
    }
    __device__ __forceinline__ uint16_t* out_of(const Seq& sq, int row) const {
        return p.a.out + (int64_t)(sq.row0 + row / p.share) * p.a.ldo +
               (int64_t)(head * p.share + row % p.share) * p.a.hso;
    }
    __device__ __forceinline__ void put_lse(const Seq& sq, int row, float ref, float sum) const {
        if (p.a.lse)
            p.a.lse[cell(sq, row)] = lse_of(ref, sum);
    }
};

// Where in its page a block of 8 tokens lies, steps of `stride` blocks on.
struct Walk {
    int idx, off, dq, dr;
    Walk() = default;
    __device__ __forceinline__ Walk(int block, int stride, int bpp)
        : idx(block / bpp), off(block % bpp), dq(stride / bpp), dr(stride % bpp) {}
    __device__ __forceinline__ void step(int bpp) {
        idx += dq;
        off += dr;
        if (off >= bpp) {
            off -= bpp;
            ++idx;
        }
    }
};

// A workgroup's place among the sequences, heads, splits and tiles; the last tiles, which see the
// most under a causal mask, start first.
struct Place {
    int tile, head, split, seq;
    __device__ __forceinline__ explicit Place(const Args& p) {
        tile = p.tiles - 1 - (int)(blockIdx.x / (uint32_t)p.units);
        int unit = (int)(blockIdx.x % (uint32_t)p.units);
        head = unit % p.a.c.heads;
        unit /= p.a.c.heads;
        split = unit % p.splits;
        seq = unit / p.splits;
    }
};

// Blocks [b0, b1) of 8 tokens of a split of tokens [lo, hi), in whole steps of `unit` blocks.
__device__ __forceinline__ void split_blocks(int lo, int hi, int split, int splits, int unit, int& b0,
                                             int& b1) {
    const int first = lo / 8, n = (hi + 7) / 8 - first;
    const int per = ((n + splits - 1) / splits + unit - 1) / unit * unit;
    b0 = first + split * per;
    b1 = b0 + per < first + n ? b0 + per : first + n;
}

// ---- few rows: the waves of a workgroup share its tokens --------------------------------------
//
// Each wave takes every fourth step of the workgroup's tokens, straight from memory to
// operands, one step loaded ahead; the waves' results join through LDS.  Scales are loaded
// once a quarter wave, one word or a few to a lane, and broadcast as DPP operands.
template <int D, int G, bool F16, int NC>
struct Tokens : State<D, G, F16, NC> {
    using S = State<D, G, F16, NC>;
    using S::W, S::NJ, S::NG, S::p, S::r, S::g, S::head, S::lo, S::hi;

    const int32_t* table;

    struct Tile {
        uint32_t k[2][W], v[NJ], s[NG];
        int tok;
        bool ok;
    };

    struct Src {
        const Tile& t;
        float ss[NG], sm[NG], s_max;

        __device__ __forceinline__ h16x8 k(int h, int w) const { return codes8(t.k[h][w]); }
        __device__ __forceinline__ h16x8 v(int j) const {
            u32x4 op;
#pragma unroll
            for (int tp = 0; tp < 4; ++tp) {
                const uint32_t w = t.v[tp * (D / 64) + j / 4];
                op[tp] = centred(j % 4 >= 2 ? w >> 8 : w, j & 1);
            }
            return __builtin_bit_cast(h16x8, op);
        }
        // Entry E of the quarter wave's words: group E / 8 of keys, then of values.
        template <int E, int... I>
        __device__ __forceinline__ void eight(float (&s)[8], float (&m)[8],
                                              std::integer_sequence<int, I...>) const {
            ((s[I] = bcast<(E + I) % 16>(ss[(E + I) / 16]), m[I] = bcast<(E + I) % 16>(sm[(E + I) / 16])),
             ...);
        }
        template <int K>
        __device__ __forceinline__ void k_scales(float (&s)[8], float (&m)[8]) const {
            eight<8 * K>(s, m, std::make_integer_sequence<int, 8>{});
        }
        template <int K>
        __device__ __forceinline__ void v_scales(float (&s)[8], float (&m)[8]) const {
            eight<8 * NG + 8 * K>(s, m, std::make_integer_sequence<int, 8>{});
        }
        __device__ __forceinline__ Src(const Tile& tile, bool mask, int lo, int hi, int r, int g)
            : t(tile), s_max(0.0f) {
            const int tok = t.tok + 8 * g + (r & 7);
            const bool in = !mask || (t.ok && tok >= lo && tok < hi);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                // 0 for tokens that no row sees
                ss[i] = in ? lo16<F16>(t.s[i]) : 0.0f;
                sm[i] = in ? hi16<F16>(t.s[i]) : 0.0f;
                // registers of values: the upper half, or the upper lanes of the only one
                if (NG == 1 ? r >= 8 : 2 * i >= NG) {
                    const float m = __builtin_fabsf(ss[i]);
                    sm[i] = __builtin_fmaf(8.0f, ss[i], sm[i]);
                    s_max = __builtin_fmaxf(s_max, m < __builtin_inff() ? m : 0.0f);
                }
            }
        }
    };

    __device__ explicit Tokens(const Args& args) : S(args) {}

    __device__ __forceinline__ int page_at(int idx) const {
        return idx < p.a.table_cols ? table[idx] : -1;
    }

    __device__ __forceinline__ Tile load(const Walk& wk, const Walk& wv, int pk, int pv, int tok) const {
        Tile t;
        const bq_kv_i4& c = p.a.c;
        t.tok = tok;
        t.ok = (uint32_t)pv < (uint32_t)c.pages;
        // a page outside the pool: page 0 is read, and no row sees it
        const int64_t ik = (uint32_t)pk < (uint32_t)c.pages ? pk : 0, iv = t.ok ? pv : 0;
        const uint8_t* k = c.k + ik * c.page_stride + (int64_t)head * c.head_stride +
                           (int64_t)wk.off * (8 * D / 2) + (r & 3) * (D / 2) + g * (D / 8);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ld_words<W>(k + h * 4 * (D / 2), t.k[h]);
        ld_words<NJ>(c.v + iv * c.page_stride + (int64_t)head * c.head_stride +
                         (int64_t)wv.off * (8 * D / 2) + r * (D / 4), t.v);
        const int64_t so = iv * c.spage_stride + (int64_t)head * c.shead_stride;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int e = 16 * i + r;
            const bool of_v = e >= 8 * NG;
            const int at = of_v ? e - 8 * NG : e;
            const uint16_t* s = (of_v ? c.vs : c.ks) + so +
                                2 * ((int64_t)(at >> 3) * c.page_size + wv.off * 8 + (at & 7));
            t.s[i] = *reinterpret_cast<const uint32_t*>(s);
        }
        return t;
    }

    // All steps over blocks of 8 tokens [b0, b1), `stride` blocks apart.
    __device__ __forceinline__ void walk(int b0, int b1, int stride) {
        if (b0 >= b1)
            return;
        const int bpp = p.bpp;
        Walk wk(b0 + (r >> 2), stride, bpp), wv(b0 + g, stride, bpp);
        Tile t = load(wk, wv, page_at(wk.idx), page_at(wv.idx), b0 * 8);
        wk.step(bpp);
        wv.step(bpp);
        int pk = page_at(wk.idx), pv = page_at(wv.idx);
        for (int b = b0; b < b1; b += stride) {
            Tile next = t;
            if (b + stride < b1) {
                next = load(wk, wv, pk, pv, (b + stride) * 8);
                wk.step(bpp);
                wv.step(bpp);
                pk = page_at(wk.idx);
                pv = page_at(wv.idx);
            }
            if (t.tok >= this->full_lo && t.tok + kStep <= this->full_hi && __all(t.ok))
                this->template step<false>(Src(t, false, lo, hi, r, g), t.tok, true);
            else
                this->template step<true>(Src(t, true, lo, hi, r, g), t.tok, t.ok);
            t = next;
        }
    }

    __device__ __forceinline__ void run(float* lds) {
        const AttnI4& a = p.a;
        const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        const Place at(p);
        head = at.head;
        const Seq sq = seq_of(a, at.seq);
        const int rows = sq.n * p.share, first = at.tile * 16 * NC;
        if (first >= rows)
            return;
        table = a.table + (int64_t)at.seq * a.ldt;
        this->load_q(sq, first, rows);
        int b0, b1;
        split_blocks(lo, hi, at.split, p.splits, 4 * kWaves, b0, b1);
        walk(b0 + 4 * wave, b1, 4 * kWaves);
        const bool whole = p.splits == 1;
        // the waves' parts: [wave][row][D + 4], then (R, sum)
        constexpr int LD = D + 4;
        float* part = lds + (wave * 16 + r) * LD;
        float* ml = lds + kWaves * 16 * LD;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float least[NG];
            const float sum = quarter_sum(this->l[c]);
#pragma unroll
            for (int k = 0; k < NG; ++k)
                least[k] = quarter_sum(this->mb[c][k]);
            if (c > 0)
                __syncthreads();
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<f32x4*>(part + 16 * j + 4 * g) = this->result(c, j, least);
            if (g == 0)
                *reinterpret_cast<f32x2*>(ml + 2 * (wave * 16 + r)) = f32x2{this->reference(c), sum};
            __syncthreads();
            const int mine = threadIdx.x >> 4, seg = threadIdx.x & 15;
            const int row = first + 16 * c + mine;
            float ref = -__builtin_inff(), w[kWaves], total = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v)
                ref = __builtin_fmaxf(ref, ml[2 * (v * 16 + mine)]);
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                w[v] = ref == -__builtin_inff()
                           ? 0.0f
                           : __builtin_amdgcn_exp2f(ml[2 * (v * 16 + mine)] - ref);
                total += w[v] * ml[2 * (v * 16 + mine) + 1];
            }
            if (row >= rows)
                continue;
            const float by = whole ? (total == 0.0f ? 0.0f : 1.0f / total) : 1.0f;
            const int64_t cell = (int64_t)at.split * a.rows * a.heads + this->cell(sq, row);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                f32x4 y{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    const f32x4 z =
                        *reinterpret_cast<const f32x4*>(lds + (v * 16 + mine) * LD + 64 * j + 4 * seg);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = __builtin_fmaf(w[v], z[i], y[i]);
                }
                if (whole)
                    put4<F16>(this->out_of(sq, row) + 64 * j + 4 * seg, y, by);
                else
                    *reinterpret_cast<f32x4*>(p.part + cell * D + 64 * j + 4 * seg) = y;
            }
            if (seg == 0) {
                if (whole)
                    this->put_lse(sq, row, ref, total);
                else
                    *reinterpret_cast<f32x2*>(p.ml + 2 * cell) = f32x2{ref, total};
            }
        }
    }
};

template <int D, int G, bool F16, int NC>
__global__ __launch_bounds__(kThreads, 2) void k_attn_tokens(Args p) {
    __shared__ __align__(16) float lds[kWaves * 16 * (D + 4) + kWaves * 16 * 2];
    Tokens<D, G, F16, NC> k(p);
    k.run(lds);
}

// ---- many rows: the waves share the tokens' operands ------------------------------------------
//
// Each wave has 16 * NC rows of its own, and all of them see the same tokens: T a turn, which the
// workgroup makes into operands once, in LDS (two buffers, one barrier a turn: while a turn's
// operands are used, the codes of the next one are unpacked and those after it loaded).  An
// operand is 64 lanes * 16 bytes in the lanes' order, so neither side meets a bank conflict; scales
// lie there in binary32.
template <int D, int G, bool F16, int NC>
struct Rows : State<D, G, F16, NC> {
    using S = State<D, G, F16, NC>;
    using S::W, S::NJ, S::NG, S::p, S::lane, S::r, S::g, S::head, S::lo, S::hi;

    static constexpr int T = D == 256 ? 32 : 64;        // tokens a turn
    static constexpr int NS = T / kStep;                // steps a turn
    static constexpr int Parts = kWaves / NS;           // waves that unpack a step
    static constexpr int KW = 2 * W / Parts;            // words of k that a lane unpacks
    static constexpr int VB = NJ / Parts;               // blocks of v that a wave unpacks
    static constexpr int SW = (2 * NG * T + kThreads - 1) / kThreads;   // words of scales to a thread
    static constexpr int kOperand = 64 * 16;            // bytes
    // a buffer: operands of k [step][h][w], of v [step][j], scales [ks, km, vs, vm][group][T], then
    // whether the pages of the 8-token blocks are there
    static constexpr int kV = NS * 2 * W * kOperand;
    static constexpr int kS = kV + NS * NJ * kOperand;
    static constexpr int kOk = kS + 4 * NG * T * 4;
    static constexpr int kBuffer = kOk + 32;

    const int32_t* table;
    int wave, wg_lo, wg_hi;

    struct Raw {
        uint32_t k[KW], v[VB < 4 ? 4 : VB], s[SW];
        bool in[SW];
        bool ok;
    };

    struct Src {
        const char* buf;
        int lane, g, sub;
        float s_max;
        __device__ __forceinline__ h16x8 k(int h, int w) const {
            return *reinterpret_cast<const h16x8*>(buf + ((sub * 2 + h) * W + w) * kOperand + lane * 16);
        }
        __device__ __forceinline__ h16x8 v(int j) const {
            return *reinterpret_cast<const h16x8*>(buf + kV + (sub * NJ + j) * kOperand + lane * 16);
        }
        __device__ __forceinline__ void eight(int which, int k, float (&s)[8]) const {
            const float* at = reinterpret_cast<const float*>(buf + kS) + (which * NG + k) * T + sub * 32 + 8 * g;
            const f32x4 a = *reinterpret_cast<const f32x4*>(at), b = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = a[i];
                s[4 + i] = b[i];
            }
        }
        template <int K>
        __device__ __forceinline__ void k_scales(float (&s)[8], float (&m)[8]) const {
            eight(0, K, s);
            eight(1, K, m);
        }
        template <int K>
        __device__ __forceinline__ void v_scales(float (&s)[8], float (&m)[8]) const {
            eight(2, K, s);
            eight(3, K, m);
        }
        __device__ __forceinline__ Src(const char* b, int lane_, int sub_)
            : buf(b), lane(lane_), g(lane_ >> 4), sub(sub_), s_max(0.0f) {
            // one token and group to a lane (NG <= 8: at most 4 rounds)
            const float* at = reinterpret_cast<const float*>(buf + kS) + 2 * NG * T + sub * 32 + (lane & 31);
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                const float m = __builtin_fabsf(at[k * T]);
                s_max = __builtin_fmaxf(s_max, m < __builtin_inff() ? m : 0.0f);
            }
        }
    };

    __device__ explicit Rows(const Args& args) : S(args) {}

    __device__ __forceinline__ int page_at(int idx) const {
        return idx < p.a.table_cols ? table[idx] : -1;
    }

    // This lane's part of a turn: step `wave / Parts`, part `wave % Parts` of its words; words of
    // scales of the whole turn.
    struct Walks {
        Walk k, v, s[SW];
    };

    __device__ __forceinline__ int step_of() const { return wave / Parts; }
    __device__ __forceinline__ int part_of() const { return wave % Parts; }
    __device__ __forceinline__ void scale_entry(int i, int& which, int& group, int& tok) const {
        const int e = (int)threadIdx.x + i * kThreads;
        tok = e % T;
        group = e / T % NG;
        which = e / (T * NG);
    }

    __device__ __forceinline__ Raw load(const Walks& w, int tok) const {
        Raw x;
        const bq_kv_i4& c = p.a.c;
        const uint32_t pages = (uint32_t)c.pages;
        const int pk = page_at(w.k.idx), pv = page_at(w.v.idx);
        const int64_t ik = (uint32_t)pk < pages ? pk : 0, iv = (uint32_t)pv < pages ? pv : 0;
        const int64_t ho = (int64_t)head * c.head_stride;
        // Parts == 2: the part is the half of the step's tokens (h); 4: h and half of the words
        const int h = part_of() & 1, w0 = Parts == 4 ? (part_of() >> 1) * (W / 2) : 0;
        ld_words<KW>(c.k + ik * c.page_stride + ho + (int64_t)w.k.off * (8 * D / 2) +
                         ((r & 3) + 4 * h) * (D / 2) + g * (D / 8) + 4 * w0, x.k);
        const uint8_t* v = c.v + iv * c.page_stride + ho + (int64_t)w.v.off * (8 * D / 2) + r * (D / 4);
        if constexpr (D == 64) {
            ld_words<4>(v, x.v);
        } else {
            // blocks [part * VB, +VB): words tp * (D / 64) + part * (VB / 4) + ..
#pragma unroll
            for (int tp = 0; tp < 4; ++tp)
#pragma unroll
                for (int i = 0; i < VB / 4; ++i)
                    x.v[tp * (VB / 4) + i] = *reinterpret_cast<const uint32_t*>(
                        v + 4 * (tp * (D / 64) + part_of() * (VB / 4) + i));
        }
        x.ok = (uint32_t)pv < pages;
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            int which, group, t;
            scale_entry(i, which, group, t);
            x.s[i] = 0;
            x.in[i] = false;
            if (which < 2) {
                const int ps = page_at(w.s[i].idx);
                x.in[i] = (uint32_t)ps < pages && tok + t >= wg_lo && tok + t < wg_hi;
                const int64_t so = ((uint32_t)ps < pages ? (int64_t)ps : 0) * c.spage_stride +
                                   (int64_t)head * c.shead_stride;
                x.s[i] = *reinterpret_cast<const uint32_t*>(
                    (which ? c.vs : c.ks) + so +
                    2 * ((int64_t)group * c.page_size + w.s[i].off * 8 + (t & 7)));
            }
        }
        return x;
    }

    __device__ __forceinline__ void unpack(const Raw& x, char* buf) const {
        const int sub = step_of(), part = part_of();
        const int h = part & 1, w0 = Parts == 4 ? (part >> 1) * (W / 2) : 0;
#pragma unroll
        for (int i = 0; i < KW; ++i)
            *reinterpret_cast<h16x8*>(buf + ((sub * 2 + h) * W + w0 + i) * kOperand + lane * 16) =
                codes8(x.k[i]);
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            u32x4 op;
            // D == 64: blocks 2 part and 2 part + 1 of the same words
            const bool shift = D == 64 ? part != 0 : i % 4 >= 2;
#pragma unroll
            for (int tp = 0; tp < 4; ++tp) {
                const uint32_t w = x.v[D == 64 ? tp : tp * (VB / 4) + i / 4];
                op[tp] = centred(shift ? w >> 8 : w, i & 1);
            }
            *reinterpret_cast<u32x4*>(buf + kV + (sub * NJ + part * VB + i) * kOperand + lane * 16) = op;
        }
        float* sc = reinterpret_cast<float*>(buf + kS);
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            int which, group, t;
            scale_entry(i, which, group, t);
            if (which < 2) {
                const float s = x.in[i] ? lo16<F16>(x.s[i]) : 0.0f, m = x.in[i] ? hi16<F16>(x.s[i]) : 0.0f;
                sc[(2 * which * NG + group) * T + t] = s;
                sc[((2 * which + 1) * NG + group) * T + t] = which ? __builtin_fmaf(8.0f, s, m) : m;
            }
        }
        if (part == 0 && r == 0)
            reinterpret_cast<int*>(buf + kOk)[sub * 4 + g] = x.ok;
    }

    __device__ __forceinline__ void run(char* lds) {
        const AttnI4& a = p.a;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        const Place at(p);
        head = at.head;
        const Seq sq = seq_of(a, at.seq);
        const int rows = sq.n * p.share, tile = at.tile * 16 * NC * kWaves, first = tile + wave * 16 * NC;
        if (tile >= rows)
            return;
        table = a.table + (int64_t)at.seq * a.ldt;
        this->range(sq, tile, 16 * NC * kWaves, rows, wg_lo, wg_hi);
        this->load_q(sq, first, rows);
        int b0, b1;
        split_blocks(wg_lo, wg_hi, at.split, p.splits, T / 8, b0, b1);
        if (b0 < b1) {
            const int bpp = p.bpp;
            Walks w;
            w.k = Walk(b0 + 4 * step_of() + (r >> 2), T / 8, bpp);
            w.v = Walk(b0 + 4 * step_of() + g, T / 8, bpp);
#pragma unroll
            for (int i = 0; i < SW; ++i) {
                int which, group, t;
                scale_entry(i, which, group, t);
                w.s[i] = Walk(b0 + t / 8, T / 8, bpp);
            }
            auto on = [&] {
                w.k.step(bpp);
                w.v.step(bpp);
#pragma unroll
                for (int i = 0; i < SW; ++i)
                    w.s[i].step(bpp);
            };
            Raw x = load(w, b0 * 8);
            on();
            unpack(x, lds);
            if (b0 + T / 8 < b1) {
                x = load(w, b0 * 8 + T);
                on();
            }
            int turn = 0;
            for (int b = b0; b < b1; b += T / 8, turn ^= 1) {
                __syncthreads();        // this turn's operands are there, the last turn's are used up
                if (b + T / 8 < b1) {
                    unpack(x, lds + (turn ^ 1) * kBuffer);
                    if (b + 2 * (T / 8) < b1) {
                        x = load(w, b * 8 + 2 * T);
                        on();
                    }
                }
                const char* buf = lds + turn * kBuffer;
#pragma unroll
                for (int sub = 0; sub < NS; ++sub) {
                    const int tok = b * 8 + sub * kStep;
                    if (tok >= hi || tok + kStep <= lo)
                        continue;
                    const bool ok = reinterpret_cast<const int*>(buf + kOk)[sub * 4 + g] != 0;
                    const Src src(buf, lane, sub);
                    if (tok >= this->full_lo && tok + kStep <= this->full_hi && __all(ok))
                        this->template step<false>(src, tok, true);
                    else
                        this->template step<true>(src, tok, ok);
                }
            }
        }
        const bool whole = p.splits == 1;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float least[NG];
            const float sum = quarter_sum(this->l[c]);
#pragma unroll
            for (int k = 0; k < NG; ++k)
                least[k] = quarter_sum(this->mb[c][k]);
            const int row = first + 16 * c + r;
            if (row >= rows)
                continue;
            const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint16_t* o = this->out_of(sq, row) + 4 * g;
            const int64_t cell = (int64_t)at.split * a.rows * a.heads + this->cell(sq, row);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const f32x4 y = this->result(c, j, least);
                if (whole)
                    put4<F16>(o + 16 * j, y, by);
                else
                    *reinterpret_cast<f32x4*>(p.part + cell * D + 16 * j + 4 * g) = y;
            }
            if (g == 0) {
                if (whole)
                    this->put_lse(sq, row, this->reference(c), sum);
                else
                    *reinterpret_cast<f32x2*>(p.ml + 2 * cell) = f32x2{this->reference(c), sum};
            }
        }
    }
};

template <int D, int G, bool F16, int NC>
__global__ __launch_bounds__(kThreads) void k_attn_rows(Args p) {
    __shared__ __align__(16) char lds[2 * Rows<D, G, F16, NC>::kBuffer];
    Rows<D, G, F16, NC> k(p);
    k.run(lds);
}

// The partial results of a row joined: a wave to a row and head.
template <int D, bool F16>
__global__ __launch_bounds__(kThreads) void k_attn_join(Args p) {
    const AttnI4& a = p.a;
    const int lane = threadIdx.x & 63;
    const int64_t at = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int64_t per = (int64_t)a.max_q * a.heads;
    const int b = (int)(at / per);
    if (b >= a.seqs)
        return;
    const int qi = (int)(at % per) / a.heads, hd = (int)(at % per) % a.heads;
    const Seq sq = seq_of(a, b);
    if (qi >= sq.n)
        return;
    const int64_t row = sq.row0 + qi, cell = row * a.heads + hd, cells = (int64_t)a.rows * a.heads;
    float ref = -__builtin_inff(), sum = 0.0f;
    for (int s = lane; s < p.splits; s += 64)
        ref = __builtin_fmaxf(ref, p.ml[2 * (s * cells + cell)]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        ref = __builtin_fmaxf(ref, __shfl_xor(ref, d));
    constexpr int N = D / 64;
    float y[N] = {};
    for (int s0 = 0; s0 < p.splits; s0 += 64) {
        float w = 0.0f, ws = 0.0f;
        if (s0 + lane < p.splits && ref != -__builtin_inff()) {
            const f32x2 m = *reinterpret_cast<const f32x2*>(p.ml + 2 * ((s0 + lane) * cells + cell));
            w = __builtin_amdgcn_exp2f(m.x - ref);
            ws = w * m.y;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            ws += __shfl_xor(ws, d);
        sum += ws;
        const int n = p.splits - s0 < 64 ? p.splits - s0 : 64;
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float by = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), s));
            const float* z = p.part + ((int64_t)(s0 + s) * cells + cell) * D + lane;
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i] = __builtin_fmaf(by, z[64 * i], y[i]);
        }
    }
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* o = a.out + row * a.ldo + (int64_t)hd * a.hso + lane;
#pragma unroll
    for (int i = 0; i < N; ++i)
        o[64 * i] = (uint16_t)pack2<F16>(y[i] * by, 0.0f);
    if (a.lse && lane == 0)
        a.lse[cell] = lse_of(ref, sum);
}

// One overload for each width, each in a file of its own.
hipError_t launch_width(std::integral_constant<int, 64>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream);
hipError_t launch_width(std::integral_constant<int, 128>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream);
hipError_t launch_width(std::integral_constant<int, 256>, const Args& a, const AttnPlan& p, bool f16,
                        hipStream_t stream);

template <int D, int G, bool F16>
hipError_t launch_group(const Args& a, const AttnPlan& p, hipStream_t st) {
    const dim3 grid((unsigned)(a.units * a.tiles)), block(kThreads);
    hipError_t e;
    if (!p.by_rows)
        e = p.cols == 1 ? launch1(k_attn_tokens<D, G, F16, 1>, grid, block, st, a)
                        : launch1(k_attn_tokens<D, G, F16, 2>, grid, block, st, a);
    else if (p.cols == 1)
        e = launch1(k_attn_rows<D, G, F16, 1>, grid, block, st, a);
    else if (D == 256 || p.cols == 2)
        e = launch1(k_attn_rows<D, G, F16, 2>, grid, block, st, a);
    else
        e = launch1(k_attn_rows<D, G, F16, D == 256 ? 2 : 4>, grid, block, st, a);
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int64_t waves = (int64_t)a.a.seqs * a.a.max_q * a.a.heads;
    return launch1(k_attn_join<D, F16>, dim3((unsigned)((waves + kWaves - 1) / kWaves)), block, st, a);
}

template <int D>
hipError_t launch_any(const Args& a, const AttnPlan& p, bool f16, hipStream_t st) {
    const int g = a.a.c.group;
    if (g == 32)
        return f16 ? launch_group<D, 32, true>(a, p, st) : launch_group<D, 32, false>(a, p, st);
    if constexpr (D == 64) {
        return f16 ? launch_group<D, 64, true>(a, p, st) : launch_group<D, 64, false>(a, p, st);
    } else {
        if (g == 64)
            return f16 ? launch_group<D, 64, true>(a, p, st) : launch_group<D, 64, false>(a, p, st);
        return f16 ? launch_group<D, 128, true>(a, p, st) : launch_group<D, 128, false>(a, p, st);
    }
}

}  // namespace attn
}  // namespace bq
