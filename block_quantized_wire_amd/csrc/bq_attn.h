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
// Codes of values are centred to c - 8, by a product with -8 or, for binary16 results, before the
// product (matrix cores cut off what is far below their largest term, which biased long binary16 sums of
// the first form by 2^-17 of a scale; bf16 sums show no bias, with 2000000 tokens of one weight the mean
// error is 2^-15 of a result's size, and the conversion would take 1% to 4% of a call): over many tokens the
// result is small beside the sums of c s and of m, and would be lost in their binary32 rounding.
// p goes in as one binary16 number where the result is bf16, whose rounding is 8 times as large;
// for binary16 results as a sum of two (22 bits in all).
//
// Steps.  A wave takes 32 tokens a step, as the rows of two 16x16x32 products with 16 * NC rows of
// q (rows of one cache head: tokens times the heads that share it).  Row 4b + i of the two is
// token 8b + i and 8b + 4 + i, so that the four lanes of a quarter wave end up with 8 whole
// tokens of their row of q: exactly the operand of the second product, V^T P^T, without a
// move between lanes.  The cache's layouts (include/blockq_kv.h) give each lane its codes in
// one run of dim/8 and one of dim/4 bytes.
//
// Softmax: R, the reference of a row, is only raised when a score passes it by 8 (a
// factor of 2^8), which a wave tests once a step; the same branch keeps the power of two that
// brings the values' sizes into the range of binary16.
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
constexpr int kMaxSplits = 256;     // of the tokens of a sequence
constexpr int kMaxDealt = 256;      // sequences whose turns are dealt out
constexpr float kRaise = 8.0f;      // a score may pass R by this, in powers of two

// Division of n < 2^28 by a d <= 2^28 known to the host: with 2^(p - 28) >= d and mul =
// ceil(2^p / d), n * mul passes n * 2^p / d by less than 2^p / d, which no quotient notices.
struct Div {
    uint32_t d, mul, p;
    static Div by(uint32_t d) {
        uint32_t p = 28;
        while (((uint64_t)1 << (p - 28)) < d)
            ++p;
        return Div{d, (uint32_t)((((uint64_t)1 << p) + d - 1) / d), p};
    }
    __device__ __forceinline__ int div(int n) const {
        return (int)((uint64_t)(uint32_t)n * mul >> p);
    }
    __device__ __forceinline__ int mod(int n) const { return n - div(n) * (int)d; }
};

struct Args {
    AttnI4 a;
    Div heads, by_splits;
    Div cells;          // cache heads * splits
    Div inner;          // by_seq: tiles, else seqs
    int32_t by_seq;     // workgroups go by sequence, then tile; else by tile, then sequence
    int32_t groups;     // workgroups: seqs * tiles * cells
    Div share;          // heads of q to one of the cache
    Div bpp;            // blocks of 8 tokens to a page
    int32_t tiles, splits;
    int32_t dealt;      // workgroups that share all turns, or 0: one to a unit
    float scale2;       // scale * log2(e)
    // partial results, relative to their R, and (R, sum of p): [splits][rows][heads][D], or where
    // the turns are dealt out [workgroup][2][16][D]
    float* part;
    float* ml;
    // where turns are dealt out: [kMaxDealt][2] a sequence's turns in one unit, all of a cache head
    // up to its end; then those of all sequences
    int32_t* found;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// The value of lane `Lane` of each row of 16 lanes.
template <int Lane>
__device__ __forceinline__ float bcast(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x150 + Lane, 0xF,
                                                              0xF, true));
}

template <int Lane>
__device__ __forceinline__ uint32_t bcast_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + Lane, 0xF, 0xF, true);
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

// Which rows of q and which tokens a sequence has; brought inside the arrays.  at0: the first row's
// place, which rows beyond max_q move too; rows further in front than max_q (2^20 at most) see the same.
struct Seq {
    int row0, n, len, at0;
};
__device__ __forceinline__ Seq seq_of(const AttnI4& a, int b) {
    Seq s;
    if (a.starts) {
        s.row0 = clampi(a.starts[b], 0, a.rows);
        const int end = clampi(a.starts[b + 1], s.row0, a.rows);
        s.n = end - s.row0;
    } else {
        s.row0 = b;
        s.n = b < a.rows ? 1 : 0;
    }
    const int64_t room = (int64_t)a.table_cols * a.c.page_size;
    s.len = clampi(a.lens[b], 0, room < a.max_len ? (int)room : a.max_len);
    s.at0 = max(s.len - s.n, -(1 << 21));
    s.n = min(s.n, a.max_q);
    return s;
}

// 8 codes as 8 operands: pairs (0, 4), (1, 5) * 16, (2, 6), (3, 7) * 16.
__device__ __forceinline__ h16x8 codes8(uint32_t w) {
    const uint32_t h = w >> 8;
    return __builtin_bit_cast(
        h16x8, u32x4{w & 0x000F000Fu, w & 0x00F000F0u, h & 0x000F000Fu, h & 0x00F000F0u});
}

// Codes of the low bits of both half-words, or of the bits above them, as numbers c - Less: 1024 + c is
// a binary16 number with c in its low bits, 64 + c one with c four bits higher.  v_and_or_b32 takes one
// constant that is not in a vector register.
template <bool Above, int Less>
__device__ __forceinline__ h16x2 numbers(uint32_t w) {
    uint32_t one = Above ? 0x54005400u : 0x64006400u;
    asm("" : "+v"(one));
    const _Float16 off = (_Float16)(-(Above ? 64.0f : 1024.0f) - Less);
    return __builtin_bit_cast(h16x2, (w & (Above ? 0x00F000F0u : 0x000F000Fu)) | one) + h16x2{off, off};
}

// Global-to-LDS load of 16 (4) bytes per lane: lane i's land at lds + 16 i (4 i).
__device__ __forceinline__ void lds_load16(const void* p, void* lds) {
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}
__device__ __forceinline__ void lds_load4(const void* p, void* lds) {
    __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
}

// 8 numbers as operands: rounded to binary16, and with Low what that leaves of them.
template <bool Low>
__device__ __forceinline__ void split8(const float (&v)[8], h16x8& hi, h16x8& lo) {
    u32x4 uh, ul;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 two{v[2 * i], v[2 * i + 1]};
        const h16x2 h = __builtin_convertvector(two, h16x2);
        uh[i] = __builtin_bit_cast(uint32_t, h);
        if constexpr (Low) {
            const f32x2 rest{two.x - (float)h.x, two.y - (float)h.y};
            ul[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, h16x2));
        }
    }
    hi = __builtin_bit_cast(h16x8, uh);
    if constexpr (Low)
        lo = __builtin_bit_cast(h16x8, ul);
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

// What is kept for 16 * NC rows of q while the tokens pass, and their scores.
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
    float R[NC], l[NC];

    __device__ explicit State(const Args& args)
        : p(args), lane(threadIdx.x & 63), r(lane & 15), g(lane >> 4) {}

    // The tokens that rows [first, first + 16 NC) of a sequence see: [lo, hi).
    __device__ __forceinline__ void range(const Seq& sq, int first, int n, int rows, int& from,
                                          int& to) const {
        const int last = (first + n < rows ? first + n : rows) - 1;
        to = first >= rows ? 0 : p.a.causal ? clampi(sq.at0 + p.share.div(last) + 1, 0, sq.len) : sq.len;
        from = p.a.window > 0 ? clampi(sq.at0 + p.share.div(first) + 1 - p.a.window, 0, to) : 0;
    }

    // Rows of q of this wave: `first` is the first of them among the sequence's rows.
    __device__ __forceinline__ void load_q(const Seq& sq, int first, int rows) {
        full_lo = 0;
        full_hi = 1 << 30;
        // Rows of q are scaled to just below 2^14, those below 2^least to less: they go without the bits that
        // this leaves them.  Where q and the scale are both very small it keeps fac a normal number: a masked
        // score is -inf * fac.
        const int least = max(-100, -135 - __builtin_amdgcn_frexp_expf(p.scale2));
        // a negative scale is that of -q
        const float sign = p.scale2 < 0.0f ? -1.0f : p.scale2 > 0.0f ? 1.0f : 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int row = first + 16 * c + r;
            const bool in = row < rows;
            const int qi = in ? p.share.div(row) : 0, hd = in ? p.share.mod(row) : 0;
            const uint16_t* x = p.a.q + (int64_t)(sq.row0 + qi) * p.a.ldq +
                                (int64_t)(head * (int)p.share.d + hd) * p.a.hsq + 8 * g;
            float f[8 * W];
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const u32x4 w = in ? ld16(x + 32 * k) : u32x4{};
                if constexpr (F16)
                    unpack_f16x8(w, f + 8 * k);
                else
                    unpack_bf16x8(w, f + 8 * k);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = __builtin_fmaxf(top, __builtin_fabsf(f[8 * k + i]));
            }
            top = quarter_max(top);
            const int e = clampi(__builtin_amdgcn_frexp_expf(top), least, 128);
            const float by = sign * __builtin_ldexpf(1.0f, 14 - e);
            fac[c] = sign == 0.0f ? 1.0f : __builtin_ldexpf(__builtin_fabsf(p.scale2), 10 + e);
            float bad = 0.0f;
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                float sum = 0.0f;
#pragma unroll
                for (int i = k * (8 * W / NG); i < (k + 1) * (8 * W / NG); ++i) {
                    f[i] *= by;
                    sum += f[i];
                }
                sum = quarter_sum(sum);
                bad += sum * 0.0f;      // a NaN or an infinity in any of the row's groups
                qs[c][k] = sum * 0x1p-24f;
            }
#pragma unroll
            for (int k = 0; k < NG; ++k)
                qs[c][k] += bad;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = i & 1 ? 0x1p-4f : 1.0f;
                    const f32x2 two{f[8 * k + i] * z, f[8 * k + i + 4] * z};
                    o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, h16x2));
                }
                q[c][k] = __builtin_bit_cast(h16x8, o);
            }
            const int at = sq.at0 + qi;     // the row's place
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
            for (int j = 0; j < NJ; ++j)
                acc[c][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // Scores, over fac, of 32 tokens: those of this quarter wave's 8 tokens.  What the source gives:
    // k(h, w), operands, and k_scales<group>, scale and least value of the 8 tokens.
    template <typename Src>
    __device__ __forceinline__ void scores(const Src& src, float (&x)[NC][8]) const {
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
            if constexpr (NG > 2)       // or all groups' scales are held at once, and registers spill
                __builtin_amdgcn_sched_barrier(0);
        });
    }
    // Scores are numbers from here on: else the compiler takes their last steps behind the branch
    // that follows, with the operands of all of them, and spills.
    static __device__ __forceinline__ void settle(float (&x)[NC][8]) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm("" : "+v"(x[c][i]));
    }
    // Whether row c sees token t of a page that is there.
    __device__ __forceinline__ bool sees(int c, int t) const {
        return t >= seen_lo[c] && t < seen_hi[c] && t < hi;
    }
    // The largest scores, and whether one passes its reference by more than kRaise.
    __device__ __forceinline__ bool tops(const float (&x)[NC][8], float (&top)[NC]) const {
        bool raise = false;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            top[c] = x[c][0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top[c] = __builtin_fmaxf(top[c], x[c][i]);
            top[c] *= fac[c];
            raise = raise || top[c] > R[c] + kRaise;
        }
        return raise;
    }
    // Raises row c's reference; what its sums are to be multiplied with.
    __device__ __forceinline__ float raised(int c, float top) {
        const float m = __builtin_fmaxf(R[c], quarter_max(top));
        const float by = R[c] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(R[c] - m);
        R[c] = m;
        return by;
    }

    template <int N, typename F>
    static __device__ __forceinline__ void unroll(F&& f) {
        unroll_at(f, std::make_integer_sequence<int, N>{});
    }
    template <typename F, int... I>
    static __device__ __forceinline__ void unroll_at(F& f, std::integer_sequence<int, I...>) {
        (f(std::integral_constant<int, I>{}), ...);
    }

    __device__ __forceinline__ int64_t cell(const Seq& sq, int row) const {
        return (int64_t)(sq.row0 + p.share.div(row)) * p.a.heads + head * (int)p.share.d + p.share.mod(row);
    }
    __device__ __forceinline__ uint16_t* out_of(const Seq& sq, int row) const {
        return p.a.out + (int64_t)(sq.row0 + p.share.div(row)) * p.a.ldo +
               (int64_t)(head * (int)p.share.d + p.share.mod(row)) * p.a.hso;
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
    __device__ __forceinline__ Walk(int block, int stride, const Div& bpp)
        : idx(bpp.div(block)), off(bpp.mod(block)), dq(bpp.div(stride)), dr(bpp.mod(stride)) {}
    __device__ __forceinline__ void step(int bpp) {
        idx += dq;
        off += dr;
        if (off >= bpp) {
            off -= bpp;
            ++idx;
        }
    }
};

// The s-th sequence of a batch, long ones first: by eighths of the longest's length, within one as
// they come.  Workgroups are started in their order, and a long one that starts last is waited for.
__device__ __forceinline__ int by_length(const AttnI4& a, int s) {
    constexpr int N = kMaxDealt / 64;
    if (a.seqs == 1 || a.seqs > kMaxDealt)
        return s;
    const int lane = threadIdx.x & 63;
    int len[N], most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int b = 64 * i + lane;
        len[i] = b < a.seqs ? clampi(a.lens[b], 0, a.max_len) : -1;
        most = len[i] > most ? len[i] : most;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int m = __shfl_xor(most, d);
        most = m > most ? m : most;
    }
    most = __builtin_amdgcn_readfirstlane(most);
    int part = 7;
    while (true) {
        // lengths of (part, part + 1] eighths; the last part takes 0 too
        const int from = (int)((int64_t)most * part >> 3), to = (int)((int64_t)most * (part + 1) >> 3);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool in = len[i] >= 0 && len[i] <= to && (len[i] > from || part == 0);
            const uint64_t m = __ballot(in);
            const int n = __popcll(m);
            if (s < n) {
                const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                                             __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
                return 64 * i + __ffsll((unsigned long long)__ballot(in && before == s)) - 1;
            }
            s -= n;
        }
        if (--part < 0)
            return 0;       // every sequence is in one part
    }
}

// A workgroup's place among the sequences, heads, splits and tiles.  Heads are next to each other;
// the last tiles, which see the most under a causal mask, start first, or where all tiles of a
// sequence see about as much, the long sequences.
struct Place {
    int tile, head, split, seq;
    __device__ __forceinline__ explicit Place(const Args& p) {
        const int n = (int)blockIdx.x;
        const int cell = p.cells.div(n), rest = n - cell * (int)p.cells.d;      // heads, splits
        const int outer = p.inner.div(cell), in = cell - outer * (int)p.inner.d;
        tile = p.tiles - 1 - (p.by_seq ? in : outer);
        seq = by_length(p.a, p.by_seq ? outer : in);
        split = p.heads.div(rest);
        head = rest - split * p.a.c.heads;
    }
};

// Blocks [b0, b1) of 8 tokens of a split of tokens [lo, hi), in whole turns of `unit` blocks; b0
// is a multiple of 4.
__device__ __forceinline__ void split_blocks(int lo, int hi, int split, const Div& splits, int unit, int& b0,
                                             int& b1) {
    const int first = lo / 32 * 4, n = (hi + 7) / 8 - first;
    const int per = (splits.div(n + (int)splits.d - 1) + unit - 1) / unit * unit;
    b0 = first + split * per;
    b1 = b0 + per < first + n ? b0 + per : first + n;
}

// Turns of 128 tokens of sequence b, over the tokens that its rows see.
constexpr int kTurn = 16;       // blocks of 8 tokens
__device__ __forceinline__ int turns_of(const AttnI4& a, int b) {
    const Seq s = seq_of(a, b);
    const int first = s.at0 + 1 - a.window;     // the first row's first token, under a window
    const int lo = a.window > 0 && first > 0 ? first : 0;
    const int blocks = (s.len + 7) / 8 - lo / 32 * 4;
    return s.n > 0 && blocks > 0 ? (blocks + kTurn - 1) / kTurn : 0;
}
// Tiles of 16 rows of sequence b.
__device__ __forceinline__ int tiles_of(const AttnI4& a, int b, const Div& share) {
    return (seq_of(a, b).n * (int)share.d + 15) / 16;
}

// `total` turns dealt out to `groups` workgroups, each one a run of them.
struct Deal {
    int each, more;     // the first `more` workgroups have one more
    __device__ __forceinline__ Deal(int total, int groups)
        : each((int)((uint32_t)total / (uint32_t)groups)), more(total - each * groups) {}
    __device__ __forceinline__ int first(int w) const { return w * each + (w < more ? w : more); }
    // the workgroup that has turn t
    __device__ __forceinline__ int of(int t) const {
        const int high = more * (each + 1);
        return t < high ? (int)((uint32_t)t / (uint32_t)(each + 1))
                        : more + (int)((uint32_t)(t - high) / (uint32_t)each);
    }
};

// Workgroups of few rows that a compute unit holds.
// Their registers decide: one that is spilled in the walk would be loaded behind the ring and drain it.  (Heads of
// 256 in groups of 64, dealt out, reload one a segment, outside the walk.)
constexpr int tokens_groups(int dim, int group, bool dealt) {
    return dim == 64 ? (dealt ? 3 : 4) : dim == 128 && group >= 64 ? 3 : dim == 256 && group == 32 ? 1 : 2;
}

// ---- few rows: the waves of a workgroup share its tokens --------------------------------------
//
// Each wave takes every fourth step of the workgroup's tokens and keeps to itself: a ring of
// `Depth` steps in LDS, filled by global-to-LDS loads (16 bytes a lane, in the cache's own order),
// so that the next steps (one at a width of 128 in groups of 64 or 128, where three workgroups share the LDS) are
// on their way without a register; no barriers until the waves'
// results meet.
// Chunks of 16 bytes are permuted within a block so that neither operand's reads meet a
// bank conflict.  Scales: one word or a few to a lane of a quarter wave, broadcast as DPP operands.
//
// Sequences of a batch differ in length, which only the device knows.  So the turns of all of them
// (one after the other, tile by tile and head by head) are dealt out evenly to as many workgroups
// as the card holds at once, each of which takes its run of turns through one unit (a sequence,
// tile and head) or several; only units that workgroups share leave partial results.
//
// Measured, one row, 64 heads on 8 of 128 numbers, bf16: 32 sequences of 701 to 8192 tokens (132 MB) 37.3 us
// and 6 of joining, dealt out, 64 as a workgroup to each unit; one of 131071 (151 MB) 39 and 6.  Of a large copy's
// 5.1 TB/s that is 75%: the first loads of a launch and the last sums take about 6 us.  Vector
// instructions fill 38% to 45% of the cycles, products 10%.
template <int D, int G, bool F16, bool Dealt>
struct Tokens : State<D, G, F16, 1> {
    static constexpr int NC = 1;
    using S = State<D, G, F16, NC>;
    using S::W, S::NJ, S::NG, S::p, S::lane, S::r, S::g, S::head, S::lo, S::hi;
    using S::acc, S::R, S::l, S::fac;

    static constexpr int kChunks = D / 4;               // of 16 bytes, in a block of 8 tokens
    static constexpr int kJ = D / 64;                   // loads of k, and of v, in a step
    static constexpr int kLoads = 2 * kJ + NG;
    static constexpr int kV = 16 * D, kS = 32 * D, kSlot = 32 * D + 256 * NG;
    // workgroups that a compute unit holds, and the steps that leave room for them
    static constexpr int kGroups = tokens_groups(D, G, Dealt);
    static constexpr int kMost = (kGroups == 1 ? 128 : 160 / kGroups - 4) * 1024 / (kWaves * kSlot);
    static constexpr int Depth = kMost > 4 ? 4 : kMost;
    static_assert(Depth >= 2, "a step is used while the next is loaded");
    static constexpr int kJoin = (kWaves * 16 * (D + 4) + kWaves * 16 * 2) * 4;
    static constexpr int kLds = kWaves * Depth * kSlot > kJoin ? kWaves * Depth * kSlot : kJoin;

    // Where chunk q of a block of k (the b-th of its step) and of v lies; each its own inverse.
    static __device__ __forceinline__ uint32_t k_slot(uint32_t q, uint32_t b) {
        if constexpr (D == 64)
            return q ^ ((b & 1) * 8 + (b >> 1 & 1));
        else if constexpr (D == 128)
            return q ^ b;
        else
            return q ^ ((q >> 4 & 1) * 4 + b);
    }
    static __device__ __forceinline__ uint32_t v_slot(uint32_t q) {
        return D == 64 ? q : D == 128 ? q ^ (q >> 4 & 1) : q ^ (q >> 4 & 3);
    }

    struct Src {
        const char* slot;
        uint32_t kw[2][W];
        float ss[NG], sm[NG], s_max;

        __device__ __forceinline__ h16x8 k(int h, int w) const { return codes8(kw[h][w]); }
        // Codes of values, read when the scores are done: registers are short before that.
        __device__ __forceinline__ void load_v(uint32_t (&vw)[NJ], int r, int g) const {
#pragma unroll
            for (int i = 0; i < NJ / 4; ++i)
                put(vw + 4 * i, slot + kV + g * 4 * D + 16 * v_slot(r * (NJ / 4) + i));
        }
        static __device__ __forceinline__ h16x8 v(const uint32_t (&vw)[NJ], int j) {
            u32x4 op;
#pragma unroll
            for (int tp = 0; tp < 4; ++tp) {
                const uint32_t w = vw[tp * (D / 64) + j / 4], x = j % 4 >= 2 ? w >> 8 : w;
                if constexpr (F16)
                    op[tp] = __builtin_bit_cast(uint32_t, j & 1 ? numbers<true, 8>(x) : numbers<false, 8>(x));
                else
                    op[tp] = x & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
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
        // `in`: some row sees the token whose words this lane has.
        __device__ __forceinline__ Src(const char* at, bool in, int r, int g) : slot(at), s_max(0.0f) {
            const uint32_t b = (uint32_t)r >> 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t row = (r & 3) + 4 * h;
                if constexpr (W == 2) {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(
                        slot + b * 4 * D + 16 * k_slot(row * 2 + (g >> 1), b) + 8 * (g & 1));
                    kw[h][0] = x.x;
                    kw[h][1] = x.y;
                } else {
#pragma unroll
                    for (int i = 0; i < W / 4; ++i)
                        put(kw[h] + 4 * i, slot + b * 4 * D +
                                               16 * k_slot(row * (D / 32) + g * (W / 4) + i, b));
                }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int e = 16 * i + r, which = e >> 3;       // groups of keys, then of values
                const uint32_t w =
                    *reinterpret_cast<const uint32_t*>(slot + kS + (which * 32 + 8 * g + (e & 7)) * 4);
                // 0 for tokens that no row sees
                ss[i] = in ? lo16<F16>(w) : 0.0f;
                sm[i] = in ? hi16<F16>(w) : 0.0f;
                // registers of values: the upper half, or the upper lanes of the only one
                if (NG == 1 ? r >= 8 : 2 * i >= NG) {
                    const float m = __builtin_fabsf(ss[i]);
                    sm[i] = __builtin_fmaf(8.0f, ss[i], sm[i]);
                    s_max = __builtin_fmaxf(s_max, m < __builtin_inff() ? m : 0.0f);
                }
            }
        }
        static __device__ __forceinline__ void put(uint32_t* w, const char* at) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = x[i];
        }
    };

    static constexpr float kDown = 18.0f;   // p is up to 2^(kRaise - kDown): 2^30 of them times 2^104 add up
    static constexpr int kTop = 15 - (int)(kRaise - kDown);     // scales times 2^k2 are up to 2^kTop
    static constexpr int kMaxK = 150;
    float mb[NC][NG];
    int k2;
    float s_lim;              // largest scale that k2 is meant for

    // 32 tokens from `tok` on.  ok: the 8 tokens' page is there.  mask (uniform): not every row sees
    // every token.  Scales of values that are not finite then go into the score of the rows that
    // see them, as a NaN, and out of the others' way.
    __device__ __forceinline__ void step(const Src& src, int tok, bool ok, bool mask) {
        float x[NC][8];
        this->scores(src, x);
        if (mask) {
            // the scales as other values than those used below, or the compiler takes the broadcasts
            // of all groups in front of this branch and spills
            Src apart = src;
#pragma unroll
            for (int i = 0; i < NG; ++i)
                asm("" : "+v"(apart.ss[i]), "+v"(apart.sm[i]));
            float bad[8];
            S::template unroll<NG>([&](auto gi) {
                constexpr int k = decltype(gi)::value;
                float s[8], m[8];
                apart.template v_scales<k>(s, m);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float z = s[i] * 0.0f + m[i] * 0.0f;      // 0, or NaN
                    bad[i] = k == 0 ? z : bad[i] + z;
                }
                if constexpr (NG > 2)
                    __builtin_amdgcn_sched_barrier(0);
            });
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c][i] = ok && this->sees(c, tok + 8 * g + i) ? x[c][i] + bad[i] : -__builtin_inff();
        }
        float top[NC];
        const bool raise = this->tops(x, top);
        if (__any(raise || src.s_max > s_lim))
            new_reference(top, src.s_max);
        uint32_t vw[NJ];
        src.load_v(vw, r, g);
        float pr[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float ref = R[c] == -__builtin_inff() ? 0.0f : R[c] + kDown;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[c][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[c][i], fac[c], -ref));
                sum += pr[c][i];
            }
            l[c] += sum;
        }
        Src fit = src;      // scales of values as they meet p
#pragma unroll
        for (int i = 0; i < NG; ++i)
            if (NG == 1 || 2 * i >= NG)
                fit.ss[i] = __builtin_ldexpf(fit.ss[i], k2);
        S::template unroll<NG>([&](auto gi) {
            constexpr int k = decltype(gi)::value;
            h16x8 ph[NC], pl[NC];
            float s[8], m[8];
            fit.template v_scales<k>(s, m);
            if (mask) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool fine = s[i] * 0.0f + m[i] * 0.0f == 0.0f;
                    s[i] = fine ? s[i] : 0.0f;
                    m[i] = fine ? m[i] : 0.0f;
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float ps[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ps[i] = pr[c][i] * s[i];
                    mb[c][k] = __builtin_fmaf(pr[c][i], m[i], mb[c][k]);
                }
                split8<F16>(ps, ph[c], pl[c]);
            }
#pragma unroll
            for (int j = k * (NJ / NG); j < (k + 1) * (NJ / NG); ++j) {
                const h16x8 o = Src::v(vw, j);
                // -8 times the power of two of an even, of an odd block's codes
                const uint32_t e = j & 1 ? 0x80808080u : 0x80088008u;
                const h16x8 eight = __builtin_bit_cast(h16x8, u32x4{e, e, e, e});
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if constexpr (F16)
                        acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, pl[c], acc[c][j], 0, 0, 0);
                    else
                        acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(eight, ph[c], acc[c][j], 0, 0, 0);
                    acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, ph[c], acc[c][j], 0, 0, 0);
                }
            }
            if constexpr (NG > 2)
                __builtin_amdgcn_sched_barrier(0);
        });
    }

    // Raises the rows' references to their largest scores, and fits 2^k to the largest scale: p times
    // scale times 2^k is up to 2^15.  The sums of p and of least values do not take 2^k: they hold
    // whatever the scales are.
    __device__ __forceinline__ void new_reference(const float (&top)[NC], float s_max) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            s_max = __builtin_fmaxf(s_max, __shfl_xor(s_max, d));
        float up = 1.0f;
        if (s_max > s_lim) {
            const int e = clampi(__builtin_amdgcn_frexp_expf(s_max), kTop - kMaxK, 107);
            up = __builtin_amdgcn_exp2f((float)(kTop - e - k2));
            k2 = kTop - e;
            s_lim = __builtin_ldexpf(1.0f, e);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float by = this->raised(c, top[c]), both = by * up;
            l[c] *= by;
#pragma unroll
            for (int k = 0; k < NG; ++k)
                mb[c][k] *= by;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][j][i] *= both;
        }
    }

    // The row's result before the division, numbers 16j + 4g .. +3.
    __device__ __forceinline__ f32x4 result(int c, int j, const float (&least)[NG]) const {
        const float by_even = __builtin_ldexpf(1.0f, (F16 ? 0 : 24) - k2);
        const float by_odd = __builtin_ldexpf(1.0f, (F16 ? 0 : 20) - k2);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = __builtin_fmaf(acc[c][j][i], j & 1 ? by_odd : by_even, least[j / (NJ / NG)]);
        return o;
    }

    // Where the blocks of this wave's next 16 steps lie, one block to a lane (four to a step): found
    // once for all of them, and handed to the loading lanes by permutes.
    const int32_t* table;
    int b0, stride, steps;
    int64_t code, scale;        // bytes from the arrays' starts
    uint64_t there;             // whether the blocks' pages are
    uint32_t oks;               // the same for the steps in the ring, 4 bits to a slot

    __device__ explicit Tokens(const Args& args) : S(args) {}

    __device__ __forceinline__ void find_pages(int n) {
        const bq_kv_i4& c = p.a.c;
        // behind the last step: that one again
        const int s = n + (lane >> 2), b = b0 + (s < steps ? s : steps - 1) * stride + (lane & 3);
        const int idx = p.bpp.div(b), o = b - idx * (int)p.bpp.d;
        const int page = idx < p.a.table_cols ? table[idx] : -1;
        const bool in = (uint32_t)page < (uint32_t)c.pages;
        // a page outside the pool: page 0 is read, and no row sees it
        const int64_t at = in ? page : 0;
        code = at * c.page_stride + (int64_t)head * c.head_stride + (int64_t)o * (4 * D);
        scale = 2 * (at * c.spage_stride + (int64_t)head * c.shead_stride) + o * 32;
        there = __ballot(in);
    }
    // The value of block `b` of the `rel`-th step found.
    static __device__ __forceinline__ int64_t from(int64_t v, int rel, uint32_t b) {
        const int at = 16 * rel + 4 * b;
        const uint32_t lo = __builtin_amdgcn_ds_bpermute(at, (int)(uint32_t)v);
        const uint32_t hi = __builtin_amdgcn_ds_bpermute(at, (int)(v >> 32));
        return (int64_t)((uint64_t)hi << 32 | lo);
    }

    // Loads step n into slot s.  The count of loads is always the same.
    __device__ __forceinline__ void issue(char* ring, int s, int n) {
        const int rel = n & 15;
        if (rel == 0)
            find_pages(n);
        const bq_kv_i4& c = p.a.c;
        char* slot = ring + s * kSlot;
        oks = (oks & ~(15u << (4 * s))) | (uint32_t)(there >> (4 * rel) & 15u) << (4 * s);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const uint32_t q = j * 64 + lane, b = q / kChunks;
            const int64_t at = from(code, rel, b);
            lds_load16(c.k + at + 16 * k_slot(q % kChunks, b), slot + 1024 * j);
            lds_load16(c.v + at + 16 * v_slot(q % kChunks), slot + kV + 1024 * j);
        }
        const int64_t at = from(scale, rel, (lane & 31) >> 3) + 4 * (lane & 7);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int which = 2 * i + (lane >> 5);
            const uint8_t* s0 = reinterpret_cast<const uint8_t*>(which < NG ? c.ks : c.vs);
            lds_load4(s0 + at + 4 * (int64_t)c.page_size * (which < NG ? which : which - NG),
                      slot + kS + 256 * i);
        }
    }

    // Steps over blocks of 8 tokens [first, end), every fourth: the first ones are sent for.
    __device__ __forceinline__ void begin(char* ring, int first, int end) {
        b0 = first;
        stride = 4 * kWaves;
        steps = first < end ? (end - first + stride - 1) / stride : 0;
        oks = 0;
        if (steps > 0) {
#pragma unroll
            for (int d = 0; d < Depth - 1; ++d)
                issue(ring, d, d);
        }
    }
    __device__ __forceinline__ void walk(char* ring) {
        int s = 0;
        for (int n = 0; n < steps; ++n) {
            // what was read of the slot that is loaded now has arrived
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(ring, s == 0 ? Depth - 1 : s - 1, n + Depth - 1);
            // this step has landed when only those after it are outstanding
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((Depth - 1) * kLoads) : "memory");
            const uint32_t ok = oks >> (4 * s) & 15u;
            const int tok = 8 * (b0 + n * stride);
            const bool mask = !(ok == 15u && tok >= this->full_lo && tok + kStep <= this->full_hi);
            const bool mine = ok >> g & 1u;
            const int t = tok + 8 * g + (r & 7);
            this->step(Src(ring + s * kSlot, !mask || (mine && t >= lo && t < hi), r, g), tok, mine, mask);
            s = s == Depth - 1 ? 0 : s + 1;
        }
        // nothing lands in LDS after the end
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // Turns [t0, t0 + n) of a unit; its result, or a partial one into `slot`.
    __device__ __forceinline__ void segment(char* lds, int seq, int cache_head, int tile, int t0, int n,
                                            int slot) {
        const AttnI4& a = p.a;
        const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        head = cache_head;
        const Seq sq = seq_of(a, seq);
        const int rows = sq.n * (int)p.share.d, first = tile * 16;
        if (first >= rows)
            return;
        table = a.table + (int64_t)seq * a.ldt;
        char* ring = lds + wave * Depth * kSlot;
        int from;
        this->range(sq, 0, rows, rows, from, hi);
        from = from / 32 * 4 + t0 * kTurn;
        const int to = from + n * kTurn, end = (hi + 7) / 8;
        begin(ring, from + 4 * wave, to < end ? to : end);
        this->range(sq, first, 16, rows, lo, hi);
        this->load_q(sq, first, rows);
        k2 = kMaxK;
        s_lim = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int k = 0; k < NG; ++k)
                mb[c][k] = 0.0f;
        walk(ring);
        const bool whole = slot < 0;
        // the waves' parts, where the rings were: [wave][row][D + 4], then (R, sum)
        constexpr int LD = D + 4;
        float* all = reinterpret_cast<float*>(lds);
        float* part = all + (wave * 16 + r) * LD;
        float* ml = all + kWaves * 16 * LD;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float least[NG];
            const float sum = quarter_sum(this->l[c]);
#pragma unroll
            for (int k = 0; k < NG; ++k)
                least[k] = quarter_sum(mb[c][k]);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<f32x4*>(part + 16 * j + 4 * g) = result(c, j, least);
            if (g == 0)
                *reinterpret_cast<f32x2*>(ml + 2 * (wave * 16 + r)) = f32x2{R[c] + kDown, sum};
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
            const int64_t cell = 16 * (int64_t)slot + mine;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                f32x4 y{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    const f32x4 z =
                        *reinterpret_cast<const f32x4*>(all + (v * 16 + mine) * LD + 64 * j + 4 * seg);
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
        __syncthreads();        // the rings may be filled again
    }

    __device__ __forceinline__ void run(char* lds, int* turns) {
        const AttnI4& a = p.a;
        if constexpr (!Dealt) {
            const Place at(p);
            segment(lds, at.seq, at.head, at.tile, 0, 1 << 23, -1);
            return;
        }
        // every wave adds up the sequences' turns: lane i finds those of i, i + 64, ..; one of them
        // leaves in LDS how many each has, and all up to its end
        int past[kMaxDealt / 64], sum = 0;
#pragma unroll
        for (int i = 0; i < kMaxDealt / 64; ++i) {
            const int b = 64 * i + lane;
            past[i] = 0;
            if (64 * i < a.seqs) {
                const int n = b < a.seqs ? turns_of(a, b) : 0;
                int v = b < a.seqs ? n * tiles_of(a, b, p.share) : 0;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int u = __shfl_up(v, d);
                    v += lane >= d ? u : 0;
                }
                past[i] = sum + v;
                sum += __builtin_amdgcn_readlane(v, 63);
                if (threadIdx.x < 64) {
                    turns[b] = n;
                    turns[kMaxDealt + b] = past[i];
                    if (blockIdx.x == 0)        // for those who join
                        *reinterpret_cast<u32x2*>(p.found + 2 * b) = u32x2{(uint32_t)n, (uint32_t)past[i]};
                }
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0)
            p.found[2 * kMaxDealt] = sum;
        const int heads = a.c.heads;
        const Deal deal(sum * heads, p.dealt);
        const int w = (int)blockIdx.x;
        int at = deal.first(w);
        const int end = deal.first(w + 1);
        if (at >= end)
            return;
        int b = 0;
#pragma unroll
        for (int i = 0; i < kMaxDealt / 64; ++i)
            if (64 * i < a.seqs)
                b += __popcll(__ballot(64 * i + lane < a.seqs && past[i] * heads <= at));
        __syncthreads();
        int count = __builtin_amdgcn_readfirstlane(turns[b]);
        int units = tiles_of(a, b, p.share) * heads;
        const int before = __builtin_amdgcn_readfirstlane(turns[kMaxDealt + b]) * heads - count * units;
        int unit = (int)((uint32_t)(at - before) / (uint32_t)count);
        int t = at - before - unit * count;
        while (true) {
            const int take = end - at < count - t ? end - at : count - t;
            const int tile = p.heads.div(unit);
            segment(lds, b, unit - tile * heads, tile, t, take,
                    take == count ? -1 : 2 * w + (t == 0 ? 1 : 0));
            at += take;
            if (at >= end)
                break;
            t = 0;
            if (++unit == units) {
                unit = 0;
                do
                    count = __builtin_amdgcn_readfirstlane(turns[++b]);
                while (count == 0);
                units = tiles_of(a, b, p.share) * heads;
            }
        }
    }
};

template <int D, int G, bool F16, bool Dealt>
__global__ __launch_bounds__(kThreads, (Tokens<D, G, F16, Dealt>::kGroups)) void k_attn_tokens(Args p) {
    __shared__ __align__(16) char lds[Tokens<D, G, F16, Dealt>::kLds];
    __shared__ int turns[Dealt ? 2 * kMaxDealt : 1];
    Tokens<D, G, F16, Dealt> k(p);
    k.run(lds, turns);
}

// ---- many rows: the waves share the tokens' operands ------------------------------------------
//
// Each of 8 waves has 16 * NC rows of its own, and all of them see the same tokens: T a turn, which
// the workgroup makes into operands once, in LDS (two buffers, one barrier a turn: while a turn's
// operands are used, the codes of the next one are unpacked and those after it loaded).  An
// operand is 64 lanes * 16 bytes in the lanes' order, so neither side meets a bank conflict.  Four
// waves unpack values, the other four keys and their scales.
//
// Values become binary16 numbers here, c s + m in one rounding, so that p needs no scale of each
// group; in the _f16 kernels a second one has what that leaves, or their results would be 40% farther from
// 64 bits than few rows' are (a third product: 8% to 14% of a call).  For that the 8 tokens of a block take a power of two 2^b that brings their
// largest to just below 2^15 (in the _f16 kernels one of 1 or less, where it is larger); a quarter wave's
// 8 tokens of p are one block, so p takes 2^(k - b) there, k the least b so far.
//
// Measured: 8192 rows and tokens, causal, 32 heads on 8 of 128 numbers, bf16, groups of 64, 792 us or 694
// TFLOP/s of the 1223 of a large product; vector instructions fill 61% of the cycles and products 27%
// of them (32 of 197 in a step of 32 rows and 32 tokens; 64 bring scales and least values into the
// scores).  LDS instructions fill 31%, without a bank conflict.
template <int D, int G, bool F16, int NC>
struct Rows : State<D, G, F16, NC> {
    using S = State<D, G, F16, NC>;
    using S::W, S::NJ, S::NG, S::p, S::lane, S::r, S::g, S::head, S::lo, S::hi;
    using S::acc, S::R, S::l, S::fac;

    static constexpr int kRowWaves = 8;
    static constexpr int T = D == 256 ? 32 : 64;        // tokens a turn
    static constexpr int NS = T / kStep;                // steps a turn
    static constexpr int Parts = 4 / NS;                // waves of a kind that unpack a step
    static constexpr int KW = 2 * W / Parts;            // words of k that a lane unpacks
    static constexpr int VB = NJ / Parts;               // blocks of v that a wave unpacks
    static constexpr int GV = 16 * VB > G ? 16 * VB / G : 1;    // groups that they are in
    static constexpr int NB = NG > 1 ? NG / 2 : 1;      // words of scales to a lane, for the largest
    static constexpr int kOperand = 64 * 16;            // bytes
    // a buffer: operands of k [step][h][w], of v [step][j], scale and least value of k [2][group][T],
    // then b and whether the page is there for each block of 8 tokens
    static constexpr int kV = NS * 2 * W * kOperand;
    static constexpr int kLow = NS * NJ * kOperand;     // _f16: what the operands of v leave of the values, behind them
    static constexpr int kS = kV + (F16 ? 2 : 1) * kLow;
    static constexpr int kB = kS + 2 * NG * T * 4;
    static constexpr int kBuffer = kB + 64;
    static_assert(NG * T <= 256, "an entry of the keys' scales to a lane");
    static constexpr float kUp = 6.0f;      // p is up to 2^(kRaise + kUp)
    static constexpr float kApart = -60.0f;
    static constexpr int kNoSize = 200;     // above every block's power of two

    const int32_t* table;
    int wave, step_of, part_of;
    int wg_lo, wg_hi;
    float k2;                   // the k above

    // What a lane has loaded of a turn.  Of values: codes, a token's scales in each of its wave's
    // groups, one or a few of all groups'; of keys: codes, an entry's scales of key and value.
    struct Raw {
        uint32_t w[4], s[2], t[NB];
        bool ok;
    };

    struct Src {
        const char* buf;
        int lane, g, sub;
        __device__ __forceinline__ h16x8 k(int h, int w) const {
            return *reinterpret_cast<const h16x8*>(buf + ((sub * 2 + h) * W + w) * kOperand + lane * 16);
        }
        __device__ __forceinline__ h16x8 v(int j) const {
            return *reinterpret_cast<const h16x8*>(buf + kV + (sub * NJ + j) * kOperand + lane * 16);
        }
        __device__ __forceinline__ h16x8 v_low(int j) const {
            return *reinterpret_cast<const h16x8*>(buf + kV + kLow + (sub * NJ + j) * kOperand + lane * 16);
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
    };

    __device__ explicit Rows(const Args& args) : S(args) {}

    __device__ __forceinline__ int page_at(int idx) const {
        return idx < p.a.table_cols ? table[idx] : -1;
    }
    __device__ __forceinline__ bool of_values() const { return wave < 4; }
    // An entry of the keys' scales: token and group; -1 where there is none for this lane.
    __device__ __forceinline__ int entry() const {
        const int e = ((wave & 3) << 6) + lane;
        return e < NG * T ? e : -1;
    }

    // Walks: the block that this lane's codes are in, and that of its entry of scales.
    __device__ __forceinline__ void start(int b0, Walk& wc, Walk& ws) const {
        wc = Walk(b0 + 4 * step_of + (of_values() ? g : r >> 2), T / 8, p.bpp);
        const int e = entry();
        ws = Walk(b0 + (e < 0 ? 0 : e % T) / 8, T / 8, p.bpp);
    }

    __device__ __forceinline__ Raw load(const Walk& wc, const Walk& ws, int tok) const {
        Raw x;
        const bq_kv_i4& c = p.a.c;
        const uint32_t pages = (uint32_t)c.pages;
        const int pc = page_at(wc.idx);
        // a page outside the pool: page 0 is read, and no row sees it
        x.ok = (uint32_t)pc < pages;
        const int64_t page = x.ok ? pc : 0;
        const int64_t code = page * c.page_stride + (int64_t)head * c.head_stride + (int64_t)wc.off * (4 * D);
        if (of_values()) {
            const uint8_t* v = c.v + code + r * (D / 4);
            if constexpr (D == 64) {
                ld_words<4>(v, x.w);
            } else {
#pragma unroll
                for (int tp = 0; tp < 4; ++tp)
                    x.w[tp] = *reinterpret_cast<const uint32_t*>(v + 4 * (tp * (D / 64) + part_of));
            }
            const uint8_t* s = reinterpret_cast<const uint8_t*>(c.vs) +
                               2 * (page * c.spage_stride + (int64_t)head * c.shead_stride) + 32 * wc.off;
            const int group = part_of * VB * 16 / G;
#pragma unroll
            for (int k = 0; k < GV; ++k)
                x.s[k] = *reinterpret_cast<const uint32_t*>(s + 4 * ((int64_t)(group + k) * c.page_size + (r & 7)));
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int e = NG == 1 ? r & 7 : 16 * i + r;
                x.t[i] = *reinterpret_cast<const uint32_t*>(s + 4 * ((int64_t)(e >> 3) * c.page_size + (e & 7)));
            }
        } else {
            const int h = part_of & 1, w0 = NS == 1 ? (part_of >> 1) * (W / 2) : 0;
            ld_words<KW>(c.k + code + ((r & 3) + 4 * h) * (D / 2) + g * (D / 8) + 4 * w0, x.w);
            const int e = entry();
            x.s[0] = x.s[1] = 0;
            if (e >= 0) {
                const int ps = page_at(ws.idx), t = e % T;
                if ((uint32_t)ps < pages && tok + t >= wg_lo && tok + t < wg_hi) {
                    const int64_t at = (int64_t)ps * c.spage_stride + (int64_t)head * c.shead_stride +
                                       2 * ((int64_t)(e / T) * c.page_size + ws.off * 8 + (t & 7));
                    x.s[0] = *reinterpret_cast<const uint32_t*>(c.ks + at);
                    x.s[1] = *reinterpret_cast<const uint32_t*>(c.vs + at);
                }
            }
        }
        return x;
    }

    // A pair of 16-bit numbers one of which is not finite.
    static __device__ __forceinline__ bool wild(uint32_t w) {
        const uint32_t e = F16 ? 0x7C007C00u : 0x7F807F80u, x = w & e;
        return (x & 0xFFFFu) == (e & 0xFFFFu) || (x >> 16) == (e >> 16);
    }

    // Whether a value of the block may be 2^15 or more: a scale of 2^10, a least value of 2^14.
    __device__ __forceinline__ bool large(const Raw& x) const {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 top{0, 0};
#pragma unroll
        for (int i = 0; i < NB; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x.t[i] & 0x7FFF7FFFu));
        return __any(top.x >= 0x6400u || top.y >= 0x7400u);
    }
    // The power of two of the block of value codes that this lane has.
    __device__ __forceinline__ int fit(const Raw& x, int tok) const {
        // the block's largest value: of |m + 8 s| + 8 |s|, which all 16 and m are within
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const float s = lo16<F16>(x.t[i]), m = hi16<F16>(x.t[i]);
            const float v = __builtin_fabsf(__builtin_fmaf(8.0f, s, m)) + 8.0f * __builtin_fabsf(s);
            const int t = tok + step_of * kStep + 8 * g + (r & 7);
            const bool out = wild(x.t[i]) || !x.ok || t < wg_lo || t >= wg_hi;
            top = max(top, out ? 0u : __float_as_uint(v));
        }
        top = row_max16(top);
        // past binary32's range: below 2^133
        const int b = 15 - (top < 0x7F800000u ? __builtin_amdgcn_frexp_expf(__uint_as_float(top)) : 133);
        // binary16's own values go as they are unless one passes the range, which a scale that was rounded up
        // can make of the largest number; a block of zeros, or one that no row sees, leaves k as it is
        if (F16)
            return b < 0 ? b : 0;
        return top == 0 ? kNoSize : min(b, 141);
    }

    __device__ __forceinline__ void unpack(const Raw& x, char* buf, int tok) const {
        if (!of_values()) {
            const int h = part_of & 1, w0 = NS == 1 ? (part_of >> 1) * (W / 2) : 0;
#pragma unroll
            for (int i = 0; i < KW; ++i)
                *reinterpret_cast<h16x8*>(buf + ((step_of * 2 + h) * W + w0 + i) * kOperand + lane * 16) =
                    codes8(x.w[i]);
            const int e = entry();
            if (e >= 0) {
                // scales of the value that are not finite reach the rows that see it in their score
                float* sc = reinterpret_cast<float*>(buf + kS);
                sc[e] = lo16<F16>(x.s[0]);
                sc[NG * T + e] = wild(x.s[1]) ? __builtin_nanf("") : hi16<F16>(x.s[0]);
            }
            return;
        }
        const int b = F16 && !large(x) ? 0 : fit(x, tok);
        // a lane scales one token's pair for each of its groups, and the quarter wave shares them
        h16x2 s2[GV][4], m2[GV][4];
        const int tok_of = tok + step_of * kStep + 8 * g + (r & 7);
        const bool seen = x.ok && tok_of >= wg_lo && tok_of < wg_hi;
        S::template unroll<GV>([&](auto gi) {
            constexpr int k = decltype(gi)::value;
            const uint32_t w = wild(x.s[k]) || !seen ? 0u : x.s[k];
            uint32_t pair;
            if constexpr (F16) {
                // b >= -6: a scale or least value loses 2^-25 at most, where the block's largest value is 2^14
                const _Float16 by = (_Float16)__builtin_ldexpf(1.0f, b);
                pair = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h16x2, w) * h16x2{by, by});
            } else {
                const f32x2 two{__builtin_ldexpf(lo16<F16>(w), b), __builtin_ldexpf(hi16<F16>(w), b)};
                pair = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, h16x2));
            }
            S::template unroll<4>([&](auto ti) {
                constexpr int i = decltype(ti)::value;
                const uint32_t even = bcast_u<2 * i>(pair), odd = bcast_u<2 * i + 1>(pair);
                s2[k][i] = __builtin_bit_cast(h16x2, __builtin_amdgcn_perm(odd, even, 0x05040100u));
                m2[k][i] = __builtin_bit_cast(h16x2, __builtin_amdgcn_perm(odd, even, 0x07060302u));
            });
        });
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int j = part_of * VB + i;
            u32x4 op, low;
#pragma unroll
            for (int tp = 0; tp < 4; ++tp) {
                // D == 64: blocks 2 part and 2 part + 1 of the same words
                const uint32_t w = x.w[tp] >> (D == 64 ? 8 * part_of + 4 * i : 4 * i);
                const h16x2 c = numbers<false, 0>(w), sc = s2[16 * i / G][tp], le = m2[16 * i / G][tp];
                const h16x2 v = __builtin_elementwise_fma(c, sc, le);
                op[tp] = __builtin_bit_cast(uint32_t, v);
                if constexpr (F16) {
                    const f32x2 rest{__builtin_fmaf((float)c.x, (float)sc.x, (float)le.x) - (float)v.x,
                                     __builtin_fmaf((float)c.y, (float)sc.y, (float)le.y) - (float)v.y};
                    low[tp] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, h16x2));
                }
            }
            char* at = buf + kV + (step_of * NJ + j) * kOperand + lane * 16;
            *reinterpret_cast<u32x4*>(at) = op;
            if constexpr (F16)
                *reinterpret_cast<u32x4*>(at + kLow) = low;
        }
        if (part_of == 0 && r == 0)
            *reinterpret_cast<f32x2*>(buf + kB + 8 * (step_of * 4 + g)) =
                f32x2{(float)b, x.ok ? 1.0f : 0.0f};
    }

    // 32 tokens: step `sub` of a turn's operands.  One body, masked or not: with two of them the
    // results are copied where they meet.
    __device__ __forceinline__ void step(const char* buf, int sub, int tok) {
        const f32x2 bo = *reinterpret_cast<const f32x2*>(buf + kB + 8 * (sub * 4 + g));
        const float b = bo.x;
        const bool ok = bo.y != 0.0f;
        const Src src{buf, lane, g, sub};
        float x[NC][8];
        this->scores(src, x);
        S::settle(x);
        if (!(tok >= this->full_lo && tok + kStep <= this->full_hi && __all(ok))) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[c][i] = ok && this->sees(c, tok + 8 * g + i) ? x[c][i] : -__builtin_inff();
        }
        float top[NC];
        const bool raise = this->tops(x, top);
        if (__any(raise || b < k2))
            new_reference(top, b);
        // A block's values may be smaller than the largest so far by any power of two.  What p takes of it
        // stays where binary32 holds p and the weights' sum, which does not go by the values: times 2^-60 p
        // is 0 as a binary16 number.
        const float apart = __builtin_fmaxf(k2 - b, kApart);
        const float up = apart + kUp;
        const float down = __builtin_amdgcn_exp2f(-apart);
        h16x8 ph[NC], pl[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float ref = (R[c] == -__builtin_inff() ? 0.0f : R[c]) - up;
            float pr[8], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[c][i], fac[c], -ref));
                sum += pr[i];
            }
            l[c] = __builtin_fmaf(sum, down, l[c]);
            split8<F16>(pr, ph[c], pl[c]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const h16x8 o = src.v(j);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if constexpr (F16) {
                    acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, pl[c], acc[c][j], 0, 0, 0);
                    acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(src.v_low(j), ph[c], acc[c][j], 0, 0, 0);
                }
                acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(o, ph[c], acc[c][j], 0, 0, 0);
            }
        }
    }

    __device__ __forceinline__ void new_reference(const float (&top)[NC], float b) {
        b = __builtin_fminf(b, __shfl_xor(b, 16));
        b = __builtin_fminf(b, __shfl_xor(b, 32));
        b = __builtin_fminf(b, k2);
        const float fit = __builtin_amdgcn_exp2f(b - k2);
        k2 = b;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const float by = this->raised(c, top[c]), both = by * fit;
            l[c] *= by;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][j][i] *= both;
        }
    }

    __device__ __forceinline__ void run(char* lds) {
        const AttnI4& a = p.a;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        step_of = NS == 2 ? (wave & 3) >> 1 : 0;
        part_of = NS == 2 ? wave & 1 : wave & 3;
        const Place at(p);
        head = at.head;
        const Seq sq = seq_of(a, at.seq);
        const int rows = sq.n * (int)p.share.d, tile = at.tile * 16 * NC * kRowWaves;
        const int first = tile + wave * 16 * NC;
        if (tile >= rows)
            return;
        table = a.table + (int64_t)at.seq * a.ldt;
        this->range(sq, tile, 16 * NC * kRowWaves, rows, wg_lo, wg_hi);
        this->range(sq, first, 16 * NC, rows, lo, hi);
        int b0, b1;
        split_blocks(wg_lo, wg_hi, at.split, p.by_splits, T / 8, b0, b1);
        Raw x;
        Walk wc, ws;
        if (b0 < b1) {
            start(b0, wc, ws);
            x = load(wc, ws, b0 * 8);
        }
        this->load_q(sq, first, rows);
        k2 = F16 ? 0.0f : (float)kNoSize;
        if (b0 < b1) {
            const int bpp = (int)p.bpp.d;
            unpack(x, lds, b0 * 8);
            if (b0 + T / 8 < b1) {
                wc.step(bpp);
                ws.step(bpp);
                x = load(wc, ws, b0 * 8 + T);
            }
            int turn = 0;
            for (int b = b0; b < b1; b += T / 8, turn ^= 1) {
                __syncthreads();        // this turn's operands are there, the last turn's are used up
                if (b + T / 8 < b1) {
                    unpack(x, lds + (turn ^ 1) * kBuffer, b * 8 + T);
                    if (b + 2 * (T / 8) < b1) {
                        wc.step(bpp);
                        ws.step(bpp);
                        x = load(wc, ws, b * 8 + 2 * T);
                    }
                }
#pragma unroll 1
                for (int sub = 0; sub < NS; ++sub) {
                    const int tok = b * 8 + sub * kStep;
                    if (tok < hi && tok + kStep > lo)
                        step(lds + turn * kBuffer, sub, tok);
                }
            }
        }
        const bool whole = p.splits == 1;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            // 2^30 weights times values of 2^100 stay in range
            const float sum = quarter_sum(l[c]) * 0x1p-24f, ref = R[c] - kUp + 24.0f;
            const int row = first + 16 * c + r;
            if (row >= rows)
                continue;
            const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint16_t* o = this->out_of(sq, row) + 4 * g;
            const int64_t cell = (int64_t)at.split * a.rows * a.heads + this->cell(sq, row);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                f32x4 y = acc[c][j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = __builtin_ldexpf(y[i], (int)-k2 - 24);
                if (whole)
                    put4<F16>(o + 16 * j, y, by);
                else
                    *reinterpret_cast<f32x4*>(p.part + cell * D + 16 * j + 4 * g) = y;
            }
            if (g == 0) {
                if (whole)
                    this->put_lse(sq, row, ref, sum);
                else
                    *reinterpret_cast<f32x2*>(p.ml + 2 * cell) = f32x2{ref, sum};
            }
        }
    }
};

template <int D, int G, bool F16, int NC>
__global__ __launch_bounds__(512, 2) void k_attn_rows(Args p) {
    __shared__ __align__(16) char lds[2 * Rows<D, G, F16, NC>::kBuffer];
    Rows<D, G, F16, NC> k(p);
    k.run(lds);
}

// The partial results of a row joined: a workgroup to a row and head.  16 bytes of a result to a
// lane, so that a workgroup reads kThreads / (D / 4) partial results at a time, each beside its
// reference, and every lane has few to read one after the other (128 of one row: 34 us with a wave
// to a row, 5 so).
template <int D, bool F16>
__global__ __launch_bounds__(kThreads) void k_attn_join(Args p) {
    constexpr int kLane = D / 4, kAt = kThreads / kLane;
    __shared__ __align__(16) float all[kAt * D];
    __shared__ float sums[kAt], refs[kAt];
    const AttnI4& a = p.a;
    const int64_t per = (int64_t)a.max_q * a.heads, at = blockIdx.x;
    const int b = (int)(at / per), cell0 = (int)(at - b * per), qi = cell0 / a.heads, hd = cell0 - qi * a.heads;
    const Seq sq = seq_of(a, b);
    if (qi >= sq.n)
        return;
    const int t = threadIdx.x;
    const int64_t row = sq.row0 + qi, cell = row * a.heads + hd, cells = (int64_t)a.rows * a.heads;
    // the partial results: `count` of them, the first at `from`, then at `next`, `step` apart
    int count = p.splits;
    int64_t from = cell, next = cell + cells, step = cells;
    if (p.dealt) {
        const int heads = a.c.heads, mine = p.found[2 * b], tiles = tiles_of(a, b, p.share);
        const int share = (int)p.share.d, r = qi * share + p.share.mod(hd);     // row of its cache head
        const int first =
            (p.found[2 * b + 1] - mine * tiles) * heads + (r / 16 * heads + p.share.div(hd)) * mine;
        const Deal deal(p.found[2 * kMaxDealt] * heads, p.dealt);
        count = 0;
        if (mine > 0) {
            const int w0 = deal.of(first), w1 = deal.of(first + mine - 1);
            if (w0 == w1)
                return;         // the workgroup has written the result
            count = w1 - w0 + 1;
            from = (int64_t)(2 * w0 + 1) * 16 + r % 16;
            next = (int64_t)(2 * w0 + 2) * 16 + r % 16;
            step = 32;
        }
    }
    const float none = -__builtin_inff();
    float ref = none, sum = 0.0f;
    f32x4 y{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = t / kLane; s < count; s += kAt) {
        const int64_t at_s = s == 0 ? from : next + (s - 1) * step;
        const f32x2 m = *reinterpret_cast<const f32x2*>(p.ml + 2 * at_s);
        const f32x4 x = *reinterpret_cast<const f32x4*>(p.part + at_s * D + 4 * (t % kLane));
        const float top = __builtin_fmaxf(ref, m.x);
        // without a reference a part is 0, or a NaN
        const float old = ref == none ? 0.0f : __builtin_amdgcn_exp2f(ref - top);
        const float w = m.x == none ? 0.0f : __builtin_amdgcn_exp2f(m.x - top);
        ref = top;
        sum = __builtin_fmaf(w, m.y, sum * old);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = __builtin_fmaf(w, x[i], y[i] * old);
    }
    *reinterpret_cast<f32x4*>(all + 4 * t) = y;
    if (t % kLane == 0) {
        sums[t / kLane] = sum;
        refs[t / kLane] = ref;
    }
    __syncthreads();
    if (t < kLane) {
        const float own = ref;
#pragma unroll
        for (int s = 0; s < kAt; ++s)
            ref = __builtin_fmaxf(ref, refs[s]);
        float w = own == none ? 0.0f : __builtin_amdgcn_exp2f(own - ref);
        sum *= w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] *= w;
#pragma unroll
        for (int s = 1; s < kAt; ++s) {
            w = refs[s] == none ? 0.0f : __builtin_amdgcn_exp2f(refs[s] - ref);
            sum = __builtin_fmaf(w, sums[s], sum);
            const f32x4 x = *reinterpret_cast<const f32x4*>(all + 4 * (s * kLane + t));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = __builtin_fmaf(w, x[i], y[i]);
        }
        put4<F16>(a.out + row * a.ldo + (int64_t)hd * a.hso + 4 * t, y, sum == 0.0f ? 0.0f : 1.0f / sum);
        if (a.lse && t == 0)
            a.lse[cell] = lse_of(ref, sum);
    }
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
    const dim3 grid((unsigned)a.groups), block(kThreads);
    hipError_t e;
    if (a.dealt)
        e = launch1(k_attn_tokens<D, G, F16, true>, dim3((unsigned)a.dealt), block, st, a);
    else if (!p.by_rows)
        e = launch1(k_attn_tokens<D, G, F16, false>, grid, block, st, a);
    else if (D == 256 || p.cols == 1)
        e = launch1(k_attn_rows<D, G, F16, 1>, grid, dim3(512), st, a);
    else
        e = launch1(k_attn_rows<D, G, F16, D == 256 ? 1 : 2>, grid, dim3(512), st, a);
    if (e != hipSuccess || (a.splits == 1 && a.dealt == 0))
        return e;
    return launch1(k_attn_join<D, F16>, dim3((unsigned)((int64_t)a.a.seqs * a.a.max_q * a.a.heads)), block,
                   st, a);
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
