// bq_kv.hip -- rows of keys and values into the 4-bit cache and back.
//
// Definition (per group of a token's row of one head): lo, hi the least and largest number;
// scale = rne16(fl32((hi - lo) / 15)); code = round-half-even(fl32((x - lo) / scale)) clamped to
// [0, 15], 0 where the scale is 0.  Back: rne16(fl32(code * scale + lo)).  lo is one of the
// 16-bit inputs, so it is held exactly.  Differences are taken in binary64, where the range of
// two bf16 numbers does not overflow, and rounded to binary32 once, as a quotient.
//
// Both directions are streams.  Eight lanes own a token's row of one head and a wave 8
// consecutive tokens, which in a prefill are one block of v's layout: its words come out whole.
// Keys: a lane has dim/8 numbers that follow each other.  Values: a lane has the numbers
// 16j + 2u and 16j + 2u + 1 of every j, so that it owns whole half-words of the block's words.
#include <type_traits>

#include "bq_device.h"
#include "bq_launch.h"

namespace bq {

namespace {

constexpr int kThreads = 256;

struct KvArgs {
    KvRows r;
    bq_kv_i4 c;
    uint32_t slots;        // pages * page_size
    int64_t units;         // rows of one token and head, tokens in whole eights
};

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

// IEEE minimum and maximum (a NaN stays) over L of the 8 lanes of a row.
template <int L>
__device__ __forceinline__ void lanes_min_max(float& lo, float& hi) {
    auto step = [&](auto ctrl) {
        constexpr int c = decltype(ctrl)::value;
        lo = __builtin_elementwise_minimum(lo, __uint_as_float(dpp<c>(__float_as_uint(lo))));
        hi = __builtin_elementwise_maximum(hi, __uint_as_float(dpp<c>(__float_as_uint(hi))));
    };
    if constexpr (L >= 2)
        step(std::integral_constant<int, 0xB1>{});      // quad_perm [1,0,3,2]
    if constexpr (L >= 4)
        step(std::integral_constant<int, 0x4E>{});      // quad_perm [2,3,0,1]
    if constexpr (L >= 8)
        step(std::integral_constant<int, 0x141>{});     // row_half_mirror
}

struct Group {
    double lo, r;          // least value, reciprocal of the scale
    uint32_t pair;         // scale and least as they are kept
    bool live;             // codes other than 0
};

template <bool F16>
__device__ __forceinline__ Group group_of(float lo, float hi) {
    Group g;
    g.lo = lo;
    const float s = (float)(((double)hi - (double)lo) / 15.0);
    uint32_t w = pack2<F16>(s, lo);
    const bool fine = __builtin_fabsf(lo) < __builtin_inff() && __builtin_fabsf(hi) < __builtin_inff();
    if (!fine)
        w = 0x7FFF7FFFu;    // two NaN in either type
    g.pair = w;
    const float held = lo16<F16>(w);
    g.live = held > 0.0f;
    g.r = recip64(g.live ? held : 1.0f);
    return g;
}

// The code of x, in the low bits.
__device__ __forceinline__ uint32_t code_of(float x, const Group& g) {
    const float t = (float)(((double)x - g.lo) * g.r);
    return rint_low_byte(__builtin_fminf(__builtin_fmaxf(t, 0.0f), 15.0f)) & 15u;
}

// The lane's row: token, head, and its place in the cache.
struct Row {
    int64_t token, code, scale;    // code bytes, scale entries
    uint32_t head, place;
    bool in;
};
template <int D>
__device__ __forceinline__ Row row_of(const KvArgs& p, int64_t unit) {
    Row r;
    // units: 8 tokens of a head, then the next head, then the next 8 tokens
    const uint32_t heads = (uint32_t)p.c.heads;
    const int64_t eight = unit >> 3;
    r.token = eight / heads * 8 + (unit & 7);
    r.head = (uint32_t)(eight % heads);
    r.in = false;
    r.place = 0;
    r.code = r.scale = 0;
    if (r.token < p.r.tokens) {
        const uint32_t slot = (uint32_t)p.r.slot[r.token];      // negative: out of range too
        if (slot < p.slots) {
            const uint32_t page = slot / (uint32_t)p.c.page_size;
            r.place = slot - page * (uint32_t)p.c.page_size;
            r.code = (int64_t)page * p.c.page_stride + (int64_t)r.head * p.c.head_stride;
            r.scale = (int64_t)page * p.c.spage_stride + (int64_t)r.head * p.c.shead_stride;
            r.in = true;
        }
    }
    return r;
}

// Byte of half-word hw of number-row r of v in the block of place.
template <int D>
__device__ __forceinline__ uint32_t v_half(uint32_t place, uint32_t r, uint32_t hw) {
    return (place >> 3) * (4 * D) + ((r * 4 + ((place & 7) >> 1)) * (D / 64) + hw) * 4 +
           (place & 1) * 2;
}

template <int D, int G, bool F16>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvArgs p) {
    constexpr int NW = D / 64;          // words of k to a lane
    constexpr int NJ = D / 16;          // pairs of v to a lane
    constexpr int NG = D / G;
    const uint32_t u = threadIdx.x & 7;
    for (int64_t unit = (blockIdx.x * (int64_t)kThreads + threadIdx.x) >> 3; unit < p.units;
         unit += (gridDim.x * (int64_t)kThreads) >> 3) {
        const Row r = row_of<D>(p, unit);
        if (!r.in)      // the 8 lanes of a row leave together
            continue;
        const uint16_t* k = p.r.k + r.token * p.r.ldk + r.head * p.r.hsk + u * (D / 8);
        const uint16_t* v = p.r.v + r.token * p.r.ldv + r.head * p.r.hsv + u * 2;
        u32x4 kw[NW];
        uint32_t vw[NJ];
#pragma unroll
        for (int i = 0; i < NW; ++i)
            kw[i] = ld16(k + 8 * i);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            vw[j] = *reinterpret_cast<const uint32_t*>(v + 16 * j);
        {
            float f[8 * NW];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                if constexpr (F16)
                    unpack_f16x8(kw[i], f + 8 * i);
                else
                    unpack_bf16x8(kw[i], f + 8 * i);
            }
            float lo = f[0], hi = f[0];
#pragma unroll
            for (int i = 1; i < 8 * NW; ++i) {
                lo = __builtin_elementwise_minimum(lo, f[i]);
                hi = __builtin_elementwise_maximum(hi, f[i]);
            }
            constexpr int L = G / (D / 8);      // lanes of a group
            lanes_min_max<L>(lo, hi);
            const Group g = group_of<F16>(lo, hi);
            uint8_t* c = p.c.k + r.code + (int64_t)r.place * (D / 2);
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                uint32_t w = 0;
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    w |= code_of(f[8 * i + n], g) << (4 * n);
                if (!g.live)
                    w = 0;
                const uint32_t at = u * NW + i;     // numbers 8 at .. 8 at + 7
                *reinterpret_cast<uint32_t*>(c + ((at & 3) * (D / 32) + (at >> 2)) * 4) = w;
            }
            if (u % L == 0)
                *reinterpret_cast<uint32_t*>(p.c.ks + r.scale +
                                             2 * ((int64_t)(u / L) * p.c.page_size + r.place)) =
                    g.pair;
        }
        uint32_t half[2][D / 64] = {};
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            constexpr int PJ = G / 16;          // pairs of a group
            float lo = lo16<F16>(vw[gi * PJ]), hi = lo;
#pragma unroll
            for (int j = gi * PJ; j < (gi + 1) * PJ; ++j) {
                const float a = lo16<F16>(vw[j]), b = hi16<F16>(vw[j]);
                lo = __builtin_elementwise_minimum(lo, __builtin_elementwise_minimum(a, b));
                hi = __builtin_elementwise_maximum(hi, __builtin_elementwise_maximum(a, b));
            }
            lanes_min_max<8>(lo, hi);
            const Group g = group_of<F16>(lo, hi);
#pragma unroll
            for (int j = gi * PJ; j < (gi + 1) * PJ; ++j) {
                const uint32_t a = code_of(lo16<F16>(vw[j]), g), b = code_of(hi16<F16>(vw[j]), g);
                half[0][j / 4] |= (g.live ? a : 0) << (4 * (j % 4));
                half[1][j / 4] |= (g.live ? b : 0) << (4 * (j % 4));
            }
            if (u == (uint32_t)gi)
                *reinterpret_cast<uint32_t*>(p.c.vs + r.scale +
                                             2 * ((int64_t)gi * p.c.page_size + r.place)) = g.pair;
        }
        uint8_t* c = p.c.v + r.code;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hw = 0; hw < D / 64; ++hw)
                *reinterpret_cast<uint16_t*>(c + v_half<D>(r.place, 2 * u + b, hw)) =
                    (uint16_t)half[b][hw];
    }
}

template <int D, int G, bool F16>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvArgs p) {
    constexpr int NW = D / 64, NJ = D / 16;
    const uint32_t u = threadIdx.x & 7;
    for (int64_t unit = (blockIdx.x * (int64_t)kThreads + threadIdx.x) >> 3; unit < p.units;
         unit += (gridDim.x * (int64_t)kThreads) >> 3) {
        const Row r = row_of<D>(p, unit);
        if (r.token >= p.r.tokens)
            continue;
        uint16_t* ko = p.r.ko + r.token * p.r.ldk + r.head * p.r.hsk + u * (D / 8);
        uint16_t* vo = p.r.vo + r.token * p.r.ldv + r.head * p.r.hsv + u * 2;
        if (!r.in) {
#pragma unroll
            for (int i = 0; i < NW; ++i)
                *reinterpret_cast<u32x4*>(ko + 8 * i) = u32x4{};
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<uint32_t*>(vo + 16 * j) = 0;
            continue;
        }
        const uint8_t* ck = p.c.k + r.code + (int64_t)r.place * (D / 2);
        const uint8_t* cv = p.c.v + r.code;
        const uint32_t* ks = reinterpret_cast<const uint32_t*>(p.c.ks + r.scale) + r.place;
        const uint32_t* vs = reinterpret_cast<const uint32_t*>(p.c.vs + r.scale) + r.place;
        constexpr int L = G / (D / 8);
        const uint32_t kp = ks[(int64_t)(u / L) * p.c.page_size];
        uint32_t kw[NW], vp[D / G], half[2][D / 64];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const uint32_t at = u * NW + i;
            kw[i] = *reinterpret_cast<const uint32_t*>(ck + ((at & 3) * (D / 32) + (at >> 2)) * 4);
        }
#pragma unroll
        for (int g = 0; g < D / G; ++g)
            vp[g] = vs[(int64_t)g * p.c.page_size];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hw = 0; hw < D / 64; ++hw)
                half[b][hw] = *reinterpret_cast<const uint16_t*>(cv + v_half<D>(r.place, 2 * u + b, hw));
        const float s = lo16<F16>(kp), m = hi16<F16>(kp);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            u32x4 w;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t c = kw[i] >> (8 * n);
                w[n] = pack2<F16>(__builtin_fmaf((float)(c & 15u), s, m),
                                  __builtin_fmaf((float)((c >> 4) & 15u), s, m));
            }
            *reinterpret_cast<u32x4*>(ko + 8 * i) = w;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float sv = lo16<F16>(vp[16 * j / G]), mv = hi16<F16>(vp[16 * j / G]);
            const float a = (float)((half[0][j / 4] >> (4 * (j % 4))) & 15u);
            const float b = (float)((half[1][j / 4] >> (4 * (j % 4))) & 15u);
            *reinterpret_cast<uint32_t*>(vo + 16 * j) =
                pack2<F16>(__builtin_fmaf(a, sv, mv), __builtin_fmaf(b, sv, mv));
        }
    }
}

KvArgs args_of(const KvRows& r, const bq_kv_i4& c) {
    return KvArgs{r, c, (uint32_t)c.pages * (uint32_t)c.page_size, (r.tokens + 7) / 8 * 8 * c.heads};
}

dim3 grid_of(int64_t units) {
    const int64_t want = (units + kThreads / 8 - 1) / (kThreads / 8), cap = 1 << 22;
    return dim3((unsigned)(want < cap ? want : cap));
}

template <bool W, int D, int G>
hipError_t go(const KvArgs& a, bool f16, hipStream_t st) {
    const dim3 grid = grid_of(a.units), block(kThreads);
    if constexpr (W)
        return f16 ? launch1(k_kv_write<D, G, true>, grid, block, st, a)
                   : launch1(k_kv_write<D, G, false>, grid, block, st, a);
    else
        return f16 ? launch1(k_kv_read<D, G, true>, grid, block, st, a)
                   : launch1(k_kv_read<D, G, false>, grid, block, st, a);
}

template <bool W>
hipError_t pick(const KvArgs& a, bool f16, hipStream_t st) {
    const int g = a.c.group;
    if (a.c.dim == 64)
        return g == 32 ? go<W, 64, 32>(a, f16, st) : go<W, 64, 64>(a, f16, st);
    if (a.c.dim == 128)
        return g == 32   ? go<W, 128, 32>(a, f16, st)
               : g == 64 ? go<W, 128, 64>(a, f16, st)
                         : go<W, 128, 128>(a, f16, st);
    return g == 32   ? go<W, 256, 32>(a, f16, st)
           : g == 64 ? go<W, 256, 64>(a, f16, st)
                     : go<W, 256, 128>(a, f16, st);
}

}  // namespace

hipError_t launch_kv_write(const KvRows& r, const bq_kv_i4& c, bool f16, hipStream_t stream) {
    return pick<true>(args_of(r, c), f16, stream);
}
hipError_t launch_kv_read(const KvRows& r, const bq_kv_i4& c, bool f16, hipStream_t stream) {
    return pick<false>(args_of(r, c), f16, stream);
}

}  // namespace bq
