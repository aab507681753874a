// bq_kv.hip -- rows of keys and values into the 4-bit cache and back.
//
// Definition (per group of a token's row of one head): lo, hi the least and largest number;
// scale = rne16(fl32((hi - lo) / 15)); code = round-half-even(fl32((x - lo) / scale)) clamped to
// [0, 15], 0 where the scale is 0.  Back: rne16(fl32(code * scale + lo)).  lo is one of the
// 16-bit inputs, so it is held exactly.  Differences are taken in binary64, where the range of
// two bf16 numbers does not overflow, and rounded to binary32 once, as a quotient.
//
// Both directions are streams.  Eight lanes own a token's row of one head and a wave 8
// consecutive tokens, which in a prefill are one block of v's layout or two.  Rows go in and out in
// runs of 128 bytes, 16 to a lane.  Keys: a lane has whole words of 8 numbers.  Values: a lane has
// the numbers 16j + 2u and 16j + 2u + 1 of every j, so that it owns whole half-words of the
// block's words; two tokens that share them put theirs together.
//
// Measured, 8 heads of 128 numbers: 16379 bf16 tokens in groups of 32 (86.5 MB) 26.6 us to write, 3.3
// TB/s, and 19.0 to read, 4.6 TB/s; 65536 binary16 tokens in groups of 128 (340 MB) 59 us to read, 5.8 TB/s,
// part of it from the last-level cache.  Bytes bound both; 32 tokens take 4.1 and 3.4 us, a launch.
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
    // the product is within 2^-52 of the quotient, which is periodic (1/15: period 4) and so at least
    // 1/30 of a step away from what binary32 rounds the other way, or exact
    const float s = (float)(((double)hi - (double)lo) * (1.0 / 15.0));
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

// A row of values between the lanes' two views of it, through LDS: 16-byte chunks u and u + 8, .. as
// they lie in memory, and pairs 16j + 2u, 16j + 2u + 1 as the cache's words want them.  Rows are
// 16 bytes * 2 apart from a multiple of the 64 banks, so that neither view meets a conflict.
template <int D>
struct Turn {
    static constexpr int kRow = 2 * D + 32;                 // bytes
    static constexpr int kBytes = kThreads / 8 * kRow;
    char* row;
    uint32_t u;
    __device__ __forceinline__ explicit Turn(char* lds)
        : row(lds + (threadIdx.x >> 3) * kRow), u(threadIdx.x & 7) {}
    __device__ __forceinline__ u32x4* chunk(int i) const {
        return reinterpret_cast<u32x4*>(row + 16 * (u + 8 * i));
    }
    __device__ __forceinline__ uint32_t* pair(int j) const {
        return reinterpret_cast<uint32_t*>(row + 4 * (u + 8 * j));
    }
    // The lanes of a row are of one wave: what they wrote is there once its LDS accesses are done.
    static __device__ __forceinline__ void done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
};

template <int D, int G, bool F16>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvArgs p) {
    constexpr int NW = D / 64;          // words of k to a lane: numbers 64i + 8u ..
    constexpr int NG = D / G;
    constexpr int HW = D / 64;          // half-words of v to a number-row
    __shared__ __align__(16) char lds[Turn<D>::kBytes];
    const Turn<D> turn(lds);
    const uint32_t u = threadIdx.x & 7;
    for (int64_t unit = (blockIdx.x * (int64_t)kThreads + threadIdx.x) >> 3; unit < p.units;
         unit += (gridDim.x * (int64_t)kThreads) >> 3) {
        const Row r = row_of<D>(p, unit);
        // the token beside this one, whose half of each word of v its lanes have: 8 lanes on
        const uint32_t key = r.in ? (uint32_t)p.r.slot[r.token] : ~0u;
        const bool paired = dpp<0x128>(key) == (key ^ 1u) && r.in;      // row_ror:8
        if (!r.in)      // the 8 lanes of a row leave together
            continue;
        const uint16_t* k = p.r.k + r.token * p.r.ldk + r.head * p.r.hsk + u * 8;
        const uint16_t* v = p.r.v + r.token * p.r.ldv + r.head * p.r.hsv + u * 8;
        u32x4 kw[NW], vc[NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            kw[i] = ld16(k + 64 * i);
            vc[i] = ld16(v + 64 * i);
        }
#pragma unroll
        for (int i = 0; i < NW; ++i)
            *turn.chunk(i) = vc[i];
        uint8_t* c = p.c.k + r.code + (int64_t)r.place * (D / 2);
        constexpr int PW = G >= 64 ? G / 64 : 1;        // words of a lane that share a group
#pragma unroll
        for (int i0 = 0; i0 < NW; i0 += PW) {
            float f[8 * PW];
#pragma unroll
            for (int i = 0; i < PW; ++i) {
                if constexpr (F16)
                    unpack_f16x8(kw[i0 + i], f + 8 * i);
                else
                    unpack_bf16x8(kw[i0 + i], f + 8 * i);
            }
            float lo = f[0], hi = f[0];
#pragma unroll
            for (int i = 1; i < 8 * PW; ++i) {
                lo = __builtin_elementwise_minimum(lo, f[i]);
                hi = __builtin_elementwise_maximum(hi, f[i]);
            }
            constexpr int L = G >= 64 ? 8 : 4;          // lanes of a group
            lanes_min_max<L>(lo, hi);
            const Group g = group_of<F16>(lo, hi);
#pragma unroll
            for (int i = 0; i < PW; ++i) {
                uint32_t w = 0;
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    w |= code_of(f[8 * i + n], g) << (4 * n);
                if (!g.live)
                    w = 0;
                const uint32_t at = 8 * (i0 + i) + u;   // numbers 8 at .. 8 at + 7
                *reinterpret_cast<uint32_t*>(c + ((at & 3) * (D / 32) + (at >> 2)) * 4) = w;
            }
            if (u % L == 0)
                *reinterpret_cast<uint32_t*>(
                    p.c.ks + r.scale +
                    2 * ((int64_t)((64 * i0 + 8 * u) / G) * p.c.page_size + r.place)) = g.pair;
        }
        Turn<D>::done();
        uint32_t half[2][HW] = {};
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            constexpr int PJ = G / 16;          // pairs of a group
            uint32_t vw[PJ];
#pragma unroll
            for (int j = 0; j < PJ; ++j)
                vw[j] = *turn.pair(gi * PJ + j);
            float lo = lo16<F16>(vw[0]), hi = lo;
#pragma unroll
            for (int j = 0; j < PJ; ++j) {
                const float a = lo16<F16>(vw[j]), b = hi16<F16>(vw[j]);
                lo = __builtin_elementwise_minimum(lo, __builtin_elementwise_minimum(a, b));
                hi = __builtin_elementwise_maximum(hi, __builtin_elementwise_maximum(a, b));
            }
            lanes_min_max<8>(lo, hi);
            const Group g = group_of<F16>(lo, hi);
#pragma unroll
            for (int i = 0; i < PJ; ++i) {
                const int j = gi * PJ + i;
                const uint32_t a = code_of(lo16<F16>(vw[i]), g), b = code_of(hi16<F16>(vw[i]), g);
                half[0][j / 4] |= (g.live ? a : 0) << (4 * (j % 4));
                half[1][j / 4] |= (g.live ? b : 0) << (4 * (j % 4));
            }
            if (u == (uint32_t)gi)
                *reinterpret_cast<uint32_t*>(p.c.vs + r.scale +
                                             2 * ((int64_t)gi * p.c.page_size + r.place)) = g.pair;
        }
        uint8_t* cv = p.c.v + r.code;
        if (paired) {
            // the even token writes both tokens' words of number-row 2u, the odd one those of 2u + 1
            const uint32_t odd = r.place & 1;
#pragma unroll
            for (int hw = 0; hw < HW; ++hw) {
                const uint32_t other = dpp<0x128>(odd ? half[0][hw] : half[1][hw]);
                const uint32_t w = odd ? other | half[1][hw] << 16 : half[0][hw] | other << 16;
                *reinterpret_cast<uint32_t*>(cv + v_half<D>(r.place & ~1u, 2 * u + odd, hw)) = w;
            }
        } else {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int hw = 0; hw < HW; ++hw)
                    *reinterpret_cast<uint16_t*>(cv + v_half<D>(r.place, 2 * u + b, hw)) =
                        (uint16_t)half[b][hw];
        }
        Turn<D>::done();
    }
}

template <int D, int G, bool F16>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvArgs p) {
    constexpr int NW = D / 64, NJ = D / 16, HW = D / 64;
    __shared__ __align__(16) char lds[Turn<D>::kBytes];
    const Turn<D> turn(lds);
    const uint32_t u = threadIdx.x & 7;
    for (int64_t unit = (blockIdx.x * (int64_t)kThreads + threadIdx.x) >> 3; unit < p.units;
         unit += (gridDim.x * (int64_t)kThreads) >> 3) {
        const Row r = row_of<D>(p, unit);
        if (r.token >= p.r.tokens)
            continue;
        uint16_t* ko = p.r.ko + r.token * p.r.ldk + r.head * p.r.hsk + u * 8;
        uint16_t* vo = p.r.vo + r.token * p.r.ldv + r.head * p.r.hsv + u * 8;
        if (!r.in) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                st16(ko + 64 * i, u32x4{});
                st16(vo + 64 * i, u32x4{});
            }
            continue;
        }
        const uint8_t* ck = p.c.k + r.code + (int64_t)r.place * (D / 2);
        const uint8_t* cv = p.c.v + r.code;
        const uint32_t* ks = reinterpret_cast<const uint32_t*>(p.c.ks + r.scale) + r.place;
        const uint32_t* vs = reinterpret_cast<const uint32_t*>(p.c.vs + r.scale) + r.place;
        uint32_t kw[NW], kp[NW], vp[D / G], half[2][HW];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const uint32_t at = 8 * i + u;      // numbers 8 at .. 8 at + 7
            kw[i] = *reinterpret_cast<const uint32_t*>(ck + ((at & 3) * (D / 32) + (at >> 2)) * 4);
            kp[i] = ks[(int64_t)(8 * at / G) * p.c.page_size];
        }
#pragma unroll
        for (int g = 0; g < D / G; ++g)
            vp[g] = vs[(int64_t)g * p.c.page_size];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int hw = 0; hw < HW; ++hw)
                half[b][hw] = *reinterpret_cast<const uint16_t*>(cv + v_half<D>(r.place, 2 * u + b, hw));
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float sv = lo16<F16>(vp[16 * j / G]), mv = hi16<F16>(vp[16 * j / G]);
            const float a = (float)((half[0][j / 4] >> (4 * (j % 4))) & 15u);
            const float b = (float)((half[1][j / 4] >> (4 * (j % 4))) & 15u);
            *turn.pair(j) = pack2<F16>(__builtin_fmaf(a, sv, mv), __builtin_fmaf(b, sv, mv));
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float s = lo16<F16>(kp[i]), m = hi16<F16>(kp[i]);
            u32x4 w;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t c = kw[i] >> (8 * n);
                w[n] = pack2<F16>(__builtin_fmaf((float)(c & 15u), s, m),
                                  __builtin_fmaf((float)((c >> 4) & 15u), s, m));
            }
            st16(ko + 64 * i, w);
        }
        Turn<D>::done();
#pragma unroll
        for (int i = 0; i < NW; ++i)
            st16(vo + 64 * i, *turn.chunk(i));
        Turn<D>::done();
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
