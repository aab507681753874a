// bq_i4.hip -- the I4 codec: 4-bit codes with one scale per group of 32, 64 or 128 columns.
//
// Definition (per group of a row): amax = max |x|; scale = rne(fl32(amax / 7)) in x's type;
// q = round-half-even(fl32(x / scale)) clamped to [-7, 7], 0 where the scale is +0; code =
// q + 8, two codes to a byte.  Back: y = rne((code - zero) * scale).
//
// A group with a NaN has the scale NaN; one with infinities +inf, its infinities q = +-7 and
// everything else q = 0.  So nothing of such a group comes back as an ordinary number.  amax is
// a maximum that keeps a NaN; between lanes it is that of the bit patterns, where infinity and
// then NaN are at the top.
//
// fl32(amax / 7) comes from the fp64 product amax * fl64(1/7): a/7 has the purely periodic
// binary expansion of period 3 unless it is exact, so it stays at least 1/14 ulp away from a
// binary32 rounding midpoint, while the product is within 2^-52.  The quotients are the
// exact fl32(x / s) of bq_device.h (quot32).
//
// Both directions are streams: the quantizer gives a lane 16 values (two 16-byte loads, one
// 8-byte store of codes; a group is 2, 4 or 8 lanes, reduced with DPP), the dequantizer 8
// (one 4-byte load, one 16-byte store).
#include "bq_device.h"
#include "bq_launch.h"

namespace bq {

namespace {

constexpr int kThreads = 256;

struct I4Args {
    const uint16_t* x;
    uint8_t* c;
    uint16_t* s;
    const uint8_t* z;
    uint16_t* y;
    int64_t ldx, ldc, lds, ldz, ldy;
    uint32_t units;      // lane units of the matrix
    uint32_t per_row;    // units in a row
};

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t h) {
    if constexpr (F16)
        return (float)__builtin_bit_cast(_Float16, h);
    else
        return __uint_as_float((uint32_t)h << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float f) {
    if constexpr (F16)
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    else
        return (uint16_t)pack_bf16x2(f, 0.0f);
}

template <bool F16>
__device__ __forceinline__ u32x4 pack8(const float f[8]) {
    if constexpr (F16) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t,
                                      h16x2{(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
        return w;
    } else {
        return pack_bf16x8(f);
    }
}

// IEEE's maximum of three values: one v_maximum3_f32.
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// The largest of the 16 values of one lane without their signs, as binary32 bits; a NaN if there is
// one.  Both forms are trees, since the chain from the loads to the codes is what a wave takes;
// binary16 finds it in the packed patterns, before the conversions.  Measured at 7168 x 43008:
// bf16 129 us, binary16 134, as with fmax, which drops a NaN; as a chain of eight steps 130 and
// 137, binary16 in the form of bf16 140.
template <bool F16>
__device__ __forceinline__ uint32_t abs_max16(u32x4 lo, u32x4 hi, const float f[16]) {
    if constexpr (F16) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = __builtin_bit_cast(u16x2, lo[i] & 0x7FFF7FFFu);
            m[4 + i] = __builtin_bit_cast(u16x2, hi[i] & 0x7FFF7FFFu);
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < d; ++i)
                m[i] = __builtin_elementwise_max(m[i], m[i + d]);
        return __float_as_uint(to_f32<true>(max(m[0].x, m[0].y)));
    } else {
        float m[6];
#pragma unroll
        for (int i = 0; i < 5; ++i)
            m[i] = max3(__builtin_fabsf(f[3 * i]), __builtin_fabsf(f[3 * i + 1]),
                        __builtin_fabsf(f[3 * i + 2]));
        m[5] = __builtin_elementwise_maximum(m[4], __builtin_fabsf(f[15]));
        return __float_as_uint(max3(max3(m[0], m[1], m[2]), m[3], m[5]));
    }
}

// Codes q + 8 of 8 values of one lane, value i in nibble i.
__device__ __forceinline__ uint32_t quant_i4x8(const float f[8], double r) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __builtin_fminf(__builtin_fmaxf(quot32(f[i], r), -7.0f), 7.0f);
        w |= ((rint_low_byte(t) + 8) & 15u) << (4 * i);
    }
    return w;
}

template <int G, bool F16>
__global__ __launch_bounds__(kThreads) void k_quant_i4(I4Args p) {
    // whole groups leave the walk together: a row has a multiple of G/16 units
    for (uint64_t at = blockIdx.x * (uint64_t)kThreads + threadIdx.x; at < p.units;
         at += gridDim.x * (uint64_t)kThreads) {
        const uint32_t u = (uint32_t)at;
        const uint32_t row = u / p.per_row, col = (u - row * p.per_row) * 16;
        const uint16_t* x = p.x + (int64_t)row * p.ldx + col;
        const u32x4 lo = ld16(x), hi = ld16(x + 8);
        float f[16];
        if constexpr (F16) {
            unpack_f16x8(lo, f);
            unpack_f16x8(hi, f + 8);
        } else {
            unpack_bf16x8(lo, f);
            unpack_bf16x8(hi, f + 8);
        }
        uint32_t b = abs_max16<F16>(lo, hi, f);
        if constexpr (G == 32)
            b = pair_max2(b);
        else if constexpr (G == 64)
            b = quad_max4(b);
        else
            b = half_row_max8(b);
        const uint16_t sh = from_f32<F16>((float)((double)__uint_as_float(b) * (1.0 / 7.0)));
        const float s = to_f32<F16>(sh);
        u32x2 w{0x88888888u, 0x88888888u};
        if (s > 0.0f) {     // neither 0 nor NaN
            // under an infinite scale the quotient of an infinity is clamped, any other rounds to 0
            const double r = recip64(__builtin_fmin((double)s, 0x1p200));
            w = u32x2{quant_i4x8(f, r), quant_i4x8(f + 8, r)};
        }
        st8(p.c + (int64_t)row * p.ldc + col / 2, w);
        if (col % G == 0)
            p.s[(int64_t)row * p.lds + col / G] = sh;
    }
}

template <int G, bool F16, bool Z>
__global__ __launch_bounds__(kThreads) void k_dequant_i4(I4Args p) {
    for (uint64_t at = blockIdx.x * (uint64_t)kThreads + threadIdx.x; at < p.units;
         at += gridDim.x * (uint64_t)kThreads) {
        const uint32_t u = (uint32_t)at;
        const uint32_t row = u / p.per_row, col = (u - row * p.per_row) * 8;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p.c + (int64_t)row * p.ldc + col / 2);
        const float s = to_f32<F16>(p.s[(int64_t)row * p.lds + col / G]);
        int z = 8;
        if constexpr (Z)
            z = p.z[(int64_t)row * p.ldz + col / G] & 15;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = (float)((int)((w >> (4 * i)) & 15u) - z) * s;
        st16(p.y + (int64_t)row * p.ldy + col, pack8<F16>(f));
    }
}

// A launch holds less than 2^32 threads: beyond 2^22 workgroups they walk on.
dim3 grid_of(uint32_t units) {
    const uint64_t want = ((uint64_t)units + kThreads - 1) / kThreads, cap = 1 << 22;
    return dim3((unsigned)(want < cap ? want : cap));
}

template <int G>
hipError_t quant(const I4Args& a, bool f16, hipStream_t st) {
    return f16 ? launch1(k_quant_i4<G, true>, grid_of(a.units), dim3(kThreads), st, a)
               : launch1(k_quant_i4<G, false>, grid_of(a.units), dim3(kThreads), st, a);
}

template <int G, bool F16>
hipError_t dequant(const I4Args& a, hipStream_t st) {
    return a.z ? launch1(k_dequant_i4<G, F16, true>, grid_of(a.units), dim3(kThreads), st, a)
               : launch1(k_dequant_i4<G, F16, false>, grid_of(a.units), dim3(kThreads), st, a);
}

}  // namespace

hipError_t launch_quant_i4(const uint16_t* x, int64_t rows, int64_t cols, int64_t ldx, int group,
                           uint8_t* c, int64_t ldc, uint16_t* scale, int64_t lds, bool f16,
                           hipStream_t stream) {
    I4Args a{};
    a.x = x;
    a.c = c;
    a.s = scale;
    a.ldx = ldx;
    a.ldc = ldc;
    a.lds = lds;
    a.per_row = (uint32_t)(cols / 16);
    a.units = (uint32_t)(rows * (cols / 16));
    return group == 32 ? quant<32>(a, f16, stream)
         : group == 64 ? quant<64>(a, f16, stream)
                       : quant<128>(a, f16, stream);
}

hipError_t launch_dequant_i4(const uint8_t* c, int64_t ldc, const uint16_t* scale, int64_t lds,
                             const uint8_t* zero, int64_t ldz, int64_t rows, int64_t cols,
                             int group, uint16_t* y, int64_t ldy, bool f16, hipStream_t stream) {
    I4Args a{};
    a.c = const_cast<uint8_t*>(c);
    a.s = const_cast<uint16_t*>(scale);
    a.z = zero;
    a.y = y;
    a.ldc = ldc;
    a.lds = lds;
    a.ldz = ldz;
    a.ldy = ldy;
    a.per_row = (uint32_t)(cols / 8);
    a.units = (uint32_t)(rows * (cols / 8));
    if (f16)
        return group == 32 ? dequant<32, true>(a, stream)
             : group == 64 ? dequant<64, true>(a, stream)
                           : dequant<128, true>(a, stream);
    return group == 32 ? dequant<32, false>(a, stream)
         : group == 64 ? dequant<64, false>(a, stream)
                       : dequant<128, false>(a, stream);
}

}  // namespace bq
