// The 4-bit form of cached latents (include/kda_mla_cache.h): 32 channels share
// a scale byte, their codes are 16 bytes.
#pragma once

#include "mla_common.hpp"

namespace kda {
namespace mla {

__host__ __device__ constexpr int mx_row_bytes(int Dc, int Dr, int elem) { return Dc / 2 + Dc / 32 + Dr * elem; }

// A block's scale and its values. (The conversions take a scale's exponent only,
// and make NaN of 255.)
struct MxScale {
    float f;
    __device__ __forceinline__ explicit MxScale(uint32_t s) : f(__uint_as_float(s << 23)) {}
    // 8 codes. A 4-bit value times a power of two is exact in bf16.
    __device__ __forceinline__ bf16x8 bf16(uint32_t c) const {
        const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 0);
        const auto a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 1);
        const auto a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 2);
        const auto a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 3);
        return bf16x8{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
    }
    __device__ __forceinline__ f32x8 f32(uint32_t c) const {
        const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f, 0);
        const auto a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f, 1);
        const auto a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f, 2);
        const auto a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, f, 3);
        return f32x8{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
    }
};

// The two codes of byte I as bf16, with a scale each: the exponents of a and b.
template <int I> __device__ __forceinline__ uint32_t mx_pair(uint32_t c, uint32_t a, uint32_t b) {
    const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, __uint_as_float(a), I));
    const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, __uint_as_float(b), I));
    return (lo & 0xffffu) | (hi & 0xffff0000u);
}

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// bf16 queries as the sum of two e4m3 numbers each, hi 2^(s - 127) + lo 2^(s - 131),
// with an s for each block of 32 channels: s puts the largest into [128, 256), hi
// rounds to 4 significant bits, and what is left of bf16's 8 fits 4 more, down to
// 2^-6: channels from 2^-13 of the largest on. Smaller ones lose at most half of
// lo's smallest step, 2^-14 2^(s - 127), 2^-21 of the largest; s is no less than 9,
// so where the largest is below 2^-111 any may lose 2^-132. A block with a NaN or
// an infinity gets s = 255, NaN.
__device__ __forceinline__ uint32_t query_max(const bf16x8& a, const bf16x8& b) {     // largest magnitude, as bits
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t x = __float_as_uint((float)a[j]) & 0x7fffffffu, y = __float_as_uint((float)b[j]) & 0x7fffffffu;
        m = x > m ? x : m;
        m = y > m ? y : m;
    }
    return m;
}
__device__ __forceinline__ uint32_t query_scale(uint32_t m) {
    const uint32_t s = m >> 23;
    return s == 255 ? 255 : s < 16 ? 9 : s - 7;          // (of tiny blocks lo's scale stays a normal number)
}
// 4 channels
__device__ __forceinline__ void query_split(const bf16x8& q, int at, uint32_t s, int& hi, int& lo) {
    const float f = __uint_as_float((254 - s) << 23);
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = (float)q[at + j] * f;
    int h = 0, l = 0;
    h = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], h, false);
    h = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], h, true);
    const auto b0 = __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
    const auto b1 = __builtin_amdgcn_cvt_pk_f32_fp8(h, true);
    l = __builtin_amdgcn_cvt_pk_fp8_f32((y[0] - b0[0]) * 16.f, (y[1] - b0[1]) * 16.f, l, false);
    l = __builtin_amdgcn_cvt_pk_fp8_f32((y[2] - b1[0]) * 16.f, (y[3] - b1[1]) * 16.f, l, true);
    hi = h;
    lo = l;
}

// Operands of a step of 128 products on 16x16 tiles, codes against e4m3: lane l
// with g = l / 16 holds of the codes the 32 products from 32 g, but of the 8-bit
// numbers the 16 from 16 g and the 16 from 64 + 16 g (measured); its scale bytes are those
// of the products from 32 g in both. So a lane has halves of blocks g / 2 and 2 + g / 2.
struct MxQuery16 {
    i32x8 hi, lo;
    uint32_t s;
    __device__ __forceinline__ void set(const bf16x8 (&q)[4], int lane) {
        auto block = [&](const bf16x8& a, const bf16x8& b) {      // the other half is in the lane 16 on
            const uint32_t m = query_max(a, b);
            const auto p = __builtin_amdgcn_permlane16_swap(m, m, false, false);
            return query_scale(p[0] > p[1] ? p[0] : p[1]);
        };
        const uint32_t s0 = block(q[0], q[1]), s1 = block(q[2], q[3]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int h, l;
            query_split(q[i / 2], 4 * (i % 2), i < 4 ? s0 : s1, h, l);
            hi[i] = h;
            lo[i] = l;
        }
        const int n = lane & 15, g = lane >> 4;
        const uint32_t a = __shfl(s0, n + 32 * (g & 1)), b = __shfl(s1, n + 32 * (g & 1));
        s = g < 2 ? a : b;
    }
};

// Codes of 4 bits (32 a lane) times e4m3 numbers; byte S of sa and sb are the scales.
template <int S> __device__ __forceinline__ f32x4 mma_mx16(const u32x4& a, const i32x8& b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};     // (4-bit operands take four registers)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, b, c, 4, 0, S, (int)sa, S, (int)sb);
}

// The scale byte of a block whose largest magnitude has these float32 bits: e + 127
// for the least e with it <= 7 * 2^e, at most 125.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255;                 // NaN or infinity
    if (amax < (27u << 23)) return 0;                    // below 2^-100
    const uint32_t s = ((amax + 0x1fffffu) >> 23) - 2;   // 1.75 * 2^x and less: x - 2, above: x - 1
    return s < 252 ? s : 252;
}

}  // namespace mla
}  // namespace kda
