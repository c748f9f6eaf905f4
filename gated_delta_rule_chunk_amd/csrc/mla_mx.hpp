// The 4-bit form of cached latents (include/kda_mla_cache.h): 32 channels share
// a scale byte, their codes are 16 bytes.
#pragma once

#include "mla_common.hpp"

namespace kda {
namespace mla {

__host__ __device__ constexpr int mx_row_bytes(int Dc, int Dr, int elem) { return Dc / 2 + Dc / 32 + Dr * elem; }

// A block's scale as float32, and its values. Byte 0 stands for zeros, 255 for NaN.
struct MxScale {
    float f;
    bool none;
    __device__ __forceinline__ explicit MxScale(uint32_t s)
        : f(__uint_as_float(s == 255 ? 0x7fc00000u : s << 23)), none(s == 0) {}
    // 8 codes. (4-bit values times a power of two are exact in bf16.)
    __device__ __forceinline__ bf16x8 bf16(uint32_t c) const {
        const f32x8 v = f32(c);
        bf16x8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (__bf16)v[j];
        return x;
    }
    __device__ __forceinline__ f32x8 f32(uint32_t c) const {
        c = none ? 0u : c;
        f32x8 x;
        const auto a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
        const auto a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1);
        const auto a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2);
        const auto a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3);
        x[0] = a0[0] * f; x[1] = a0[1] * f; x[2] = a1[0] * f; x[3] = a1[1] * f;
        x[4] = a2[0] * f; x[5] = a2[1] * f; x[6] = a3[0] * f; x[7] = a3[1] * f;
        return x;
    }
};

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
