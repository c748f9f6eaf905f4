// Rows to and from a cache that holds the latents in 4 bits (layout:
// include/kda_mla_cache.h).
#include "launchers.hpp"
#include "mla_mx.hpp"

namespace kda {
namespace {

using namespace mla;

// Offsets in a page of row r's codes, scale bytes and shared part.
struct Row {
    int64_t codes, scales, rope;
};
__device__ __forceinline__ Row row_at(int Dc, int Dr, int elem, int ps, int r) {
    return {(int64_t)r * (Dc / 2), (((int64_t)Dc / 2) << ps) + (int64_t)r * (Dc / 32),
            (((int64_t)Dc / 2 + Dc / 32) << ps) + (int64_t)r * (Dr * elem)};
}
// the last sequence that starts at or before row i of a packed tensor; its own rows only
__device__ __forceinline__ bool sequence_of(const int32_t* cu, int N, int64_t i, int& n, int64_t& t) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i) lo = mid; else hi = mid;
    }
    n = lo;
    t = i - cu[lo];
    return t >= 0 && i < cu[lo + 1];
}
template <class T> __device__ __forceinline__ f32x8 load8f(const T* p) {
    if constexpr (sizeof(T) == 2) {
        float f[8];
        unpack8(*reinterpret_cast<const uint4*>(p), f);
        return f32x8{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
    } else {
        return load8(p);
    }
}

// A thread for 8 channels of a new row, four for a block of 32; threads behind
// them for 16 bytes of the shared part each.
template <class T, int DC, int DR> __global__ __launch_bounds__(256) void mla_append_mx_kernel(MlaAppendArgs a, int64_t units) {
    constexpr int U = DC / 8 + DR / kChunk<T>;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= units) return;
    const int64_t i = x / U;
    const int u = (int)(x % U);
    int n, b = 0;
    int64_t t;
    if (a.cu) {
        if (!sequence_of(a.cu, a.N, i, n, t)) return;
    } else {
        n = b = (int)(i / a.T);
        t = i % a.T;
    }
    const int have = a.lens[n];
    if (have < 0) return;                                        // padding row
    const int64_t pos = (int64_t)have + t, pg = pos >> a.page_shift;
    int e = -1;
    if (pg < a.max_pages) e = a.table[(int64_t)n * a.max_pages + pg];
    if (e < 0 || e >= a.n_pages) {
        if (u == 0) atomicAdd(a.status, 1u);
        return;
    }
    char* page = static_cast<char*>(a.cache) + e * ((int64_t)mx_row_bytes(DC, DR, sizeof(T)) << a.page_shift);
    const Row at = row_at(DC, DR, sizeof(T), a.page_shift, (int)(pos & ((1 << a.page_shift) - 1)));
    const int64_t row = a.cu ? i : t;
    if (u >= DC / 8) {
        const int c = (u - DC / 8) * kChunk<T>;
        *reinterpret_cast<u32x4*>(page + at.rope + c * sizeof(T)) =
            *reinterpret_cast<const u32x4*>(static_cast<const T*>(a.kr) + b * a.kr_batch + row * a.kr_row + c);
        return;
    }
    const f32x8 v = load8f(static_cast<const T*>(a.latent) + b * a.lat_batch + row * a.lat_row + 8 * u);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t y = __float_as_uint(v[j]) & 0x7fffffffu;
        m = y > m ? y : m;
    }
    // the block's four threads are neighbours in a wave and all here
    uint32_t o = __shfl_xor(m, 1);
    m = o > m ? o : m;
    o = __shfl_xor(m, 2);
    m = o > m ? o : m;
    const uint32_t s = mx_scale_byte(m);
    uint32_t c = 0;
    if (s != 0 && s != 255) {
        // rounds to the nearest, ties to even, and past 6 to 6
        const float f = __uint_as_float(s << 23);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], f, 3);
    }
    *reinterpret_cast<uint32_t*>(page + at.codes + 4 * u) = c;
    if ((u & 3) == 0) *reinterpret_cast<uint8_t*>(page + at.scales + (u >> 2)) = (uint8_t)s;
}

template <class T, int DC, int DR> __global__ __launch_bounds__(256) void mla_read_mx_kernel(MlaReadArgs a, int64_t units) {
    constexpr int U = DC / 8 + DR / kChunk<T>;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= units) return;
    const int64_t i = x / U;
    const int u = (int)(x % U);
    int n;
    int64_t t;
    const bool mine = sequence_of(a.cu, a.N, i, n, t);
    if (!mine && !a.zero_rest) return;
    int e = -1;
    int64_t pos = 0;
    if (mine) {
        pos = (a.starts ? (int64_t)a.starts[n] : 0) + t;
        const int64_t pg = pos >> a.page_shift;
        if (pos >= 0 && pg < a.max_pages) e = a.table[(int64_t)n * a.max_pages + pg];
        if (e >= a.n_pages) e = -1;
        if (e < 0 && u == 0) atomicAdd(a.status, 1u);
    }
    const char* page = static_cast<const char*>(a.cache) + e * ((int64_t)mx_row_bytes(DC, DR, sizeof(T)) << a.page_shift);
    const Row at = row_at(DC, DR, sizeof(T), a.page_shift, (int)(pos & ((1 << a.page_shift) - 1)));
    if (u >= DC / 8) {
        const int c = (u - DC / 8) * kChunk<T>;
        u32x4 v = {0, 0, 0, 0};
        if (e >= 0) v = *reinterpret_cast<const u32x4*>(page + at.rope + c * sizeof(T));
        *reinterpret_cast<u32x4*>(static_cast<T*>(a.rope) + i * DR + c) = v;
        return;
    }
    uint32_t c = 0, s = 0;
    if (e >= 0) {
        c = *reinterpret_cast<const uint32_t*>(page + at.codes + 4 * u);
        s = *reinterpret_cast<const uint8_t*>(page + at.scales + (u >> 2));
    }
    const MxScale f(s);
    T* to = static_cast<T*>(a.latent) + i * DC + 8 * u;
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<bf16x8*>(to) = f.bf16(c);
    } else {
        const f32x8 v = f.f32(c);
        *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
}

template <class T, int DC, int DR> hipError_t append(const MlaAppendArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.B * a.T * (DC / 8 + DR / kChunk<T>);
    mla_append_mx_kernel<T, DC, DR><<<dim3((unsigned)((units + 255) / 256)), 256, 0, s>>>(a, units);
    return hipGetLastError();
}
template <class T, int DC, int DR> hipError_t read(const MlaReadArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.T * (DC / 8 + DR / kChunk<T>);
    mla_read_mx_kernel<T, DC, DR><<<dim3((unsigned)((units + 255) / 256)), 256, 0, s>>>(a, units);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mla_append_mx(const MlaAppendArgs& a, hipStream_t s) {
    if (a.bf16) return a.Dc == 512 ? (a.Dr ? append<__bf16, 512, 64>(a, s) : append<__bf16, 512, 0>(a, s))
                                   : (a.Dr ? append<__bf16, 256, 64>(a, s) : append<__bf16, 256, 0>(a, s));
    return a.Dc == 512 ? (a.Dr ? append<float, 512, 64>(a, s) : append<float, 512, 0>(a, s))
                       : (a.Dr ? append<float, 256, 64>(a, s) : append<float, 256, 0>(a, s));
}
hipError_t launch_mla_read_mx(const MlaReadArgs& a, hipStream_t s) {
    if (a.bf16) return a.Dc == 512 ? (a.Dr ? read<__bf16, 512, 64>(a, s) : read<__bf16, 512, 0>(a, s))
                                   : (a.Dr ? read<__bf16, 256, 64>(a, s) : read<__bf16, 256, 0>(a, s));
    return a.Dc == 512 ? (a.Dr ? read<float, 512, 64>(a, s) : read<float, 512, 0>(a, s))
                       : (a.Dr ? read<float, 256, 64>(a, s) : read<float, 256, 0>(a, s));
}

}  // namespace kda
