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

// Workgroups of kRows rows. A thread of each row finds its place in the cache, for
// all of them in LDS; a thread has 8 channels of every kStep-th row, four threads a
// block of 32, and 16 bytes of the shared part of one row: all its loads are under
// way at once. Bound by memory: 28 000 new rows of 512 + 64 bf16 channels are written
// in 12 us (3.6 TB/s), 37 000 read back in 12 (4.8, in part from the last-level
// cache); a thread for each 16 bytes, which found its row's place itself, took 18 and 20.
constexpr int kRows = 16;
template <class T, int DC, int DR> struct Split {
    static constexpr int kUnits = DC / 8, kStep = 256 / kUnits, kPasses = kRows / kStep, kRope = DR / kChunk<T>;
    static_assert(kRows % kStep == 0 && kRows * kRope <= 256, "a thread has one piece of the shared part at most");
};
constexpr int64_t kZeros = -1, kSkip = -2;                        // in place of a page's offset

template <class T, int DC, int DR> __global__ __launch_bounds__(256) void mla_append_mx_kernel(MlaAppendArgs a, uint32_t rows) {
    using S = Split<T, DC, DR>;
    __shared__ int64_t page_of[kRows];
    __shared__ int slot[kRows];
    const int tid = threadIdx.x, u = tid % S::kUnits, r0 = tid / S::kUnits;
    const uint32_t i0 = blockIdx.x * kRows;
    auto source = [&](const void* base, uint32_t i, int64_t row, int64_t batch) {
        const uint32_t b = a.cu ? 0 : i / (uint32_t)a.T, t = a.cu ? i : i - b * (uint32_t)a.T;
        return static_cast<const T*>(base) + b * batch + t * row;
    };
    f32x8 v[S::kPasses];
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
        const uint32_t i = i0 + r0 + p * S::kStep;
        v[p] = f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < rows) v[p] = load8f(source(a.latent, i, a.lat_row, a.lat_batch) + 8 * u);
    }
    u32x4 k = {0, 0, 0, 0};
    if constexpr (DR > 0) {
        const uint32_t i = i0 + tid / S::kRope;
        if (tid < kRows * S::kRope && i < rows)
            k = *reinterpret_cast<const u32x4*>(source(a.kr, i, a.kr_row, a.kr_batch) + tid % S::kRope * kChunk<T>);
    }
    if (tid < kRows) {
        const uint32_t i = i0 + tid;
        int64_t at = kSkip, pos = 0;
        int n = 0;
        int64_t t = 0;
        bool mine = i < rows;
        if (mine) {
            if (a.cu) {
                mine = sequence_of(a.cu, a.N, i, n, t);
            } else {
                n = (int)(i / (uint32_t)a.T);
                t = i - (uint32_t)n * (uint32_t)a.T;
            }
        }
        const int have = mine ? a.lens[n] : -1;                   // negative: padding row
        if (have >= 0) {
            pos = have + t;
            const int64_t pg = pos >> a.page_shift;
            int e = -1;
            if (pg < a.max_pages) e = a.table[(int64_t)n * a.max_pages + pg];
            if (e < 0 || e >= a.n_pages) atomicAdd(a.status, 1u);
            else at = e * ((int64_t)mx_row_bytes(DC, DR, sizeof(T)) << a.page_shift);
        }
        page_of[tid] = at;
        slot[tid] = (int)(pos & ((1 << a.page_shift) - 1));
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
        const int r = r0 + p * S::kStep;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t y = __float_as_uint(v[p][j]) & 0x7fffffffu;
            m = y > m ? y : m;
        }
        uint32_t o = __shfl_xor(m, 1);
        m = o > m ? o : m;
        o = __shfl_xor(m, 2);
        m = o > m ? o : m;
        const uint32_t s = mx_scale_byte(m);
        uint32_t c = 0;
        if (s != 0 && s != 255) {
            // rounds to the nearest, ties to even, and past 6 to 6
            const float f = __uint_as_float(s << 23);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[p][0], v[p][1], f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[p][2], v[p][3], f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[p][4], v[p][5], f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[p][6], v[p][7], f, 3);
        }
        if (page_of[r] < 0) continue;
        char* const page = static_cast<char*>(a.cache) + page_of[r];
        const Row at = row_at(DC, DR, sizeof(T), a.page_shift, slot[r]);
        *reinterpret_cast<uint32_t*>(page + at.codes + 4 * u) = c;
        if ((u & 3) == 0) *reinterpret_cast<uint8_t*>(page + at.scales + (u >> 2)) = (uint8_t)s;
    }
    if constexpr (DR > 0) {
        const int r = tid / S::kRope;
        if (tid < kRows * S::kRope && page_of[r] >= 0)
            *reinterpret_cast<u32x4*>(static_cast<char*>(a.cache) + page_of[r] +
                                      row_at(DC, DR, sizeof(T), a.page_shift, slot[r]).rope + 16 * (tid % S::kRope)) = k;
    }
}

template <class T, int DC, int DR> __global__ __launch_bounds__(256) void mla_read_mx_kernel(MlaReadArgs a, uint32_t rows) {
    using S = Split<T, DC, DR>;
    __shared__ int64_t page_of[kRows];
    __shared__ int slot[kRows];
    const int tid = threadIdx.x, u = tid % S::kUnits, r0 = tid / S::kUnits;
    const uint32_t i0 = blockIdx.x * kRows;
    if (tid < kRows) {
        const uint32_t i = i0 + tid;
        int64_t at = kSkip, pos = 0, t;
        int n;
        if (i < rows) {
            if (sequence_of(a.cu, a.N, i, n, t)) {
                pos = (a.starts ? (int64_t)a.starts[n] : 0) + t;
                const int64_t pg = pos >> a.page_shift;
                int e = -1;
                if (pos >= 0 && pg < a.max_pages) e = a.table[(int64_t)n * a.max_pages + pg];
                if (e < 0 || e >= a.n_pages) {
                    atomicAdd(a.status, 1u);
                    at = kZeros;
                } else {
                    at = e * ((int64_t)mx_row_bytes(DC, DR, sizeof(T)) << a.page_shift);
                }
            } else if (a.zero_rest) {
                at = kZeros;
            }
        }
        page_of[tid] = at;
        slot[tid] = (int)(pos & ((1 << a.page_shift) - 1));
    }
    __syncthreads();
    uint32_t c[S::kPasses], s[S::kPasses];
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
        const int r = r0 + p * S::kStep;
        c[p] = s[p] = 0;
        if (page_of[r] < 0) continue;
        const char* const page = static_cast<const char*>(a.cache) + page_of[r];
        const Row at = row_at(DC, DR, sizeof(T), a.page_shift, slot[r]);
        c[p] = *reinterpret_cast<const uint32_t*>(page + at.codes + 4 * u);
        s[p] = *reinterpret_cast<const uint8_t*>(page + at.scales + (u >> 2));
    }
    if constexpr (DR > 0) {
        const int r = tid / S::kRope;
        if (tid < kRows * S::kRope && page_of[r] != kSkip) {
            u32x4 k = {0, 0, 0, 0};
            if (page_of[r] >= 0)
                k = *reinterpret_cast<const u32x4*>(static_cast<const char*>(a.cache) + page_of[r] +
                                                    row_at(DC, DR, sizeof(T), a.page_shift, slot[r]).rope + 16 * (tid % S::kRope));
            *reinterpret_cast<u32x4*>(static_cast<T*>(a.rope) + (int64_t)(i0 + r) * DR + tid % S::kRope * kChunk<T>) = k;
        }
    }
#pragma unroll
    for (int p = 0; p < S::kPasses; ++p) {
        const int r = r0 + p * S::kStep;
        if (page_of[r] == kSkip) continue;
        const MxScale f(s[p]);
        T* to = static_cast<T*>(a.latent) + (int64_t)(i0 + r) * DC + 8 * u;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<bf16x8*>(to) = f.bf16(c[p]);
        } else {
            const f32x8 v = f.f32(c[p]);
            *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
}

template <class T, int DC, int DR> hipError_t append(const MlaAppendArgs& a, hipStream_t s) {
    const uint32_t rows = (uint32_t)a.B * (uint32_t)a.T;
    mla_append_mx_kernel<T, DC, DR><<<dim3((rows + kRows - 1) / kRows), 256, 0, s>>>(a, rows);
    return hipGetLastError();
}
template <class T, int DC, int DR> hipError_t read(const MlaReadArgs& a, hipStream_t s) {
    mla_read_mx_kernel<T, DC, DR><<<dim3(((uint32_t)a.T + kRows - 1) / kRows), 256, 0, s>>>(a, (uint32_t)a.T);
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
