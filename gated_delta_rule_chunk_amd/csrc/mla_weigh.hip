// The attention weight that cached rows gather: w_j = decay w_j + sum over the
// rows of queries (token, head) of exp(s_ij - lse_i), s as in mla_step.hip.
//
// A wave holds 32 cache rows (keys) in registers, as the first operand of
// 32x32 tiles of the matrix instructions, and meets all rows of queries that
// its workgroup keeps in LDS: no exchange between waves, and each cache row is
// read once. Scores come out with a lane holding one query and 16 keys, so
// that a key's weight is a sum down a register, over the lanes at the very end.
#include "mla_mx.hpp"
#include "mla_step.hpp"

namespace kda {
namespace {

constexpr int kWaves = 8;       // of a workgroup, 32 keys each
constexpr int kUnit = 32 * kWaves;
// rows of queries in LDS at a time, at most
template <class T> constexpr int kQueries = sizeof(T) == 2 ? 128 : 64;

// Columns in the order of the products: step st multiplies, in half hf of the
// lanes, the 8 channels from 64 (st / 4) + 8 (st % 4) + 32 hf, so that a lane's
// part of four steps is one block of 32 of the 4-bit cache.
template <class T, int RC> __device__ __forceinline__ Frag<T> read_query(const char* lds, int r, int st, int hf) {
    const char* p = lds + r * (RC * 16);
    const int sw = swizzle<RC>(r), k = 8 * (st / 4) + st % 4;
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const bf16x8*>(p + chunk_at<RC>(k, 4 * hf, sw));
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(2 * k, 8 * hf, sw));
        const f32x4 b = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(2 * k, 8 * hf + 1, sw));
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
}

// A lane's key, read from global memory (zeros where it does not exist).
template <class T, int DC, int DR, bool MX> struct Key {
    const char* row;            // rows of T: the row; 4 bits: its codes
    const char* scales;
    const char* rope;
    bool have;

    __device__ __forceinline__ Frag<T> zero() const {
        Frag<T> z;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = (T)0.f;
        return z;
    }
    __device__ __forceinline__ Frag<T> operand(int st, int hf) const {
        if (!have) return zero();
        const int c = 64 * (st / 4) + 8 * (st % 4) + 32 * hf;
        if constexpr (!MX) return load8(reinterpret_cast<const T*>(row) + c);
        if (st >= DC / 16) return load8(reinterpret_cast<const T*>(rope) + (c - DC));
        const MxScale f(*reinterpret_cast<const uint8_t*>(scales + c / 32));
        const uint32_t x = *reinterpret_cast<const uint32_t*>(row + c / 2);
        if constexpr (sizeof(T) == 2) return f.bf16(x);
        else return f.f32(x);
    }
};

template <class T, int DC, int DR, bool MX>
__global__ __launch_bounds__(64 * kWaves, 2) void mla_weigh_kernel(MlaWeighArgs x, int chunk, int parts) {
    constexpr int D = DC + DR, RC = D / kChunk<T>, NS = D / 16;
    constexpr bool kKeep = sizeof(T) == 2;                // float32's keys are read again for every block of queries
    extern __shared__ __attribute__((aligned(1024))) char smem[];
    float* const lse2 = reinterpret_cast<float*>(smem + chunk * (RC * 16));     // lse / log 2 of the rows in LDS
    int* const last = reinterpret_cast<int*>(lse2 + chunk);                     // the last key that each sees
    __shared__ float sums[kWaves][32];
    const MlaStepArgs& a = x.s;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int M = a.Tq * a.H, ps = a.page_shift;
    const float c = a.scale * kLog2e;

    Scan sq = scan_tiles<kUnit>(a, 0, lane);
    int total = sq.all();
    for (int b = 64; b < a.Nb; b += 64) total += scan_tiles<kUnit>(a, b, lane).all();
    const int per = (int)(((unsigned)total + (unsigned)parts - 1) / (unsigned)parts);
    int at = (int)blockIdx.x * per;
    if (at >= total) return;
    const int end = total - at < per ? total : at + per;
    int b0 = 0, before = 0, loaded = -1;                  // loaded: whose queries are in LDS
    for (; at < end; ++at) {
        while (at >= before + sq.all()) {
            before += sq.all();
            b0 += 64;
            sq = scan_tiles<kUnit>(a, b0, lane);
        }
        const int l = __ffsll((unsigned long long)__ballot(before + sq.sum > at)) - 1;
        const int b = b0 + l;
        const int len = __builtin_amdgcn_readlane(sq.len, l), rows = __builtin_amdgcn_readlane(sq.rows, l);
        const int u = at - before - (__builtin_amdgcn_readlane(sq.sum, l) - __builtin_amdgcn_readlane(sq.cnt, l));
        if (u == 0 && threadIdx.x == 0 && len > rows) atomicAdd(a.status, 1u);
        const int key0 = u * kUnit + w * 32, key = key0 + n;

        Key<T, DC, DR, MX> k;
        int e = -1;
        if (key < rows) e = a.table[(int64_t)b * a.max_pages + (key >> ps)];
        k.have = e >= 0 && e < a.n_pages;
        const int64_t pr = key & ((1 << ps) - 1);
        // a missing page is counted at its first row
        const uint64_t bad = __ballot(key < rows && !k.have && hf == 0 && pr == 0);
        if (bad && lane == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
        if constexpr (MX) {
            const char* page = static_cast<const char*>(a.cache) + e * ((int64_t)mx_row_bytes(DC, DR, sizeof(T)) << ps);
            k.row = page + pr * (DC / 2);
            k.scales = page + (((int64_t)DC / 2) << ps) + pr * (DC / 32);
            k.rope = page + (((int64_t)DC / 2 + DC / 32) << ps) + pr * (DR * (int)sizeof(T));
        } else {
            k.row = static_cast<const char*>(a.cache) + (((int64_t)e << ps) + pr) * (RC * 16);
        }
        const bool holes = __any(key < rows && !k.have);
        Frag<T> kf[kKeep ? NS : 1];
        if constexpr (kKeep) {
#pragma unroll
            for (int s = 0; s < NS; ++s) kf[s] = k.operand(s, hf);
        }
        float sum[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[r] = 0.f;
        for (int m0 = 0; m0 < M; m0 += chunk) {
            if (M > chunk || loaded != b) {
                __syncthreads();
                for (int i = threadIdx.x; i < chunk * RC; i += 64 * kWaves) {
                    const int r = i / RC, q = i % RC, m = m0 + r;
                    u32x4 v = {0, 0, 0, 0};
                    if (m < M) {
                        const int tok = m / a.H, head = m - tok * a.H, ch = q * kChunk<T>;
                        const T* p = ch < DC ? static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h + ch
                                             : static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h + (ch - DC);
                        v = *reinterpret_cast<const u32x4*>(p);
                    }
                    *reinterpret_cast<u32x4*>(smem + r * (RC * 16) + ((q ^ swizzle<RC>(r)) << 4)) = v;
                }
                for (int r = threadIdx.x; r < chunk; r += 64 * kWaves) {
                    const int m = m0 + r, see = len - a.Tq + m / a.H;
                    lse2[r] = m < M ? x.lse[(int64_t)b * M + m] * kLog2e : 0.f;
                    last[r] = m >= M ? -1 : see < rows - 1 ? see : rows - 1;
                }
                __syncthreads();
                loaded = b;
            }
            if (key0 >= rows) continue;
            const int some = M - m0 < chunk ? M - m0 : chunk;
            for (int r0 = 0; r0 < some; r0 += 32) {
                f32x16 s = zero16();
#pragma unroll
                for (int st = 0; st < NS; ++st)
                    s = mma(kKeep ? kf[kKeep ? st : 0] : k.operand(st, hf), read_query<T, RC>(smem, r0 + n, st, hf), s);
                settle(s);
                const float z = lse2[r0 + n];
                if (holes || key0 + 32 > len - a.Tq + 1 || key0 + 32 > rows || r0 + 32 > some) {
                    const uint64_t there = __ballot(k.have);
                    const int lim = last[r0 + n] - key0 - 4 * hf;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int i = 8 * (r / 4) + r % 4;
                        const bool on = i <= lim && (there >> (i + 4 * hf) & 1);
                        sum[r] += on ? __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -z)) : 0.f;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) sum[r] += __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -z));
                }
            }
        }
        if (key0 >= rows) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) sum[r] += __shfl_xor(sum[r], d);
            if (n == 0) sums[w][8 * (r / 4) + 4 * hf + r % 4] = sum[r];
        }
        wait_lds();
        if (lane < 32 && key < rows) {
            const int64_t i = ((int64_t)b * a.max_pages << ps) + key;
            float old = 0.f;
            if (x.decay != 0.f && key < len - x.fresh) old = x.decay * x.w_in[i];
            x.w_out[i] = old + sums[w][lane];
        }
        wait_lds();
    }
}

template <class T, int DC, int DR, bool MX> hipError_t launch_weigh(const MlaWeighArgs& x, hipStream_t s) {
    const MlaStepArgs& a = x.s;
    const int M = a.Tq * a.H;
    int chunk = (M + 31) / 32 * 32;
    if (chunk > kQueries<T>) chunk = kQueries<T>;
    const int64_t cap = (int64_t)a.max_pages << a.page_shift, units = a.Nb * ((cap + kUnit - 1) / kUnit);
    const int parts = (int)(units < 256 ? units : 256);
    const int lds = chunk * ((DC + DR) * (int)sizeof(T) + 8);
    const void* f = reinterpret_cast<const void*>(&mla_weigh_kernel<T, DC, DR, MX>);
    if (const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) return e;
    mla_weigh_kernel<T, DC, DR, MX><<<dim3((unsigned)parts), 64 * kWaves, lds, s>>>(x, chunk, parts);
    return hipGetLastError();
}
template <class T, bool MX> hipError_t weigh_dims(const MlaWeighArgs& x, hipStream_t s) {
    if (x.s.Dc == 512) return x.s.Dr ? launch_weigh<T, 512, 64, MX>(x, s) : launch_weigh<T, 512, 0, MX>(x, s);
    return x.s.Dr ? launch_weigh<T, 256, 64, MX>(x, s) : launch_weigh<T, 256, 0, MX>(x, s);
}

}  // namespace

hipError_t launch_mla_weigh(const MlaWeighArgs& x, hipStream_t s) {
    if (x.mx) return x.s.bf16 ? weigh_dims<__bf16, true>(x, s) : weigh_dims<float, true>(x, s);
    return x.s.bf16 ? weigh_dims<__bf16, false>(x, s) : weigh_dims<float, false>(x, s);
}

}  // namespace kda
