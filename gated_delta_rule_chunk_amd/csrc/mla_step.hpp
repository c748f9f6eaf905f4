// What the calls over cached rows share (mla_step.hip, mla_step_mx.hip,
// mla_weigh.hip): 16x16 tiles, the list of tiles of all sequences, its parts, and
// the kernel that joins their results.
#pragma once

#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

constexpr int kTile = 32;       // cache rows a tile
// waves of 16 rows of queries a workgroup, at most (float32: what LDS holds)
template <class T, int DC> constexpr int max_waves() { return sizeof(T) == 4 && DC == 512 ? 6 : 8; }

// Layout of a step of 32 products on 16x16 tiles (mla_common.hpp has the 32x32
// ones): lane l with n = l % 16, g = l / 16 holds A row n and B column n,
// products 8 g .. 8 g + 7, and accumulator register r is row 4 g + r, column
// n. Two blocks of scores (keys 0-15, 16-31) make, as they stand, the B
// operand over 32 keys whose product j of group g is key 4 g + j (j < 4) or 16
// + 4 g + j - 4.
__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}
// The position of a tile's chunks: chunk c of row r lies at c ^ swizzle16(r).
// LDS serves a read of 16 bytes per lane in quarters of 16 lanes, of which one
// is the lanes 0-3, 12-15 and 20-27: here rows 0-3 and 12-15 of a group's chunk
// and rows 4-11 of its neighbour's. It serves the transposed read of 8 bytes
// per lane in halves: chunk pairs of eight consecutive rows. float32's column
// read takes four chunks of four rows, four rows apart. Each of these takes
// every bank once.
template <class T, int RC> __device__ __forceinline__ int swizzle16(int r) {
    if constexpr (sizeof(T) == 4) {
        static_assert(RC % 16 == 0, "whole bank cycles");
        return r & 15;
    } else {
        return RC % 16 == 0 ? (r & 7) << 1 : r & 6;   // 8 mod 16: odd rows are half a bank cycle away already
    }
}
// A operand over the columns: tile row r, columns 32 step + 8 g .. + 7
template <class T, int RC> __device__ __forceinline__ Frag<T> read_rows16(const char* lds, int r, int step, int g) {
    const char* p = lds + r * (RC * 16);
    const int sw = swizzle16<T, RC>(r);
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const bf16x8*>(p + chunk_at<RC>(4 * step, g, sw));
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(8 * step, 2 * g, sw));
        const f32x4 b = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(8 * step, 2 * g + 1, sw));
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
}
// A operand over 32 rows of a tile in the order above: row n = column col0 + n
template <class T, int RC> __device__ __forceinline__ Frag<T> read_cols16(const char* lds, int col0, int lane) {
    const int g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
        bf16x8 f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = 16 * u + 4 * g + ((lane >> 2) & 3);
            const char* p = lds + r * (RC * 16) + (lane & 1) * 8 + chunk_at<RC>(col0 >> 3, (lane & 3) >> 1, swizzle16<T, RC>(r));
            const bf16x4 b = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)p));
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * u + j] = b[j];
        }
        return f;
    } else {
        f32x8 f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = 16 * (j >> 2) + 4 * g + (j & 3);
            f[j] = *reinterpret_cast<const float*>(lds + r * (RC * 16) + (lane & 3) * 4 +
                                                   chunk_at<RC>(col0 >> 2, (lane & 15) >> 2, swizzle16<T, RC>(r)));
        }
        return f;
    }
}
// over the four lanes of a query row
__device__ __forceinline__ float group_max(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return half_max(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
}
__device__ __forceinline__ float group_sum(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return half_sum(__uint_as_float(p[0]) + __uint_as_float(p[1]));
}
// four consecutive columns
__device__ __forceinline__ void store4(__bf16* p, const f32x4& x, float mul) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2_bf16(x[0] * mul, x[1] * mul), pack2_bf16(x[2] * mul, x[3] * mul));
}
__device__ __forceinline__ void store4(float* p, const f32x4& x, float mul) {
    *reinterpret_cast<f32x4*>(p) = f32x4{x[0] * mul, x[1] * mul, x[2] * mul, x[3] * mul};
}

// The list of tiles, 64 sequences at a time, one per lane: the length, by which
// tokens see, rows of the cache (the length cut to what the page table holds),
// tiles, and tiles up to and with the sequence's.
struct Scan {
    int len, rows, cnt, sum;
    __device__ __forceinline__ int all() const { return __builtin_amdgcn_readlane(sum, 63); }
};
template <int TILE = kTile> __device__ __forceinline__ Scan scan_tiles(const MlaStepArgs& a, int b0, int lane) {
    Scan x;
    const int cap = a.max_pages << a.page_shift, n = b0 + lane < a.Nb ? a.lens[b0 + lane] : 0;
    x.len = n < 0 ? 0 : n;
    x.rows = x.len < cap ? x.len : cap;
    x.cnt = (x.rows + TILE - 1) / TILE;
    x.sum = x.cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(x.sum, d);
        x.sum += lane >= d ? v : 0;
    }
    return x;
}
// Tiles a part: an even share
__device__ __forceinline__ int part_tiles(const MlaStepArgs& a, int total) {
    const int x = (int)(((unsigned)total + (unsigned)a.parts - 1) / (unsigned)a.parts);
    return __builtin_amdgcn_readfirstlane(x > 1 ? x : 1);
}

// Partial result j (0: of a sequence begun in an earlier part, 1: of one that
// goes on in the next) of a part and row of queries: maximum, sum, 2 unused, Dc values.
__device__ __forceinline__ float* partial(const MlaStepArgs& a, int group, int part, int j, int row) {
    return a.part + ((((int64_t)group * a.parts + part) * 2 + j) * (16 * a.waves) + row) * (a.Dc + 4);
}

// Joins the parts of sequences that span several; writes zeros for sequences
// without cache rows. A workgroup takes a.join_rows rows of queries of one
// sequence. Up to kFewParts parts, each of its four waves takes rows of its own;
// of more, they take the parts of a row in turn, and their sums meet in LDS.
// Bound by latency: a row is two dependent reads. Rows of a wave's own against
// shared ones: 3 parts (128 sequences, 96 heads) 20 against 39 us; 16 parts of
// one sequence 5.1 against 4.1 us.
constexpr int kFewParts = 8;
constexpr int kMaxParts = 256;  // mla_step_plan makes no more

// A wave's part of a row of queries over parts p0 + at, + step, ...: the sums of
// all columns, not yet divided by l.
template <int DC, int MOST>
__device__ __forceinline__ void join_row(const MlaStepArgs& a, int row, int p0, int p1, int at, int step, int lane,
                                         f32x4 (&s)[DC / 256], float& m, float& l) {
    const int group = row / (16 * a.waves), r = row % (16 * a.waves);
    float pm[MOST / 64], pl[MOST / 64];        // all under way together
#pragma unroll
    for (int k = 0; k < MOST / 64; ++k) {
        const int p = p0 + 64 * k + lane;
        pm[k] = -INFINITY;
        pl[k] = 0.f;
        if (p <= p1) {
            const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
            pm[k] = x[0];
            pl[k] = x[1];
        }
    }
    m = pm[0];
#pragma unroll
    for (int k = 1; k < MOST / 64; ++k) m = fmaxf(m, pm[k]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float ms = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < MOST / 64; ++k) l += pl[k] * __builtin_amdgcn_exp2f(pm[k] - ms);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
#pragma unroll
    for (int v = 0; v < DC / 256; ++v) s[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = p0 + at; p <= p1; p += step) {
        const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
        const float f = __builtin_amdgcn_exp2f(x[0] - ms);
#pragma unroll
        for (int v = 0; v < DC / 256; ++v) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(x + 4 + 256 * v + 4 * lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[v][j] += f * y[j];
        }
    }
}
template <class T, int DC, int MOST = kMaxParts, int TILE = kTile>
__global__ __launch_bounds__(256) void mla_step_join_kernel(MlaStepArgs a, int blocks) {
    __shared__ __attribute__((aligned(16))) float sums[4][DC];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int M = a.Tq * a.H, b = blockIdx.x / blocks, row0 = blockIdx.x % blocks * a.join_rows;
    const int row1 = row0 + a.join_rows < M ? row0 + a.join_rows : M;
    int first = 0, total = 0, tiles = 0;
    for (int b0 = 0; b0 < a.Nb; b0 += 64) {
        const Scan sq = scan_tiles<TILE>(a, b0, lane);
        if (b >= b0 && b < b0 + 64) {
            tiles = __builtin_amdgcn_readlane(sq.cnt, b - b0);
            first = total + __builtin_amdgcn_readlane(sq.sum, b - b0) - tiles;
        }
        total += sq.all();
    }
    T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC;
    float* lp = a.lse ? a.lse + (int64_t)b * M : nullptr;
    if (tiles == 0) {
        for (int d = threadIdx.x; d < (row1 - row0) * DC; d += 256) op[(int64_t)row0 * DC + d] = (T)0.f;
        if (lp)
            for (int i = row0 + threadIdx.x; i < row1; i += 256) lp[i] = -INFINITY;
        return;
    }
    const int per = part_tiles(a, total), p0 = first / per, p1 = (first + tiles - 1) / per;
    if (p0 == p1) return;
    f32x4 s[DC / 256];
    float m, l;
    auto inverse = [&] { return l > 0.f ? 1.f / l : l == 0.f ? 0.f : l; };
    auto put_lse = [&](int row) {
        if (lp) lp[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
    };
    if (p1 - p0 < kFewParts) {
        for (int row = row0 + w; row < row1; row += 4) {
            join_row<DC, MOST>(a, row, p0, p1, 0, 1, lane, s, m, l);
            const float inv = inverse();
#pragma unroll
            for (int v = 0; v < DC / 256; ++v) store4(op + (int64_t)row * DC + 256 * v + 4 * lane, s[v], inv);
            if (lane == 0) put_lse(row);
        }
        return;
    }
    for (int row = row0; row < row1; ++row) {
        join_row<DC, MOST>(a, row, p0, p1, w, 4, lane, s, m, l);
#pragma unroll
        for (int v = 0; v < DC / 256; ++v) *reinterpret_cast<f32x4*>(&sums[w][256 * v + 4 * lane]) = s[v];
        __syncthreads();
        const float inv = inverse();
        for (int d = threadIdx.x; d < DC; d += 256)
            op[(int64_t)row * DC + d] = (T)((((sums[0][d] + sums[1][d]) + sums[2][d]) + sums[3][d]) * inv);
        if (threadIdx.x == 0) put_lse(row);
        __syncthreads();
    }
}

}  // namespace
}  // namespace kda
