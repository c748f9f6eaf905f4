// Latent attention, absorbed form: new tokens' queries against a paged cache
// of latents. A cache row is c (Dc) then r (Dr), shared by the heads:
//   s = scale (q_latent . c + q_rope . r),  p = softmax s,  o = sum p c.
//
// The rows of queries (token, head) of one sequence all read the same cache
// rows, so a workgroup takes up to 128 of them and a run of the cache, and
// every cache row is read from HBM once per 128 rows of queries. The cache goes
// from global memory to LDS in tiles of 32 rows, two buffers. Two waves share
// a block of 32 rows of queries: each forms the scores over half of the
// columns (its half of the queries stays in registers) and, after they have
// exchanged these sums through LDS, the output of half of the Dc columns, so
// that its accumulators (Dc / 4 registers) leave room for two waves per SIMD.
//
// The work is split over the cache by its true lengths, which only the device
// knows: the 32-row tiles of all sequences form one list, cut into equal
// parts, one per workgroup. A workgroup walks through the sequences of its
// part; a sequence that lies in one part is finished there, one that spans
// several leaves (maximum, sum, output) of each part in the workspace, and a
// second kernel joins them. Parts are at least min_tiles long, so that short
// caches do not drown in partial results. Bound by the cache's bytes for many
// rows of cache, by latency for few.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

constexpr int kTile = 32;       // cache rows a tile
// blocks of 32 rows of queries a workgroup, at most: what LDS holds
template <class T, int DC> constexpr int max_blocks() { return sizeof(T) == 4 && DC == 512 ? 2 : 4; }

// The list of tiles: number of tiles of sequence b
__device__ __forceinline__ int row_len(const MlaStepArgs& a, int b) {
    const int cap = a.max_pages << a.page_shift, n = a.lens[b];
    return n < 0 ? 0 : n > cap ? cap : n;
}

// Inclusive sums of the tile counts of sequences b0 .. b0 + 63, one per lane.
__device__ __forceinline__ int scan_tiles(const MlaStepArgs& a, int b0, int lane, int& cnt) {
    cnt = b0 + lane < a.Nb ? (row_len(a, b0 + lane) + kTile - 1) / kTile : 0;
    int sum = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d);
        sum += lane >= d ? v : 0;
    }
    return sum;
}
__device__ __forceinline__ int64_t all_tiles(const MlaStepArgs& a, int lane) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.Nb; b0 += 64) {
        int cnt;
        total += __builtin_amdgcn_readlane(scan_tiles(a, b0, lane, cnt), 63);
    }
    return total;
}
__device__ __forceinline__ int64_t part_tiles(const MlaStepArgs& a, int64_t total) {
    const int64_t per = (total + a.parts - 1) / a.parts;
    return per > a.min_tiles ? per : a.min_tiles;
}

// Partial result j (0: of a sequence begun in an earlier part, 1: of one that
// goes on in the next) of row m of the part: maximum, sum, Dc values.
__device__ __forceinline__ float* partial(const MlaStepArgs& a, int group, int64_t part, int j, int row) {
    const int64_t rows = 32 * a.blocks;
    return a.part + ((((int64_t)group * a.parts + part) * 2 + j) * rows + row) * (a.Dc + 4);
}

template <class T, int DC, int DR>
__global__ __launch_bounds__(512, 2) void mla_step_kernel(MlaStepArgs a) {
    constexpr int D = DC + DR, RC = D / kChunk<T>, kBuf = kTile * RC * 16;
    constexpr int NS = D / 32, ND = DC / 64;          // this wave's steps of the scores, blocks of the output
    // float32 queries do not fit the registers beside the output: they are
    // read again for every tile (its products take 16 times as long as bf16's)
    constexpr bool kKeepQ = sizeof(T) == 2;
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    __shared__ __attribute__((aligned(16))) float part_sc[2 * max_blocks<T, DC>()][4][64][4];     // the waves' scores over their columns
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5, half = w & 1;
    const int group = blockIdx.x % a.groups;
    const int64_t part = blockIdx.x / a.groups;
    const int64_t total = all_tiles(a, lane), per = part_tiles(a, total);
    int64_t at = part * per;                                     // next tile of the list
    const int64_t end = at + per < total ? at + per : total;
    if (at >= end) return;
    const int row = group * 32 * a.blocks + 32 * (w >> 1) + n32, M = a.Tq * a.H;   // this lane's row of queries
    const int mrow = row < M ? row : M - 1;
    const int tok = mrow / a.H, head = mrow % a.H;
    const float c = a.scale * kLog2e;
    const int ps = a.page_shift;

    int b0 = 0, cnt, sum = scan_tiles(a, 0, lane, cnt);
    int64_t before = 0;                                          // tiles of the sequences before b0
    while (at < end) {
        while (at >= before + __builtin_amdgcn_readlane(sum, 63)) {
            before += __builtin_amdgcn_readlane(sum, 63);
            b0 += 64;
            sum = scan_tiles(a, b0, lane, cnt);
        }
        const int l = __ffsll((unsigned long long)__ballot(before + sum > at)) - 1;
        const int b = b0 + l;
        const int tiles = __builtin_amdgcn_readlane(cnt, l);
        const int64_t first = before + __builtin_amdgcn_readlane(sum, l) - tiles;   // the sequence's place in the list
        const int t0 = (int)(at - first), t1 = end - first < tiles ? (int)(end - first) : tiles;
        at = first + t1;
        const int len = row_len(a, b);

        if (t0 == 0 && w == 0 && lane == 0 && group == 0 && a.lens[b] > len) atomicAdd(a.status, 1u);

        // queries
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h + 16 * half + 8 * hf;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h + 16 * half + 8 * hf;
        // this wave's steps: every second one
        auto load_q = [&](int s) { return 2 * s < DC / 16 ? load8(qlp + 32 * s) : load8(qrp + 32 * s - DC); };
        Frag<T> qf[kKeepQ ? NS : 1];
        if constexpr (kKeepQ) {
#pragma unroll
            for (int s = 0; s < NS; ++s) qf[s] = load_q(s);
        }
        f32x16 acc[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = zero16();
        float m = -INFINITY, lsum = 0.f;

        // Page table entries of 64 pages, one per lane; -1 for no such page.
        const int32_t* table = a.table + (int64_t)b * a.max_pages;
        int pbase = -64, pages = 0;
        auto fetch_pages = [&](int p) {
            if (p >= pbase + 64) {
                pbase = p;
                const int i = p + lane;
                int e = i < a.max_pages ? table[i] : -1;
                const bool used = i <= (len - 1) >> ps;
                if (e < 0 || e >= a.n_pages) e = -1;
                const uint64_t bad = __ballot(used && e < 0);
                if (bad && w == 0 && lane == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
                pages = e;
            }
        };
        // Tile t's two page entries (pages of 16 rows: its halves), as first
        // cache row of each, and which of them exist.
        auto tile_pages = [&](int t, int64_t& r0, int64_t& r1, int& have) {
            const int k0 = t * kTile;
            fetch_pages(k0 >> ps);
            const int e0 = __builtin_amdgcn_readlane(pages, (k0 >> ps) - pbase);
            int e1 = e0;
            if (ps == 4) {
                // a second page that the sequence does not reach is not needed
                const int p1 = (k0 >> 4) + 1;
                if (k0 + 16 < len) {
                    fetch_pages(p1);
                    e1 = __builtin_amdgcn_readlane(pages, p1 - pbase);
                } else {
                    e1 = -1;
                }
                r0 = (int64_t)(e0 < 0 ? 0 : e0) << 4;
                r1 = (int64_t)(e1 < 0 ? 0 : e1) << 4;
            } else {
                r0 = ((int64_t)(e0 < 0 ? 0 : e0) << ps) + (k0 & ((1 << ps) - 1));
                r1 = r0 + 16;
            }
            have = (e0 >= 0) | (e1 >= 0) << 1;
        };
        auto load = [&](int t, char* buf, int64_t r0, int64_t r1) {
            const int rmax = len - 1 - t * kTile;
            const char* base = static_cast<const char*>(a.cache);
            for (int i = w; i < kTile * RC / 64; i += 2 * a.blocks) {
                const int s = i * 64 + lane;
                const int r = s / RC, cc = (s % RC) ^ swizzle<RC>(r);
                const int rr = r < rmax ? r : rmax;
                const int64_t at_row = rr < 16 ? r0 + rr : r1 + (rr - 16);
                load_lds16(base + at_row * (D * (int)sizeof(T)) + cc * 16, buf + i * 1024);
            }
        };
        int64_t r0, r1;
        int have, next_have = 0;
        tile_pages(t0, r0, r1, have);
        load(t0, smem[0], r0, r1);
        wait_loads();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const char* buf = smem[(t - t0) & 1];
            if (t + 1 < t1) {
                tile_pages(t + 1, r0, r1, next_have);
                load(t + 1, smem[(t + 1 - t0) & 1], r0, r1);
            }
            f32x16 sc = zero16();
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const Frag<T> kf = read_rows<T, RC>(buf, n32, 2 * s, hf, half);
                sc = mma(kf, kKeepQ ? qf[kKeepQ ? s : 0] : load_q(s), sc);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(part_sc[w][g][lane]) =
                    f32x4{sc[4 * g], sc[4 * g + 1], sc[4 * g + 2], sc[4 * g + 3]};
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the sums are in LDS
            wg_barrier();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(part_sc[w ^ 1][g][lane]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[4 * g + j] += x[j];
            }
            // keys that this lane's token sees in the tile: the first lim + 1
            const int k0 = t * kTile;
            if (k0 + kTile > len - a.Tq + 1 || have != 3) {
                const int lim = len - a.Tq + tok - k0 - 4 * hf;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int k = 8 * (r / 4) + r % 4;
                    sc[r] = k > lim || !(have >> (r / 8) & 1) ? -INFINITY : sc[r];
                }
            }
            float mx = sc[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sc[r]);
            mx = half_max(mx);
            // The running maximum moves only when some row's grows by more
            // than 2^8: until then its terms reach at most 2^8, exact enough
            // in float32, and the output needs no rescaling (256 products a
            // lane and tile).
            if (__any((mx - m) * c > 8.f || (m == -INFINITY && mx > -INFINITY))) {
                const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
                const float al = __builtin_amdgcn_exp2f((m - ms) * c);
                lsum *= al;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= al;
                m = mn;
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
            float ts = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r], c, -mc));
                ts += sc[r];
            }
            lsum += ts;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<T> pf = to_frag<T>(sc, s);
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    acc[d] = mma(read_cols<T, RC>(buf + half * (DC / 2) * sizeof(T), 16 * s, 32 * d, lane), pf, acc[d]);
            }
            have = next_have;
            wait_loads();
            wg_barrier();
        }
        const float lt = half_sum(lsum);
        const bool live = row < M;
        if (t0 == 0 && t1 == tiles) {
            const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;
            const int64_t orow = (int64_t)b * M + mrow;
            T* op = static_cast<T*>(a.o) + orow * DC + half * (DC / 2);
#pragma unroll
            for (int d = 0; d < ND; ++d) store_tile<T>(op + 32 * d, acc[d], inv, hf, live);
            if (a.lse && live && hf == 0 && half == 0)
                a.lse[orow] = lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            float* p = partial(a, group, part, t0 > 0 ? 0 : 1, 32 * (w >> 1) + n32);
            if (hf == 0 && half == 0) {
                p[0] = m * c;
                p[1] = lt;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) store_tile<float>(p + 4 + half * (DC / 2) + 32 * d, acc[d], 1.f, hf, true);
        }
    }
}

// Joins the parts of a row of queries, one wave each; writes zeros for rows of
// sequences without cache rows.
template <class T> __global__ __launch_bounds__(256) void mla_step_join_kernel(MlaStepArgs a, int64_t rows) {
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= rows) return;
    const int M = a.Tq * a.H, b = (int)(i / M), row = (int)(i % M);
    const int64_t per = part_tiles(a, all_tiles(a, lane));
    int64_t first = 0;
    int tiles = 0;
    for (int b0 = 0; b0 <= b; b0 += 64) {
        int cnt;
        const int sum = scan_tiles(a, b0, lane, cnt);
        if (b < b0 + 64) {
            tiles = __builtin_amdgcn_readlane(cnt, b - b0);
            first += __builtin_amdgcn_readlane(sum, b - b0) - tiles;
        } else {
            first += __builtin_amdgcn_readlane(sum, 63);
        }
    }
    T* op = static_cast<T*>(a.o) + i * a.Dc;
    if (tiles == 0) {
        for (int d = lane; d < a.Dc; d += 64) op[d] = (T)0.f;
        if (a.lse && lane == 0) a.lse[i] = -INFINITY;
        return;
    }
    const int64_t p0 = first / per, p1 = (first + tiles - 1) / per;
    if (p0 == p1) return;
    const int group = row / (32 * a.blocks), r = row % (32 * a.blocks);
    float m = -INFINITY, l = 0.f;
    for (int64_t p = p0; p <= p1; ++p) {
        const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
        const float mx = x[0], mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
        l = l * __builtin_amdgcn_exp2f(m - ms) + x[1] * __builtin_amdgcn_exp2f(mx - ms);
        m = mn;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    for (int d = 4 * lane; d < a.Dc; d += 256) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        for (int64_t p = p0; p <= p1; ++p) {
            const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
            const float f = __builtin_amdgcn_exp2f(x[0] - ms);
            const f32x4 v = *reinterpret_cast<const f32x4*>(x + 4 + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += f * v[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) op[d + j] = (T)(s[j] * inv);
    }
    if (a.lse && lane == 0) a.lse[i] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// One thread per 16-byte chunk of a new token.
template <class T> __global__ __launch_bounds__(256) void mla_append_kernel(MlaAppendArgs a, int64_t chunks) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= chunks) return;
    const int D = a.Dc + a.Dr, RC = D / kChunk<T>;
    const int64_t i = x / RC;
    const int col = (int)(x % RC) * kChunk<T>;
    int n, t, b;
    if (a.cu) {
        // the last sequence that starts at or before token i
        int lo = 0, hi = a.N;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= i) lo = mid; else hi = mid;
        }
        if (i < a.cu[lo] || i >= a.cu[lo + 1]) return;
        n = lo;
        t = (int)i - a.cu[lo];
        b = 0;
    } else {
        n = b = (int)(i / a.T);
        t = (int)(i % a.T);
    }
    const int have = a.lens[n];
    if (have < 0) return;                                        // padding row
    const int64_t pos = (int64_t)have + t, pg = pos >> a.page_shift;
    int e = -1;
    if (pg < a.max_pages) e = a.table[(int64_t)n * a.max_pages + pg];
    if (e < 0 || e >= a.n_pages) {
        if (col == 0) atomicAdd(a.status, 1u);
        return;
    }
    const int64_t row = a.cu ? i : t;
    const T* src = col < a.Dc ? static_cast<const T*>(a.latent) + b * a.lat_batch + row * a.lat_row + col
                              : static_cast<const T*>(a.kr) + b * a.kr_batch + row * a.kr_row + (col - a.Dc);
    T* dst = static_cast<T*>(a.cache) + (((int64_t)e << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * D + col;
    *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
}

template <class T, int DC, int DR> hipError_t launch(const MlaStepArgs& a, hipStream_t s) {
    mla_step_kernel<T, DC, DR><<<dim3((unsigned)(a.groups * a.parts)), 128 * a.blocks, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)a.Nb * a.Tq * a.H;
    mla_step_join_kernel<T><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a, rows);
    return hipGetLastError();
}
template <class T> hipError_t launch_dims(const MlaStepArgs& a, hipStream_t s) {
    if (a.Dc == 512) return a.Dr ? launch<T, 512, 64>(a, s) : launch<T, 512, 0>(a, s);
    return a.Dr ? launch<T, 256, 64>(a, s) : launch<T, 256, 0>(a, s);
}

}  // namespace

size_t mla_step_plan(MlaStepArgs& a) {
    const int64_t blocks = ((int64_t)a.Tq * a.H + 31) / 32;             // of 32 rows of queries
    const int64_t most_blocks = a.bf16 ? 4 : a.Dc == 512 ? max_blocks<float, 512>() : 4;
    a.groups = (int32_t)((blocks + most_blocks - 1) / most_blocks);
    a.blocks = (int32_t)((blocks + a.groups - 1) / a.groups);
    a.min_tiles = 4;
    const int64_t most = (int64_t)a.Nb * ((((int64_t)a.max_pages << a.page_shift) + kTile - 1) / kTile);
    int64_t parts = 256 / a.groups;
    if (parts < 32) parts = 32;
    if (parts > (most + a.min_tiles - 1) / a.min_tiles) parts = (most + a.min_tiles - 1) / a.min_tiles;
    a.parts = (int32_t)(parts > 1 ? parts : 1);
    return (size_t)a.groups * a.parts * 2 * (32 * a.blocks) * (a.Dc + 4) * sizeof(float);
}

hipError_t launch_mla_step(const MlaStepArgs& a, hipStream_t s) {
    return a.bf16 ? launch_dims<__bf16>(a, s) : launch_dims<float>(a, s);
}

hipError_t launch_mla_append(const MlaAppendArgs& a, hipStream_t s) {
    const int64_t per = (int64_t)(a.Dc + a.Dr) * (a.bf16 ? 2 : 4) / 16, chunks = (int64_t)a.B * a.T * per;
    if (chunks == 0) return hipSuccess;
    const dim3 grid((unsigned)((chunks + 255) / 256));
    if (a.bf16) mla_append_kernel<__bf16><<<grid, 256, 0, s>>>(a, chunks);
    else mla_append_kernel<float><<<grid, 256, 0, s>>>(a, chunks);
    return hipGetLastError();
}

}  // namespace kda
