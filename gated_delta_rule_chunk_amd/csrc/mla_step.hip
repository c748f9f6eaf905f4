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
// second kernel joins them. Parts are long enough that a short cache does not
// drown in partial results (part_tiles). Bound by the cache's bytes for many
// rows of cache, by latency for few.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

constexpr int kTile = 32;       // cache rows a tile
// blocks of 32 rows of queries a workgroup, at most: what LDS holds
template <class T, int DC> constexpr int max_blocks() { return sizeof(T) == 4 && DC == 512 ? 2 : 4; }

// The list of tiles: rows of the cache that sequence b has
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
__device__ __forceinline__ int all_tiles(const MlaStepArgs& a, int lane) {
    int total = 0;
    for (int b0 = 0; b0 < a.Nb; b0 += 64) {
        int cnt;
        total += __builtin_amdgcn_readlane(scan_tiles(a, b0, lane, cnt), 63);
    }
    return total;
}
// Tiles a part: an even share, but no fewer than keeps the partial results
// (a part's cost of writing and joining them against the time of a tile).
__device__ __forceinline__ int part_tiles(const MlaStepArgs& a, int total) {
    const int per = (int)(((unsigned)total + (unsigned)a.parts - 1) / (unsigned)a.parts);
    const int least = (int)__builtin_ceilf(__builtin_sqrtf((float)total) * a.part_cost);
    const int x = per > least ? per : least;
    return __builtin_amdgcn_readfirstlane(x > 1 ? x : 1);
}

// Partial result j (0: of a sequence begun in an earlier part, 1: of one that
// goes on in the next) of a part and row of queries: maximum, sum, 2 unused, Dc values.
__device__ __forceinline__ float* partial(const MlaStepArgs& a, int group, int part, int j, int row) {
    return a.part + ((((int64_t)group * a.parts + part) * 2 + j) * (32 * a.blocks) + row) * (a.Dc + 4);
}

// A tile's 32 rows of RC chunks to LDS (layout: mla_common.hpp). Rows 0-15 lie
// at lo and 16-31 at hi, 16 consecutive rows each. Lane l of instruction i
// fills chunk 64 i + l of the tile; as a row's chunks are permuted within
// their groups only, its source is that chunk with its low bits exchanged.
// With EDGE, rows past rmax are not read (row rmax stands in), and halves
// whose page does not exist (bits of have) are zeros: a hidden row's weight is
// 0, but what it multiplies has to be finite.
template <int RC, int WAVES, bool EDGE>
__device__ __forceinline__ void load_cache_tile(char* lds, const char* lo, const char* hi, int rmax, int have, int w,
                                                int lane) {
    constexpr int kInstr = kTile * RC / 64, kHalf = kInstr / 2;
    asm volatile("" : "+v"(lane));   // addresses are formed here for each tile, not kept in registers
#pragma unroll
    for (int k = 0; k < (kInstr + WAVES - 1) / WAVES; ++k) {
        const int i = k * WAVES + w;
        if (kInstr % WAVES != 0 && i >= kInstr) break;
        const int s = i * 64 + lane;
        int r;
        if constexpr (RC % 64 == 0) {                     // an instruction stays in one row
            r = i / (RC / 64);
        } else {                                          // a row has RC / 8 groups of 8 chunks
            r = (int)((8u * (unsigned)i + ((unsigned)lane >> 3)) / (unsigned)(RC / 8));
        }
        const int src = s ^ swizzle<RC>(r);
        if constexpr (EDGE) {
            const int half = i >= kHalf && rmax >= 16;    // where its rows come from
            if (have >> half & 1) {
                const int rr = r > rmax ? rmax : r;
                load_lds16((rr < 16 ? lo : hi - 16 * RC * 16) + (src + (rr - r) * RC) * 16, lds + i * 1024);
            } else {
                *reinterpret_cast<u32x4*>(lds + i * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
            }
        } else {
            load_lds16s((i >= kHalf ? hi - 16 * RC * 16 : lo), src * 16, lds + i * 1024);
        }
    }
}

template <class T, int DC, int DR, int BLK>
__global__ __launch_bounds__(128 * BLK, BLK > 2 ? 2 : 1) void mla_step_kernel(MlaStepArgs a) {
    constexpr int D = DC + DR, RC = D / kChunk<T>, kBuf = kTile * RC * 16, WAVES = 2 * BLK;
    constexpr int NS = D / 32, ND = DC / 64;          // this wave's steps of the scores, blocks of the output
    // float32 queries do not fit the registers beside the output: they are
    // read again for every tile (its products take 16 times as long as bf16's)
    constexpr bool kKeepQ = sizeof(T) == 2;
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    __shared__ __attribute__((aligned(16))) float part_sc[WAVES][4][64][4];     // the waves' scores over their columns
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5, half = w & 1;
    const int group = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    const int total = all_tiles(a, lane), per = part_tiles(a, total);
    int at = part * per;                                         // next tile of the list
    const int end = total - at < per ? total : at + per;
    if (at >= total) return;
    const int M = a.Tq * a.H;
    const float c = a.scale * kLog2e;
    const int ps = a.page_shift;

    int b0 = 0, cnt, sum = scan_tiles(a, 0, lane, cnt);
    int before = 0;                                              // tiles of the sequences before b0
    while (at < end) {
        while (at >= before + __builtin_amdgcn_readlane(sum, 63)) {
            before += __builtin_amdgcn_readlane(sum, 63);
            b0 += 64;
            sum = scan_tiles(a, b0, lane, cnt);
        }
        const int l = __ffsll((unsigned long long)__ballot(before + sum > at)) - 1;
        const int b = b0 + l;
        const int tiles = __builtin_amdgcn_readlane(cnt, l);
        const int first = before + __builtin_amdgcn_readlane(sum, l) - tiles;       // the sequence's place in the list
        const int t0 = at - first, t1 = end - first < tiles ? end - first : tiles;
        at = first + t1;
        const int len = __builtin_amdgcn_readfirstlane(row_len(a, b));
        if (t0 == 0 && w == 0 && lane == 0 && group == 0 && a.lens[b] > len) atomicAdd(a.status, 1u);

        // queries: row group * 32 BLK + 32 (w / 2) + n32 of the (token, head) pairs
        const int row = group * 32 * BLK + 32 * (w >> 1) + n32, mrow = row < M ? row : M - 1;
        const int tok = mrow / a.H;
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + (mrow - tok * a.H) * a.ql_h + 16 * half +
                       8 * hf;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + (mrow - tok * a.H) * a.qr_h + 16 * half +
                       8 * hf;
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
        auto page = [&](int p) -> int {
            if (p >= pbase + 64) {
                pbase = p;
                const int i = p + lane;
                int e = i < a.max_pages ? table[i] : -1;
                if (e < 0 || e >= a.n_pages) e = -1;
                // counted once: where the page's first row is this part's
                const int64_t r = (int64_t)i << ps;
                const uint64_t bad = __ballot(e < 0 && r < len && r >= t0 * kTile && r < (int64_t)t1 * kTile);
                if (bad && group == 0 && w == 0 && lane == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
                pages = e;
            }
            return __builtin_amdgcn_readlane(pages, p - pbase);
        };
        // Issues tile t's loads; returns which of its halves exist.
        auto load = [&](int t, char* buf) -> int {
            const int k0 = t * kTile;
            const int e0 = page(k0 >> ps);
            int e1 = e0;
            int64_t r0, r1;                                       // first cache row of each half
            if (ps == 4) {
                e1 = k0 + 16 < len ? page((k0 >> 4) + 1) : -1;    // a page not reached is not looked up
                r0 = (int64_t)(e0 < 0 ? 0 : e0) << 4;
                r1 = (int64_t)(e1 < 0 ? 0 : e1) << 4;
            } else {
                r0 = ((int64_t)(e0 < 0 ? 0 : e0) << ps) + (k0 & ((1 << ps) - 1));
                r1 = r0 + 16;
            }
            const char* lo = static_cast<const char*>(a.cache) + r0 * (RC * 16);
            const char* hi = static_cast<const char*>(a.cache) + r1 * (RC * 16);
            const int have = (e0 >= 0) | (e1 >= 0) << 1;
            if (have == 3 && k0 + kTile <= len) load_cache_tile<RC, WAVES, false>(buf, lo, hi, 0, 0, w, lane);
            else load_cache_tile<RC, WAVES, true>(buf, lo, hi, len - 1 - k0, have, w, lane);
            return have;
        };
        int have = load(t0, smem[0]), next_have = 0;
        wait_loads_and_lds();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const char* buf = smem[(t - t0) & 1];
            if (t + 1 < t1) next_have = load(t + 1, smem[(t + 1 - t0) & 1]);
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
            // in float32, and the output needs no rescaling (Dc / 4 products
            // a lane and tile).
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
            wait_loads_and_lds();
            wg_barrier();
        }
        const float lt = half_sum(lsum);
        int ln = lane;
        asm volatile("" : "+v"(ln));                              // formed again here, not kept over the loop
        const int orow = group * 32 * BLK + 32 * (w >> 1) + (ln & 31);
        const bool live = orow < M;
        if (t0 == 0 && t1 == tiles) {
            const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;
            const int64_t at_o = (int64_t)b * M + (live ? orow : M - 1);
            T* op = static_cast<T*>(a.o) + at_o * DC + half * (DC / 2);
#pragma unroll
            for (int d = 0; d < ND; ++d) store_tile<T>(op + 32 * d, acc[d], inv, hf, live);
            if (a.lse && live && hf == 0 && half == 0)
                a.lse[at_o] = lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            float* p = partial(a, group, part, t0 > 0 ? 0 : 1, 32 * (w >> 1) + (ln & 31));
            if (hf == 0 && half == 0) {
                p[0] = m * c;
                p[1] = lt;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) store_tile<float>(p + 4 + half * (DC / 2) + 32 * d, acc[d], 1.f, hf, true);
        }
    }
}

// Joins the parts of a row of queries; writes zeros for rows of sequences
// without cache rows. A workgroup takes one row: its four waves take the parts
// in turn, each over all columns, and their sums meet in LDS.
template <class T, int DC> __global__ __launch_bounds__(256) void mla_step_join_kernel(MlaStepArgs a) {
    __shared__ __attribute__((aligned(16))) float sums[4][DC];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int M = a.Tq * a.H, b = blockIdx.x / M, row = blockIdx.x % M;
    int first = 0, total = 0, tiles = 0;
    for (int b0 = 0; b0 < a.Nb; b0 += 64) {
        int cnt;
        const int sum = scan_tiles(a, b0, lane, cnt);
        if (b >= b0 && b < b0 + 64) {
            tiles = __builtin_amdgcn_readlane(cnt, b - b0);
            first = total + __builtin_amdgcn_readlane(sum, b - b0) - tiles;
        }
        total += __builtin_amdgcn_readlane(sum, 63);
    }
    T* op = static_cast<T*>(a.o) + (int64_t)blockIdx.x * DC;
    if (tiles == 0) {
        for (int d = threadIdx.x; d < DC; d += 256) op[d] = (T)0.f;
        if (a.lse && threadIdx.x == 0) a.lse[blockIdx.x] = -INFINITY;
        return;
    }
    const int per = part_tiles(a, total), p0 = first / per, p1 = (first + tiles - 1) / per;
    if (p0 == p1) return;
    const int group = row / (32 * a.blocks), r = row % (32 * a.blocks);
    float m = -INFINITY;
    for (int p = p0 + lane; p <= p1; p += 64) m = fmaxf(m, partial(a, group, p, p > p0 ? 0 : 1, r)[0]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int p = p0 + lane; p <= p1; p += 64) {
        const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
        l += x[1] * __builtin_amdgcn_exp2f(x[0] - ms);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
    constexpr int V = DC / 256;
    f32x4 s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = p0 + w; p <= p1; p += 4) {
        const float* x = partial(a, group, p, p > p0 ? 0 : 1, r);
        const float f = __builtin_amdgcn_exp2f(x[0] - ms);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(x + 4 + 256 * v + 4 * lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[v][j] += f * y[j];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) *reinterpret_cast<f32x4*>(&sums[w][256 * v + 4 * lane]) = s[v];
    __syncthreads();
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    for (int d = threadIdx.x; d < DC; d += 256)
        op[d] = (T)((((sums[0][d] + sums[1][d]) + sums[2][d]) + sums[3][d]) * inv);
    if (a.lse && threadIdx.x == 0)
        a.lse[blockIdx.x] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
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
    const dim3 grid((unsigned)(a.groups * a.parts));
    if (a.blocks == 1) mla_step_kernel<T, DC, DR, 1><<<grid, 128, 0, s>>>(a);
    else if (a.blocks == 2) mla_step_kernel<T, DC, DR, 2><<<grid, 256, 0, s>>>(a);
    if constexpr (max_blocks<T, DC>() > 2) {
        if (a.blocks == 3) mla_step_kernel<T, DC, DR, 3><<<grid, 384, 0, s>>>(a);
        else if (a.blocks == 4) mla_step_kernel<T, DC, DR, 4><<<grid, 512, 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    mla_step_join_kernel<T, DC><<<dim3((unsigned)((int64_t)a.Nb * a.Tq * a.H)), 256, 0, s>>>(a);
    return hipGetLastError();
}
template <class T> hipError_t launch_dims(const MlaStepArgs& a, hipStream_t s) {
    if (a.Dc == 512) return a.Dr ? launch<T, 512, 64>(a, s) : launch<T, 512, 0>(a, s);
    return a.Dr ? launch<T, 256, 64>(a, s) : launch<T, 256, 0>(a, s);
}

}  // namespace

// The split over workgroups. A block of 32 rows of queries costs the same
// whether its rows are used, so the blocks are spread evenly over as few
// groups as hold them. One workgroup of three or four blocks fills a compute
// unit, two of one block fit.
size_t mla_step_plan(MlaStepArgs& a) {
    const int64_t blocks = ((int64_t)a.Tq * a.H + 31) / 32;
    const int64_t most_blocks = a.bf16 ? 4 : a.Dc == 512 ? max_blocks<float, 512>() : max_blocks<float, 256>();
    a.groups = (int32_t)((blocks + most_blocks - 1) / most_blocks);
    a.blocks = (int32_t)((blocks + a.groups - 1) / a.groups);
    const int64_t most = (int64_t)a.Nb * ((((int64_t)a.max_pages << a.page_shift) + kTile - 1) / kTile);
    int64_t parts = (a.blocks == 1 ? 512 : 256) / a.groups;
    if (parts < 32) parts = 32;
    if (parts > most) parts = most;
    a.parts = (int32_t)(parts > 1 ? parts : 1);
    // writing and joining a part's results, in tiles: about 1/16 a tile for 96
    // rows of 512 columns; the sum of both costs is least at sqrt(total) / 4
    a.part_cost = 0.25f;
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
