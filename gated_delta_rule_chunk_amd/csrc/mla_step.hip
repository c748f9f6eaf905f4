// Latent attention, absorbed form: new tokens' queries against a paged cache
// of latents. A cache row is c (Dc) then r (Dr), shared by the heads:
//   s = scale (q_latent . c + q_rope . r),  p = softmax s,  o = sum p c.
//
// The rows of queries (token, head) of one sequence all read the same cache
// rows, so a workgroup takes up to 128 of them and a run of the cache, and
// every cache row is read from HBM once per 128 rows of queries. The cache goes
// from global memory to LDS in tiles, the next one under way while one is at
// work.
// Two waves share a block of 32 rows of queries: each forms the scores and
// probabilities of 16 of them, and, after they have exchanged these (1 or 2 KB)
// through LDS, the outputs of all 32 over half of the Dc columns. So a value
// operand read from LDS, the costliest access here (it is read transposed),
// serves two products, nothing is computed twice, and queries, scores and
// outputs (Dc / 4 registers) leave room for two waves per SIMD.
//
// The work is split over the cache by its true lengths, which only the device
// knows: the tiles of all sequences form one list, cut into equal
// parts, one per workgroup. A workgroup walks through the sequences of its
// part; a sequence that lies in one part is finished there, one that spans
// several leaves (maximum, sum, output) of each part in the workspace, and a
// second kernel joins them.
//
// Measured, bf16, 96 heads, Dc = 512, Dr = 64. 128 sequences of 4096 to 8192
// rows (922 MB): 237-280 us and 20 us for the join, 3.3-3.9 TB/s; the cache's tiles
// alone load in 187 us. A tile takes 4600 clocks: SIMDs 0 and 1 hold two of the
// six waves (2200 clocks of matrix instructions), LDS delivers for 1500, and at
// the clock that this load leaves, 1.9-2.2 GHz, that is the time. One sequence of
// 100001 rows (115 MB): 42 us, of which 28 are its 13 tiles a workgroup, and 14
// us for the join of 256 parts (47 MB). One of 1000 rows: 11 and 5 us, latency.
// The batch with two and four new tokens each, by the call: 456 and 741 us, 0.65
// and 0.78 of the matrix cores' floor.
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
__device__ __forceinline__ Scan scan_tiles(const MlaStepArgs& a, int b0, int lane) {
    Scan x;
    const int cap = a.max_pages << a.page_shift, n = b0 + lane < a.Nb ? a.lens[b0 + lane] : 0;
    x.len = n < 0 ? 0 : n;
    x.rows = x.len < cap ? x.len : cap;
    x.cnt = (x.rows + kTile - 1) / kTile;
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

// A tile's rows of RC chunks come to LDS (layout: mla_common.hpp) as two halves
// of 16 consecutive cache rows. Lane l of a half's instruction j fills chunk
// 64 j + l of it; as a row's chunks are permuted within their groups only, its
// source is that chunk with its low bits exchanged.
template <class T, int RC> struct CacheTile {
    static constexpr int kInstr = 16 * RC / 64;           // a half
    static __device__ __forceinline__ int row(int j, int lane) {
        if constexpr (RC % 64 == 0) return j / (RC / 64); // an instruction stays in one row
        // a row has RC / 8 groups of 8 chunks
        return (int)((8u * (unsigned)j + ((unsigned)lane >> 3)) / (unsigned)(RC / 8));
    }
    static __device__ __forceinline__ int source(int j, int lane) {
        return (j * 64 + lane) ^ swizzle16<T, RC>(row(j, lane));
    }
};
// Loads a wave issues for a tile, and the x-th of them, if `on`: for a tile whose
// rows all exist.
template <class T, int RC, int WAVES> constexpr int tile_loads() {
    return (CacheTile<T, RC>::kInstr + WAVES - 1) / WAVES * 2;
}
template <class T, int RC, int WAVES>
__device__ __forceinline__ void load_of_tile(int x, bool on, char* lds, const char* lo, const char* hi, int w, int lane) {
    using C = CacheTile<T, RC>;
    const int q = x & 1, j = (x >> 1) * WAVES + w;
    load_lds16s_if(on && (C::kInstr % WAVES == 0 || j < C::kInstr), q ? hi : lo, C::source(j, lane) * 16,
                   lds + (q * C::kInstr + j) * 1024);
}
// A whole tile of which rows past rmax are not read (row rmax stands in), and
// halves whose page does not exist (bits of have) are zeros: a hidden row's
// weight is 0, but what it multiplies has to be finite.
template <class T, int RC, int WAVES>
__device__ __forceinline__ void load_edge_tile(char* lds, const char* lo, const char* hi, int rmax, int have, int w,
                                               int lane) {
    using C = CacheTile<T, RC>;
    asm volatile("" : "+v"(lane));   // addresses are formed here for each tile, not kept in registers
    for (int j = w; j < C::kInstr; j += WAVES) {
        const int src = C::source(j, lane), r = C::row(j, lane);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            char* to = lds + (q * C::kInstr + j) * 1024;
            const int f = 16 * q <= rmax ? q : 0;         // the half its rows come from
            if (have >> f & 1) {
                const int last = rmax - 16 * f, rr = f < q || r > last ? last : r;
                load_lds16((f ? hi : lo) + (src + (rr - r) * RC) * 16, to);
            } else {
                *reinterpret_cast<u32x4*>(to + lane * 16) = u32x4{0, 0, 0, 0};
            }
        }
    }
}

template <class T, int DC, int DR, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES > 4 ? 2 : 1) void mla_step_kernel(MlaStepArgs a) {
    constexpr int D = DC + DR, RC = D / kChunk<T>, kBuf = kTile * RC * 16;
    constexpr int NS = D / 32, ND = DC / 32;          // steps of the scores, blocks of the output's half
    // Not all queries fit the registers beside an output of 512 columns and what
    // is under way: the first kLdsQ steps' of bf16 stay in LDS. float32's stay in
    // registers where they fit beside the output or with one wave per SIMD;
    // otherwise they are read again for every tile (64 sequences of 4096 rows, 64
    // heads: kept 208, read again 271 us for Dc = 256, 361 and 521 for 512). So
    // are those of six waves of Dc = 512, which spill 20 registers besides: 96
    // heads take 698 us, and 128, in two groups of four waves, 676.
    constexpr bool kKeepQ = sizeof(T) == 2 || DC == 256 || WAVES <= 4;
    constexpr int kLdsQ = sizeof(T) == 2 && DC == 512 ? 8 : 0;
    // bf16: the next tile's loads go out one by one under the products of the
    // scores. All at once, a wave waits about 150 clocks for each. float32's
    // products leave no registers for them, and take far longer than the loads.
    constexpr bool kSpread = sizeof(T) == 2;
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    // what the two waves of a row block tell each other: probabilities as
    // operands, the factor of the running maximum's move (later 1 / sum)
    __shared__ __attribute__((aligned(32))) Frag<T> probs[WAVES][64];
    __shared__ float factor[WAVES][16];
    __shared__ __attribute__((aligned(16))) Frag<T> lds_q[kLdsQ ? WAVES : 1][kLdsQ ? kLdsQ : 1][kLdsQ ? 64 : 1];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = w & 1;
    const int group = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    Scan sq = scan_tiles(a, 0, lane);
    int total = sq.all();
    for (int b = 64; b < a.Nb; b += 64) total += scan_tiles(a, b, lane).all();
    const int per = part_tiles(a, total);
    int at = part * per;                                         // next tile of the list
    const int end = total - at < per ? total : at + per;
    if (at >= total) return;
    const int M = a.Tq * a.H;
    const float c = a.scale * kLog2e;
    const int ps = a.page_shift;

    int b0 = 0, before = 0;                                      // sq's first sequence, tiles before it
    while (at < end) {
        while (at >= before + sq.all()) {
            before += sq.all();
            b0 += 64;
            sq = scan_tiles(a, b0, lane);
        }
        const int l = __ffsll((unsigned long long)__ballot(before + sq.sum > at)) - 1;
        const int b = b0 + l;
        const int tiles = __builtin_amdgcn_readlane(sq.cnt, l), len = __builtin_amdgcn_readlane(sq.len, l);
        const int rows = __builtin_amdgcn_readlane(sq.rows, l);
        const int first = before + __builtin_amdgcn_readlane(sq.sum, l) - tiles;    // the sequence's place in the list
        const int t0 = at - first, t1 = end - first < tiles ? end - first : tiles;
        at = first + t1;
        if (t0 == 0 && group == 0 && w == 0 && lane == 0 && len > rows) atomicAdd(a.status, 1u);

        // queries: row 16 WAVES group + 16 w + n of the (token, head) pairs
        const int row = (group * WAVES + w) * 16 + (lane & 15), mrow = row < M ? row : M - 1;
        const int tok = mrow / a.H, head = mrow - tok * a.H;
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h + 8 * (lane >> 4);
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h + 8 * (lane >> 4);
        auto load_q = [&](int s) { return s < DC / 32 ? load8(qlp + 32 * s) : load8(qrp + 32 * s - DC); };
        f32x4 acc[2][ND];                                         // of this wave's rows, of the other wave's
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[0][d] = acc[1][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, lsum = 0.f;

        // A tile: which of its halves exist, where they lie, whether all its rows do
        struct Tile {
            int have;
            bool whole;
            const char *lo, *hi;
        };
        // Page table entries of 64 pages, one per lane; -1 for no such page or one
        // past the rows. A tile's halves lie in one page or, where pages have
        // 16 rows, in an even one and the next: of the same 64.
        const int32_t* table = a.table + (int64_t)b * a.max_pages;
        int pbase = -64, pages = 0;
        auto entry = [&](int p) {
            const int i = p + lane;
            return i < a.max_pages && (int64_t)i << ps < rows ? table[i] : 0;
        };
        auto keep = [&](int p, int e) {
            pbase = p;
            const int64_t r = (int64_t)(p + lane) << ps;
            if (e < 0 || e >= a.n_pages) e = -1;
            // counted once: where the page's first row is this part's
            const uint64_t bad = __ballot(e < 0 && r >= t0 * kTile && r < (int64_t)t1 * kTile);
            if (bad && group == 0 && w == 0 && lane == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
            pages = r < rows ? e : -1;
        };
        // the first entries and the queries are under way together
        const int p0 = t0 * kTile >> ps, e = entry(p0);
        Frag<T> qf[kKeepQ ? NS : 1];
        if constexpr (kKeepQ) {
#pragma unroll
            for (int s = 0; s < NS; ++s) qf[s] = load_q(s);
        }
        keep(p0, e);
        auto find = [&](int t) {
            const int k0 = t * kTile, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            const int e0 = __builtin_amdgcn_readlane(pages, p - pbase);
            const int e1 = __builtin_amdgcn_readlane(pages, ((k0 + 16) >> ps) - pbase);
            const int mask = (1 << ps) - 1;
            Tile x;
            x.have = (e0 >= 0 ? 1 : 0) | (e1 >= 0 ? 2 : 0);
            x.whole = x.have == 3 && k0 + kTile <= rows;
            // (a missing page's address is not used)
            x.lo = static_cast<const char*>(a.cache) + (((int64_t)e0 << ps) + (k0 & mask)) * (RC * 16);
            x.hi = static_cast<const char*>(a.cache) + (((int64_t)e1 << ps) + ((k0 + 16) & mask)) * (RC * 16);
            return x;
        };
        auto load_edge = [&](const Tile& x, int t, char* to) {
            const int rmax = rows - 1 - t * kTile;
            load_edge_tile<T, RC, WAVES>(to, x.lo, x.hi, rmax < kTile - 1 ? rmax : kTile - 1, x.have, w, lane);
        };
        constexpr int kLoads = tile_loads<T, RC, WAVES>();
        auto load_whole = [&](const Tile& x, char* to) {
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // addresses are formed here, not kept in registers
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_of_tile<T, RC, WAVES>(i, true, to, x.lo, x.hi, w, ln);
        };
        Tile next = find(t0);
        if (next.whole) load_whole(next, smem[0]);
        else load_edge(next, t0, smem[0]);
        int have = next.have;
        if constexpr (kKeepQ) {
#pragma unroll
            for (int s = 0; s < kLdsQ; ++s) lds_q[w][s][lane] = qf[s];
        }
        wait_loads_and_lds();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const char* buf = smem[(t - t0) & 1];
            char* const to = smem[(t + 1 - t0) & 1];
            next.whole = false;
            if (t + 1 < t1) {
                next = find(t + 1);
                if (!next.whole) load_edge(next, t + 1, to);
                else if (!kSpread) load_whole(next, to);
            }
            // LDS addresses are formed anew for each tile: kept over the loop,
            // they push operands out of the registers
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4;
            f32x4 sc[2], odd[2];                                  // 16 keys each, in two chains
#pragma unroll
            for (int q = 0; q < 2; ++q) sc[q] = odd[q] = f32x4{0.f, 0.f, 0.f, 0.f};
            {
                // operands in the order of their use: for the steps whose
                // queries are in LDS, these and the two blocks of keys, for
                // the others the keys
                Frag<T> q;
                auto keys = [&](int s, int h) { return read_rows16<T, RC>(buf, 16 * h + (ln & 15), s, g); };
                auto read = [&](int i) -> Frag<T> {
                    if (i < 3 * kLdsQ) return i % 3 == 0 ? lds_q[w][kLdsQ ? i / 3 : 0][ln] : keys(i / 3, i % 3 - 1);
                    return keys((i - kLdsQ) / 2, (i - kLdsQ) % 2);
                };
                ReadAhead<T, 2 * NS + kLdsQ, 6> ahead;
                ahead.start(read);
                ahead.template run<1, 1>(read, [&](int i, const Frag<T>& x) {
                    if (i < 3 * kLdsQ && i % 3 == 0) {
                        q = x;
                        return;
                    }
                    const int s = i < 3 * kLdsQ ? i / 3 : (i - kLdsQ) / 2;
                    const int h = i < 3 * kLdsQ ? i % 3 - 1 : (i - kLdsQ) % 2;
                    if (i >= 3 * kLdsQ && h == 0) q = kKeepQ ? qf[kKeepQ ? s : 0] : load_q(s);
                    f32x4& y = s % 2 ? odd[h] : sc[h];
                    y = mma16(x, q, y);
                    if constexpr (kSpread) {              // load l behind product l kProducts / kLoads
                        constexpr int kProducts = 2 * NS;
                        static_assert(kLoads <= kProducts, "one a product");
                        const int n = 2 * s + h, l = (n * kLoads + kProducts - 1) / kProducts;
                        if (l < ((n + 1) * kLoads + kProducts - 1) / kProducts)
                            load_of_tile<T, RC, WAVES>(l, next.whole, to, next.lo, next.hi, w, ln);
                    }
                }, [](int i) { return i >= 3 * kLdsQ || i % 3 != 0; });
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[q][r] += odd[q][r];
            // keys that this lane's token sees in the tile: the first lim + 1
            const int k0 = t * kTile;
            if (k0 + kTile > len - a.Tq + 1 || k0 + kTile > rows || have != 3) {
                const int last = len - a.Tq + tok < rows - 1 ? len - a.Tq + tok : rows - 1, lim = last - k0 - 4 * g;
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        sc[q][r] = 16 * q + r > lim || !(have >> q & 1) ? -INFINITY : sc[q][r];
            }
            float mx = sc[0][0];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, sc[q][r]);
            mx = group_max(mx);
            // The running maximum moves only when it grows by more than 2^8
            // (from -inf at first): until then its terms reach at most 2^8,
            // exact enough in float32, and the output needs no rescaling (the
            // published conditional rescaling of the online softmax).
            float al = 1.f;
            if ((mx - m) * c > 8.f) {
                al = __builtin_amdgcn_exp2f((m - mx) * c);
                lsum *= al;
                m = mx;
            }
            const float mc = m == -INFINITY ? 0.f : m * c;        // nothing seen yet: all terms are 0
            Frag<T> pf;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[q][r], c, -mc));
                    lsum += p;
                    pf[4 * q + r] = (T)p;      // bf16: the one rounding of the probabilities, as operands
                }
            probs[w][ln] = pf;
            if (g == 0) factor[w][ln] = al;
            wait_lds();
            wg_barrier();
            auto read = [&](int i) {
                return read_cols16<T, RC>(buf + half * (DC / 2) * sizeof(T), 16 * i, ln);
            };
            ReadAhead<T, ND, 4> ahead;
            ahead.start(read);
            const Frag<T> po = probs[w ^ 1][ln];
            const float ao = factor[w ^ 1][ln & 15];
            if (__any(al != 1.f || ao != 1.f)) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[0][d][r] *= al;
                        acc[1][d][r] *= ao;
                    }
            }
            ahead.template run<2>(read, [&](int i, const Frag<T>& x) {
                acc[0][i] = mma16(x, pf, acc[0][i]);
                acc[1][i] = mma16(x, po, acc[1][i]);
            });
            have = next.have;
            wait_loads_and_lds();
            wg_barrier();
        }
        const float lt = group_sum(lsum);
        int ln = lane;                                            // the same here
        asm volatile("" : "+v"(ln));
        const int g = ln >> 4, r0 = (group * WAVES + w) * 16 + (ln & 15), r1 = r0 + (half ? -16 : 16);
        if (t0 == 0 && t1 == tiles) {
            const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;   // no visible key: 0; NaN stays NaN
            if (g == 0) factor[w][ln] = inv;
            wait_lds();
            wg_barrier();
            const float io = factor[w ^ 1][ln & 15];
            T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC + half * (DC / 2) + 4 * g;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                if (r0 < M) store4(op + (int64_t)r0 * DC + 16 * d, acc[0][d], inv);
                if (r1 < M) store4(op + (int64_t)r1 * DC + 16 * d, acc[1][d], io);
            }
            if (a.lse && r0 < M && g == 0)
                a.lse[(int64_t)b * M + r0] =
                    lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
            wait_lds();
            wg_barrier();                                         // the next sequence writes factor again
        } else {
            const int j = t0 > 0 ? 0 : 1;
            float* p = partial(a, group, part, j, 16 * w + (ln & 15));
            float* x = partial(a, group, part, j, 16 * (w ^ 1) + (ln & 15));
            if (g == 0) {
                p[0] = m * c;
                p[1] = lt;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                store4(p + 4 + half * (DC / 2) + 16 * d + 4 * g, acc[0][d], 1.f);
                store4(x + 4 + half * (DC / 2) + 16 * d + 4 * g, acc[1][d], 1.f);
            }
        }
    }
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
template <int DC>
__device__ __forceinline__ void join_row(const MlaStepArgs& a, int row, int p0, int p1, int at, int step, int lane,
                                         f32x4 (&s)[DC / 256], float& m, float& l) {
    const int group = row / (16 * a.waves), r = row % (16 * a.waves);
    float pm[kMaxParts / 64], pl[kMaxParts / 64];        // all under way together
#pragma unroll
    for (int k = 0; k < kMaxParts / 64; ++k) {
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
    for (int k = 1; k < kMaxParts / 64; ++k) m = fmaxf(m, pm[k]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float ms = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxParts / 64; ++k) l += pl[k] * __builtin_amdgcn_exp2f(pm[k] - ms);
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
template <class T, int DC> __global__ __launch_bounds__(256) void mla_step_join_kernel(MlaStepArgs a, int blocks) {
    __shared__ __attribute__((aligned(16))) float sums[4][DC];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int M = a.Tq * a.H, b = blockIdx.x / blocks, row0 = blockIdx.x % blocks * a.join_rows;
    const int row1 = row0 + a.join_rows < M ? row0 + a.join_rows : M;
    int first = 0, total = 0, tiles = 0;
    for (int b0 = 0; b0 < a.Nb; b0 += 64) {
        const Scan sq = scan_tiles(a, b0, lane);
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
            join_row<DC>(a, row, p0, p1, 0, 1, lane, s, m, l);
            const float inv = inverse();
#pragma unroll
            for (int v = 0; v < DC / 256; ++v) store4(op + (int64_t)row * DC + 256 * v + 4 * lane, s[v], inv);
            if (lane == 0) put_lse(row);
        }
        return;
    }
    for (int row = row0; row < row1; ++row) {
        join_row<DC>(a, row, p0, p1, w, 4, lane, s, m, l);
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

// One thread per 16-byte chunk of a new token. Bound by HBM, few tokens by the
// launch: 28000 tokens of 1152 bytes (65 MB read and written) 14-15.7 us, 4.1-4.6
// TB/s (a plain copy: 4.8); 128 tokens 3 us.
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
    if (a.waves == 2) mla_step_kernel<T, DC, DR, 2><<<grid, 128, 0, s>>>(a);
    else if (a.waves == 4) mla_step_kernel<T, DC, DR, 4><<<grid, 256, 0, s>>>(a);
    else if (a.waves == 6) mla_step_kernel<T, DC, DR, 6><<<grid, 384, 0, s>>>(a);
    else if constexpr (max_waves<T, DC>() > 6) mla_step_kernel<T, DC, DR, 8><<<grid, 512, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int blocks = (a.Tq * a.H + a.join_rows - 1) / a.join_rows;
    mla_step_join_kernel<T, DC><<<dim3((unsigned)((int64_t)a.Nb * blocks)), 256, 0, s>>>(a, blocks);
    return hipGetLastError();
}
template <class T> hipError_t launch_dims(const MlaStepArgs& a, hipStream_t s) {
    if (a.Dc == 512) return a.Dr ? launch<T, 512, 64>(a, s) : launch<T, 512, 0>(a, s);
    return a.Dr ? launch<T, 256, 64>(a, s) : launch<T, 256, 0>(a, s);
}

}  // namespace

// The split over workgroups. The blocks of 32 rows of queries are spread evenly
// over as few groups as hold them, two waves a block: every group reads the
// cache. A cache so short that there is a compute unit for each tile and group
// gets more of them, as time is then what one tile and its results take (32
// tiles, 96 heads: 11.2 us in three groups, 14.9 in one; a cache of 3126 tiles
// would be read three times).
size_t mla_step_plan(MlaStepArgs& a) {
    const int64_t rows = (int64_t)a.Tq * a.H, blocks = (rows + 31) / 32;
    const int64_t most = (int64_t)a.Nb * ((((int64_t)a.max_pages << a.page_shift) + kTile - 1) / kTile);
    const int most_blocks = (!a.bf16 && a.Dc == 512 ? max_waves<float, 512>() : 8) / 2;
    int64_t per = most_blocks;                                    // blocks a workgroup
    while (per > 1 && (blocks + per - 2) / (per - 1) * most <= 256) --per;
    a.groups = (int32_t)((blocks + per - 1) / per);
    a.waves = (int32_t)((blocks + a.groups - 1) / a.groups) * 2;
    int64_t parts = kMaxParts / a.groups;
    if (parts < 32) parts = 32;
    if (parts > most) parts = most;
    a.parts = (int32_t)(parts > 1 ? parts : 1);
    // the join: about 1024 workgroups, most of which find nothing to join
    const int64_t j = (a.Nb * rows + 1023) / 1024;
    a.join_rows = (int32_t)(j < rows ? j : rows);
    return (size_t)a.groups * a.parts * 2 * (16 * a.waves) * (a.Dc + 4) * sizeof(float);
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
