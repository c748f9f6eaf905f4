// The attention weight that cached rows gather: w_j = decay w_j + sum over the
// rows of queries (token, head) of exp(s_ij - lse_i), s as in mla_step.hip.
#include "mla_mx_tile.hpp"

namespace kda {
namespace {

// float32. A wave holds 32 cache rows (keys), a lane a half of one, as the first
// operand of 32x32 tiles of the matrix instructions, and meets all rows of queries
// that its workgroup keeps in LDS: no exchange between waves, and each cache row is
// read from memory once (and from the caches for every further 32 rows of queries).
// Scores come out with a lane holding one query and 16 keys, so that a key's weight
// is a sum down a register, over the lanes at the very end.
// 32 sequences of 4096, 96 heads, 512 + 64 channels: 189 us over the 4-bit cache (206
// with the keys held in registers, where they spill), 203 over float32 rows; products
// at 72 TFLOP/s, one chain of them a wave.
constexpr int kUnit = 32 * kWaves;
constexpr int kQueries = 64;    // rows of queries in LDS at a time, at most

// Columns in the order of the products: step st multiplies, in half hf of the
// lanes, the 8 channels from 64 (st / 4) + 8 (st % 4) + 32 hf, so that a lane's
// part of four steps is one block of 32 of the 4-bit cache.
template <int RC> __device__ __forceinline__ f32x8 read_query(const char* lds, int r, int st, int hf) {
    const char* p = lds + r * (RC * 16);
    const int sw = swizzle<RC>(r), k = 8 * (st / 4) + st % 4;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(2 * k, 8 * hf, sw));
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(2 * k, 8 * hf + 1, sw));
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// A lane's key, read from global memory (zeros where it does not exist).
template <int DC, bool MX> struct Key {
    const char* row;            // rows of float32: the row; 4 bits: its codes
    const char* scales;
    const char* rope;
    bool have;

    __device__ __forceinline__ f32x8 operand(int st, int hf) const {
        if (!have) return f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int c = 64 * (st / 4) + 8 * (st % 4) + 32 * hf;
        if constexpr (!MX) return load8(reinterpret_cast<const float*>(row) + c);
        if (st >= DC / 16) return load8(reinterpret_cast<const float*>(rope) + (c - DC));
        return MxScale(*reinterpret_cast<const uint8_t*>(scales + c / 32)).f32(*reinterpret_cast<const uint32_t*>(row + c / 2));
    }
};

template <int DC, int DR, bool MX>
__global__ __launch_bounds__(64 * kWaves, 2) void mla_weigh_f32_kernel(MlaWeighArgs x, int chunk, int parts) {
    using T = float;
    constexpr int D = DC + DR, RC = D / kChunk<T>, NS = D / 16;
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

        Key<DC, MX> k;
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
                int half = hf;
                // keys of 512 channels are read again for every 32 rows: they do not fit the registers
                if constexpr (DC == 512) asm volatile("" : "+v"(half));
#pragma unroll
                for (int st = 0; st < NS; ++st) s = mma(k.operand(st, half), read_query<RC>(smem, r0 + n, st, half), s);
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

// bf16. Tiles of 64 keys come to LDS, the next one under way while one is at work
// (of 4 bits as they are: the scores run on the codes). A wave takes the rows of
// queries by sets of 16, whose operands it holds in registers: of up to eight sets
// one each for as long as the sequence lasts (where there are fewer, two or four
// waves share a set's keys: 32 sequences of 8192, 12 rows 26 us against 37 by one,
// bf16 rows 51 against 65; 48 rows 39 and 38, 59 and 67), of more each wave takes every eighth in turn. A lane
// holds one row of queries and four keys of a group of 16, so that weights sum up in
// registers, over the 16 lanes of a group at the tile's end, over the waves through
// LDS. The order of all sums goes by the sizes alone.
// 128 sequences of 4096 to 8192 bf16 rows, 96 heads: 215 us, the rows at 4.2 TB/s,
// 89% of a copy's rate. 24 tokens of 96 heads over the 4-bit cache, 26 000 keys:
// 73 us, 940 TFLOP/s, matrix cores 57% busy; with one tile a turn, where all
// queries came from the L2 cache for each, 87.
constexpr int kSets = 8;                                          // sets that stay in registers, one a wave

// A set's operands. For many sets over 4-bit keys they are split (mla_mx.hpp) once
// for the whole call, by the kernel below, and lie in the workspace in the order of the lanes.
template <int DC, int DR> constexpr int kSetBytes = DC / 128 * 4096 + 256 + DR / 32 * 1024;
template <int DC, int DR, bool MX> struct Queries {
    static constexpr int NM = DC / 128, NS = DR / 32;
    MxQuery16 qm[MX ? NM : 1];
    uint32_t qs;
    bf16x8 qf[MX ? (NS ? NS : 1) : (DC + DR) / 32];
    float z;                                                      // the row's lse / log 2
    int last;                                                     // the last key that it sees, -1 behind the last row

    __device__ __forceinline__ void row(const MlaWeighArgs& x, int b, int set, int lane, int len, int rows) {
        const MlaStepArgs& a = x.s;
        const int M = a.Tq * a.H, m = 16 * set + (lane & 15), mm = m < M ? m : M - 1;
        z = x.lse[(int64_t)b * M + mm] * kLog2e;
        const int see = len - a.Tq + mm / a.H;
        last = m >= M ? -1 : see < rows - 1 ? see : rows - 1;
    }
    __device__ __forceinline__ void load(const MlaStepArgs& a, int b, int set, int lane) {
        const int M = a.Tq * a.H, m = 16 * set + (lane & 15), mm = m < M ? m : M - 1, g = lane >> 4;
        const int tok = mm / a.H, head = mm - tok * a.H;
        const __bf16* ql = static_cast<const __bf16*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h;
        const __bf16* qr = static_cast<const __bf16*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h;
        if constexpr (MX) {
            bf16x8 q[NM][4];
#pragma unroll
            for (int s = 0; s < NM; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[s][i] = load8(ql + 32 * (NM * ((g >> 1) + 2 * (i >> 1)) + s) + 16 * (g & 1) + 8 * (i & 1));
#pragma unroll
            for (int s = 0; s < NS; ++s) qf[s] = load8(qr + 32 * s + 8 * g);
            qs = 0;
#pragma unroll
            for (int s = 0; s < NM; ++s) {
                qm[s].set(q[s], lane);
                qs |= qm[s].s << 8 * s;
            }
        } else {
#pragma unroll
            for (int s = 0; s < (DC + DR) / 32; ++s) qf[s] = s < DC / 32 ? load8(ql + 32 * s + 8 * g) : load8(qr + 32 * s - DC + 8 * g);
        }
    }
    // split ones from and to the workspace
    __device__ __forceinline__ void load_split(const char* p, int lane) {
#pragma unroll
        for (int s = 0; s < NM; ++s) {
            const char* const f = p + s * 4096 + lane * 16;
            const u32x4 h0 = *reinterpret_cast<const u32x4*>(f), h1 = *reinterpret_cast<const u32x4*>(f + 1024);
            const u32x4 l0 = *reinterpret_cast<const u32x4*>(f + 2048), l1 = *reinterpret_cast<const u32x4*>(f + 3 * 1024);
            qm[s].hi = i32x8{(int)h0[0], (int)h0[1], (int)h0[2], (int)h0[3], (int)h1[0], (int)h1[1], (int)h1[2], (int)h1[3]};
            qm[s].lo = i32x8{(int)l0[0], (int)l0[1], (int)l0[2], (int)l0[3], (int)l1[0], (int)l1[1], (int)l1[2], (int)l1[3]};
        }
        qs = *reinterpret_cast<const uint32_t*>(p + NM * 4096 + lane * 4);
#pragma unroll
        for (int s = 0; s < NS; ++s) qf[s] = *reinterpret_cast<const bf16x8*>(p + NM * 4096 + 256 + s * 1024 + lane * 16);
    }
    __device__ __forceinline__ void store_split(char* p, int lane) const {
#pragma unroll
        for (int s = 0; s < NM; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                char* const f = p + s * 4096 + i * 1024 + lane * 16;
                *reinterpret_cast<u32x4*>(f) = u32x4{(uint32_t)qm[s].hi[4 * i], (uint32_t)qm[s].hi[4 * i + 1],
                                                     (uint32_t)qm[s].hi[4 * i + 2], (uint32_t)qm[s].hi[4 * i + 3]};
                *reinterpret_cast<u32x4*>(f + 2048) = u32x4{(uint32_t)qm[s].lo[4 * i], (uint32_t)qm[s].lo[4 * i + 1],
                                                            (uint32_t)qm[s].lo[4 * i + 2], (uint32_t)qm[s].lo[4 * i + 3]};
            }
        *reinterpret_cast<uint32_t*>(p + NM * 4096 + lane * 4) = qs;
#pragma unroll
        for (int s = 0; s < NS; ++s) *reinterpret_cast<bf16x8*>(p + NM * 4096 + 256 + s * 1024 + lane * 16) = qf[s];
    }
};
template <int DC, int DR> __global__ __launch_bounds__(256) void mla_split_queries_kernel(MlaWeighArgs x, int sets, int64_t all) {
    const int lane = threadIdx.x & 63;
    const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= all) return;
    Queries<DC, DR, true> q;
    q.load(x.s, (int)(i / sets), (int)(i % sets), lane);
    q.store_split(x.split + i * kSetBytes<DC, DR>, lane);
}

// A tile of rows of bf16 (mx_fetch is the 4-bit one; the same arguments)
template <int RC>
__device__ __forceinline__ int rows_fetch(char* to, const char* cache, int pages, uint64_t exist, int pbase, int ps, int k0,
                                          int rows, int w, int lane) {
    constexpr int kInstr = 16 * RC / 64;                          // of 1 KB a quarter of 16 rows
    const int quarter = w & 3, j0 = w >> 2;
    int have = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) have |= (int)(exist >> (((k0 + 16 * q) >> ps) - pbase) & 1) << q;
    const int kq = k0 + 16 * quarter, row = kq & ((1 << ps) - 1);
    const int64_t page = __builtin_amdgcn_readlane(pages, (kq >> ps) - pbase);
    const char* const from = cache + ((page << ps) + row) * (RC * 16);       // (a missing page's is not used)
    char* const at = to + quarter * (RC * 256);
    const bool whole = have == 15 && k0 + kRows <= rows;
    const int left = have >> quarter & 1 ? rows - kq : 0;         // rows of the quarter to be read
    int ln = lane;
    asm volatile("" : "+v"(ln));                                  // offsets are formed here, not kept in registers
#pragma unroll
    for (int i = 0; i < kInstr / 2; ++i) {
        const int j = j0 + 2 * i, r = (j * 64 + ln) / RC, off = ((j * 64 + ln) ^ swizzle16<__bf16, RC>(r)) * 16;
        if (whole) load_lds16s(from, off, at + j * 1024);
        else *reinterpret_cast<u32x4*>(at + j * 1024 + ln * 16) =
                r < left ? *reinterpret_cast<const u32x4*>(from + off) : u32x4{0, 0, 0, 0};
    }
    return have;
}

// over the 16 lanes of a row
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0xB1, 0xf, 0xf, true));       // lane ^ 1
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x4E, 0xf, 0xf, true));       // lane ^ 2
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 0xf, 0xf, true));      // 7 - lane % 8
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 0xf, 0xf, true));      // 15 - lane
    return v;
}

// KS waves a set; MANY: more sets than waves (KS = 1)
template <int DC, int DR, bool MX, int KS, bool MANY>
__global__ __launch_bounds__(64 * kWaves, 2) void mla_weigh_bf16_kernel(MlaWeighArgs x, int parts) {
    using Raw = RawTile<DC, DR>;
    // tiles a turn: queries that pass by meet two, where LDS holds two more
    constexpr int RC = (DC + DR) / 8, NG = 4 / KS, KT = MANY && MX ? 2 : 1, kBytes = MX ? Raw::kBytes : kRows * RC * 16;
    __shared__ __attribute__((aligned(1024))) char tile[2][KT][kBytes];
    __shared__ __attribute__((aligned(16))) float sums[2][kWaves / KS][KT][kRows];
    const MlaStepArgs& a = x.s;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = w % KS, slot = w / KS, ps = a.page_shift, sets = (a.Tq * a.H + 15) / 16;
    const float c = a.scale * kLog2e;
    const int64_t page_bytes = (int64_t)mx_row_bytes(DC, DR, 2) << ps;

    Scan sq = scan_tiles<kRows>(a, 0, lane);
    int total = sq.all();
    for (int b = 64; b < a.Nb; b += 64) total += scan_tiles<kRows>(a, b, lane).all();
    const int per = (int)(((unsigned)total + (unsigned)parts - 1) / (unsigned)parts);
    int at = (int)blockIdx.x * per;
    if (at >= total) return;
    const int end = total - at < per ? total : at + per;
    int b0 = 0, before = 0;
    while (at < end) {
        while (at >= before + sq.all()) {
            before += sq.all();
            b0 += 64;
            sq = scan_tiles<kRows>(a, b0, lane);
        }
        const int l = __ffsll((unsigned long long)__ballot(before + sq.sum > at)) - 1;
        const int b = b0 + l;
        const int tiles = __builtin_amdgcn_readlane(sq.cnt, l), len = __builtin_amdgcn_readlane(sq.len, l);
        const int rows = __builtin_amdgcn_readlane(sq.rows, l);
        const int first = before + __builtin_amdgcn_readlane(sq.sum, l) - tiles;    // the sequence's place in the list
        const int t0 = at - first, t1 = end - first < tiles ? end - first : tiles;
        at = first + t1;
        if (t0 == 0 && threadIdx.x == 0 && len > rows) atomicAdd(a.status, 1u);

        // page table entries of 64 pages, as in mla_step_mx.hip
        const int32_t* table = a.table + (int64_t)b * a.max_pages;
        int pbase = -64, pages = 0;
        uint64_t exist = 0;
        auto entry = [&](int p) {
            const int i = p + lane;
            return i < a.max_pages && (int64_t)i << ps < rows ? table[i] : 0;
        };
        auto keep = [&](int p, int e) {
            pbase = p;
            const int64_t r = (int64_t)(p + lane) << ps;
            if (e < 0 || e >= a.n_pages) e = -1;
            // counted once: where the page's first row is this part's
            const uint64_t bad = __ballot(e < 0 && r >= t0 * kRows && r < (int64_t)t1 * kRows && r < rows);
            if (bad && threadIdx.x == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
            pages = r < rows ? e : -1;
            exist = __ballot(pages >= 0);
        };
        auto fetch = [&](int t, char* to) {
            const int k0 = t * kRows, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            if constexpr (MX)
                return mx_fetch<DC, DR>(to, static_cast<const char*>(a.cache), page_bytes, pages, exist, pbase, ps, k0, rows, w, lane);
            else return rows_fetch<RC>(to, static_cast<const char*>(a.cache), pages, exist, pbase, ps, k0, rows, w, lane);
        };
        const int p0 = t0 * kRows >> ps;
        keep(p0, entry(p0));
        int have[KT], next[KT];
        auto fetch_turn = [&](int t, char (*to)[kBytes], int (&h)[KT]) {
#pragma unroll
            for (int j = 0; j < KT; ++j) h[j] = t + j < t1 ? fetch(t + j, to[j]) : 0;
        };
        fetch_turn(t0, tile[0], have);
        Queries<DC, DR, MX> q[MANY && KT == 1 ? 2 : 1];
        auto load = [&](Queries<DC, DR, MX>& y, int set) {
            if (set >= sets) return;
            y.row(x, b, set, lane, len, rows);
            if constexpr (MX && MANY) y.load_split(x.split + ((int64_t)b * sets + set) * kSetBytes<DC, DR>, lane);
            else y.load(a, b, set, lane);
        };
        if constexpr (!MANY) load(q[0], slot);
        wait_loads_and_lds();
        wg_barrier();
        for (int t = t0, i = 0; t < t1; t += KT, i ^= 1) {
            const int k0 = t * kRows;
            fetch_turn(t + KT, tile[i ^ 1], next);
            // the waves that write the weights read the old ones now
            const int mine = kWaves - 1 - w, key = k0 + kRows * mine + lane;
            const bool writes = mine < KT && t + mine < t1 && key < rows;
            const int64_t at_key = ((int64_t)b * a.max_pages << ps) + key;
            float old = 0.f;
            if (writes && x.decay != 0.f && key < len - x.fresh) old = x.decay * x.w_in[at_key];
            float sum[KT][NG][4];
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int h = 0; h < NG; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum[j][h][r] = 0.f;
            // all rows see all keys of a turn but at its sequence's end
            const bool edge = k0 + KT * kRows > len - a.Tq + 1 || k0 + KT * kRows > rows || have[0] != 15 || have[KT - 1] != 15;
            auto add = [&](const Queries<DC, DR, MX>& y, bool tail) {
                const int key0 = 16 * NG * kg;
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    if (j > 0 && t + j >= t1) break;
                    const char* const buf = tile[i][j];
                    f32x4 sc[NG];
                    if constexpr (MX) {
                        mx_scores<DC, DR, NG>(buf, key0, lane, y.qm, y.qs, y.qf, sc);
                    } else {
                        int ln = lane;
                        asm volatile("" : "+v"(ln));
#pragma unroll
                        for (int h = 0; h < NG; ++h) sc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < (DC + DR) / 32; ++s)
#pragma unroll
                            for (int h = 0; h < NG; ++h)
                                sc[h] = mma16(read_rows16<__bf16, RC>(buf, key0 + 16 * h + (ln & 15), s, ln >> 4), y.qf[s], sc[h]);
#pragma unroll
                        for (int h = 0; h < NG; ++h) asm volatile("" : "+v"(sc[h]));
                    }
                    settle(sc[0], sc[NG - 1]);
                    if constexpr (NG == 4) settle(sc[1], sc[2]);
                    if (edge || tail) {
                        const int lim = y.last - k0 - kRows * j - key0 - 4 * (lane >> 4);
#pragma unroll
                        for (int h = 0; h < NG; ++h)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                sum[j][h][r] += 16 * h + r <= lim && (have[j] >> (NG * kg + h) & 1)
                                                    ? __builtin_amdgcn_exp2f(__builtin_fmaf(sc[h][r], c, -y.z)) : 0.f;
                    } else {
#pragma unroll
                        for (int h = 0; h < NG; ++h)
#pragma unroll
                            for (int r = 0; r < 4; ++r) sum[j][h][r] += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[h][r], c, -y.z));
                    }
                }
            };
            // (the rows behind the last are in the last set)
            if constexpr (MANY && KT == 1) {
                load(q[0], w);
                for (int s = w; s < sets; s += 2 * kWaves) {
                    load(q[1], s + kWaves);
                    add(q[0], s == sets - 1);
                    if (s + kWaves < sets) {
                        load(q[0], s + 2 * kWaves);
                        add(q[1], s + kWaves == sets - 1);
                    }
                }
            } else if constexpr (MANY) {
                for (int s = w; s < sets; s += kWaves) {
                    load(q[0], s);
                    add(q[0], s == sets - 1);
                }
            } else if (slot < sets) {
                add(q[0], slot == sets - 1);
            }
            if (MANY || slot < sets) {
#pragma unroll
                for (int j = 0; j < KT; ++j)
#pragma unroll
                    for (int h = 0; h < NG; ++h) {
                        f32x4 v;
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = row_sum(sum[j][h][r]);
                        if ((lane & 15) == 0)
                            *reinterpret_cast<f32x4*>(&sums[i][slot][j][16 * (NG * kg + h) + 4 * (lane >> 4)]) = v;
                    }
            }
            wait_loads_and_lds();
            wg_barrier();
            if (writes) {
                const int n = MANY ? kWaves : sets;
                float v = 0.f;
                for (int s = 0; s < n; ++s) v += sums[i][s][mine][lane];
                x.w_out[at_key] = old + v;
            }
#pragma unroll
            for (int j = 0; j < KT; ++j) have[j] = next[j];
        }
        wait_lds();
        wg_barrier();                                             // the next sequence's first tile overwrites a buffer
    }
}

template <int DC, int DR, bool MX> hipError_t launch_weigh_f32(const MlaWeighArgs& x, hipStream_t s) {
    const MlaStepArgs& a = x.s;
    const int M = a.Tq * a.H;
    int chunk = (M + 31) / 32 * 32;
    if (chunk > kQueries) chunk = kQueries;
    const int64_t cap = (int64_t)a.max_pages << a.page_shift, units = a.Nb * ((cap + kUnit - 1) / kUnit);
    const int parts = (int)(units < 256 ? units : 256);
    const int lds = chunk * ((DC + DR) * 4 + 8);
    const void* f = reinterpret_cast<const void*>(&mla_weigh_f32_kernel<DC, DR, MX>);
    if (const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) return e;
    mla_weigh_f32_kernel<DC, DR, MX><<<dim3((unsigned)parts), 64 * kWaves, lds, s>>>(x, chunk, parts);
    return hipGetLastError();
}
template <int DC, int DR, bool MX> hipError_t launch_weigh_bf16(const MlaWeighArgs& x, hipStream_t s) {
    const MlaStepArgs& a = x.s;
    const int sets = (a.Tq * a.H + 15) / 16;
    const int64_t cap = (int64_t)a.max_pages << a.page_shift, units = a.Nb * ((cap + kRows - 1) / kRows);
    const int parts = (int)(units < 256 ? units : 256);           // one a compute unit
    const dim3 grid((unsigned)parts);
    if (sets <= 2) mla_weigh_bf16_kernel<DC, DR, MX, 4, false><<<grid, 64 * kWaves, 0, s>>>(x, parts);
    else if (sets <= 4) mla_weigh_bf16_kernel<DC, DR, MX, 2, false><<<grid, 64 * kWaves, 0, s>>>(x, parts);
    else if (sets <= kSets) mla_weigh_bf16_kernel<DC, DR, MX, 1, false><<<grid, 64 * kWaves, 0, s>>>(x, parts);
    else {
        if constexpr (MX) {
            const int64_t all = (int64_t)a.Nb * sets;
            mla_split_queries_kernel<DC, DR><<<dim3((unsigned)((all + 3) / 4)), 256, 0, s>>>(x, sets, all);
            if (const hipError_t e = hipGetLastError()) return e;
        }
        mla_weigh_bf16_kernel<DC, DR, MX, 1, true><<<grid, 64 * kWaves, 0, s>>>(x, parts);
    }
    return hipGetLastError();
}
template <int DC, int DR> hipError_t launch_weigh(const MlaWeighArgs& x, hipStream_t s) {
    if (x.s.bf16) return x.mx ? launch_weigh_bf16<DC, DR, true>(x, s) : launch_weigh_bf16<DC, DR, false>(x, s);
    return x.mx ? launch_weigh_f32<DC, DR, true>(x, s) : launch_weigh_f32<DC, DR, false>(x, s);
}

}  // namespace

size_t mla_weigh_workspace(const MlaWeighArgs& x) {
    const int64_t sets = ((int64_t)x.s.Tq * x.s.H + 15) / 16;
    if (!x.mx || !x.s.bf16 || sets <= kSets) return 0;
    const int bytes = x.s.Dc == 512 ? (x.s.Dr ? kSetBytes<512, 64> : kSetBytes<512, 0>)
                                    : (x.s.Dr ? kSetBytes<256, 64> : kSetBytes<256, 0>);
    return (size_t)(x.s.Nb * sets) * bytes;
}

hipError_t launch_mla_weigh(const MlaWeighArgs& x, hipStream_t s) {
    if (x.s.Dc == 512) return x.s.Dr ? launch_weigh<512, 64>(x, s) : launch_weigh<512, 0>(x, s);
    return x.s.Dr ? launch_weigh<256, 64>(x, s) : launch_weigh<256, 0>(x, s);
}

}  // namespace kda
