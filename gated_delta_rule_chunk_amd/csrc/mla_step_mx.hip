// Latent attention, absorbed form, over a cache that holds the latents in 4 bits
// (include/kda_mla_cache.h): s = scale (q_latent . c + q_rope . r), p = softmax s,
// o = sum p c.
//
// As in mla_step.hip the tiles of 32 cache rows of all sequences form one list,
// cut into equal parts by the lengths on the device, and a second kernel joins
// the parts. A tile's codes come to registers a tile ahead, 32 channels a
// thread, and are written to LDS as T. Four waves share a block of 32 rows of
// queries: each forms the scores of 16 rows and 16 keys, the two that share
// rows agree on the running maximum, and each multiplies the probabilities of
// all 32 rows with a quarter of the columns. So neither queries, scores nor outputs
// (Dc / 8 registers) take more than a third of a SIMD's registers, and three
// blocks (96 rows) leave each SIMD three waves.
#include "mla_mx.hpp"
#include "mla_step.hpp"

namespace kda {
namespace {

// blocks of 32 rows of queries a workgroup, at most (float32: as queries and outputs fit the registers)
__host__ __device__ constexpr int most_blocks(bool bf16, int dc) { return bf16 ? 3 : dc == 256 ? 2 : 1; }
// two workgroups of one block a compute unit
constexpr int kMostParts = 512;

// Where the parts of a tile as it lies in memory come to in LDS: codes, shared
// parts, scale bytes, each as Q times 16 rows. A row of codes is 16 or 8
// chunks of 16 bytes, one of the shared part 8; chunk c lies at c ^ swz(r).
// The scores' operand reads take, of 16 lanes that LDS serves at a time, 8 rows of
// chunk c and 8 other rows of chunk c ^ 4, c ^ 2 (codes) or c ^ 1 (shared part):
// rows 0-3 and 12-15, and 4-11. Under these permutations each takes every bank once.
template <int DC, int DR, int Q = 2> struct RawTile {
    static constexpr int NB = DC / 32;
    static constexpr int kCodes = 16 * DC / 2, kRope = 16 * DR * 2, kScales = 16 * NB;      // bytes of 16 rows
    static constexpr int kBytes = Q * (kCodes + kRope + 256);
    static constexpr int kCodeLoads = kCodes / 1024, kRopeLoads = kRope / 1024, kLoads = Q * (kCodeLoads + kRopeLoads + 1);
    static __device__ __forceinline__ int swz_codes(int r) {
        if constexpr (NB == 16) return (r & 7) << 1 | ((r >> 3 ^ r >> 2) & 1);
        else return (r >> 1 & 3) << 1 | ((r >> 3 ^ r >> 2) & 1);
    }
    static __device__ __forceinline__ int swz_rope(int r) { return r >> 1 & 7; }
    static __device__ __forceinline__ int codes(int r, int c) { return r * (DC / 2) + ((c ^ swz_codes(r & 15)) << 4); }
    static __device__ __forceinline__ int rope(int r, int c) { return Q * kCodes + r * (DR * 2) + ((c ^ swz_rope(r & 15)) << 4); }
    static __device__ __forceinline__ int scales(int r) { return Q * (kCodes + kRope) + (r >> 4) * 256 + (r & 15) * NB; }

    // Load x of the tile's kLoads: its place in LDS, and where a lane's bytes
    // come from in the page (rows from `row` on): one instruction of 16 bytes a lane, or (scales) 4.
    static __device__ __forceinline__ bool is_scales(int x) { return x / Q >= kCodeLoads + kRopeLoads; }
    static __device__ __forceinline__ int place(int x) {
        const int q = x % Q, j = x / Q;
        if (is_scales(x)) return Q * (kCodes + kRope) + q * 256;
        return j < kCodeLoads ? q * kCodes + j * 1024 : Q * kCodes + q * kRope + (j - kCodeLoads) * 1024;
    }
    // its plane's offset in a page, bytes of a row there
    static __device__ __forceinline__ int64_t plane(int x, int ps) {
        const int j = x / Q;
        return is_scales(x) ? ((int64_t)DC / 2) << ps : j < kCodeLoads ? 0 : ((int64_t)DC / 2 + NB) << ps;
    }
    static __device__ __forceinline__ int row_bytes(int x) { return is_scales(x) ? NB : x / Q < kCodeLoads ? DC / 2 : DR * 2; }
    // row (of the 16) and byte offset from its first row of a lane's part
    static __device__ __forceinline__ void source(int x, int lane, int& r, int& off) {
        const int j = x / Q;
        if (is_scales(x)) {
            r = lane / (NB / 4);
            off = lane * 4;
        } else if (j < kCodeLoads) {
            const int p = j * 64 + lane;
            r = p / NB;
            off = r * (DC / 2) + (((p % NB) ^ swz_codes(r)) << 4);
        } else {
            const int p = (j - kCodeLoads) * 64 + lane;
            r = p / 8;
            off = r * 128 + (((p % 8) ^ swz_rope(r)) << 4);
        }
    }
};

// bf16. A tile goes from memory to LDS as it is; there the scores read the codes,
// as operands of the scaled matrix instructions, and every thread turns a block of
// 32 channels into bf16, for the outputs, once for all rows of queries. While a
// tile's scores are formed the outputs of the one before are, so that between two
// barriers there is always work for the matrix cores; the next tile loads
// meanwhile.
template <int DC, int DR, int RB>
__global__ __launch_bounds__(256 * RB, RB == 3 ? 3 : 2) void mla_mx_step_bf16_kernel(MlaStepArgs a) {
    using T = __bf16;
    using Raw = RawTile<DC, DR>;
    constexpr int ND = DC / 64, NT = 256 * RB, NB = DC / 32, NM = DC / 128, NS = DR / 32;
    // one block: latents as bf16 once only, so that more workgroups fit a compute unit and cover each other's waits
    constexpr int kWide = RB == 1 ? 1 : 2;
    __shared__ __attribute__((aligned(1024))) char raw[2][Raw::kBytes];
    __shared__ __attribute__((aligned(1024))) char wide[kWide][kTile * DC * 2];
    __shared__ __attribute__((aligned(32))) T probs[RB][2][64][8];
    __shared__ float tops[RB][2][2][16], factor[RB][2][16];
    constexpr int kAhead = 2;                                 // operands of the outputs under way
    // three waves a SIMD: of 512 channels the last steps' lo do not fit the registers
    constexpr int kLdsQ = RB == 3 && DC == 512 ? 1 : 0;
    __shared__ __attribute__((aligned(16))) bf16x8 lds_qf[kLdsQ ? 2 * RB : 1][kLdsQ && NS ? NS : 1][kLdsQ && NS ? 64 : 1];
    __shared__ __attribute__((aligned(16))) u32x4 lds_q[kLdsQ ? 2 * RB : 1][kLdsQ ? kLdsQ : 1][2][kLdsQ ? 64 : 1];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rb = w >> 2, quarter = w & 3, rh = w & 1, kh = quarter >> 1;
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
    const int64_t page_bytes = (int64_t)mx_row_bytes(DC, DR, sizeof(T)) << ps;

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
        if (t0 == 0 && group == 0 && tid == 0 && len > rows) atomicAdd(a.status, 1u);

        // queries: row 32 (RB group + rb) + 16 rh + n of the (token, head) pairs
        const int mrow = min(((group * RB + rb) * 2 + rh) * 16 + (lane & 15), M - 1);
        const int tok = mrow / a.H, head = mrow - tok * a.H;
        const int last = min(len - a.Tq + tok, rows - 1);         // the last key that this lane's token sees
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h;
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
            if (bad && group == 0 && tid == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
            pages = r < rows ? e : -1;
        };
        // the first entries and the queries are under way together
        const int p0 = t0 * kTile >> ps, e = entry(p0);
        // step s multiplies the blocks s, s + NM, s + 2 NM and s + 3 NM
        MxQuery16 qm[NM];
        uint32_t qs = 0;                                          // their scale bytes
#pragma unroll
        for (int s = 0; s < NM; ++s) {
            bf16x8 x[4];
            const int g = lane >> 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = load8(qlp + 32 * (NM * ((g >> 1) + 2 * (i >> 1)) + s) + 16 * (g & 1) + 8 * (i & 1));
            qm[s].set(x, lane);
            qs |= qm[s].s << 8 * s;
            __builtin_amdgcn_sched_barrier(0);                    // one after the other: their sources take registers, too
        }
#pragma unroll
        for (int s = NM - kLdsQ; s < NM; ++s)                     // (the waves that share rows write the same)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                lds_q[2 * rb + rh][s - (NM - kLdsQ)][i][lane] =
                    u32x4{(uint32_t)qm[s].lo[4 * i], (uint32_t)qm[s].lo[4 * i + 1], (uint32_t)qm[s].lo[4 * i + 2],
                          (uint32_t)qm[s].lo[4 * i + 3]};
        bf16x8 qf[NS ? NS : 1];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            qf[s] = load8(qrp + 32 * s + 8 * (lane >> 4));
            if constexpr (kLdsQ) lds_qf[2 * rb + rh][s][lane] = qf[s];
        }
        keep(p0, e);

        constexpr int kMine = (Raw::kLoads + 4 * RB - 1) / (4 * RB);                    // loads a wave issues for a tile
        // Sends tile t on its way to LDS; returns which of its halves exist. Rows
        // past the length and of missing pages are zeros there: their weights are
        // 0, but what these multiply has to be finite.
        auto fetch = [&](int t, char* to) {
            const int k0 = t * kTile, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            const int e0 = __builtin_amdgcn_readlane(pages, p - pbase);
            const int e1 = __builtin_amdgcn_readlane(pages, ((k0 + 16) >> ps) - pbase);
            const int mask = (1 << ps) - 1, have = (e0 >= 0 ? 1 : 0) | (e1 >= 0 ? 2 : 0);
            const char* const lo = static_cast<const char*>(a.cache) + e0 * page_bytes;      // (a missing page's is not used)
            const char* const hi = static_cast<const char*>(a.cache) + e1 * page_bytes;
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // offsets are formed here, not kept in registers
            if (have == 3 && k0 + kTile <= rows) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int x = w + 4 * RB * i, q = x & 1;
                    if (Raw::kLoads % (4 * RB) && x >= Raw::kLoads) break;
                    const char* const from = (q ? hi : lo) + Raw::plane(x, ps) + (int64_t)((k0 + 16 * q) & mask) * Raw::row_bytes(x);
                    int r, off;
                    Raw::source(x, ln, r, off);
                    if (!Raw::is_scales(x)) load_lds16s(from, off, to + Raw::place(x));
                    else if (NB == 16 || ln < 32) load_lds4s(from, off, to + Raw::place(x));
                }
                return have;
            }
            for (int x = w; x < Raw::kLoads; x += 4 * RB) {
                const int q = x & 1;
                const char* const from = (q ? hi : lo) + Raw::plane(x, ps) + (int64_t)((k0 + 16 * q) & mask) * Raw::row_bytes(x);
                int r, off;
                Raw::source(x, ln, r, off);
                char* const at = to + Raw::place(x);
                const bool there = (have >> q & 1) && k0 + 16 * q + r < rows;
                if (!Raw::is_scales(x))
                    *reinterpret_cast<u32x4*>(at + 16 * ln) = there ? *reinterpret_cast<const u32x4*>(from + off) : u32x4{0, 0, 0, 0};
                else if (NB == 16 || ln < 32)
                    *reinterpret_cast<uint32_t*>(at + 4 * ln) = there ? *reinterpret_cast<const uint32_t*>(from + off) : 0u;
            }
            return have;
        };
        // A tile's latents as bf16: blocks of 16 columns, 32 rows of 32 bytes each,
        // which the transposing reads take in the order of the lanes. Eight of 16
        // lanes (a row each) write the second half of a row when the others write the first, so that
        // they take all banks.
        auto widen = [&](const char* from, char* to) {
            int td = tid;
            asm volatile("" : "+v"(td));
            const int r = td & 31, odd_half = r >> 3 & 1;
#pragma unroll
            for (int i = 0; i < (kTile * NB + NT - 1) / NT; ++i) {
                const int blk = i * (NT / 32) + (td >> 5);
                if (kTile * NB % NT && blk >= NB) break;
                const u32x4 c = *reinterpret_cast<const u32x4*>(from + Raw::codes(r, blk));
                const MxScale f(*reinterpret_cast<const uint8_t*>(from + Raw::scales(r) + blk));
                char* const at = to + blk * 2048 + r * 32 + 16 * odd_half;
                char* const other = to + blk * 2048 + r * 32 + 16 * (odd_half ^ 1);
                *reinterpret_cast<bf16x8*>(at) = f.bf16(odd_half ? c[1] : c[0]);
                *reinterpret_cast<bf16x8*>(other) = f.bf16(odd_half ? c[0] : c[1]);
                *reinterpret_cast<bf16x8*>(at + 1024) = f.bf16(odd_half ? c[3] : c[2]);
                *reinterpret_cast<bf16x8*>(other + 1024) = f.bf16(odd_half ? c[2] : c[3]);
            }
        };
        f32x4 acc[2][ND];                                         // of the block's two sets of 16 rows
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[0][d] = acc[1][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, lsum = 0.f;
        // 16 keys of a tile against the wave's 16 rows, in two chains
        f32x4 sc, odd;
        auto scores = [&](const char* buf) {
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // LDS addresses are formed here, not kept over the loop
            const int g = ln >> 4, kr = 16 * kh + (ln & 15);
            sc = odd = f32x4{0.f, 0.f, 0.f, 0.f};
            uint32_t ks;
            if constexpr (NM == 4) ks = *reinterpret_cast<const uint32_t*>(buf + Raw::scales(kr) + 4 * g);
            else ks = *reinterpret_cast<const uint16_t*>(buf + Raw::scales(kr) + 2 * g);
            auto product = [&](auto S) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(buf + Raw::codes(kr, NM * g + S.value));
                sc = mma_mx16<S.value>(x, qm[S.value].hi, sc, ks, qs);
                i32x8 lo = qm[S.value].lo;
                if constexpr (S.value >= NM - kLdsQ) {
                    const auto& q = lds_q[2 * rb + rh][S.value - (NM - kLdsQ)];
                    const u32x4 l0 = q[0][ln], l1 = q[1][ln];
                    lo = i32x8{(int)l0[0], (int)l0[1], (int)l0[2], (int)l0[3], (int)l1[0], (int)l1[1], (int)l1[2], (int)l1[3]};
                }
                odd = mma_mx16<S.value>(x, lo, odd, ks, qs - 0x04040404u);              // (no byte is below 4; NaN's stays large)
            };
            product(std::integral_constant<int, 0>{});
            product(std::integral_constant<int, 1>{});
            if constexpr (NM == 4) {
                __builtin_amdgcn_sched_barrier(0);                // operands of two steps at a time
                product(std::integral_constant<int, 2>{});
                product(std::integral_constant<int, 3>{});
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                f32x4& y = s % 2 ? odd : sc;
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(buf + Raw::rope(kr, 4 * s + g));
                y = mma16(x, kLdsQ ? lds_qf[2 * rb + rh][s][ln] : qf[s], y);
            }
        };
        // 32 keys' probabilities times a quarter of the columns
        auto outputs = [&](const char* buf) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            Frag<T> p[2];
            float f[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                p[s] = *reinterpret_cast<const Frag<T>*>(&probs[rb][s][ln][0]);
                f[s] = factor[rb][s][ln & 15];
            }
            if (__any(f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[0][d][r] *= f[0];
                        acc[1][d][r] *= f[1];
                    }
            }
            auto read = [&](int d) -> Frag<T> {
                const char* const from = buf + (quarter * ND + d) * 1024 + ln * 8;
                const bf16x4 lo4 = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)from));
                const bf16x4 hi4 = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)(from + 512)));
                return __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
            };
            ReadAhead<T, ND, kAhead> ahead;
            ahead.start(read);
            ahead.template run<2>(read, [&](int d, const Frag<T>& v) {
                acc[0][d] = mma16(v, p[0], acc[0][d]);
                acc[1][d] = mma16(v, p[1], acc[1][d]);
            });
        };
        int now = fetch(t0, raw[0]);
        wait_loads_and_lds();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const int odd_tile = (t - t0) & 1;
            int next = 0;
            if (t + 1 < t1) next = fetch(t + 1, raw[odd_tile ^ 1]);
            if (kWide == 2) widen(raw[odd_tile], wide[kWide - 1 & odd_tile]);
            scores(raw[odd_tile]);
            settle(sc, odd);                                      // (here: or the compiler moves the products behind the outputs, and spills)
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[r] += odd[r];
            asm volatile("" : "+v"(sc));
            if (t > t0) outputs(wide[kWide - 1 & (odd_tile ^ 1)]);
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4;
            // of the tile the first lim + 1 keys
            const int k0 = t * kTile;
            if (k0 + kTile > len - a.Tq + 1 || k0 + kTile > rows || now != 3) {
                const int lim = last - k0 - 4 * g - 16 * kh;
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[r] = r > lim || !(now >> kh & 1) ? -INFINITY : sc[r];
            }
            float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            mx = group_max(mx);
            if (g == 0) tops[rb][rh][kh][ln] = mx;
            wait_lds();
            wg_barrier();
            mx = fmaxf(mx, tops[rb][rh][kh ^ 1][ln & 15]);
            // the running maximum moves as in mla_step.hip
            float al = 1.f;
            if ((mx - m) * c > 8.f) {
                al = __builtin_amdgcn_exp2f((m - mx) * c);
                lsum *= al;
                m = mx;
            }
            const float m0 = m == -INFINITY ? 0.f : m;            // nothing seen yet: all terms are 0
            T pf[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float p = __builtin_amdgcn_exp2f((sc[r] - m0) * c);
                lsum += p;
                pf[r] = (T)p;                  // bf16: the one rounding of the probabilities, as operands
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) probs[rb][rh][ln][4 * kh + r] = pf[r];
            if (g == 0 && kh == 0) factor[rb][rh][ln] = al;
            if (kWide == 1) widen(raw[odd_tile], wide[0]);        // all have read the tile before
            now = next;
            wait_loads_and_lds();
            wg_barrier();
        }
        outputs(wide[kWide - 1 & ((t1 - 1 - t0) & 1)]);
        // sums of both halves of the keys
        float lt = group_sum(lsum);
        wait_lds();
        wg_barrier();
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int g = ln >> 4, r0 = (group * RB + rb) * 32 + (ln & 15), r1 = r0 + 16, row = rh ? r1 : r0;
        if (g == 0) tops[rb][rh][kh][ln] = lt;
        wait_lds();
        wg_barrier();
        lt = tops[rb][rh][0][ln & 15] + tops[rb][rh][1][ln & 15];
        if (t0 == 0 && t1 == tiles) {
            float inv[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float x = tops[rb][s][0][ln & 15] + tops[rb][s][1][ln & 15];
                inv[s] = x > 0.f ? 1.f / x : x == 0.f ? 0.f : x;  // no visible key: 0; NaN stays NaN
            }
            T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC + quarter * (DC / 4) + 4 * g;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                if (r0 < M) store4(op + (int64_t)r0 * DC + 16 * d, acc[0][d], inv[0]);
                if (r1 < M) store4(op + (int64_t)r1 * DC + 16 * d, acc[1][d], inv[1]);
            }
            if (a.lse && row < M && g == 0 && kh == 0)
                a.lse[(int64_t)b * M + row] =
                    lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            const int j = t0 > 0 ? 0 : 1;
            float* const x0 = partial(a, group, part, j, 32 * rb + (ln & 15));
            float* const x1 = partial(a, group, part, j, 32 * rb + 16 + (ln & 15));
            if (g == 0 && kh == 0 && row < M) {
                float* const p = rh ? x1 : x0;
                p[0] = m * c;
                p[1] = lt;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                if (r0 < M) store4(x0 + 4 + quarter * (DC / 4) + 16 * d + 4 * g, acc[0][d], 1.f);
                if (r1 < M) store4(x1 + 4 + quarter * (DC / 4) + 16 * d + 4 * g, acc[1][d], 1.f);
            }
        }
        wait_lds();
        wg_barrier();                                             // the next sequence writes tops again
    }
}


// bf16, over 32 rows of queries. Eight waves share up to six sets of 16 rows and
// tiles of 64 keys. A wave a set forms its scores, so that a row's maximum and sum
// stay in one wave; every wave multiplies all rows' probabilities with an eighth of
// the columns, so that each value operand is read from LDS once. A tile's scores
// are formed along with the outputs of the one before; the softmax and the widening
// come between, the next tile's loads are under way all the while.
template <int DC, int DR, int S>
__global__ __launch_bounds__(512, 2) void mla_mx_step_many_kernel(MlaStepArgs a) {
    using T = __bf16;
    using Raw = RawTile<DC, DR, 4>;
    constexpr int kRows = 64, kWaves = 8, ND = DC / 16 / kWaves, NB = DC / 32, NM = DC / 128, NS = DR / 32;
    __shared__ __attribute__((aligned(1024))) char raw[2][Raw::kBytes];
    __shared__ __attribute__((aligned(1024))) char wide[kRows * DC * 2];
    __shared__ __attribute__((aligned(16))) Frag<T> probs[2][S][64];     // of 32 keys each
    __shared__ float factor[S][16];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool scorer = w < S;
    const int group = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    Scan sq = scan_tiles<kRows>(a, 0, lane);
    int total = sq.all();
    for (int b = 64; b < a.Nb; b += 64) total += scan_tiles<kRows>(a, b, lane).all();
    const int per = part_tiles(a, total);
    int at = part * per;                                         // next tile of the list
    const int end = total - at < per ? total : at + per;
    if (at >= total) return;
    const int M = a.Tq * a.H;
    const float c = a.scale * kLog2e;
    const int ps = a.page_shift;
    const int64_t page_bytes = (int64_t)mx_row_bytes(DC, DR, sizeof(T)) << ps;

    int b0 = 0, before = 0;                                      // sq's first sequence, tiles before it
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
        if (t0 == 0 && group == 0 && tid == 0 && len > rows) atomicAdd(a.status, 1u);

        // queries: row 32 (RB group + rb) + 16 rh + n of the (token, head) pairs
        const int mrow = min((group * S + (scorer ? w : 0)) * 16 + (lane & 15), M - 1);
        const int tok = mrow / a.H, head = mrow - tok * a.H;
        const int last = min(len - a.Tq + tok, rows - 1);         // the last key that this lane's token sees
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h;
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
            const uint64_t bad = __ballot(e < 0 && r >= t0 * kRows && r < (int64_t)t1 * kRows);
            if (bad && group == 0 && tid == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
            pages = r < rows ? e : -1;
        };
        // the first entries and the queries are under way together
        const int p0 = t0 * kRows >> ps, e = entry(p0);
        // step s multiplies the blocks s, s + NM, s + 2 NM and s + 3 NM
        MxQuery16 qm[NM];
        uint32_t qs = 0;                                          // their scale bytes
#pragma unroll
        for (int s = 0; s < NM; ++s) {
            bf16x8 x[4];
            const int g = lane >> 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = load8(qlp + 32 * (NM * ((g >> 1) + 2 * (i >> 1)) + s) + 16 * (g & 1) + 8 * (i & 1));
            qm[s].set(x, lane);
            qs |= qm[s].s << 8 * s;
            __builtin_amdgcn_sched_barrier(0);                    // one after the other: their sources take registers, too
        }
        bf16x8 qf[NS ? NS : 1];
#pragma unroll
        for (int s = 0; s < NS; ++s) qf[s] = load8(qrp + 32 * s + 8 * (lane >> 4));
        keep(p0, e);

        constexpr int kMine = (Raw::kLoads + kWaves - 1) / kWaves;                      // loads a wave issues for a tile
        // Sends tile t on its way to LDS; returns which of its quarters exist. Rows
        // past the length and of missing pages are zeros there: their weights are
        // 0, but what these multiply has to be finite.
        auto fetch = [&](int t, char* to) {
            const int k0 = t * kRows, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            const int mask = (1 << ps) - 1;
            auto page = [&](int q) { return __builtin_amdgcn_readlane(pages, ((k0 + 16 * q) >> ps) - pbase); };
            int have = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) have |= page(q) >= 0 ? 1 << q : 0;
            const bool whole = have == 15 && k0 + kRows <= rows;
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // offsets are formed here, not kept in registers
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int x = w + kWaves * i, q = x & 3;
                if (Raw::kLoads % kWaves && x >= Raw::kLoads) break;
                // (a missing page's address is not used)
                const char* const from = static_cast<const char*>(a.cache) + page(q) * page_bytes + Raw::plane(x, ps) +
                                         (int64_t)((k0 + 16 * q) & mask) * Raw::row_bytes(x);
                char* const at = to + Raw::place(x);
                int r, off;
                Raw::source(x, ln, r, off);
                if (whole) {
                    if (!Raw::is_scales(x)) load_lds16s(from, off, at);
                    else if (NB == 16 || ln < 32) load_lds4s(from, off, at);
                } else {
                    const bool there = (have >> q & 1) && k0 + 16 * q + r < rows;
                    if (!Raw::is_scales(x))
                        *reinterpret_cast<u32x4*>(at + 16 * ln) = there ? *reinterpret_cast<const u32x4*>(from + off) : u32x4{0, 0, 0, 0};
                    else if (NB == 16 || ln < 32)
                        *reinterpret_cast<uint32_t*>(at + 4 * ln) = there ? *reinterpret_cast<const uint32_t*>(from + off) : 0u;
                }
            }
            return have;
        };
        // A tile's latents as bf16: for 32 rows each as in the kernel above
        auto widen = [&](const char* from) {
            int td = tid;
            asm volatile("" : "+v"(td));
            const int r = td & 63, odd_half = r >> 3 & 1;
#pragma unroll
            for (int i = 0; i < NB / kWaves; ++i) {
                const int blk = i * kWaves + (td >> 6);
                const u32x4 c = *reinterpret_cast<const u32x4*>(from + Raw::codes(r, blk));
                const MxScale f(*reinterpret_cast<const uint8_t*>(from + Raw::scales(r) + blk));
                char* const to = wide + (r >> 5) * (32 * DC * 2) + blk * 2048 + (r & 31) * 32;
                char* const at = to + 16 * odd_half;
                char* const other = to + 16 * (odd_half ^ 1);
                *reinterpret_cast<bf16x8*>(at) = f.bf16(odd_half ? c[1] : c[0]);
                *reinterpret_cast<bf16x8*>(other) = f.bf16(odd_half ? c[0] : c[1]);
                *reinterpret_cast<bf16x8*>(at + 1024) = f.bf16(odd_half ? c[3] : c[2]);
                *reinterpret_cast<bf16x8*>(other + 1024) = f.bf16(odd_half ? c[2] : c[3]);
            }
        };
        f32x4 acc[S][ND];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[s][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, lsum = 0.f;
        // The products of the scores of a tile, in chains of 16 keys, each step's
        // operands read under the one before.
        f32x4 sc[4];
        auto products = [&](const char* buf) {
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // LDS addresses are formed here, not kept over the loop
            const int g = ln >> 4, n = ln & 15;
            uint32_t ks[4];
            u32x4 x[2][4];
            auto read = [&](int i) {
#pragma unroll
                for (int h = 0; h < 4; ++h) x[i & 1][h] = *reinterpret_cast<const u32x4*>(buf + Raw::codes(16 * h + n, NM * g + i));
            };
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                sc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
                if constexpr (NM == 4) ks[h] = *reinterpret_cast<const uint32_t*>(buf + Raw::scales(16 * h + n) + 4 * g);
                else ks[h] = *reinterpret_cast<const uint16_t*>(buf + Raw::scales(16 * h + n) + 2 * g);
            }
            read(0);
            bf16x8 y[4];
            auto rope = [&](int s) {
#pragma unroll
                for (int h = 0; h < 4; ++h) y[h] = *reinterpret_cast<const bf16x8*>(buf + Raw::rope(16 * h + n, 4 * s + g));
            };
            auto step = [&](auto I) {
                constexpr int i = I.value;
                if constexpr (i + 1 < NM) read(i + 1);
                else if constexpr (NS > 0) rope(0);
#pragma unroll
                for (int h = 0; h < 4; ++h) sc[h] = mma_mx16<i>(x[i & 1][h], qm[i].hi, sc[h], ks[h], qs);
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    sc[h] = mma_mx16<i>(x[i & 1][h], qm[i].lo, sc[h], ks[h], qs - 0x04040404u);         // (no byte is below 4; NaN's stays large)
                __builtin_amdgcn_sched_barrier(0);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            if constexpr (NM == 4) {
                step(std::integral_constant<int, 2>{});
                step(std::integral_constant<int, 3>{});
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
#pragma unroll
                for (int h = 0; h < 4; ++h) sc[h] = mma16(y[h], qf[s], sc[h]);
                if (s + 1 < NS) rope(s + 1);
            }
            // (sends the products on their way here: the compiler would move them behind what follows)
            asm volatile("" : "+v"(sc[0]), "+v"(sc[1]), "+v"(sc[2]), "+v"(sc[3]));
        };
        // the probabilities of tile t for the wave's set
        auto softmax = [&](int t, int have) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4, n = ln & 15;
            settle(sc[0], sc[1]);
            settle(sc[2], sc[3]);
            // of the tile a lane's token sees the first lim + 1 keys
            const int k0 = t * kRows;
            if (k0 + kRows > len - a.Tq + 1 || k0 + kRows > rows || have != 15) {
                const int lim = last - k0 - 4 * g;
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[h][r] = 16 * h + r > lim || !(have >> h & 1) ? -INFINITY : sc[h][r];
            }
            float mx = sc[0][0];
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, sc[h][r]);
            mx = group_max(mx);
            // the running maximum moves as in mla_step.hip
            float al = 1.f;
            if ((mx - m) * c > 8.f) {
                al = __builtin_amdgcn_exp2f((m - mx) * c);
                lsum *= al;
                m = mx;
            }
            const float m0 = m == -INFINITY ? 0.f : m;            // nothing seen yet: all terms are 0
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                Frag<T> pf;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f((sc[2 * u + h][r] - m0) * c);
                        lsum += p;
                        pf[4 * h + r] = (T)p;  // the one rounding of the probabilities, as operands
                    }
                probs[u][w][ln] = pf;
            }
            if (g == 0) factor[w][n] = al;
        };
        // all rows' outputs over the wave's columns
        auto outputs = [&] {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            float f[S];
            bool move = false;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                f[s] = factor[s][ln & 15];
                move |= f[s] != 1.f;
            }
            if (__any(move)) {
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[s][d][r] *= f[s];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {                         // 32 keys each
                Frag<T> p[S];
#pragma unroll
                for (int s = 0; s < S; ++s) p[s] = probs[u][s][ln];
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const char* const x = wide + u * (32 * DC * 2) + (w * ND + d) * 1024 + ln * 8;
                    const bf16x4 lo4 = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)x));
                    const bf16x4 hi4 = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)(x + 512)));
                    const bf16x8 v = __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                    for (int s = 0; s < S; ++s) acc[s][d] = mma16(v, p[s], acc[s][d]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // Tile t lies in raw[(t - t0) % 2].
        int h1 = fetch(t0, raw[0]);
        wait_loads_and_lds();
        wg_barrier();
        int h2 = t0 + 1 < t1 ? fetch(t0 + 1, raw[1]) : 0;
        if (scorer) {
            products(raw[0]);
            softmax(t0, h1);
        }
        widen(raw[0]);
        wait_loads_and_lds();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const int i = (t - t0) & 1;
            const bool more = t + 1 < t1;
            h1 = h2;
            if (t + 2 < t1) h2 = fetch(t + 2, raw[i]);
            if (more && scorer) products(raw[i ^ 1]);
            outputs();
            wait_lds();
            wg_barrier();
            if (more) {
                if (scorer) softmax(t + 1, h1);
                widen(raw[i ^ 1]);
                wait_loads_and_lds();
                wg_barrier();
            }
        }
        // every wave needs the rows' sums
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int g = ln >> 4, n = ln & 15, r0 = group * S * 16 + n, col = w * (DC / kWaves) + 4 * g;
        const float lt = group_sum(lsum);
        if (scorer && g == 0) factor[w][n] = lt;
        wait_lds();
        wg_barrier();
        if (t0 == 0 && t1 == tiles) {
            T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC + col;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float x = factor[s][n];
                const float inv = x > 0.f ? 1.f / x : x == 0.f ? 0.f : x;      // no visible key: 0; NaN stays NaN
                if (r0 + 16 * s < M) {
#pragma unroll
                    for (int d = 0; d < ND; ++d) store4(op + (int64_t)(r0 + 16 * s) * DC + 16 * d, acc[s][d], inv);
                }
            }
            if (a.lse && scorer && g == 0 && r0 + 16 * w < M)
                a.lse[(int64_t)b * M + r0 + 16 * w] =
                    lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            const int j = t0 > 0 ? 0 : 1;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float* const x = partial(a, group, part, j, 16 * s + n);
                if (r0 + 16 * s < M) {
                    if (w == s && g == 0) {
                        x[0] = m * c;
                        x[1] = lt;
                    }
#pragma unroll
                    for (int d = 0; d < ND; ++d) store4(x + 4 + col + 16 * d, acc[s][d], 1.f);
                }
            }
        }
        wait_lds();
        wg_barrier();                                             // the next sequence writes factor again
    }
}

// float32: a tile's codes come to registers a tile ahead, 32 channels a thread,
// and go to LDS as float32 rows, which scores and outputs read.
template <int DC, int DR, int RB> __global__ __launch_bounds__(256 * RB, RB) void mla_mx_step_f32_kernel(MlaStepArgs a) {
    using T = float;
    constexpr int D = DC + DR, RC = D / kChunk<T>, NS = D / 32, ND = DC / 64, NT = 256 * RB;
    constexpr int NB = DC / 32, RR = DR / kChunk<T>;          // blocks of 32 channels, 16-byte chunks of the shared part
    constexpr int CI = (kTile * NB + NT - 1) / NT, RI = (kTile * RR + NT - 1) / NT;     // of them a thread
    __shared__ __attribute__((aligned(1024))) char smem[2][kTile * RC * 16];
    __shared__ __attribute__((aligned(32))) T probs[RB][2][64][8];
    __shared__ float tops[RB][2][2][16], factor[RB][2][16];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rb = w >> 2, quarter = w & 3, rh = w & 1, kh = quarter >> 1;
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
    const int64_t page_bytes = (int64_t)mx_row_bytes(DC, DR, sizeof(T)) << ps;

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
        if (t0 == 0 && group == 0 && tid == 0 && len > rows) atomicAdd(a.status, 1u);

        // queries: row 32 (RB group + rb) + 16 rh + n of the (token, head) pairs
        const int row = ((group * RB + rb) * 2 + rh) * 16 + (lane & 15), mrow = row < M ? row : M - 1;
        const int tok = mrow / a.H, head = mrow - tok * a.H;
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h;
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
            if (bad && group == 0 && tid == 0) atomicAdd(a.status, (unsigned)__popcll(bad));
            pages = r < rows ? e : -1;
        };
        // the first entries and the queries are under way together
        const int p0 = t0 * kTile >> ps, e = entry(p0);
        Frag<T> qf[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int ch = 32 * s + 8 * (lane >> 4);
            qf[s] = ch < DC ? load8(qlp + ch) : load8(qrp + ch - DC);
        }
        keep(p0, e);

        // A tile on its way: this thread's blocks and chunks. Rows past the length
        // and of missing pages are zeros: hidden rows' weights are 0, but what they multiply has to be finite.
        u32x4 codes[CI], shared_part[RI ? RI : 1];
        uint32_t scale[CI];
        int have = 0;
        auto fetch = [&](int t) {
            const int k0 = t * kTile, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            const int e0 = __builtin_amdgcn_readlane(pages, p - pbase);
            const int e1 = __builtin_amdgcn_readlane(pages, ((k0 + 16) >> ps) - pbase);
            const int mask = (1 << ps) - 1;
            const char* const lo = static_cast<const char*>(a.cache) + e0 * page_bytes;
            const char* const hi = static_cast<const char*>(a.cache) + e1 * page_bytes;
            have = (e0 >= 0 ? 1 : 0) | (e1 >= 0 ? 2 : 0);
            int td = tid;
            asm volatile("" : "+v"(td));                          // nothing that goes by the thread is kept over the loop
#pragma unroll
            for (int i = 0; i < CI; ++i) {
                const int x = i * NT + td, r = x / NB, blk = x % NB;
                codes[i] = u32x4{0, 0, 0, 0};
                scale[i] = 0;
                if (r < kTile && k0 + r < rows && (have >> (r >> 4) & 1)) {
                    const char* const page = r >> 4 ? hi : lo;
                    const int64_t pr = (k0 + r) & mask;
                    codes[i] = *reinterpret_cast<const u32x4*>(page + pr * (DC / 2) + blk * 16);
                    scale[i] = *reinterpret_cast<const uint8_t*>(page + ((int64_t)(DC / 2) << ps) + pr * NB + blk);
                }
            }
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int x = i * NT + td, r = x / (RR ? RR : 1), ch = x % (RR ? RR : 1);
                shared_part[i] = u32x4{0, 0, 0, 0};
                if (r < kTile && k0 + r < rows && (have >> (r >> 4) & 1))
                    shared_part[i] = *reinterpret_cast<const u32x4*>(
                        (r >> 4 ? hi : lo) + ((int64_t)(DC / 2 + NB) << ps) + ((int64_t)((k0 + r) & mask) * RR + ch) * 16);
            }
        };
        auto put = [&](char* to) {
            int td = tid;
            asm volatile("" : "+v"(td));
#pragma unroll
            for (int i = 0; i < CI; ++i) {
                const int x = i * NT + td, r = x / NB, blk = x % NB, sw = swizzle16<T, RC>(r);
                if (kTile * NB % NT && r >= kTile) break;
                const MxScale f(scale[i]);
                char* const p = to + r * (RC * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x8 v = f.f32(codes[i][j]);
                    *reinterpret_cast<f32x4*>(p + (((8 * blk + 2 * j) ^ sw) << 4)) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4*>(p + (((8 * blk + 2 * j + 1) ^ sw) << 4)) = f32x4{v[4], v[5], v[6], v[7]};
                }
            }
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const int x = i * NT + td, r = x / (RR ? RR : 1), ch = x % (RR ? RR : 1);
                if (kTile * RR % NT && r >= kTile) break;
                *reinterpret_cast<u32x4*>(to + r * (RC * 16) + (((DC / kChunk<T> + ch) ^ swizzle16<T, RC>(r)) << 4)) = shared_part[i];
            }
        };
        f32x4 acc[2][ND];                                         // of the block's two sets of 16 rows
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[0][d] = acc[1][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, lsum = 0.f;
        fetch(t0);
        put(smem[0]);
        int now = have;
        if (t0 + 1 < t1) fetch(t0 + 1);
        wait_lds();
        wg_barrier();
        for (int t = t0; t < t1; ++t) {
            const char* const buf = smem[(t - t0) & 1];
            int ln = lane;
            asm volatile("" : "+v"(ln));                          // LDS addresses are formed here, not kept over the loop
            const int g = ln >> 4;
            f32x4 sc = {0.f, 0.f, 0.f, 0.f}, odd = sc;            // 16 keys, in two chains
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                f32x4& y = s % 2 ? odd : sc;
                y = mma16(read_rows16<T, RC>(buf, 16 * kh + (ln & 15), s, g), qf[s], y);
            }
            settle(sc, odd);
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[r] += odd[r];
            // keys that this lane's token sees in the tile: the first lim + 1
            const int k0 = t * kTile;
            if (k0 + kTile > len - a.Tq + 1 || k0 + kTile > rows || now != 3) {
                const int last = len - a.Tq + tok < rows - 1 ? len - a.Tq + tok : rows - 1, lim = last - k0 - 4 * g - 16 * kh;
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[r] = r > lim || !(now >> kh & 1) ? -INFINITY : sc[r];
            }
            float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            mx = group_max(mx);
            if (g == 0) tops[rb][rh][kh][ln] = mx;
            wait_lds();
            wg_barrier();
            mx = fmaxf(mx, tops[rb][rh][kh ^ 1][ln & 15]);
            // the running maximum moves as in mla_step.hip
            float al = 1.f;
            if ((mx - m) * c > 8.f) {
                al = __builtin_amdgcn_exp2f((m - mx) * c);
                lsum *= al;
                m = mx;
            }
            const float m0 = m == -INFINITY ? 0.f : m;            // nothing seen yet: all terms are 0
            T pf[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float p = __builtin_amdgcn_exp2f((sc[r] - m0) * c);
                lsum += p;
                pf[r] = (T)p;                  // bf16: the one rounding of the probabilities, as operands
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) probs[rb][rh][ln][4 * kh + r] = pf[r];
            if (g == 0 && kh == 0) factor[rb][rh][ln] = al;
            // the next tile: its buffer's readers have passed the barrier
            if (t + 1 < t1) {
                put(smem[(t + 1 - t0) & 1]);
                now = have;
                if (t + 2 < t1) fetch(t + 2);
            }
            wait_lds();
            wg_barrier();
            Frag<T> p[2];
            float f[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                p[s] = *reinterpret_cast<const Frag<T>*>(&probs[rb][s][ln][0]);
                f[s] = factor[rb][s][ln & 15];
            }
            if (__any(f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[0][d][r] *= f[0];
                        acc[1][d][r] *= f[1];
                    }
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const Frag<T> v = read_cols16<T, RC>(buf, quarter * (DC / 4) + 16 * d, ln);
                acc[0][d] = mma16(v, p[0], acc[0][d]);
                acc[1][d] = mma16(v, p[1], acc[1][d]);
            }
        }
        // sums of both halves of the keys
        float lt = group_sum(lsum);
        wait_lds();
        wg_barrier();
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int g = ln >> 4, r0 = (group * RB + rb) * 32 + (ln & 15), r1 = r0 + 16;
        if (g == 0) tops[rb][rh][kh][ln] = lt;
        wait_lds();
        wg_barrier();
        lt = tops[rb][rh][0][ln & 15] + tops[rb][rh][1][ln & 15];
        if (t0 == 0 && t1 == tiles) {
            float inv[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float x = tops[rb][s][0][ln & 15] + tops[rb][s][1][ln & 15];
                inv[s] = x > 0.f ? 1.f / x : x == 0.f ? 0.f : x;  // no visible key: 0; NaN stays NaN
            }
            T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC + quarter * (DC / 4) + 4 * g;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                if (r0 < M) store4(op + (int64_t)r0 * DC + 16 * d, acc[0][d], inv[0]);
                if (r1 < M) store4(op + (int64_t)r1 * DC + 16 * d, acc[1][d], inv[1]);
            }
            if (a.lse && row < M && g == 0 && kh == 0)
                a.lse[(int64_t)b * M + row] =
                    lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            const int j = t0 > 0 ? 0 : 1;
            float* const x0 = partial(a, group, part, j, 32 * rb + (ln & 15));
            float* const x1 = partial(a, group, part, j, 32 * rb + 16 + (ln & 15));
            if (g == 0 && kh == 0 && row < M) {
                float* const p = rh ? x1 : x0;
                p[0] = m * c;
                p[1] = lt;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                if (r0 < M) store4(x0 + 4 + quarter * (DC / 4) + 16 * d + 4 * g, acc[0][d], 1.f);
                if (r1 < M) store4(x1 + 4 + quarter * (DC / 4) + 16 * d + 4 * g, acc[1][d], 1.f);
            }
        }
        wait_lds();
        wg_barrier();                                             // the next sequence writes tops again
    }
}

template <class T, int DC, int DR> hipError_t launch_mx(const MlaStepArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.groups * a.parts));
    if constexpr (sizeof(T) == 2) {
        if (a.waves == 2) mla_mx_step_bf16_kernel<DC, DR, 1><<<grid, 256, 0, s>>>(a);
        else if (a.waves == 4) mla_mx_step_many_kernel<DC, DR, 4><<<grid, 512, 0, s>>>(a);
        else mla_mx_step_many_kernel<DC, DR, 6><<<grid, 512, 0, s>>>(a);
    } else {
        if (a.waves == 2) mla_mx_step_f32_kernel<DC, DR, 1><<<grid, 256, 0, s>>>(a);
        else if constexpr (most_blocks(false, DC) > 1) mla_mx_step_f32_kernel<DC, DR, 2><<<grid, 512, 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int blocks = (a.Tq * a.H + a.join_rows - 1) / a.join_rows;
    if (sizeof(T) == 2 && a.waves > 2)
        mla_step_join_kernel<T, DC, kMostParts, 64><<<dim3((unsigned)((int64_t)a.Nb * blocks)), 256, 0, s>>>(a, blocks);
    else mla_step_join_kernel<T, DC, kMostParts><<<dim3((unsigned)((int64_t)a.Nb * blocks)), 256, 0, s>>>(a, blocks);
    return hipGetLastError();
}
template <class T> hipError_t launch_mx_dims(const MlaStepArgs& a, hipStream_t s) {
    if (a.Dc == 512) return a.Dr ? launch_mx<T, 512, 64>(a, s) : launch_mx<T, 512, 0>(a, s);
    return a.Dr ? launch_mx<T, 256, 64>(a, s) : launch_mx<T, 256, 0>(a, s);
}

}  // namespace

// The split over workgroups: blocks of 32 rows of queries spread evenly over as few
// groups as hold them; a cache so short that there is a compute unit for each
// tile and group gets more of them.
size_t mla_step_mx_plan(MlaStepArgs& a) {
    const int64_t rows = (int64_t)a.Tq * a.H, blocks = (rows + 31) / 32;
    const int64_t most = (int64_t)a.Nb * ((((int64_t)a.max_pages << a.page_shift) + kTile - 1) / kTile);
    int64_t per = most_blocks(a.bf16, a.Dc);                      // blocks a workgroup
    while (per > 1 && (blocks + per - 2) / (per - 1) * most <= 256) --per;
    a.groups = (int32_t)((blocks + per - 1) / per);
    a.waves = (int32_t)((blocks + a.groups - 1) / a.groups) * 2;
    int64_t parts = (a.bf16 && a.waves == 2 ? kMostParts : 256) / a.groups;
    if (parts < 32) parts = 32;
    if (parts > most) parts = most;
    a.parts = (int32_t)(parts > 1 ? parts : 1);
    const int64_t j = (a.Nb * rows + 1023) / 1024;                // the join: as in mla_step.hip
    a.join_rows = (int32_t)(j < rows ? j : rows);
    return (size_t)a.groups * a.parts * 2 * (16 * a.waves) * (a.Dc + 4) * sizeof(float);
}

hipError_t launch_mla_step_mx(const MlaStepArgs& a, hipStream_t s) {
    return a.bf16 ? launch_mx_dims<__bf16>(a, s) : launch_mx_dims<float>(a, s);
}

}  // namespace kda
