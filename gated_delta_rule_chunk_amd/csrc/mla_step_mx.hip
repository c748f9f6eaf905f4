// Latent attention, absorbed form, over a cache that holds the latents in 4 bits
// (include/kda_mla_cache.h): s = scale (q_latent . c + q_rope . r), p = softmax s,
// o = sum p c.
//
// As in mla_step.hip the tiles of cache rows of all sequences (64 rows, float32
// 32) form one list, cut into equal parts by the lengths on the device, and a
// second kernel joins the parts.
#include "mla_mx_tile.hpp"
#include "mla_step.hpp"

namespace kda {
namespace {

// float32: blocks of 32 rows of queries a workgroup, at most (as queries and outputs fit the registers)
__host__ __device__ constexpr int most_blocks(int dc) { return dc == 256 ? 2 : 1; }
// bf16: workgroups a compute unit, as registers and LDS allow; a part for each
__host__ __device__ constexpr int residents(int dc, int sets) { return sets == 1 || (sets == 2 && dc == 256) ? 2 : 1; }
// bf16. Eight waves share up to six sets of 16 rows of queries and tiles of 64 keys,
// which come straight to LDS as they lie in memory, two ahead of the outputs.
// Scores run on the codes (mla_mx_tile.hpp). A set has one wave for them, or two or
// four that take 16-key groups of the tile each and tell each other their maxima;
// every wave multiplies all rows' probabilities with an eighth of the columns, whose
// codes it turns and widens to bf16 in registers, each once a tile. A tile's
// scores are formed before the outputs of the one before.
// Bound, with six sets, by matrix (36%) and vector instructions (43% of the cycles),
// which two waves a SIMD seldom overlap: 3.2 us a tile, 128 sequences of 4096 to
// 8192, 96 heads in 205-220 us, 760 TFLOP/s. Measured and not kept, same case: a
// widened copy of the tile in LDS for the outputs (217), four tile buffers (227),
// half of the waves a phase behind the others (213). With one set, by vector
// instructions (66%): 64 sequences of 8192 to 16384, 12 heads in 83 us, 2.5 TB/s;
// two workgroups a compute unit (one: 100 us). The matrix cores take bf16, so the
// probabilities are rounded once, as operands, their sum is not: o is off by
// 0.0017-0.0018 of its norm, where its own rounding alone leaves 0.0017.
template <int DC, int DR, int S>
__global__ __launch_bounds__(512, 2 * residents(DC, S)) void mla_mx_step_bf16_kernel(MlaStepArgs a) {
    using T = __bf16;
    using Raw = RawTile<DC, DR>;
    // waves of a set, 16-key groups of each
    constexpr int KS = S == 6 ? 1 : S == 4 ? 2 : 4, NG = 4 / KS;
    constexpr int ND = DC / 16 / kWaves, NB = DC / 32, NM = DC / 128, NS = DR / 32;
    constexpr int PB = KS == 1 ? 2 : 1;                          // one barrier a tile, or two
    __shared__ __attribute__((aligned(1024))) char raw[3][Raw::kBytes];
    __shared__ __attribute__((aligned(16))) s16x4 probs[PB][2][S][64][2];   // of 32 keys each: operands
    // A tile's scales by blocks: as numbers, or (one set) as the exponents of bf16.
    using Scale = std::conditional_t<(S > 1), uint32_t, uint16_t>;
    constexpr int kExponent = S > 1 ? 23 : 7;
    __shared__ __attribute__((aligned(16))) Scale scales[PB][NB][kRows];
    __shared__ float factor[PB][S][16], tops[S][KS][16];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool scorer = w < S * KS;
    const int set = scorer ? w / KS : 0, kg = w % KS;
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

        // queries: row 16 (S group + set) + n of the (token, head) pairs
        const int mrow = min((group * S + set) * 16 + (lane & 15), M - 1);
        const int tok = mrow / a.H, head = mrow - tok * a.H;
        const int last = min(len - a.Tq + tok, rows - 1);         // the last key that this lane's token sees
        const T* qlp = static_cast<const T*>(a.ql) + b * a.ql_b + tok * a.ql_t + head * a.ql_h;
        const T* qrp = static_cast<const T*>(a.qr) + b * a.qr_b + tok * a.qr_t + head * a.qr_h;
        // Page table entries of 64 pages, one per lane; -1 for no such page or one
        // past the rows. A tile's quarters lie in pages of the same 64.
        const int32_t* table = a.table + (int64_t)b * a.max_pages;
        int pbase = -64, pages = 0;
        uint64_t exist = 0;                                       // which of them do
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
            exist = __ballot(pages >= 0);
        };
        // the first entries and the queries are under way together
        const int p0 = t0 * kRows >> ps, e = entry(p0);
        // step s multiplies the blocks s, s + NM, s + 2 NM and s + 3 NM
        bf16x8 q[NM][4];
#pragma unroll
        for (int s = 0; s < NM; ++s) {
            const int g = lane >> 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[s][i] = load8(qlp + 32 * (NM * ((g >> 1) + 2 * (i >> 1)) + s) + 16 * (g & 1) + 8 * (i & 1));
        }
        bf16x8 qf[NS ? NS : 1];
#pragma unroll
        for (int s = 0; s < NS; ++s) qf[s] = load8(qrp + 32 * s + 8 * (lane >> 4));
        __builtin_amdgcn_sched_barrier(0);                        // all are under way
        keep(p0, e);

        auto fetch = [&](int t, char* to) {
            const int k0 = t * kRows, p = k0 >> ps;
            if (p >= pbase + 64) keep(p, entry(p));
            return mx_fetch<DC, DR>(to, static_cast<const char*>(a.cache), page_bytes, pages, exist, pbase, ps, k0, rows, w, lane);
        };
        // Tile t lies in raw[(t - t0) % 3].
        int h0 = fetch(t0, raw[0]);
        MxQuery16 qm[NM];
        uint32_t qs = 0;                                          // their scale bytes
#pragma unroll
        for (int s = 0; s < NM; ++s) {
            qm[s].set(q[s], lane);
            qs |= qm[s].s << 8 * s;
            __builtin_amdgcn_sched_barrier(0);
        }
        // a tile's scale bytes, turned: outputs take four keys of a block together
        auto turn = [&](const char* from, int b) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int q = kWaves - 1 - w;                         // (the last waves have no scores, or the fewest)
            if (q < NB / 4) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(from + Raw::scales(ln) + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) scales[b][4 * q + i][ln] = (Scale)((x >> 8 * i & 255) << kExponent);
            }
        };
        f32x4 acc[S][ND];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[s][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, lsum = 0.f;
        f32x4 sc[NG];
        float mx = -INFINITY;
        auto products = [&](const char* buf) { mx_scores<DC, DR, NG>(buf, 16 * NG * kg, lane, qm, qs, qf, sc); };
        // hides what the rows of tile t do not see; their maxima over the wave's keys
        auto maxima = [&](int t, int have) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4, n = ln & 15;
            settle(sc[0], sc[NG - 1]);
            if constexpr (NG == 4) settle(sc[1], sc[2]);
            // of the tile a lane's token sees the first lim + 1 keys
            const int k0 = t * kRows;
            if (k0 + kRows > len - a.Tq + 1 || k0 + kRows > rows || have != 15) {
                const int lim = last - k0 - 4 * g - 16 * NG * kg;
#pragma unroll
                for (int h = 0; h < NG; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[h][r] = 16 * h + r > lim || !(have >> (NG * kg + h) & 1) ? -INFINITY : sc[h][r];
            }
            mx = sc[0][0];
#pragma unroll
            for (int h = 0; h < NG; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, sc[h][r]);
            mx = group_max(mx);
            if (KS > 1 && g == 0) tops[set][kg][n] = mx;
        };
        // the probabilities of the wave's keys
        auto softmax = [&](int b) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4, n = ln & 15;
            if constexpr (KS > 1) {
#pragma unroll
                for (int i = 0; i < KS; ++i) mx = fmaxf(mx, tops[set][i][n]);
            }
            // the running maximum moves as in mla_step.hip
            float al = 1.f;
            if ((mx - m) * c > (S > 1 ? 8.f : 0.f)) {
                al = __builtin_amdgcn_exp2f((m - mx) * c);
                lsum *= al;
                m = mx;
            }
            const float m0 = m == -INFINITY ? 0.f : m;            // nothing seen yet: all terms are 0
#pragma unroll
            for (int h = 0; h < NG; ++h) {
                float p[4];
                bf16x4 pf;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[r] = __builtin_amdgcn_exp2f((sc[h][r] - m0) * c);
                    lsum += p[r];
                    pf[r] = (T)p[r];           // the one rounding of the probabilities, as operands
                }
                s16x4 bits = __builtin_bit_cast(s16x4, pf);
                if constexpr (S == 1) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) bits[r] = p[r] < 0x1p-126f ? -32768 : bits[r] - (127 << 7);
                }
                probs[b][(NG * kg + h) >> 1][set][ln][(NG * kg + h) & 1] = bits;
            }
            if (g == 0 && kg == 0) factor[b][set][n] = al;
        };
        // All rows' outputs over the wave's columns. A transposing read gives a lane
        // one column of the 16 keys that it holds in both steps of 32, in their order.
        // The conversions take one scale, where the two codes of a byte are of two
        // keys: a pair takes two conversions, a half of each. For one set it costs
        // less to scale the probabilities, which then are at most 1 (a maximum moves
        // at once): as bf16's bits, 127 << 7 less, a scale's exponent is added, and
        // what is negative then is 0, as are those of zeros, -32768, at any scale.
        // (A block of NaN needs none: it made its row's sum NaN.) 64 sequences of
        // 16384, 12 heads: 92 us with scaled pairs, 83 with scaled probabilities.
        auto outputs = [&](const char* buf, int b) {
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int g = ln >> 4, key = 16 * (ln >> 2 & 3) + 4 * g + (ln & 3);
            typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
            i32x2 codes[ND];
#pragma unroll
            for (int d = 0; d < ND; ++d)
                codes[d] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                    (KDA_LDS i32x2*)(buf + Raw::codes(key, (w * ND + d) >> 1) + 8 * ((w * ND + d) & 1)));
            float f[S];
            bool move = false;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                f[s] = factor[b][s][ln & 15];
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
                typedef int16_t s16x8 __attribute__((ext_vector_type(8)));
                s16x8 p[S];
#pragma unroll
                for (int s = 0; s < S; ++s) p[s] = *reinterpret_cast<const s16x8*>(&probs[b][u][s][ln][0]);
                if constexpr (S == 1) {
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        const Scale* const at = &scales[b][(w * ND + d) >> 1][32 * u + 4 * g];
                        const s16x4 e0 = *reinterpret_cast<const s16x4*>(at), e1 = *reinterpret_cast<const s16x4*>(at + 16);
                        const s16x8 y = p[0] + __builtin_shufflevector(e0, e1, 0, 1, 2, 3, 4, 5, 6, 7);
                        acc[0][d] = mma16(MxScale(127).bf16(codes[d][u]),
                                          __builtin_bit_cast(bf16x8, __builtin_elementwise_max(y, (s16x8)0)), acc[0][d]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    continue;
                }
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    uint32_t v[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {                 // 16 keys of the tile each
                        const Scale* const at = &scales[b][(w * ND + d) >> 1][32 * u + 16 * h + 4 * g];
                        const u32x4 e = *reinterpret_cast<const u32x4*>(at);
                        v[2 * h] = h ? mx_pair<2>(codes[d][u], e[0], e[1]) : mx_pair<0>(codes[d][u], e[0], e[1]);
                        v[2 * h + 1] = h ? mx_pair<3>(codes[d][u], e[2], e[3]) : mx_pair<1>(codes[d][u], e[2], e[3]);
                    }
#pragma unroll
                    for (int s = 0; s < S; ++s) acc[s][d] = mma16(__builtin_bit_cast(bf16x8, u32x4{v[0], v[1], v[2], v[3]}), __builtin_bit_cast(bf16x8, p[s]), acc[s][d]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        wait_loads_and_lds();
        wg_barrier();
        // From a tile before the first on, which has no outputs: the first one's scores
        // are no code of their own (one sequence of 100001: 46 -> 44 us).
        for (int t = t0 - 1, i = 2; t < t1; ++t) {
            const int now = (t - t0) & (PB - 1), i1 = i == 2 ? 0 : i + 1, i2 = 3 - i - i1, have = h0;
            const bool more = t + 1 < t1;
            if (t + 2 < t1) h0 = fetch(t + 2, raw[i2]);
            if (more && scorer) {
                products(raw[i1]);
                if (t < t0) settle(sc[0], sc[NG - 1]);            // (no outputs follow)
            }
            if (t >= t0) outputs(raw[i], now);
            if (more) {
                if (scorer) maxima(t + 1, have);
                if constexpr (KS > 1) {
                    wait_lds();
                    wg_barrier();
                }
                turn(raw[i1], now ^ (PB - 1));
                if (scorer) softmax(now ^ (PB - 1));
                wait_loads_and_lds();
                wg_barrier();
            }
            i = i1;
        }
        // every wave needs the rows' sums
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int g = ln >> 4, n = ln & 15, r0 = group * S * 16 + n, col = w * (DC / kWaves) + 4 * g;
        const float part_sum = group_sum(lsum);
        if (scorer && g == 0) tops[set][kg][n] = part_sum;
        wait_lds();
        wg_barrier();
        auto sum_of = [&](int s) {
            float x = tops[s][0][n];
#pragma unroll
            for (int i = 1; i < KS; ++i) x += tops[s][i][n];
            return x;
        };
        const float lt = sum_of(set);
        if (t0 == 0 && t1 == tiles) {
            T* op = static_cast<T*>(a.o) + (int64_t)b * M * DC + col;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float x = sum_of(s);
                const float inv = x > 0.f ? 1.f / x : x == 0.f ? 0.f : x;      // no visible key: 0; NaN stays NaN
                if (r0 + 16 * s < M) {
#pragma unroll
                    for (int d = 0; d < ND; ++d) store4(op + (int64_t)(r0 + 16 * s) * DC + 16 * d, acc[s][d], inv);
                }
            }
            if (a.lse && scorer && kg == 0 && g == 0 && r0 + 16 * set < M)
                a.lse[(int64_t)b * M + r0 + 16 * set] =
                    lt == 0.f ? -INFINITY : (m * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
        } else {
            const int j = t0 > 0 ? 0 : 1;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float* const x = partial(a, group, part, j, 16 * s + n);
                if (r0 + 16 * s < M) {
                    if (scorer && set == s && kg == 0 && g == 0) {
                        x[0] = m * c;
                        x[1] = lt;
                    }
#pragma unroll
                    for (int d = 0; d < ND; ++d) store4(x + 4 + col + 16 * d, acc[s][d], 1.f);
                }
            }
        }
        wait_lds();
        wg_barrier();                                             // the next sequence writes tops again
    }
}

// float32: a tile's codes come to registers a tile ahead, 32 channels a thread,
// and go to LDS as float32 rows, which scores and outputs read. Four waves share a
// block of 32 rows of queries: each forms the scores of 16 rows and 16 keys, the two
// that share rows agree on the running maximum, and each multiplies the
// probabilities of all 32 rows with a quarter of the columns. Two blocks for Dc =
// 256; one for 512, where queries and outputs take the registers of two. 8
// sequences of 1024 to 2047, 3 new tokens, 16 heads, Dc = 256 in 25 us, bound by the
// latency of two tiles in a row.
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
                pf[r] = p;
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
        if (a.waves == 1) mla_mx_step_bf16_kernel<DC, DR, 1><<<grid, 64 * kWaves, 0, s>>>(a);
        else if (a.waves == 2) mla_mx_step_bf16_kernel<DC, DR, 2><<<grid, 64 * kWaves, 0, s>>>(a);
        else if (a.waves == 4) mla_mx_step_bf16_kernel<DC, DR, 4><<<grid, 64 * kWaves, 0, s>>>(a);
        else mla_mx_step_bf16_kernel<DC, DR, 6><<<grid, 64 * kWaves, 0, s>>>(a);
    } else {
        if (a.waves == 2) mla_mx_step_f32_kernel<DC, DR, 1><<<grid, 256, 0, s>>>(a);
        else if constexpr (most_blocks(DC) > 1) mla_mx_step_f32_kernel<DC, DR, 2><<<grid, 512, 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int blocks = (a.Tq * a.H + a.join_rows - 1) / a.join_rows;
    mla_step_join_kernel<T, DC, sizeof(T) == 2 ? 2 * kMaxParts : kMaxParts, sizeof(T) == 2 ? kRows : kTile>
        <<<dim3((unsigned)((int64_t)a.Nb * blocks)), 256, 0, s>>>(a, blocks);
    return hipGetLastError();
}
template <class T> hipError_t launch_mx_dims(const MlaStepArgs& a, hipStream_t s) {
    if (a.Dc == 512) return a.Dr ? launch_mx<T, 512, 64>(a, s) : launch_mx<T, 512, 0>(a, s);
    return a.Dr ? launch_mx<T, 256, 64>(a, s) : launch_mx<T, 256, 0>(a, s);
}

}  // namespace

// The split over workgroups: sets of 16 rows of queries (float32: blocks of 32,
// which a.waves counts as two) spread evenly over as few groups as hold them; a
// cache so short that there is a compute unit for each tile and group gets more.
size_t mla_step_mx_plan(MlaStepArgs& a) {
    const int64_t rows = (int64_t)a.Tq * a.H, tile = a.bf16 ? kRows : kTile;
    const int64_t most = (int64_t)a.Nb * ((((int64_t)a.max_pages << a.page_shift) + tile - 1) / tile);
    const int64_t sets = (rows + 15) / 16;
    if (a.bf16) {
        int64_t per = 6;                                          // sets a workgroup
        while (per > 1 && (sets + per - 2) / (per - 1) * most <= 256) --per;
        a.groups = (int32_t)((sets + per - 1) / per);
        const int64_t n = (sets + a.groups - 1) / a.groups;
        a.waves = (int32_t)(n <= 2 ? n : n <= 4 ? 4 : 6);
        a.groups = (int32_t)((sets + a.waves - 1) / a.waves);
    } else {
        const int64_t blocks = (sets + 1) / 2;
        int64_t per = most_blocks(a.Dc);
        while (per > 1 && (blocks + per - 2) / (per - 1) * most <= 256) --per;
        a.groups = (int32_t)((blocks + per - 1) / per);
        a.waves = (int32_t)((blocks + a.groups - 1) / a.groups) * 2;
    }
    int64_t parts = kMaxParts * (a.bf16 ? residents(a.Dc, a.waves) : 1) / a.groups;
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
