// Second kernel of the expanded latent attention's backward (mla_bwd.hip): a
// block of keys walks over the queries that see it, dk and dv in registers.
// In a header because the two element types want different registers for
// their accumulators: mla_dkv_bf16.hip and mla_bwd.hip.
// One wave per SIMD: keys, values and the two accumulators of 32 keys take 240
// of its registers, so its matrix and vector instructions do not overlap and the
// matrix cores are busy 37-39% of the time. The split kernels of 128 + 64 channels
// spill, float32's 4 registers, bf16's 1. Two things that shorten other loops
// here lengthen this one (bf16, 4096 tokens, 96 heads): the next tile's loads
// issued among the products 1517 against 1303 us, the scores' operands read a
// fixed six ahead 1400.
#pragma once

#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace mla {

template <class T, int DN, int DR, bool SPLIT>
__global__ __launch_bounds__(256, 1) void mla_dkv_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BQ = sizeof(T) == 2 && !SPLIT ? 64 : 32, QB = BQ / 32, BK = SPLIT ? 32 : 128;
    constexpr int CN = DN / kChunk<T>, CR = DR / kChunk<T>, NV = DN / 32, NK = DQ / 32;
    constexpr int kQ = BQ * CN * 16, kTileBytes = 2 * kQ + BQ * CR * 16;       // q's own part, d_o, q's shared part
    constexpr int kBuf = SPLIT ? larger(kTileBytes, (NV + NK) * 4096) : kTileBytes;    // split: also the exchange
    constexpr int kLoaders = SPLIT ? 1 : 4;
    __shared__ __attribute__((aligned(1024))) char smem[SPLIT ? 4 : 2][kBuf];
    // lse (base 2) and D of the tile's rows; split: in registers, row n32 on lane n32
    __shared__ __attribute__((aligned(16))) float stat[SPLIT ? 1 : 2][2][SPLIT ? 1 : BQ];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5, lw = SPLIT ? 0 : w;
    int h;
    int64_t slot;
    const int part = SPLIT ? (int)(blockIdx.x / (slots * a.H)) : 0;
    head_and_slot(blockIdx.x - part * slots * a.H, slots, a.H, h, slot);
    int n, k0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuk, a.N, a.Tk, BK, slot, lane, n, ks, Lk, k0)) return;
    const bool rest = a.cuk && n == a.N;
    if (rest && !a.zero_rest) return;
    seq_range(a.cuq, a.N, rest ? 0 : n, a.Tq, qs, Lq);
    if (rest) Lq = 0;
    const int off = Lk - Lq;
    const int wk0 = k0 + 32 * lw, j = wk0 + n32, jc = j < Lk ? j : Lk - 1;
    // the first query that sees the block's first key, down to a tile's start
    int first = 0;
    if (a.causal && k0 - off > 0) first = (k0 - off) / BQ * BQ;
    const int tiles = first < Lq ? (Lq - first + BQ - 1) / BQ : 0;

    Frag<T> kf[DQ / 16], vf[DN / 16];
    const int64_t kvrow = (ks + jc) * a.H + h;
    {
        const T* p = static_cast<const T*>(a.kv) + kvrow * 2 * DN + 8 * hf;
#pragma unroll
        for (int s = 0; s < DN / 16; ++s) {
            kf[s] = load8(p + 16 * s);
            vf[s] = load8(p + DN + 16 * s);
        }
        if constexpr (DR > 0) {
            const T* r = static_cast<const T*>(a.kr) + 8 * hf +
                         (a.cuk ? (ks + jc) * a.kr_row : n * a.kr_batch + jc * a.kr_row);
#pragma unroll
            for (int s = 0; s < DR / 16; ++s) kf[DN / 16 + s] = load8(r + 16 * s);
        }
    }
    f32x16 dk[DQ / 32], dv[DN / 32];
#pragma unroll
    for (int d = 0; d < DQ / 32; ++d) dk[d] = zero16();
#pragma unroll
    for (int d = 0; d < DN / 32; ++d) dv[d] = zero16();
    const float c = a.scale * kLog2e;
    const int64_t qst = (int64_t)a.H * DQ * sizeof(T), ost = (int64_t)a.H * DN * sizeof(T);
    const char* qp = static_cast<const char*>(a.q) + (qs * a.H + h) * DQ * (int64_t)sizeof(T);
    const char* dp_ = static_cast<const char*>(a.d_o) + (qs * a.H + h) * DN * (int64_t)sizeof(T);
    const int64_t srow = ((a.cuq ? 0 : (int64_t)n * a.H) + h) * a.Tq + (a.cuq ? qs : 0);

    TileLoad<CN, BQ, kLoaders> lq, ld;
    TileLoad<DR ? CR : 8, BQ, kLoaders> lr;
    lq.init(qst, lw, lane);
    ld.init(ost, lw, lane);
    if constexpr (DR > 0) lr.init(qst, lw, lane);
    auto load = [&](int t, char* buf) {
        const int r0 = first + t * BQ, rmax = Lq - 1 - r0;
        lq.load(buf, qp + r0 * qst, qst, rmax, lw, lane);
        ld.load(buf + kQ, dp_ + r0 * ost, ost, rmax, lw, lane);
        if constexpr (DR > 0) lr.load(buf + 2 * kQ, qp + DN * sizeof(T) + r0 * qst, qst, rmax, lw, lane);
    };
    // Rows past the sequence and rows without a visible key get lse = +inf,
    // which makes all their terms zero.
    auto row_lse = [&](int r) {
        const float x = r < Lq ? a.lse[srow + r] * kLog2e : INFINITY;
        return x == -INFINITY ? INFINITY : x;
    };
    auto row_delta = [&](int r) {
        if (r >= Lq) return 0.f;
        const float* d = a.delta + srow + r;
        float x = *d;
        if constexpr (sizeof(T) == 2)
            for (int p = 1; p < a.delta_parts; ++p) x += *(d += (int64_t)a.B * a.H * a.Tq);
        return x;
    };
    // stats(qb, g, l2, de): lse and D of rows 8 g + 4 hf .. + 3 of query block qb
    auto compute = [&](int t, const char* buf, auto stats) {
#pragma unroll
        for (int qb = 0; qb < QB; ++qb) {
            const int r0 = first + t * BQ + 32 * qb;       // query r0 sees keys <= r0 + off
            if (a.causal && wk0 > r0 + 31 + off) continue;
            f32x16 sc = zero16(), dp = zero16();
#pragma unroll
            for (int s = 0; s < DQ / 16; ++s) {
                if (s < DN / 16) {
                    sc = mma(read_rows<T, CN>(buf, 32 * qb + n32, s, hf), kf[s], sc);
                    dp = mma(read_rows<T, CN>(buf + kQ, 32 * qb + n32, s, hf), vf[s < DN / 16 ? s : 0], dp);
                } else if constexpr (DR > 0) {
                    sc = mma(read_rows<T, CR>(buf + 2 * kQ, 32 * qb + n32, s - DN / 16, hf), kf[s], sc);
                }
            }
            if constexpr (sizeof(T) == 2) sched_reads_under_mma<6, 1, (DQ + DN) / 16 - 6>();
            if (a.causal && wk0 + 31 > r0 + off) {
                const int lim = j - off - r0 - 4 * hf;     // rows below it do not see this lane's key
#pragma unroll
                for (int r = 0; r < 16; ++r) sc[r] = 8 * (r / 4) + r % 4 < lim ? -INFINITY : sc[r];
            }
            // operands of a step: d_o for dv, then q for dk
            auto read = [&](int i) -> Frag<T> {
                const int s = i / (NV + NK), d = i % (NV + NK);
                if (d < NV) return read_cols<T, CN>(buf + kQ, 32 * qb + 16 * s, 32 * d, lane);
                if constexpr (DR > 0)
                    if (d >= 2 * NV) return read_cols<T, CR>(buf + 2 * kQ, 32 * qb + 16 * s, 32 * (d - 2 * NV), lane);
                return read_cols<T, CN>(buf, 32 * qb + 16 * s, 32 * (d - NV), lane);
            };
            ReadAhead<T, 2 * (NV + NK), 4> ahead;
            ahead.start(read);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 l2, de;
                stats(qb, g, l2, de);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * g + e;
                    sc[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r], c, -l2[e]));
                    dp[r] = sc[r] * (dp[r] - de[e]);
                }
            }
            const Frag<T> pf[2] = {to_frag<T>(sc, 0), to_frag<T>(sc, 1)};
            const Frag<T> sf[2] = {to_frag<T>(dp, 0), to_frag<T>(dp, 1)};
            ahead.run(read, [&](int i, const Frag<T>& x) {
                const int s = i / (NV + NK), d = i % (NV + NK);
                if (d < NV) dv[d] = mma(x, pf[s], dv[d]);
                else dk[d - NV] = mma(x, sf[s], dk[d - NV]);
            });
        }
    };
    const bool live = j < Lk;
    T* p = static_cast<T*>(a.dkv) + kvrow * 2 * DN;
    float* r = nullptr;
    if constexpr (DR > 0) r = a.dkr_part + ((((int64_t)part * a.H + h) * a.B + (a.cuk ? 0 : n)) * a.Tk + (a.cuk ? ks + jc : jc)) * DR;
    // block d of the results: dk, then dv
    float* f = SPLIT && a.k_parts > 1 ? a.dkv_part + ((int64_t)part * a.B * a.Tk * a.H + kvrow) * 2 * DN : nullptr;
    auto store = [&](int d, const f32x16& x) {
        if (SPLIT && f && (d < NV || d >= NK)) {
            store_tile<float>(f + (d < NV ? 32 * d : DN + 32 * (d - NK)), x, d < NV ? a.scale : 1.f, hf, live);
            return;
        }
        if (d < NV) store_tile<T>(p + 32 * d, x, a.scale, hf, live);
        else if (d < NK) store_tile<float>(r + 32 * (d - NV), x, a.scale, hf, live);
        else store_tile<T>(p + DN + 32 * (d - NK), x, 1.f, hf, live);
    };
    if constexpr (SPLIT) {
        for (int t = w + 4 * part; t < tiles; t += 4 * a.k_parts) {
            load(t, smem[w]);
            const int row = first + t * BQ + n32;
            const float ls = row_lse(row), dl = row_delta(row);
            wait_loads_and_lds();
            compute(t, smem[w], [&](int, int g, f32x4& l2, f32x4& de) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l2[e] = __shfl(ls, 8 * g + 4 * hf + e);
                    de[e] = __shfl(dl, 8 * g + 4 * hf + e);
                }
            });
            wait_loads_and_lds();
        }
#pragma unroll
        for (int d = 0; d < NK; ++d) put_block(smem[w], d, dk[d], lane);
#pragma unroll
        for (int d = 0; d < NV; ++d) put_block(smem[w], NK + d, dv[d], lane);
        wait_loads_and_lds();
        wg_barrier();
        const float one[4] = {1.f, 1.f, 1.f, 1.f};
        for (int d = w; d < NK + NV; d += 4) store(d, sum_blocks(smem[0], kBuf, d, one, lane));
    } else {
        const int sr = threadIdx.x % BQ, sk = threadIdx.x / BQ;   // what this thread fetches of the statistics
        auto fetch = [&](int t) -> float {
            if (sk == 0) return row_lse(first + t * BQ + sr);
            return sk == 1 ? row_delta(first + t * BQ + sr) : 0.f;
        };
        if (tiles > 0) {
            load(0, smem[0]);
            const float x = fetch(0);
            if (sk < 2) stat[0][sk][sr] = x;
        }
        wait_loads_and_lds();
        wg_barrier();
        for (int t = 0; t < tiles; ++t) {
            float x = 0.f;
            if (t + 1 < tiles) {
                x = fetch(t + 1);
                load(t + 1, smem[(t + 1) & 1]);
            }
            compute(t, smem[t & 1], [&](int qb, int g, f32x4& l2, f32x4& de) {
                l2 = *reinterpret_cast<const f32x4*>(&stat[t & 1][0][32 * qb + 8 * g + 4 * hf]);
                de = *reinterpret_cast<const f32x4*>(&stat[t & 1][1][32 * qb + 8 * g + 4 * hf]);
            });
            if (t + 1 < tiles && sk < 2) stat[(t + 1) & 1][sk][sr] = x;
            wait_loads_and_lds();
            wg_barrier();
        }
#pragma unroll
        for (int d = 0; d < NK; ++d) store(d, dk[d]);
#pragma unroll
        for (int d = 0; d < NV; ++d) store(NK + d, dv[d]);
    }
}

template <class T, int DN, int DR> hipError_t launch_dkv(const MlaArgs& a, hipStream_t s) {
    if (a.Tk == 0) return hipSuccess;
    int64_t slots = tile_slots(a.cuk, a.B, a.N, a.Tk, 128);
    if (slots * a.H < kSmallLaunch<T>) {
        slots = tile_slots(a.cuk, a.B, a.N, a.Tk, 32);
        mla_dkv_kernel<T, DN, DR, true><<<dim3((unsigned)(slots * a.H * a.k_parts)), 256, 0, s>>>(a, slots);
    } else {
        mla_dkv_kernel<T, DN, DR, false><<<dim3((unsigned)(slots * a.H)), 256, 0, s>>>(a, slots);
    }
    return hipGetLastError();
}
template <class T> hipError_t launch_dkv_dims(const MlaArgs& a, hipStream_t s) {
    if (a.Dn == 128) return a.Dr ? launch_dkv<T, 128, 64>(a, s) : launch_dkv<T, 128, 0>(a, s);
    return a.Dr ? launch_dkv<T, 64, 64>(a, s) : launch_dkv<T, 64, 0>(a, s);
}

}  // namespace mla
}  // namespace kda
