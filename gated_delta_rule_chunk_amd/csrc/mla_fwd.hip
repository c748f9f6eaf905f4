// Latent attention, expanded form: softmax attention whose keys are a part
// per head and a part shared by the heads,
//   s_ij = scale (q_i[:Dn] . k_j + q_i[Dn:] . r_j),  p = softmax_j s,  o_i = sum_j p_ij v_j,
// over the visible keys j <= i + Lk - Lq (causal) or all, one pass over the
// keys with the running maximum and sum of the softmax.
//
// A workgroup takes 128 queries of one head (a wave 32 of them) and walks the
// keys in tiles of BN. The key and value tiles go straight from
// global memory to LDS, two buffers, the next tile in flight while one is
// computed; queries, scores, probabilities and outputs stay in registers (the
// scores are formed transposed: mla_common.hpp). In bf16 the probabilities are
// rounded once, as operands, their sum is not: the matrix cores take bf16, and
// the result is off by 0.0020-0.0023 of its norm where its own rounding alone
// leaves 0.0017. Bound by the matrix cores and
// the exponentials, 2 (2 Dn + Dr) products per score: a wave's own matrix and
// vector instructions hardly overlap, those of the two waves on a SIMD do.
// Measured, bf16, causal, 4096 tokens, 96 heads of 128 + 64 channels: 484-565
// us, 910-1060 TFLOP/s over the visible pairs (a plain 8192^3 product of the
// library: 1131), matrix cores busy 55% of the time, no bank conflicts.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

template <class T, int DN, int DR, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void mla_fwd_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BN = sizeof(T) == 2 && !SPLIT ? 64 : 32, KB = BN / 32, BM = SPLIT ? 32 : 128;
    constexpr int CK = DN / kChunk<T>, CR = DR / kChunk<T>;             // chunks per row
    constexpr int kK = BN * CK * 16, kR = BN * CR * 16, kTileBytes = 2 * kK + kR;
    // two buffers; or one a wave, which the exchange (accumulators, maxima, sums) uses later
    constexpr int kBuf = SPLIT ? larger(kTileBytes, DN * 128 + 256) : kTileBytes;
    constexpr int kLoaders = SPLIT ? 1 : 4;                             // waves that load a tile together
    __shared__ __attribute__((aligned(1024))) char smem[SPLIT ? 4 : 2][kBuf];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5, lw = SPLIT ? 0 : w;
    int h;
    int64_t slot;
    head_and_slot(blockIdx.x, slots, a.H, h, slot);
    slot = slots - 1 - slot;                            // a sequence's longest rows of keys first
    int n, q0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuq, a.N, a.Tq, BM, slot, lane, n, qs, Lq, q0)) return;
    const bool rest = a.cuq && n == a.N;                // rows behind the last sequence: zeros, if anything
    if (rest && !a.zero_rest) return;
    seq_range(a.cuk, a.N, rest ? 0 : n, a.Tk, ks, Lk);
    if (rest) Lk = 0;
    const int off = Lk - Lq;                            // row i sees keys j <= i + off
    const int wq0 = q0 + 32 * lw;
    const int last = (q0 + BM < Lq ? q0 + BM : Lq) - 1;
    int keys = Lk;                                      // keys that any row of the tile sees
    if (a.causal) keys = last + off + 1 < Lk ? last + off + 1 : Lk;
    const int tiles = keys > 0 ? (keys + BN - 1) / BN : 0;

    const int64_t kvs = (int64_t)a.H * 2 * DN * sizeof(T);
    const char* kvp = static_cast<const char*>(a.kv) + ks * kvs + (int64_t)h * 2 * DN * sizeof(T);
    const int64_t krs = a.kr_row * sizeof(T);
    const char* krp = nullptr;
    if constexpr (DR > 0)
        krp = static_cast<const char*>(a.kr) + (a.cuk ? ks * krs : (int64_t)n * a.kr_batch * (int64_t)sizeof(T));

    const int i = wq0 + n32;                            // this lane's row
    const bool live = i < Lq;
    const int64_t qrow = (qs + (live ? i : Lq - 1)) * a.H + h;
    Frag<T> qf[DQ / 16];
    {
        const T* p = static_cast<const T*>(a.q) + qrow * DQ + 8 * hf;
#pragma unroll
        for (int s = 0; s < DQ / 16; ++s) qf[s] = load8(p + 16 * s);
    }
    f32x16 acc[DN / 32];
#pragma unroll
    for (int d = 0; d < DN / 32; ++d) acc[d] = zero16();
    float m = -INFINITY, l = 0.f;
    const float c = a.scale * kLog2e;

    TileLoad<CK, BN, kLoaders> lk;
    TileLoad<DR ? CR : 8, BN, kLoaders> lr;
    lk.init(kvs, lw, lane);
    if constexpr (DR > 0) lr.init(krs, lw, lane);
    auto load = [&](int t, char* buf) {
        const int k0 = t * BN, rmax = Lk - 1 - k0;
        lk.load(buf, kvp + k0 * kvs, kvs, rmax, lw, lane);
        lk.load(buf + kK, kvp + DN * sizeof(T) + k0 * kvs, kvs, rmax, lw, lane);
        if constexpr (DR > 0) lr.load(buf + 2 * kK, krp + k0 * krs, krs, rmax, lw, lane);
    };
    auto compute = [&](int t, const char* buf) {
        const int k0 = t * BN;
        // rows of this wave all before the tile's first key: nothing to do
        if (a.causal && k0 > wq0 + 31 + off) return;
        f32x16 sc[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) sc[kb] = zero16();
#pragma unroll
        for (int s = 0; s < DQ / 16; ++s)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                if (s < DN / 16) {
                    sc[kb] = mma(read_rows<T, CK>(buf, 32 * kb + n32, s, hf), qf[s], sc[kb]);
                } else if constexpr (DR > 0) {
                    sc[kb] = mma(read_rows<T, CR>(buf + 2 * kK, 32 * kb + n32, s - DN / 16, hf), qf[s], sc[kb]);
                }
            }
        if constexpr (sizeof(T) == 2) sched_reads_under_mma<larger(DQ / 32, 2), 1, DQ / 16 * KB - larger(DQ / 32, 2)>();
        // hide keys past the sequence or after the row
        if (k0 + BN > Lk || (a.causal && k0 + BN - 1 > wq0 + off)) {
            int lim = Lk - 1 - k0;
            if (a.causal) lim = i + off - k0 < lim ? i + off - k0 : lim;
            lim -= 4 * hf;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sc[kb][r] = 32 * kb + 8 * (r / 4) + r % 4 > lim ? -INFINITY : sc[kb][r];
        }
        float mx = sc[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, sc[kb][r]);
        mx = half_max(mx);
        // The running maximum moves only when some row's grows by more than
        // 2^8 (from -inf at first): until then its terms reach at most 2^8,
        // exact enough in float32, and the output needs no rescaling (the
        // published conditional rescaling of the online softmax).
        if (__any((mx - m) * c > 8.f)) {
            const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: all terms are 0
            const float al = __builtin_amdgcn_exp2f((m - ms) * c);
            l *= al;
            m = mn;
#pragma unroll
            for (int d = 0; d < DN / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] *= al;
        }
        const char* vb = buf + kK;
        auto read = [&](int x) { return read_cols<T, CK>(vb, 16 * (x / (DN / 32)), 32 * (x % (DN / 32)), lane); };
        ReadAhead<T, KB * DN / 16, 3> ahead;
        ahead.start(read);
        const float mc = m == -INFINITY ? 0.f : m * c;
        float sum = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[kb][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[kb][r], c, -mc));
                sum += sc[kb][r];
            }
        l += sum;
        Frag<T> pf[2 * KB];
#pragma unroll
        for (int s = 0; s < 2 * KB; ++s) pf[s] = to_frag<T>(sc[s / 2], s % 2);
        ahead.run(read, [&](int x, const Frag<T>& v) {
            acc[x % (DN / 32)] = mma(v, pf[x / (DN / 32)], acc[x % (DN / 32)]);
        });
    };
    T* op = static_cast<T*>(a.o) + qrow * DN;
    auto put_lse = [&](float mm, float lt) {
        if (a.lse && live && hf == 0)
            a.lse[((a.cuq ? 0 : (int64_t)n * a.H) + h) * a.Tq + (a.cuq ? qs + i : i)] =
                lt == 0.f ? -INFINITY : (mm * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
    };
    if constexpr (SPLIT) {
        for (int t = w; t < tiles; t += 4) {
            load(t, smem[w]);
            wait_loads_and_lds();
            compute(t, smem[w]);
            wait_loads_and_lds();
        }
        float* ml = reinterpret_cast<float*>(smem[w] + DN * 128);
        const float lw_sum = half_sum(l);
        if (hf == 0) {
            ml[n32] = m;
            ml[32 + n32] = lw_sum;
        }
#pragma unroll
        for (int d = 0; d < DN / 32; ++d) put_block(smem[w], d, acc[d], lane);
        wait_loads_and_lds();
        wg_barrier();
        float f[4], mm = -INFINITY, lt = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            f[v] = reinterpret_cast<const float*>(smem[v] + DN * 128)[n32];
            mm = fmaxf(mm, f[v]);
        }
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            f[v] = __builtin_amdgcn_exp2f((f[v] - ms) * c);
            lt += f[v] * reinterpret_cast<const float*>(smem[v] + DN * 128)[32 + n32];
        }
        const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;   // no visible key: 0; NaN stays NaN
        if (w < DN / 32) store_tile<T>(op + 32 * w, sum_blocks(smem[0], kBuf, w, f, lane), inv, hf, live);
        if (w == 0) put_lse(mm, lt);
    } else {
        if (tiles > 0) load(0, smem[0]);
        wait_loads_and_lds();
        wg_barrier();
        auto step = [&](int t, const char* buf, char* next) {
            if (t + 1 < tiles) load(t + 1, next);
            compute(t, buf);
            wait_loads_and_lds();
            wg_barrier();
        };
        for (int t = 0; t < tiles; t += 2) {
            step(t, smem[0], smem[1]);
            if (t + 1 < tiles) step(t + 1, smem[1], smem[0]);
        }
        const float lt = half_sum(l);
        const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;
#pragma unroll
        for (int d = 0; d < DN / 32; ++d) store_tile<T>(op + 32 * d, acc[d], inv, hf, live);
        put_lse(m, lt);
    }
}

template <class T, int DN, int DR> hipError_t launch(const MlaArgs& a, hipStream_t s) {
    int64_t slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 128);
    if (slots * a.H < kSmallLaunch<T>) {
        slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 32);
        mla_fwd_kernel<T, DN, DR, true><<<dim3((unsigned)(slots * a.H)), 256, 0, s>>>(a, slots);
    } else {
        mla_fwd_kernel<T, DN, DR, false><<<dim3((unsigned)(slots * a.H)), 256, 0, s>>>(a, slots);
    }
    return hipGetLastError();
}

template <class T> hipError_t launch_dims(const MlaArgs& a, hipStream_t s) {
    if (a.Dn == 128) return a.Dr ? launch<T, 128, 64>(a, s) : launch<T, 128, 0>(a, s);
    return a.Dr ? launch<T, 64, 64>(a, s) : launch<T, 64, 0>(a, s);
}

}  // namespace

hipError_t launch_mla_fwd(const MlaArgs& a, hipStream_t s) {
    return a.bf16 ? launch_dims<__bf16>(a, s) : launch_dims<float>(a, s);
}

}  // namespace kda
