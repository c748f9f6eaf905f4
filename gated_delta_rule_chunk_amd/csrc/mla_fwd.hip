// Latent attention, expanded form: softmax attention whose keys are a part
// per head and a part shared by the heads,
//   s_ij = scale (q_i[:Dn] . k_j + q_i[Dn:] . r_j),  p = softmax_j s,  o_i = sum_j p_ij v_j,
// over the visible keys j <= i + Lk - Lq (causal) or all, one pass over the
// keys with the running maximum and sum of the softmax.
//
// A workgroup takes 4 x 32 x QB queries of one head (a wave 32 QB of them) and
// walks the keys in tiles of BN. The key and value tiles go straight from
// global memory to LDS, two buffers, the next tile in flight while one is
// computed; queries, scores, probabilities and outputs stay in registers (the
// scores are formed transposed: mla_common.hpp). Bound by the matrix cores and
// the exponentials: 2 (2 Dn + Dr) products per score.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

template <class T> constexpr int kFwdKeys = sizeof(T) == 2 ? 64 : 32;   // keys a tile

template <class T, int DN, int DR, int QB>
__global__ __launch_bounds__(256, QB == 1 && sizeof(T) == 2 ? 2 : 1) void mla_fwd_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BN = kFwdKeys<T>, KB = BN / 32, BM = 128 * QB;
    constexpr int CK = DN / kChunk<T>, CR = DR / kChunk<T>;             // chunks per row
    constexpr int kK = BN * CK * 16, kR = BN * CR * 16, kBuf = 2 * kK + kR;
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5;
    int h;
    int64_t slot;
    head_and_slot(slots, a.H, h, slot);
    slot = slots - 1 - slot;                            // a sequence's longest rows of keys first
    int n, q0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuq, a.N, a.Tq, BM, slot, lane, n, qs, Lq, q0)) return;
    const bool rest = a.cuq && n == a.N;                // rows behind the last sequence: zeros, if anything
    if (rest && !a.zero_rest) return;
    seq_range(a.cuk, a.N, rest ? 0 : n, a.Tk, ks, Lk);
    if (rest) Lk = 0;
    const int off = Lk - Lq;                            // row i sees keys j <= i + off
    const int wq0 = q0 + 32 * QB * w;
    const int last = (q0 + BM < Lq ? q0 + BM : Lq) - 1;
    int keys = Lk;                                      // keys that any row of the tile sees
    if (a.causal) keys = last + off + 1 < Lk ? last + off + 1 : Lk;
    const int tiles = keys > 0 ? (keys + BN - 1) / BN : 0;

    const T* qp = static_cast<const T*>(a.q);
    const int64_t kvs = (int64_t)a.H * 2 * DN * sizeof(T);
    const char* kvp = static_cast<const char*>(a.kv) + ks * kvs + (int64_t)h * 2 * DN * sizeof(T);
    const int64_t krs = a.kr_row * sizeof(T);
    const char* krp = nullptr;
    if constexpr (DR > 0)
        krp = static_cast<const char*>(a.kr) + (a.cuk ? ks * krs : (int64_t)n * a.kr_batch * (int64_t)sizeof(T));

    Frag<T> qf[QB][DQ / 16];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        int i = wq0 + 32 * b + n32;
        i = i < Lq ? i : Lq - 1;
        const T* p = qp + ((qs + i) * a.H + h) * DQ + 8 * hf;
#pragma unroll
        for (int s = 0; s < DQ / 16; ++s) qf[b][s] = load8(p + 16 * s);
    }
    f32x16 acc[QB][DN / 32];
    float m[QB], l[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        m[b] = -INFINITY;
        l[b] = 0.f;
#pragma unroll
        for (int d = 0; d < DN / 32; ++d) acc[b][d] = zero16();
    }
    const float c = a.scale * kLog2e;

    TileLoad<CK, BN, 4> lk;
    TileLoad<DR ? CR : 8, BN, 4> lr;
    lk.init(kvs, w, lane);
    if constexpr (DR > 0) lr.init(krs, w, lane);
    auto load = [&](int t, char* buf) {
        const int k0 = t * BN, rmax = Lk - 1 - k0;
        lk.load(buf, kvp + k0 * kvs, kvs, rmax, w, lane);
        lk.load(buf + kK, kvp + DN * sizeof(T) + k0 * kvs, kvs, rmax, w, lane);
        if constexpr (DR > 0) lr.load(buf + 2 * kK, krp + k0 * krs, krs, rmax, w, lane);
    };
    auto tile_step = [&](int t, const char* buf, char* next) {
        if (t + 1 < tiles) load(t + 1, next);
        const int k0 = t * BN;
        // rows of this wave all before the tile's first key: nothing to do
        if (!a.causal || k0 <= wq0 + 32 * QB - 1 + off) {
            f32x16 sc[QB][KB];
#pragma unroll
            for (int b = 0; b < QB; ++b)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) sc[b][kb] = zero16();
#pragma unroll
            for (int s = 0; s < DQ / 16; ++s)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    Frag<T> kf;
                    if (s < DN / 16) {
                        kf = read_rows<T, CK>(buf, 32 * kb + n32, s, hf);
                    } else if constexpr (DR > 0) {
                        kf = read_rows<T, CR>(buf + 2 * kK, 32 * kb + n32, s - DN / 16, hf);
                    }
#pragma unroll
                    for (int b = 0; b < QB; ++b) sc[b][kb] = mma(kf, qf[b][s], sc[b][kb]);
                }
            if constexpr (sizeof(T) == 2) sched_reads_under_mma<6, 1, DQ / 16 * KB - 6>();
            // hide keys past the sequence or after the row
            if (k0 + BN > Lk || (a.causal && k0 + BN - 1 > wq0 + off)) {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    int lim = Lk - 1 - k0;
                    if (a.causal) {
                        const int x = wq0 + 32 * b + n32 + off - k0;
                        lim = x < lim ? x : lim;
                    }
                    lim -= 4 * hf;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            sc[b][kb][r] = 32 * kb + 8 * (r / 4) + r % 4 > lim ? -INFINITY : sc[b][kb][r];
                }
            }
            float mx[QB];
            bool grown = false;
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                mx[b] = sc[b][0][0];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 16; ++r) mx[b] = fmaxf(mx[b], sc[b][kb][r]);
                mx[b] = half_max(mx[b]);
                grown |= (mx[b] - m[b]) * c > 8.f;
            }
            // The running maximum moves only when some row's grows by more
            // than 2^8 (from -inf at first): until then its terms reach at
            // most 2^8, exact enough in float32, and the output needs no
            // rescaling.
            if (__any(grown)) {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    const float mn = fmaxf(m[b], mx[b]);
                    const float ms = mn == -INFINITY ? 0.f : mn;      // nothing seen yet: all terms are 0
                    const float al = __builtin_amdgcn_exp2f((m[b] - ms) * c);
                    l[b] *= al;
                    m[b] = mn;
#pragma unroll
                    for (int d = 0; d < DN / 32; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[b][d][r] *= al;
                }
            }
            const char* vb = buf + kK;
            auto read = [&](int i) {
                return read_cols<T, CK>(vb, 16 * (i / (DN / 32)), 32 * (i % (DN / 32)), lane);
            };
            ReadAhead<T, KB * DN / 16, 3> ahead;
            ahead.start(read);
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                const float mc = m[b] == -INFINITY ? 0.f : m[b] * c;
                float sum = 0.f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][kb][r], c, -mc));
                        sc[b][kb][r] = p;
                        sum += p;
                    }
                l[b] += sum;
            }
            Frag<T> pf[QB][2 * KB];
#pragma unroll
            for (int b = 0; b < QB; ++b)
#pragma unroll
                for (int s = 0; s < 2 * KB; ++s) pf[b][s] = to_frag<T>(sc[b][s / 2], s % 2);
            ahead.template run<QB>(read, [&](int i, const Frag<T>& x) {
                const int s = i / (DN / 32), d = i % (DN / 32);
#pragma unroll
                for (int b = 0; b < QB; ++b) acc[b][d] = mma(x, pf[b][s], acc[b][d]);
            });
        }
        wait_loads_and_lds();
        wg_barrier();
    };
    if (tiles > 0) load(0, smem[0]);
    wait_loads_and_lds();
    wg_barrier();
    for (int t = 0; t < tiles; t += 2) {
        tile_step(t, smem[0], smem[1]);
        if (t + 1 < tiles) tile_step(t + 1, smem[1], smem[0]);
    }
    T* op = static_cast<T*>(a.o);
#pragma unroll
    for (int b = 0; b < QB; ++b) {
        const int i = wq0 + 32 * b + n32;
        const float lt = half_sum(l[b]);
        const float inv = lt > 0.f ? 1.f / lt : lt == 0.f ? 0.f : lt;   // no visible key: 0; NaN stays NaN
        const bool live = i < Lq;
        T* p = op + ((qs + (live ? i : 0)) * a.H + h) * DN;
#pragma unroll
        for (int d = 0; d < DN / 32; ++d) store_tile<T>(p + 32 * d, acc[b][d], inv, hf, live);
        if (a.lse && live && hf == 0) {
            const float v = lt == 0.f ? -INFINITY : (m[b] * c + __builtin_amdgcn_logf(lt)) * 0.6931471805599453f;
            const int64_t row = a.cuq ? qs + i : i;
            a.lse[((a.cuq ? 0 : (int64_t)n * a.H) + h) * a.Tq + row] = v;
        }
    }
}

template <class T, int DN, int DR, int QB> hipError_t launch(const MlaArgs& a, hipStream_t s) {
    const int64_t slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 128 * QB);
    const int64_t items = slots * a.H;
    if (items == 0) return hipSuccess;
    mla_fwd_kernel<T, DN, DR, QB><<<dim3((unsigned)items), 256, 0, s>>>(a, slots);
    return hipGetLastError();
}

template <class T> hipError_t launch_dims(const MlaArgs& a, hipStream_t s) {
    if (a.Dn == 128) return a.Dr ? launch<T, 128, 64, 1>(a, s) : launch<T, 128, 0, 1>(a, s);
    return a.Dr ? launch<T, 64, 64, 1>(a, s) : launch<T, 64, 0, 1>(a, s);
}

}  // namespace

hipError_t launch_mla_fwd(const MlaArgs& a, hipStream_t s) {
    return a.bf16 ? launch_dims<__bf16>(a, s) : launch_dims<float>(a, s);
}

}  // namespace kda
