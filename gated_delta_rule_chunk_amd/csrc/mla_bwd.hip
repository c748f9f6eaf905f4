// Backward of the expanded latent attention. With s_ij, p_ij, o_i as in the
// forward and lse_i = log sum_j exp s_ij:
//   p_ij = exp(s_ij - lse_i),  D_i = d_o_i . o_i,  ds_ij = p_ij (d_o_i . v_j - D_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij d_o_i,
// with k_j the key's own and shared parts together; the shared part's gradient
// is the sum of its share over the heads.
//
// Two kernels, each with every sum in one wave's registers, so that no result
// depends on an order of arrival: the first walks a block of queries over the
// keys (D on the way, dq), the second a block of keys over the queries (dk,
// dv). The scores are formed twice (two of the seven products per pair);
// adding dq from the second kernel's workgroups instead would take an atomic
// per query row, key tile and column, more bytes than the scores cost
// products. A third kernel sums the shared part over the heads, in their
// order, from float32 shares. Bound by the matrix cores.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

template <class T> constexpr int kBwdKeys = sizeof(T) == 2 ? 64 : 32;     // keys a tile (dq)
template <class T> constexpr int kBwdRows = sizeof(T) == 2 ? 64 : 32;     // queries a tile (dk, dv)

template <class T, int DN, int DR>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void mla_dq_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BN = kBwdKeys<T>, KB = BN / 32, BM = 128;
    constexpr int CK = DN / kChunk<T>, CR = DR / kChunk<T>;
    constexpr int kK = BN * CK * 16, kR = BN * CR * 16, kBuf = 2 * kK + kR;
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5;
    const int64_t item = xcd_item(slots * a.H);
    if (item < 0) return;
    const int h = (int)(item / slots);
    int n, q0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuq, a.N, a.Tq, BM, slots - 1 - item % slots, lane, n, qs, Lq, q0)) return;
    const bool rest = a.cuq && n == a.N;
    if (rest && !a.zero_rest) return;
    seq_range(a.cuk, a.N, rest ? 0 : n, a.Tk, ks, Lk);
    if (rest) Lk = 0;
    const int off = Lk - Lq;
    const int wq0 = q0 + 32 * w;
    const int last = (q0 + BM < Lq ? q0 + BM : Lq) - 1;
    int keys = Lk;
    if (a.causal) keys = last + off + 1 < Lk ? last + off + 1 : Lk;
    const int tiles = keys > 0 ? (keys + BN - 1) / BN : 0;

    const int64_t kvs = (int64_t)a.H * 2 * DN * sizeof(T);
    const char* kvp = static_cast<const char*>(a.kv) + ks * kvs + (int64_t)h * 2 * DN * sizeof(T);
    const int64_t krs = a.kr_row * sizeof(T);
    const char* krp = nullptr;
    if constexpr (DR > 0)
        krp = static_cast<const char*>(a.kr) + (a.cuk ? ks * krs : (int64_t)n * a.kr_batch * (int64_t)sizeof(T));

    const int i = wq0 + n32, ic = i < Lq ? i : Lq - 1;
    const bool live = i < Lq;
    const int64_t qrow = (qs + ic) * a.H + h;
    const int64_t srow = ((a.cuq ? 0 : (int64_t)n * a.H) + h) * a.Tq + (a.cuq ? qs + ic : ic);
    Frag<T> qf[DQ / 16], df[DN / 16];
    float delta = 0.f;
    {
        const T* p = static_cast<const T*>(a.q) + qrow * DQ + 8 * hf;
#pragma unroll
        for (int s = 0; s < DQ / 16; ++s) qf[s] = load8(p + 16 * s);
        const T* d = static_cast<const T*>(a.d_o) + qrow * DN + 8 * hf;
        const T* o = static_cast<const T*>(a.o) + qrow * DN + 8 * hf;
#pragma unroll
        for (int s = 0; s < DN / 16; ++s) {
            df[s] = load8(d + 16 * s);
            const Frag<T> of = load8(o + 16 * s);
#pragma unroll
            for (int j = 0; j < 8; ++j) delta += (float)df[s][j] * (float)of[j];
        }
        delta = half_sum(delta);
        if (live && hf == 0 && !rest) a.delta[srow] = delta;
    }
    f32x16 acc[DQ / 32];
#pragma unroll
    for (int d = 0; d < DQ / 32; ++d) acc[d] = zero16();
    const float c = a.scale * kLog2e;
    // a row without a visible key has lse -inf; all its terms are hidden below
    const float lse = rest ? 0.f : a.lse[srow], l2 = lse == -INFINITY ? 0.f : lse * kLog2e;

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
    if (tiles > 0) load(0, smem[0]);
    wait_loads_and_lds();
    wg_barrier();
    for (int t = 0; t < tiles; ++t) {
        const char* buf = smem[t & 1];
        if (t + 1 < tiles) load(t + 1, smem[(t + 1) & 1]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int k0 = t * BN + 32 * kb;
            if (a.causal && k0 > wq0 + 31 + off) continue;
            f32x16 sc = zero16(), dp = zero16();
#pragma unroll
            for (int s = 0; s < DQ / 16; ++s) {
                if (s < DN / 16) {
                    sc = mma(read_rows<T, CK>(buf, 32 * kb + n32, s, hf), qf[s], sc);
                    dp = mma(read_rows<T, CK>(buf + kK, 32 * kb + n32, s, hf), df[s < DN / 16 ? s : 0], dp);
                } else if constexpr (DR > 0) {
                    sc = mma(read_rows<T, CR>(buf + 2 * kK, 32 * kb + n32, s - DN / 16, hf), qf[s], sc);
                }
            }
            if constexpr (sizeof(T) == 2) sched_reads_under_mma<6, 1, (DQ + DN) / 16 - 6>();
            if (k0 + 32 > Lk || (a.causal && k0 + 31 > wq0 + off)) {
                int lim = Lk - 1 - k0;
                if (a.causal) {
                    const int x = i + off - k0;
                    lim = x < lim ? x : lim;
                }
                lim -= 4 * hf;
#pragma unroll
                for (int r = 0; r < 16; ++r) sc[r] = 8 * (r / 4) + r % 4 > lim ? -INFINITY : sc[r];
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r], c, -l2));
                sc[r] = p * (dp[r] - delta);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<T> f = to_frag<T>(sc, s);
#pragma unroll
                for (int d = 0; d < DQ / 32; ++d) {
                    if (d < DN / 32) {
                        acc[d] = mma(read_cols<T, CK>(buf, 32 * kb + 16 * s, 32 * d, lane), f, acc[d]);
                    } else if constexpr (DR > 0) {
                        acc[d] = mma(read_cols<T, CR>(buf + 2 * kK, 32 * kb + 16 * s, 32 * d - DN, lane), f, acc[d]);
                    }
                }
            }
            if constexpr (sizeof(T) == 2) sched_reads_over_valu<8, 90, 2, DQ / 16 - 4>();
        }
        wait_loads_and_lds();
        wg_barrier();
    }
    T* p = static_cast<T*>(a.dq) + qrow * DQ;
#pragma unroll
    for (int d = 0; d < DQ / 32; ++d) store_tile<T>(p + 32 * d, acc[d], a.scale, hf, live);
}

template <class T, int DN, int DR>
__global__ __launch_bounds__(256, 1) void mla_dkv_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BQ = kBwdRows<T>, QB = BQ / 32, BK = 128;
    constexpr int CN = DN / kChunk<T>, CR = DR / kChunk<T>;
    constexpr int kQ = BQ * CN * 16, kBuf = 2 * kQ + BQ * CR * 16;    // q's own part, d_o, q's shared part
    __shared__ __attribute__((aligned(1024))) char smem[2][kBuf];
    __shared__ __attribute__((aligned(16))) float stat[2][2][BQ];     // lse (base 2) and D of the tile's rows
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5;
    const int64_t item = xcd_item(slots * a.H);
    if (item < 0) return;
    const int h = (int)(item / slots);
    int n, k0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuk, a.N, a.Tk, BK, item % slots, lane, n, ks, Lk, k0)) return;
    const bool rest = a.cuk && n == a.N;
    if (rest && !a.zero_rest) return;
    seq_range(a.cuq, a.N, rest ? 0 : n, a.Tq, qs, Lq);
    if (rest) Lq = 0;
    const int off = Lk - Lq;
    const int wk0 = k0 + 32 * w, j = wk0 + n32, jc = j < Lk ? j : Lk - 1;
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

    TileLoad<CN, BQ, 4> lq, ld;
    TileLoad<DR ? CR : 8, BQ, 4> lr;
    lq.init(qst, w, lane);
    ld.init(ost, w, lane);
    if constexpr (DR > 0) lr.init(qst, w, lane);
    auto load = [&](int t, char* buf) {
        const int r0 = first + t * BQ, rmax = Lq - 1 - r0;
        lq.load(buf, qp + r0 * qst, qst, rmax, w, lane);
        ld.load(buf + kQ, dp_ + r0 * ost, ost, rmax, w, lane);
        if constexpr (DR > 0) lr.load(buf + 2 * kQ, qp + DN * sizeof(T) + r0 * qst, qst, rmax, w, lane);
    };
    // Rows past the sequence and rows without a visible key get lse = +inf,
    // which makes all their terms zero.
    auto load_stat = [&](int t, float& x) {
        const int r = first + t * BQ + (threadIdx.x & (BQ - 1));
        if ((int)threadIdx.x < BQ) {
            x = r < Lq ? a.lse[srow + r] * kLog2e : INFINITY;
            if (x == -INFINITY) x = INFINITY;
        } else if ((int)threadIdx.x < 2 * BQ) {
            x = r < Lq ? a.delta[srow + r] : 0.f;
        }
    };
    auto put_stat = [&](int b, float x) {
        if ((int)threadIdx.x < 2 * BQ) stat[b][threadIdx.x / BQ][threadIdx.x % BQ] = x;
    };
    float x = 0.f;
    if (tiles > 0) {
        load(0, smem[0]);
        load_stat(0, x);
        put_stat(0, x);
    }
    wait_loads_and_lds();
    wg_barrier();
    for (int t = 0; t < tiles; ++t) {
        const char* buf = smem[t & 1];
        if (t + 1 < tiles) {
            load_stat(t + 1, x);
            load(t + 1, smem[(t + 1) & 1]);
        }
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
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 l2 = *reinterpret_cast<const f32x4*>(&stat[t & 1][0][32 * qb + 8 * g + 4 * hf]);
                const f32x4 de = *reinterpret_cast<const f32x4*>(&stat[t & 1][1][32 * qb + 8 * g + 4 * hf]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * g + e;
                    sc[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r], c, -l2[e]));
                    dp[r] = sc[r] * (dp[r] - de[e]);
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<T> pf = to_frag<T>(sc, s), sf = to_frag<T>(dp, s);
#pragma unroll
                for (int d = 0; d < DN / 32; ++d)
                    dv[d] = mma(read_cols<T, CN>(buf + kQ, 32 * qb + 16 * s, 32 * d, lane), pf, dv[d]);
#pragma unroll
                for (int d = 0; d < DQ / 32; ++d) {
                    if (d < DN / 32) {
                        dk[d] = mma(read_cols<T, CN>(buf, 32 * qb + 16 * s, 32 * d, lane), sf, dk[d]);
                    } else if constexpr (DR > 0) {
                        dk[d] = mma(read_cols<T, CR>(buf + 2 * kQ, 32 * qb + 16 * s, 32 * d - DN, lane), sf, dk[d]);
                    }
                }
            }
            if constexpr (sizeof(T) == 2) sched_reads_over_valu<16, 110, 2, (DQ + DN) / 16 - 4>();
        }
        if (t + 1 < tiles) put_stat((t + 1) & 1, x);
        wait_loads_and_lds();
        wg_barrier();
    }
    const bool live = j < Lk;
    T* p = static_cast<T*>(a.dkv) + kvrow * 2 * DN;
#pragma unroll
    for (int d = 0; d < DN / 32; ++d) {
        store_tile<T>(p + 32 * d, dk[d], a.scale, hf, live);
        store_tile<T>(p + DN + 32 * d, dv[d], 1.f, hf, live);
    }
    if constexpr (DR > 0) {
        float* r = a.dkr_part + (((int64_t)h * a.B + (a.cuk ? 0 : n)) * a.Tk + (a.cuk ? ks + jc : jc)) * DR;
#pragma unroll
        for (int d = 0; d < DR / 32; ++d) store_tile<float>(r + 32 * d, dk[DN / 32 + d], a.scale, hf, live);
    }
}

// Sums the shared key part's shares over the heads, in their order: four
// columns a thread.
template <class T> __global__ __launch_bounds__(256) void mla_dkr_kernel(MlaArgs a, int64_t quads) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= quads) return;
    const int64_t per = (int64_t)a.B * a.Tk * a.Dr;
    if (a.cuk && !a.zero_rest) {
        int64_t s;
        int len;
        seq_range(a.cuk, a.N, a.N, a.Tk, s, len);
        if (x * 4 / a.Dr >= s) return;
    }
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const float* p = a.dkr_part + 4 * x;
#pragma unroll 8
    for (int h = 0; h < a.H; ++h) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + h * per);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += v[j];
    }
    T* o = static_cast<T*>(a.dkr) + 4 * x;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (T)sum[j];
}

template <class T, int DN, int DR> hipError_t launch(const MlaArgs& a, hipStream_t s) {
    hipError_t e;
    int64_t slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 128), items = slots * a.H;
    if (a.Tq > 0) {
        mla_dq_kernel<T, DN, DR><<<dim3((unsigned)((items + 7) / 8 * 8)), 256, 0, s>>>(a, slots);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.Tk == 0) return hipSuccess;
    slots = tile_slots(a.cuk, a.B, a.N, a.Tk, 128), items = slots * a.H;
    mla_dkv_kernel<T, DN, DR><<<dim3((unsigned)((items + 7) / 8 * 8)), 256, 0, s>>>(a, slots);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (DR > 0) {
        const int64_t quads = (int64_t)a.B * a.Tk * DR / 4;
        mla_dkr_kernel<T><<<dim3((unsigned)((quads + 255) / 256)), 256, 0, s>>>(a, quads);
        e = hipGetLastError();
    }
    return e;
}
template <class T> hipError_t launch_dims(const MlaArgs& a, hipStream_t s) {
    if (a.Dn == 128) return a.Dr ? launch<T, 128, 64>(a, s) : launch<T, 128, 0>(a, s);
    return a.Dr ? launch<T, 64, 64>(a, s) : launch<T, 64, 0>(a, s);
}

}  // namespace

hipError_t launch_mla_bwd(const MlaArgs& a, hipStream_t s) {
    return a.bf16 ? launch_dims<__bf16>(a, s) : launch_dims<float>(a, s);
}

}  // namespace kda
