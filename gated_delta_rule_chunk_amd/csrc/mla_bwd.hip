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
// order, from float32 shares; in launches of few workgroups several of them
// share a block, and it sums their results too. Bound by the matrix cores; measured, bf16,
// causal, 4096 tokens, 96 heads of 128 + 64 channels: 745-790 us for dq (512
// products a score and head: 1050-1110 TFLOP/s), 1140-1330 us for dk and dv (640:
// 780-910 TFLOP/s), 18 us for the sum over the heads (100 MB read, 5.6 TB/s).
// Rounding: bf16 operands are rounded once, p and ds among them. An independent
// error of up to 2^-8 of each ds (0.0017 in the mean square) leaves dq with about
// the error that its own rounding has, 0.0024 of its norm together.
// D from o as the forward rounded it to bf16 would be off by up to 2^-8 of the
// magnitudes in it, for all keys of a row alike: 0.003 of the norm of dq and dk
// in sequences of 2 to 8 tokens, 0.006 in long ones whose weights are nearly all
// on one key. As sum_j p_ij = 1, the sum of a row's ds says what D is off by, so
// the first kernel hands D + sum_j ds_ij to the second one, and walks tiles of
// up to 128 keys, where that error weighs most, twice, the first time for D
// alone. What is left is dq of rows of more keys with such weights: taking it
// out would take the walk's products again (a second walk for all: 0.7 ms of
// 2.5) or sum_j p_ij k_j beside dq, whose registers are full. The backward takes
// as long as without, within 1%, at 4096 tokens and 96 heads (1960-1995 us), 512
// tokens and 16 heads times 8 (102), and packed ragged batches; 64 sequences of
// 100 tokens, 16 heads, all walked twice, 127 against 115 us.
#include "launchers.hpp"
#include "mla_common.hpp"
#include "mla_dkv.hpp"

namespace kda {
namespace {

using namespace mla;

template <class T, int DN, int DR, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(T) == 2 && !SPLIT ? 2 : 1) void mla_dq_kernel(MlaArgs a, int64_t slots) {
    constexpr int DQ = DN + DR, BN = sizeof(T) == 2 && !SPLIT ? 64 : 32, KB = BN / 32, BM = SPLIT ? 32 : 128;
    constexpr int CK = DN / kChunk<T>, CR = DR / kChunk<T>;
    constexpr int kK = BN * CK * 16, kR = BN * CR * 16, kTileBytes = 2 * kK + kR;
    constexpr int kBuf = SPLIT ? larger(kTileBytes, DQ * 128) : kTileBytes;    // split: also the exchange
    constexpr int kLoaders = SPLIT ? 1 : 4;
    constexpr bool kRounded = sizeof(T) == 2;                                  // o has lost what D needs
    __shared__ __attribute__((aligned(1024))) char smem[SPLIT ? 4 : 2][kBuf];
    __shared__ float dsum[2][SPLIT ? 4 : 1][32];                               // split: the waves' sums for D
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n32 = lane & 31, hf = lane >> 5, lw = SPLIT ? 0 : w;
    int h;
    int64_t slot;
    const int part = SPLIT ? (int)(blockIdx.x / (slots * a.H)) : 0;
    head_and_slot(blockIdx.x - part * slots * a.H, slots, a.H, h, slot);
    int n, q0, Lq, Lk;
    int64_t qs, ks;
    if (!tile_of(a.cuq, a.N, a.Tq, BM, slots - 1 - slot, lane, n, qs, Lq, q0)) return;
    const bool rest = a.cuq && n == a.N;
    if (rest && !a.zero_rest) return;
    seq_range(a.cuk, a.N, rest ? 0 : n, a.Tk, ks, Lk);
    if (rest) Lk = 0;
    const int off = Lk - Lq;
    const int wq0 = q0 + 32 * lw;
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
    const int64_t srow0 = ((a.cuq ? 0 : (int64_t)n * a.H) + h) * a.Tq + (a.cuq ? qs : 0), srow = srow0 + ic;
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
    }
    // this lane's row, for addresses that are formed after the loop and not kept over it
    auto row_again = [&] {
        int r = ic;
        if constexpr (kRounded) asm volatile("" : "+v"(r));
        return r;
    };
    auto put_delta = [&](float x) {
        if (live && hf == 0 && !rest && part < a.delta_parts && w == (SPLIT ? 0 : w))
            a.delta[(int64_t)part * a.B * a.H * a.Tq + srow0 + row_again()] = x;
    };
    if constexpr (!kRounded) put_delta(delta);
    f32x16 acc[DQ / 32];
#pragma unroll
    for (int d = 0; d < DQ / 32; ++d) acc[d] = zero16();
    float more = 0.f;                                   // sum of this lane's ds: what D is off by
    const float c = a.scale * kLog2e;
    // a row without a visible key has lse -inf; all its terms are hidden below
    const float lse = rest ? 0.f : a.lse[srow], l2 = lse == -INFINITY ? 0.f : lse * kLog2e;

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
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int k0 = t * BN + 32 * kb;
            if (a.causal && k0 > wq0 + 31 + off) continue;
            // LDS addresses are formed anew for each block: kept over the
            // loop, they push operands out of the registers
            int ln = lane;
            asm volatile("" : "+v"(ln));
            const int ln32 = ln & 31, lhf = ln >> 5;
            f32x16 sc = zero16(), dp = zero16();
#pragma unroll
            for (int s = 0; s < DQ / 16; ++s) {
                if (s < DN / 16) {
                    sc = mma(read_rows<T, CK>(buf, 32 * kb + ln32, s, lhf), qf[s], sc);
                    dp = mma(read_rows<T, CK>(buf + kK, 32 * kb + ln32, s, lhf), df[s < DN / 16 ? s : 0], dp);
                } else if constexpr (DR > 0) {
                    sc = mma(read_rows<T, CR>(buf + 2 * kK, 32 * kb + ln32, s - DN / 16, lhf), qf[s], sc);
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
            auto read = [&](int i) -> Frag<T> {
                const int s = i / (DQ / 32), d = i % (DQ / 32);
                if constexpr (DR > 0)
                    if (d >= DN / 32) return read_cols<T, CR>(buf + 2 * kK, 32 * kb + 16 * s, 32 * d - DN, ln);
                return read_cols<T, CK>(buf, 32 * kb + 16 * s, 32 * d, ln);
            };
            ReadAhead<T, DQ / 16, 3> ahead;
            ahead.start(read);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r], c, -l2));
                sc[r] = p * (dp[r] - delta);
                if constexpr (kRounded) more += sc[r];
            }
            const Frag<T> f[2] = {to_frag<T>(sc, 0), to_frag<T>(sc, 1)};
            ahead.run(read, [&](int i, const Frag<T>& x) {
                acc[i % (DQ / 32)] = mma(x, f[i / (DQ / 32)], acc[i % (DQ / 32)]);
            });
        }
    };
    // Tiles of up to 128 keys are walked twice, the first time for D.
    int pass = tiles <= 128 / BN ? 0 : 1;
    auto again = [&](float x) {                         // D's correction, from all of a row's products
        if (pass == 0) {
            delta += x;
            more = 0.f;
#pragma unroll
            for (int d = 0; d < DQ / 32; ++d) acc[d] = zero16();
        }
        return pass++ == 0;
    };
    if constexpr (SPLIT) {
        auto walk = [&](int t0, int step) {
            for (int t = t0; t < tiles; t += step) {
                load(t, smem[w]);
                wait_loads_and_lds();
                compute(t, smem[w]);
                wait_loads_and_lds();
            }
        };
        float x;
        if constexpr (kRounded) {
            do {                                        // (a first walk is a whole one, parts or not)
                walk(w + (pass ? 4 * part : 0), pass ? 4 * a.q_parts : 4);
                more = half_sum(more);
                if (hf == 0) dsum[pass][w][n32] = more;
                wait_loads_and_lds();
                wg_barrier();
                x = ((dsum[pass][0][n32] + dsum[pass][1][n32]) + dsum[pass][2][n32]) + dsum[pass][3][n32];
            } while (again(x));
            put_delta((part == 0 ? delta : 0.f) + x);
        } else {
            walk(w + 4 * part, 4 * a.q_parts);
        }
#pragma unroll
        for (int d = 0; d < DQ / 32; ++d) put_block(smem[w], d, acc[d], lane);
        wait_loads_and_lds();
        wg_barrier();
        const float one[4] = {1.f, 1.f, 1.f, 1.f};
        const int64_t out = (qs + row_again()) * a.H + h;
        T* p = static_cast<T*>(a.dq) + out * DQ;
        float* f = a.q_parts > 1 ? a.dq_part + (((int64_t)part * a.B * a.Tq * a.H) + out) * DQ : nullptr;
        for (int d = w; d < DQ / 32; d += 4) {
            const f32x16 x = sum_blocks(smem[0], kBuf, d, one, lane);
            if (f) store_tile<float>(f + 32 * d, x, a.scale, hf, live);
            else store_tile<T>(p + 32 * d, x, a.scale, hf, live);
        }
    } else {
        auto walk = [&] {
            // the compiler does not know where a walk begins: what it would form
            // in front of both walks and keep pushes operands out of the registers
            // (a quarter of the kernel's time with one workgroup a compute unit)
            int t0 = 0;
            if constexpr (kRounded) asm volatile("" : "+s"(t0));
            if (tiles > 0) load(t0, smem[t0]);
            wait_loads_and_lds();
            wg_barrier();
            for (int t = t0; t < tiles; ++t) {
                if (t + 1 < tiles) load(t + 1, smem[(t + 1) & 1]);
                compute(t, smem[t & 1]);
                wait_loads_and_lds();
                wg_barrier();
            }
        };
        if constexpr (kRounded) {
            do {
                walk();
                more = half_sum(more);
            } while (again(more));
            put_delta(delta + more);
        } else {
            walk();
        }
        T* p = static_cast<T*>(a.dq) + ((qs + row_again()) * a.H + h) * DQ;
#pragma unroll
        for (int d = 0; d < DQ / 32; ++d) store_tile<T>(p + 32 * d, acc[d], a.scale, hf, live);
    }
}

// The float32 shares of a gradient (the heads' of the shared key part; those of
// workgroups that shared a block) summed in their order: up to three gradients
// a launch, four columns a thread.
struct Shares {
    const float* in;            // [n] of quads * 4
    void* out;
    int32_t n, row_quads, T;
    const int32_t* cu;          // packed: rows behind the last sequence are left alone, unless they are zeroed
    int64_t quads;
    int64_t blocks;             // workgroups of this one and of those before it
};
struct SharesArgs {
    Shares of[3];
    int32_t N;
    bool zero_rest;
};
template <class T> __global__ __launch_bounds__(256) void mla_sum_kernel(SharesArgs a) {
    const int which = (int)blockIdx.x < a.of[0].blocks ? 0 : (int)blockIdx.x < a.of[1].blocks ? 1 : 2;
    const Shares& g = a.of[which];
    const int64_t x = ((int64_t)blockIdx.x - (which ? a.of[which - 1].blocks : 0)) * 256 + threadIdx.x;
    if (x >= g.quads) return;
    if (g.cu && !a.zero_rest) {
        int64_t s;
        int len;
        seq_range(g.cu, a.N, a.N, g.T, s, len);
        if (x / g.row_quads >= s) return;
    }
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const float* p = g.in + 4 * x;
#pragma unroll 8
    for (int i = 0; i < g.n; ++i) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + 4 * i * g.quads);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += v[j];
    }
    T* o = static_cast<T*>(g.out) + 4 * x;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (T)sum[j];
}

template <class T, int DN, int DR> hipError_t launch_dq(const MlaArgs& a, hipStream_t s) {
    if (a.Tq == 0) return hipSuccess;
    int64_t slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 128);
    if (slots * a.H < kSmallLaunch<T>) {
        slots = tile_slots(a.cuq, a.B, a.N, a.Tq, 32);
        mla_dq_kernel<T, DN, DR, true><<<dim3((unsigned)(slots * a.H * a.q_parts)), 256, 0, s>>>(a, slots);
    } else {
        mla_dq_kernel<T, DN, DR, false><<<dim3((unsigned)(slots * a.H)), 256, 0, s>>>(a, slots);
    }
    return hipGetLastError();
}
template <class T> hipError_t launch_dq_dims(const MlaArgs& a, hipStream_t s) {
    if (a.Dn == 128) return a.Dr ? launch_dq<T, 128, 64>(a, s) : launch_dq<T, 128, 0>(a, s);
    return a.Dr ? launch_dq<T, 64, 64>(a, s) : launch_dq<T, 64, 0>(a, s);
}
template <class T> hipError_t launch_sums(const MlaArgs& a, hipStream_t s) {
    SharesArgs x{};
    x.N = a.N;
    x.zero_rest = a.zero_rest;
    int64_t blocks = 0;
    const auto add = [&](Shares& g, const float* in, void* out, int n, int row, int T_, const int32_t* cu) {
        g.in = in; g.out = out; g.n = n; g.row_quads = row; g.T = T_; g.cu = cu;
        g.quads = in ? (int64_t)a.B * T_ * row : 0;
        g.blocks = blocks += (g.quads + 255) / 256;
    };
    add(x.of[0], a.dkr ? a.dkr_part : nullptr, a.dkr, a.k_parts * a.H, a.Dr / 4, a.Tk, a.cuk);
    add(x.of[1], a.k_parts > 1 ? a.dkv_part : nullptr, a.dkv, a.k_parts, a.H * a.Dn / 2, a.Tk, a.cuk);
    add(x.of[2], a.q_parts > 1 ? a.dq_part : nullptr, a.dq, a.q_parts, a.H * (a.Dn + a.Dr) / 4, a.Tq, a.cuq);
    if (blocks == 0) return hipSuccess;
    mla_sum_kernel<T><<<dim3((unsigned)blocks), 256, 0, s>>>(x);
    return hipGetLastError();
}

}  // namespace

// Workgroups that share a block of queries (keys), each with every so many
// groups of four tiles of the other side: as many as find a compute unit, if the
// walk is long enough to be worth a sum of their shares. Measured, 128 + 64
// channels, causal, the backward with and without: float32 500 tokens, 8 heads
// 71 : 107 us, 1000 tokens, 1 head 70 : 186, 200 tokens 47 : 63. bf16 1000
// tokens, 1 head 35 : 50, 4000 tokens 98 : 154, but 500 tokens, 8 heads 39 : 35.
// T is the rows of all packed sequences: the host does not know their lengths,
// and their mean misjudges a long one among short ones. Total against mean, 1
// head: float32 1000 tokens and 15 times 8 70 : 188, 16 of 64 48 : 44, 4 of 256
// 49 : 46; bf16 2000 and 20 times 50 59 : 86, 32 of 64 26 : 21, 2 of 2000 63 : 62.
static int walk_parts(bool bf16, int64_t workgroups, int T) {
    const int tiles = (T + 31) / 32, least = bf16 ? 16 : 4;
    int p = 1;
    while (p < 4 && workgroups > 0 && workgroups * p * 2 <= 256 && tiles > least * p) p *= 2;
    return p;
}
size_t mla_bwd_plan(MlaArgs& a) {
    a.q_parts = walk_parts(a.bf16, tile_slots(a.cuq, a.B, a.N, a.Tq, 32) * a.H, a.Tk);
    a.k_parts = walk_parts(a.bf16, tile_slots(a.cuk, a.B, a.N, a.Tk, 32) * a.H, a.Tq);
    const int64_t nq = (int64_t)a.B * a.H * a.Tq, nk = (int64_t)a.B * a.H * a.Tk;
    float* p = a.delta;
    const auto take = [&](int64_t n) {
        float* x = p;
        if (p) p += n;
        return x;
    };
    a.delta_parts = a.bf16 ? a.q_parts : 1;
    const int64_t sizes[] = {(a.q_parts * nq + 3) / 4 * 4, a.k_parts * nk * a.Dr,
                             a.q_parts > 1 ? a.q_parts * nq * (a.Dn + a.Dr) : 0,
                             a.k_parts > 1 ? a.k_parts * nk * 2 * a.Dn : 0};
    a.delta = take(sizes[0]);
    a.dkr_part = take(sizes[1]);
    a.dq_part = take(sizes[2]);
    a.dkv_part = take(sizes[3]);
    return (size_t)(sizes[0] + sizes[1] + sizes[2] + sizes[3]) * sizeof(float);
}

hipError_t launch_mla_bwd(const MlaArgs& a, hipStream_t s) {
    hipError_t e = a.bf16 ? launch_dq_dims<__bf16>(a, s) : launch_dq_dims<float>(a, s);
    if (e == hipSuccess) e = a.bf16 ? launch_mla_dkv_bf16(a, s) : launch_dkv_dims<float>(a, s);
    if (e == hipSuccess) e = a.bf16 ? launch_sums<__bf16>(a, s) : launch_sums<float>(a, s);
    return e;
}

}  // namespace kda
