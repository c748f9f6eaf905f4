// Device helpers shared by the latent-attention kernels (gfx950 only).
//
// All matrix products run on 32x32 tiles with 16 products per element and
// instruction group ("step"), for bf16 one v_mfma_f32_32x32x16_bf16, for
// float32 eight v_mfma_f32_32x32x2f32 on the same logical operands. Operand
// layout of a step, for lane l with n = l % 32, hf = l / 32: A row n and B
// column n, products 8 hf .. 8 hf + 7. Accumulator register r of lane l is
// row 8 (r / 4) + 4 hf + r % 4, column n.
//
// The scores are formed transposed (rows = keys, columns = queries), so a
// lane's 16 accumulator registers all belong to one query: the softmax needs
// one exchange with lane l ^ 32 and no shared memory. Registers 8 s .. 8 s + 7
// are then, as they stand, the B operand of a step over 16 keys if the A
// operand takes its products in the same order: product j of half hf is key
// 4 hf + j for j < 4 and 8 + 4 hf + j - 4 for j >= 4 ("register order").
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace kda {
namespace mla {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#define KDA_LDS __attribute__((address_space(3)))

template <class T> struct Elem;
template <> struct Elem<__bf16> {
    using Frag = bf16x8;
};
template <> struct Elem<float> {
    using Frag = f32x8;
};
template <class T> using Frag = typename Elem<T>::Frag;
// elements of T in a 16-byte chunk
template <class T> constexpr int kChunk = 16 / (int)sizeof(T);

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.f;
    return z;
}

// LDS tiles: rows of RC 16-byte chunks (RC a multiple of 8) with no padding,
// chunk c of row r at position c ^ swizzle(r), so that the 16 rows of an
// operand read, and the 4 chunks of 4 or 8 consecutive rows of a transposed
// read, lie in different banks. Loads straight from global memory fill LDS in
// the order of the lanes, so padding is not possible; the source address of
// each lane carries the permutation instead.
template <int RC> __device__ __forceinline__ int swizzle(int r) {
    if constexpr (RC % 16 == 0) {
        return ((r & 3) << 2) | ((r >> 2) & 3);
    } else {   // 8 mod 16: odd rows are half a bank cycle away already
        return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    }
}

// 16 bytes per lane from global memory to LDS at `lds` (uniform) + 16 * lane.
// Written as an instruction so that the compiler, which cannot tell the two
// buffers apart, does not wait for the next tile before it reads this one;
// wait_loads_and_lds() and the barrier order them. It has no register output.
// The compiler inserts no wait states here either, so the asm brings them: one
// between the write of m0, the place in LDS, and the load. Nothing else in these
// kernels uses m0 (the compiler takes no reserved register as a clobber).
__device__ __forceinline__ void load_lds16(const char* g, char* lds) {
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(KDA_LDS char*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(base), "v"(g) : "memory");
}
// the same from g (uniform) + off bytes. A load needs five wait states after a
// vector instruction has written its scalar address (readfirstlane does), but
// none after a scalar one, whose own read of it the hardware orders: the
// address is copied, which is m0's wait state too.
__device__ __forceinline__ void load_lds16s(const char* g, int off, char* lds) {
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(KDA_LDS char*)lds);
    const uint64_t u = reinterpret_cast<uint64_t>(g);
    const uint64_t from = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
    uint64_t t;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
                 : "=&s"(t)
                 : "s"(base), "v"(off), "s"(from)
                 : "memory");
}
// the same where `on` (uniform): no branch, which would end the compiler's
// scheduling region. All lanes of the wave are active here.
__device__ __forceinline__ void load_lds16s_if(bool on, const char* g, int off, char* lds) {
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(KDA_LDS char*)lds);
    const uint64_t u = reinterpret_cast<uint64_t>(g);
    const uint64_t from = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
    const uint32_t lanes = __builtin_amdgcn_readfirstlane(on ? 0xffffffffu : 0u);
    uint64_t t;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\ts_mov_b32 exec_lo, %4\n\ts_mov_b32 exec_hi, %4\n\t"
                 "global_load_lds_dwordx4 %2, %0\n\ts_mov_b64 exec, -1"
                 : "=&s"(t)
                 : "s"(base), "v"(off), "s"(from), "s"(lanes)
                 : "memory");
}

// Rows [0, ROWS) of a tile from global rows `stride` bytes apart to LDS, WAVES
// waves (this one w), not waited for. Each instruction covers 64 / RC (or a
// part of) rows; the swizzle repeats every 16 rows, so a lane's offset in the
// tile takes P values only, kept in registers, and the row of an instruction
// goes into the uniform base: no vector arithmetic per tile.
template <int RC, int ROWS, int WAVES> struct TileLoad {
    static constexpr int NT = 64 * WAVES, kInstr = ROWS * RC / NT;
    static_assert(ROWS * RC % NT == 0 && NT % RC == 0, "whole rows an instruction of all waves");
    static constexpr int R = NT / RC;                     // rows an instruction of all waves
    static constexpr int P = R >= 16 ? 1 : 16 / R < kInstr ? 16 / R : kInstr;
    int off[P];

    __device__ __forceinline__ void init(int64_t stride, int w, int lane) {
        const int s = w * 64 + lane;
#pragma unroll
        for (int i = 0; i < P; ++i) off[i] = (s / RC) * (int)stride + (((s % RC) ^ swizzle<RC>(i * R + s / RC)) << 4);
    }
    // all rows exist
    __device__ __forceinline__ void full(char* lds, const char* g, int64_t stride, int w) const {
#pragma unroll
        for (int i = 0; i < kInstr; ++i) load_lds16s(g + i * R * stride, off[i % P], lds + (i * NT + w * 64) * 16);
    }
    // rows past rmax are not read: row rmax stands in
    __device__ __forceinline__ void edge(char* lds, const char* g, int64_t stride, int rmax, int w, int lane) const {
        asm volatile("" : "+v"(lane));                    // nothing of this is kept over the tiles
        const int s = w * 64 + lane;
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int r = i * R + s / RC, rr = r < rmax ? r : rmax;
            load_lds16(g + rr * stride + (((s % RC) ^ swizzle<RC>(r)) << 4), lds + (i * NT + w * 64) * 16);
        }
    }
    __device__ __forceinline__ void load(char* lds, const char* g, int64_t stride, int rmax, int w, int lane) const {
        if (rmax >= ROWS - 1) full(lds, g, stride, w);
        else edge(lds, g, stride, rmax, w, lane);
    }
};

// Scheduling: AHEAD LDS reads first, then EACH reads after every one of MMAS
// matrix instructions, so that operands are under way while the ones before
// them are used.
template <int AHEAD, int EACH, int MMAS> __device__ __forceinline__ void sched_reads_under_mma() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < MMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, EACH, 0);
    }
}

// Operands that are read from LDS kAhead at a time in front of their products:
// start() issues the first reads, before the vector arithmetic that the
// products wait for, and run() multiplies (use(i, operand) for operand i of N)
// and keeps reading ahead. read(i) is operand i.
template <class T, int N, int AHEAD> struct ReadAhead {
    static constexpr int kAhead = sizeof(T) == 2 ? AHEAD : 2;
    Frag<T> ring[kAhead];

    template <class Read> __device__ __forceinline__ void start(Read read) {
        static_assert(N >= kAhead, "operands");
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ring[i] = read(i);
        __builtin_amdgcn_sched_barrier(0);
    }
    // MMAS products with each operand of READS LDS reads, of which has(i) has any
    template <int MMAS = 1, int READS = 2, class Read, class Use, class Has>
    __device__ __forceinline__ void run(Read read, Use use, Has has) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            use(i, ring[i % kAhead]);
            if (i + kAhead < N) ring[i % kAhead] = read(i + kAhead);
        }
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < N - kAhead; ++i) {
                if (has(i)) __builtin_amdgcn_sched_group_barrier(0x008, MMAS, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    template <int MMAS = 1, int READS = 2, class Read, class Use> __device__ __forceinline__ void run(Read read, Use use) {
        run<MMAS, READS>(read, use, [](int) { return true; });
    }
};

// Byte offset in a row of chunk k + x (k a multiple of 2 known when compiling,
// x the lane's part, below 8 with k's bits clear) under swizzle sw. Written so
// that few registers serve many k: chunks are permuted within groups of 16
// (or 8), and the group goes into the instruction's offset.
template <int RC> __device__ __forceinline__ int chunk_at(int k, int x, int sw) {
    constexpr int G = RC % 16 == 0 ? 16 : 8;
    return (((x ^ sw) ^ (k & (G - 1))) << 4) + (k / G * G) * 16;
}

// Operand of one step over the columns: row r, products = columns
// 16 step + 8 hf .. + 7. (The x argument: 2 * half more for steps that two
// waves take in turn, with step = 2 * (step of the wave).)
template <class T, int RC>
__device__ __forceinline__ Frag<T> read_rows(const char* lds, int r, int step, int hf, int odd = 0) {
    const char* p = lds + r * (RC * 16);
    const int sw = swizzle<RC>(r);
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const bf16x8*>(p + chunk_at<RC>(2 * step, 2 * odd + hf, sw));
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(4 * step, 4 * odd + 2 * hf, sw));
        const f32x4 b = *reinterpret_cast<const f32x4*>(p + chunk_at<RC>(4 * step, 4 * odd + 2 * hf + 1, sw));
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
}

// Operand of one step over the rows: operand row n = column col0 + n of the
// tile, products = rows row0 .. row0 + 15 in register order (above). bf16
// uses the transposing LDS read: each 16 lanes read a 4 x 16 block, 8 bytes
// per lane, and lane i of them receives column i.
template <class T, int RC> __device__ __forceinline__ Frag<T> read_cols(const char* lds, int row0, int col0, int lane) {
    if constexpr (sizeof(T) == 2) {
        bf16x8 f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = 8 * u + 4 * (lane >> 5) + ((lane >> 2) & 3);      // row0 is a multiple of 16
            const int x = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            const char* p = lds + r * (RC * 16) + (lane & 1) * 8 + row0 * (RC * 16) +
                            chunk_at<RC>(col0 >> 3, x, swizzle<RC>(r));
            const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KDA_LDS s16x4*)p);
            const bf16x4 b = __builtin_bit_cast(bf16x4, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[4 * u + j] = b[j];
        }
        return f;
    } else {
        f32x8 f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
            f[j] = *reinterpret_cast<const float*>(lds + r * (RC * 16) + (lane & 3) * 4 + row0 * (RC * 16) +
                                                   chunk_at<RC>(col0 >> 2, (lane & 31) >> 2, swizzle<RC>(r)));
        }
        return f;
    }
}

// Eight consecutive elements of a row in global memory.
template <class T> __device__ __forceinline__ Frag<T> load8(const T* p) {
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const bf16x8*>(p);
    } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
}

// Accumulator registers 8 s .. 8 s + 7 as an operand. bf16 rounds here, once,
// to the nearest: the matrix cores take bf16, and the statistics stay float32.
template <class T> __device__ __forceinline__ Frag<T> to_frag(const f32x16& x, int s) {
    Frag<T> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (T)x[8 * s + j];
    return f;
}

// max / sum over a lane and its other half
__device__ __forceinline__ float half_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Stores a 32 x 32 accumulator (transposed: lane column n = output row, rows
// = 32 consecutive output columns) times mul to p = that row's first of the
// 32 columns. The two halves of a lane pair exchange registers so that each
// stores 8 consecutive columns. Every lane takes part in the exchange; only
// lanes with `live` store.
template <class T>
__device__ __forceinline__ void store_tile(T* p, const f32x16& acc, float mul, int hf, bool live) {
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
        if constexpr (sizeof(T) == 2) {
            const uint32_t a0 = pack2_bf16(acc[4 * g] * mul, acc[4 * g + 1] * mul);
            const uint32_t a1 = pack2_bf16(acc[4 * g + 2] * mul, acc[4 * g + 3] * mul);
            const uint32_t b0 = pack2_bf16(acc[4 * g + 4] * mul, acc[4 * g + 5] * mul);
            const uint32_t b1 = pack2_bf16(acc[4 * g + 6] * mul, acc[4 * g + 7] * mul);
            const auto x0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
            const auto x1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
            if (live) *reinterpret_cast<u32x4*>(p + 8 * (g + hf)) = u32x4{x0[0], x1[0], x0[1], x1[1]};
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const f32x4 v = {acc[4 * (g + k)] * mul, acc[4 * (g + k) + 1] * mul, acc[4 * (g + k) + 2] * mul,
                                 acc[4 * (g + k) + 3] * mul};
                if (live) *reinterpret_cast<f32x4*>(p + 8 * (g + k) + 4 * hf) = v;
            }
        }
    }
}

__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    asm volatile("" ::: "memory");
}

constexpr int larger(int a, int b) { return a > b ? a : b; }

// The workgroup barrier without a fence: every wave has waited for its own
// loads and LDS accesses before it (wait_loads_and_lds).
__device__ __forceinline__ void wg_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// Waits for this wave's loads into LDS and for its own LDS accesses. (The
// builtin, so that the compiler knows of it.)
__device__ __forceinline__ void wait_loads_and_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0), lgkmcnt(0)
    asm volatile("" ::: "memory");
}

// Split kernels: where a launch would leave compute units idle, the four waves
// of a workgroup take the same 32 rows and every fourth tile of the other side
// each, with a tile buffer of their own, and their sums meet in LDS at the end.
// A launch counts as small below one workgroup of 128 rows per compute unit; in
// float32, whose products hide the loads that are not overlapped here, below 1.75.
// Measured, causal, split against whole in us, forward, backward:
//   workgroups          128               256               384               512
//   2048 tokens, 128 + 64 channels
//     bf16      32 : 48, 120 : 158   43 : 48, 212 : 159   62 : 52, 318 : 169   81 : 56, 420 : 193
//     float32 121 : 332, 405 : 1258 242 : 334, 803 : 1275 365 : 336, 1215 : 1289 482 : 365, 1599 : 1399
//   2048 tokens, 64 channels
//     bf16      17 : 30, 53 : 102    20 : 32, 86 : 103    29 : 33, 127 : 109   34 : 33, 167 : 111
//     float32   54 : 146, 186 : 497  82 : 146, 279 : 498 117 : 182, 407 : 555 152 : 193, 525 : 603
//   8 sequences of 512, 128 + 64 channels
//     bf16      16 : 17, 69 : 56     26 : 18, 113 : 60    36 : 24, 166 : 92    42 : 26, 201 : 100
//     float32   65 : 89, 214 : 342   99 : 93, 328 : 349  140 : 159, 471 : 602 171 : 180, 581 : 686
// The two sides cross at other numbers for each direction, width and length; one
// per type serves them all, and leaves up to a third to some near it: bf16
// backwards of 512 tokens are faster whole at 128, bf16 forwards of 2048 split
// at 256, float32 ones of 64 channels split at 512.
template <class T> constexpr int64_t kSmallLaunch = sizeof(T) == 4 ? 448 : 256;

// A wave's accumulator block d to and from its exchange region
__device__ __forceinline__ void put_block(char* region, int d, const f32x16& x, int lane) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(region + ((d * 4 + g) * 64 + lane) * 16) =
            f32x4{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]};
}
// block d of the four regions, `stride` bytes apart, each times its factor
__device__ __forceinline__ f32x16 sum_blocks(const char* regions, int stride, int d, const float (&f)[4], int lane) {
    f32x16 s = zero16();
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(regions + v * stride + ((d * 4 + g) * 64 + lane) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[4 * g + j] += f[v] * x[j];
        }
    return s;
}

// Which head and which slot of the tile list workgroup `item` takes. Workgroups are
// dealt round-robin over the 8 XCDs, each with an L2 of its own, and start in
// the order of their index. Heads go fastest, so that with a multiple of 8 of
// them every head stays on one XCD, where its tiles share the L2; a sequence's slots
// go by falling work, so that no long tile starts last (heads one after the other,
// each from its longest tile, left a fifth of the wave slots empty at 4096
// tokens); and 32 heads go at a time, 4 on an XCD, so that enough of a head's
// tiles walk through the same keys together. Sequences follow one another as the
// caller packed them (the dq kernel and the forward take the last one first), so
// a long one may still start last: the tiles of twelve ragged sequences of up to
// 1100 tokens, 24 heads, would end about a fifth sooner in falling order.
__device__ __forceinline__ void head_and_slot(int64_t item, int64_t slots, int H, int& h, int64_t& slot) {
    const int g = (int)(item / (32 * slots)) * 32, n = H - g < 32 ? H - g : 32;
    const int64_t r = item - g * slots;
    h = g + (int)(r % n);
    slot = r / n;
}

// Start and length of sequence n (dense: rows of T; packed: offsets cu,
// clipped to [0, T] so that no value in it leads outside the tensor). Packed
// sequence N is the rows behind the last one.
__device__ __forceinline__ void seq_range(const int32_t* cu, int N, int n, int T, int64_t& start, int& len) {
    if (!cu) {
        start = (int64_t)n * T;
        len = T;
        return;
    }
    int a = cu[n], b = n < N ? cu[n + 1] : T;
    a = a < 0 ? 0 : a > T ? T : a;
    b = b < a ? a : b > T ? T : b;
    start = a;
    len = b - a;
}

// Packed sequences (the rows behind the last one counted as a sequence more)
// cut into tiles of `tile` rows: the sequence and tile of slot t in the list
// of all tiles; false past its end, which is at most T / tile + N + 1. A wave
// takes 64 sequences at a time (their tile counts summed over the lanes).
__device__ __forceinline__ bool find_tile(const int32_t* cu, int N, int T, int tile, int64_t t, int lane, int& n, int& k) {
    int64_t before = 0;
    for (int n0 = 0; n0 <= N; n0 += 64) {
        int cnt = 0;
        if (n0 + lane <= N) {
            int64_t s;
            int len;
            seq_range(cu, N, n0 + lane, T, s, len);
            cnt = (len + tile - 1) / tile;
        }
        int sum = cnt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            sum += lane >= d ? v : 0;
        }
        const int total = __builtin_amdgcn_readlane(sum, 63);
        if (t < before + total) {
            const int l = __ffsll((unsigned long long)__ballot(before + sum > t)) - 1;
            n = n0 + l;
            k = (int)(t - before) - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(cnt, l));
            return true;
        }
        before += total;
    }
    return false;
}

// Tile `slot` of the list of all tiles of `tile` rows over B dense or N packed
// sequences of [.., T, ..]: its sequence n, that sequence's start and length,
// the tile's first row r0; false past the end of the list.
__device__ __forceinline__ bool tile_of(const int32_t* cu, int N, int T, int tile, int64_t slot, int lane, int& n,
                                        int64_t& start, int& len, int& r0) {
    int k;
    if (cu) {
        if (!find_tile(cu, N, T, tile, slot, lane, n, k)) return false;
    } else {
        const int per = (T + tile - 1) / tile;
        n = (int)(slot / per);
        k = (int)(slot % per);
    }
    seq_range(cu, N, n, T, start, len);
    r0 = k * tile;
    return true;
}
// length of that list, at most
inline int64_t tile_slots(const int32_t* cu, int B, int N, int T, int tile) {
    return cu ? (int64_t)T / tile + N + 1 : B * (((int64_t)T + tile - 1) / tile);
}

}  // namespace mla
}  // namespace kda
