// Eviction of cached rows by their gathered weights (include/kda_mla_cache.h has
// the rule). The rows that stay are selected by their weights' bits, eleven at a
// time from the top (a radix select); what moves where is listed; the rows move,
// with their weights: only those that stay of the pages that go, never more than
// half of the rows looked at. Up to kOne rows a sequence, one workgroup a sequence
// reads the weights once, into registers, and decides in one launch; of longer
// sequences a workgroup has a part, in a launch for each step.
// 128 sequences of 4096 to 8192 bf16 rows of 1152 bytes, to 4096 each: decided in 19 us
// (latency: three passes over LDS, each with four barriers), 148 000 rows moved in 82
// (4.2 TB/s read and written; a copy's 4.8). One sequence of 100 001 float32 rows of
// 1 KB, to 50 000: begin 5, three passes 5 each, count 6, list 8, 24 000 rows moved 16,
// together 50, against 194 by one workgroup: bound by the latency of seven launches
// of dependent reads. In a graph, with what moves: a sequence of 1024 rows 19 us in one
// decision, 35 in steps; of 16384 35 and 37; 64 of 16384 56 and 74.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 2048, kPasses = 3;
constexpr int kKeys = 16, kOne = kThreads * kKeys;         // weights in a thread's registers; rows of one workgroup's sequence
constexpr int kPart = 2 * kThreads;                         // rows of a part: a multiple of this
constexpr int kMost = 1024;                                 // parts of a sequence, at most
constexpr int kMove = 32;                                  // rows that a workgroup moves at a time

__host__ __device__ __forceinline__ int64_t capacity(const MlaEvictArgs& x) { return (int64_t)x.max_pages << x.page_shift; }
__host__ __device__ __forceinline__ int64_t part_rows(int64_t cap) {
    return (cap + (int64_t)kPart * kMost - 1) / ((int64_t)kPart * kMost) * kPart;
}
__host__ __device__ __forceinline__ int parts_of(int64_t cap) {
    return cap <= kOne ? 0 : (int)((cap + part_rows(cap) - 1) / part_rows(cap));
}

// A sequence's state and lists in the workspace.
struct Counts {
    int low, low_equal, high, high_equal;                   // rows above and at the last key that stays, by side
};
struct Work {
    int32_t* state;                                         // length, pages that go, moves, -; the key so far and how many rows of it stay, by passes: [4..11]
    int32_t *dst, *src;                                     // rows by their places in the new page table
    float* val;                                             // the weights that move
    // longer sequences:
    int32_t* hold;                                          // the page table, while it changes in place
    int32_t* bins;                                          // [kPasses][kBins]
    Counts *counts, *waves;                                 // [parts]; [parts][kWaves] of the part's waves before
};
constexpr int kState = 12;
__host__ __device__ __forceinline__ int64_t words_a_sequence(int64_t cap, int64_t max_pages) {
    const int64_t P = parts_of(cap);
    return kState + 3 * (cap / 2) + (P ? (max_pages + 3) / 4 * 4 + kPasses * kBins + P * 4 * (1 + kWaves) : 0);
}
__device__ __forceinline__ Work work_of(const MlaEvictArgs& x, int n) {
    const int64_t cap = capacity(x), most = cap / 2;
    Work w;
    w.state = x.work + n * words_a_sequence(cap, x.max_pages);
    w.dst = w.state + kState;
    w.src = w.dst + most;
    w.val = reinterpret_cast<float*>(w.src + most);
    w.hold = w.src + 2 * most;
    w.bins = w.hold + (x.max_pages + 3) / 4 * 4;
    w.counts = reinterpret_cast<Counts*>(w.bins + kPasses * kBins);
    w.waves = w.counts + parts_of(cap);
    return w;
}

// What goes: E of pages a .. b - 1, of `used`.
struct Range {
    int len, a, b, E, used;
    __device__ __forceinline__ Range(const MlaEvictArgs& x, int length) {
        const int ps = x.page_shift;
        len = length < 0 ? 0 : length;
        a = (int)(((int64_t)x.first + (1 << ps) - 1) >> ps);
        b = (len > x.recent ? len - x.recent : 0) >> ps;
        E = len > x.keep ? (len - x.keep) >> ps : 0;
        if (E > b - a) E = b - a;
        if (E < 0) E = 0;
        used = (int)(((int64_t)len + (1 << ps) - 1) >> ps);
    }
    // rows looked at; rows of the pages that stay, and as many stay
    __device__ __forceinline__ int rows(int ps) const { return (b - a) << ps; }
    __device__ __forceinline__ int low(int ps) const { return (b - a - E) << ps; }
};
// Larger weights have larger keys; NaN the largest; -0 is 0. No key is 0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (!(w == w)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ int shift_of(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ int width_of(int pass) { return pass == 2 ? 10 : 11; }

// The bin that holds the want-th largest key, and how many keys are above it.
// All kThreads threads; ends with a barrier.
__device__ __forceinline__ void find_bin(const int* bins, int want, int& bin, int& above) {
    __shared__ int part[kWaves], found[2];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int2 c = *reinterpret_cast<const int2*>(bins + 2 * tid);
    int s = c.x + c.y;                                      // becomes: keys in this thread's bins and above
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_down(s, d);
        s += lane + d < 64 ? v : 0;
    }
    if (lane == 0) part[w] = s;
    __syncthreads();
    for (int v = w + 1; v < kWaves; ++v) s += part[v];
    const int above1 = s - c.x - c.y, above0 = s - c.x;
    if (above1 < want && above0 >= want) {
        found[0] = 2 * tid + 1;
        found[1] = above1;
    }
    if (above0 < want && s >= want) {
        found[0] = 2 * tid;
        found[1] = above0;
    }
    __syncthreads();
    bin = found[0];
    above = found[1];
    __syncthreads();
}

// 64 rows of a wave, the first one j: their counts
__device__ __forceinline__ void count(Counts& c, uint32_t k, int j, int low, uint32_t last) {
    const uint64_t gt = __ballot(k > last), eq = __ballot(k == last);
    const int some = low - j;
    const uint64_t mask = some <= 0 ? 0 : some >= 64 ? ~0ull : (1ull << some) - 1;
    c.low += __popcll(gt & mask);
    c.low_equal += __popcll(eq & mask);
    c.high += __popcll(gt & ~mask);
    c.high_equal += __popcll(eq & ~mask);
}
__device__ __forceinline__ void add(Counts& c, const Counts& y) {
    c.low += y.low;
    c.low_equal += y.low_equal;
    c.high += y.high;
    c.high_equal += y.high_equal;
}
// Of equal rows the first `want` stay: those on the low side first. The rows
// that leave holes and those that move, of the rows counted in c (from the first
// row on, `lows` of them on the low side).
__device__ __forceinline__ int holes_of(const Counts& c, int lows, int want) {
    return lows - c.low - (c.low_equal < want ? c.low_equal : want);
}
__device__ __forceinline__ int movers_of(const Counts& c, int want) {
    const int all = c.low_equal + c.high_equal;
    return c.high + (all < want ? all : want) - (c.low_equal < want ? c.low_equal : want);
}
// lists 64 rows of a wave
struct Listing {
    int holes, movers, ties;
    __device__ __forceinline__ void rows(const Work& wk, float v, uint32_t k, int j, int low, uint32_t last, int want,
                                         int base, int back, int lane) {
        const uint64_t under = (1ull << lane) - 1, eq = __ballot(k == last);
        const bool stays = k > last || (k == last && ties + __popcll(eq & under) < want);
        const bool hole = !stays && j < low, mover = stays && j >= low;          // (behind the last row: k = 0, j >= low)
        const uint64_t hm = __ballot(hole), mm = __ballot(mover);
        if (hole) wk.dst[holes + __popcll(hm & under)] = base + j;
        if (mover) {
            const int i = movers + __popcll(mm & under);
            wk.src[i] = base + j + back;
            wk.val[i] = v;
        }
        ties += __popcll(eq);
        holes += __popcll(hm);
        movers += __popcll(mm);
    }
};

// Weights j0 .. j1 - 1 that stay where they are (but for the holes, which the moves fill afterwards).
__device__ __forceinline__ void copy_weights(const MlaEvictArgs& x, int n, const Range& g, int64_t j0, int64_t j1) {
    const float* from = x.w_in + n * capacity(x);
    float* to = x.w_out + n * capacity(x);
    if (from == to) return;
    const int stay = g.E ? (g.b - g.E) << x.page_shift : g.len;
    for (int64_t j = j0 + threadIdx.x; j < j1; j += kThreads)
        if (j < stay || j >= g.len) to[j] = from[j];
}

__global__ __launch_bounds__(kThreads) void mla_evict_plan_kernel(MlaEvictArgs x) {
    __shared__ __attribute__((aligned(16))) int bins[kBins];
    __shared__ Counts waves[kWaves];
    static_assert(kOne / 16 <= kThreads, "a thread has an entry of the page table");
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, ps = x.page_shift;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int length = x.lens[n];
    const int32_t* table = x.table + (int64_t)n * x.max_pages;
    const int page = tid < x.max_pages ? table[tid] : 0;
    Range g(x, length);
    const Work wk = work_of(x, n);
    // a wave takes a run of rows. A length past the page table is found below: reads end with it.
    const int R = g.E && g.len <= capacity(x) ? g.rows(ps) : 0, low = g.low(ps);
    const float* wr = x.w_in + n * capacity(x) + ((int64_t)g.a << ps);
    const int run = (R + kThreads - 1) / kThreads * 64, j0 = w * run;
    float v[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
        const int j = j0 + 64 * i + lane;
        v[i] = 64 * i < run && j < R ? wr[j] : 0.f;
    }
    auto key = [&](int i) { return j0 + 64 * i + lane < R ? key_of(v[i]) : 0; };
    bool fault = g.len > capacity(x) || (g.E && tid >= g.a && tid < g.b && (page < 0 || page >= x.n_pages));
    fault = __syncthreads_or(fault);                        // counted once; the sequence stays as it is
    if (fault && tid == 0) atomicAdd(x.status, 1u);
    if (fault) g.E = 0;
    int moves = 0;
    if (g.E && low) {
        uint32_t last = 0;
        int want = low;
#pragma unroll 1
        for (int pass = 0; pass < kPasses; ++pass) {
            const int shift = shift_of(pass), width = width_of(pass);
            bins[tid] = 0;
            bins[tid + kThreads] = 0;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (64 * i >= run) break;
                const uint32_t k = key(i);
                if (k && (pass == 0 || k >> (shift + width) == last)) atomicAdd(&bins[k >> shift & ((1 << width) - 1)], 1);
            }
            __syncthreads();
            int bin, above;
            find_bin(bins, want, bin, above);
            last = last << width | (uint32_t)bin;
            want -= above;
        }
        Counts c{};
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (64 * i >= run) break;
            count(c, key(i), j0 + 64 * i, low, last);
        }
        if (lane == 0) waves[w] = c;
        __syncthreads();
        Counts before{}, all{};
        for (int u = 0; u < kWaves; ++u) {
            if (u == w) before = all;
            add(all, waves[u]);
        }
        moves = movers_of(all, want);
        Listing to{holes_of(before, j0 < low ? j0 : low, want), movers_of(before, want), before.low_equal + before.high_equal};
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (64 * i >= run) break;
            to.rows(wk, v[i], key(i), j0 + 64 * i + lane, low, last, want, g.a << ps, (g.used - g.b) << ps, lane);
        }
    }
    copy_weights(x, n, g, 0, capacity(x));
    // the page table: where this thread's entry goes
    if (tid < x.max_pages && (g.E || x.table_out != x.table)) {
        const int stay = g.b - g.E, p = !g.E || tid < stay || tid >= g.used ? tid : tid < g.b ? tid + g.used - g.b : tid - g.E;
        x.table_out[(int64_t)n * x.max_pages + p] = page;
    }
    if (tid == 0) {
        wk.state[0] = g.len;
        wk.state[1] = g.E;
        wk.state[2] = moves;
        x.lens_out[n] = g.E ? g.len - (g.E << ps) : length;
    }
}

// Long sequences: the same in steps.
// A fault is counted once and leaves the sequence as it is.
__device__ __forceinline__ Range checked(const MlaEvictArgs& x, int n) {
    Range g(x, x.lens[n]);
    const int32_t* table = x.table + (int64_t)n * x.max_pages;
    bool fault = g.len > capacity(x);
    if (!fault && g.E)
        for (int p = g.a + threadIdx.x; p < g.b; p += kThreads) fault |= table[p] < 0 || table[p] >= x.n_pages;
    fault = __syncthreads_or(fault);
    if (fault && threadIdx.x == 0) atomicAdd(x.status, 1u);
    if (fault) g.E = 0;
    return g;
}

__global__ __launch_bounds__(kThreads) void mla_evict_begin_kernel(MlaEvictArgs x) {
    const int n = blockIdx.x;
    const Range g = checked(x, n);
    const Work wk = work_of(x, n);
    for (int i = threadIdx.x; i < kPasses * kBins; i += kThreads) wk.bins[i] = 0;
    if (threadIdx.x == 0) {
        wk.state[0] = g.len;
        wk.state[1] = g.E;
        wk.state[2] = 0;
        wk.state[4] = 0;
        wk.state[5] = g.low(x.page_shift);
    }
}
struct Part {
    Range g;
    Work wk;
    int n, p, R, low;
    int64_t j0, j1;                                         // its rows among those looked at
    const float* wr;
    __device__ __forceinline__ Part(const MlaEvictArgs& x) : g(x, 0) {
        const int64_t cap = capacity(x), rows = part_rows(cap);
        const int P = parts_of(cap);
        n = (int)(blockIdx.x / (unsigned)P);
        p = (int)(blockIdx.x % (unsigned)P);
        wk = work_of(x, n);
        g = Range(x, wk.state[0]);
        if (!wk.state[1]) g.E = 0;
        R = g.E ? g.rows(x.page_shift) : 0;
        low = g.E ? g.low(x.page_shift) : 0;
        if (!low) R = 0;                                    // nothing to select
        j0 = p * rows < R ? p * rows : R;
        j1 = j0 + rows < R ? j0 + rows : R;
        wr = x.w_in + n * cap + ((int64_t)g.a << x.page_shift);
    }
    // the key so far and how many rows of it stay, after `pass` passes; kept for the next launch
    __device__ __forceinline__ void key(int pass, uint32_t& last, int& want) const {
        int32_t* s = wk.state + 4 + 2 * (pass ? pass - 1 : 0);
        last = (uint32_t)s[0];
        want = s[1];
        if (!pass) return;
        int bin, above;
        find_bin(wk.bins + (pass - 1) * kBins, want, bin, above);
        last = last << width_of(pass - 1) | (uint32_t)bin;
        want -= above;
        if (p == 0 && threadIdx.x == 0) {
            s[2] = (int32_t)last;
            s[3] = want;
        }
    }
};
__global__ __launch_bounds__(kThreads) void mla_evict_bins_kernel(MlaEvictArgs x, int pass) {
    __shared__ int bins[kBins];
    const Part y(x);
    if (y.j0 >= y.j1) return;
    uint32_t last;
    int want;
    y.key(pass, last, want);
    bins[threadIdx.x] = 0;
    bins[threadIdx.x + kThreads] = 0;
    __syncthreads();
    const int shift = shift_of(pass), width = width_of(pass);
    for (int64_t j = y.j0 + threadIdx.x; j < y.j1; j += kPart) {
        const bool two = j + kThreads < y.j1;
        const float v0 = y.wr[j], v1 = two ? y.wr[j + kThreads] : 0.f;
        const uint32_t k0 = key_of(v0), k1 = key_of(v1);
        if (pass == 0 || k0 >> (shift + width) == last) atomicAdd(&bins[k0 >> shift & ((1 << width) - 1)], 1);
        if (two && (pass == 0 || k1 >> (shift + width) == last)) atomicAdd(&bins[k1 >> shift & ((1 << width) - 1)], 1);
    }
    __syncthreads();
    int* all = y.wk.bins + pass * kBins;                    // whole numbers: any order gives the same
    for (int i = threadIdx.x; i < kBins; i += kThreads)
        if (bins[i]) atomicAdd(&all[i], bins[i]);
}
__global__ __launch_bounds__(kThreads) void mla_evict_count_kernel(MlaEvictArgs x) {
    __shared__ Counts waves[kWaves];
    const Part y(x);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (y.j0 >= y.j1) {
        if (threadIdx.x == 0) y.wk.counts[y.p] = Counts{};
        return;
    }
    uint32_t last;
    int want;
    y.key(kPasses, last, want);
    const int64_t run = part_rows(capacity(x)) / kWaves, j0 = y.j0 + w * run;
    Counts c{};
    for (int64_t j = j0; j < j0 + run && j < y.j1; j += 128) {
        const int64_t i = j + lane;
        const uint32_t k0 = i < y.j1 ? key_of(y.wr[i]) : 0, k1 = i + 64 < y.j1 ? key_of(y.wr[i + 64]) : 0;
        count(c, k0, (int)j, y.low, last);
        count(c, k1, (int)j + 64, y.low, last);
    }
    if (lane == 0) waves[w] = c;
    __syncthreads();
    if (threadIdx.x <= kWaves) {                            // of the waves before this one; of all
        Counts sum{};
        for (int v = 0; v < kWaves; ++v)
            if (v < (int)threadIdx.x) add(sum, waves[v]);
        (threadIdx.x == kWaves ? y.wk.counts[y.p] : y.wk.waves[y.p * kWaves + threadIdx.x]) = sum;
    }
}
// The page table: pages from b on close up, the emptied ones come behind them.
__device__ __forceinline__ void write_table(const MlaEvictArgs& x, int n, const Range& g, int32_t* hold) {
    const int32_t* table = x.table + (int64_t)n * x.max_pages;
    int32_t* out = x.table_out + (int64_t)n * x.max_pages;
    const int tid = threadIdx.x, stay = g.b - g.E;
    if (out != table) {
        for (int p = tid; p < x.max_pages; p += kThreads)
            out[p] = !g.E || p < stay || p >= g.used ? table[p] : p < g.used - g.E ? table[p + g.E] : table[p - (g.used - g.b)];
    } else if (g.E) {
        for (int p = stay + tid; p < g.used; p += kThreads) hold[p] = table[p];
        __syncthreads();
        for (int p = stay + tid; p < g.used; p += kThreads) out[p] = p < g.used - g.E ? hold[p + g.E] : hold[p - (g.used - g.b)];
    }
}
__global__ __launch_bounds__(kThreads) void mla_evict_list_kernel(MlaEvictArgs x) {
    __shared__ Counts sums[kWaves][2];
    const Part y(x);
    const int64_t cap = capacity(x), rows = part_rows(cap);
    const int P = parts_of(cap), ps = x.page_shift, lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (y.R) {
        const uint32_t last = (uint32_t)y.wk.state[4 + 2 * kPasses];
        const int want = y.wk.state[5 + 2 * kPasses];
        // of the parts before this one, and of all: a thread has one (at most kMost = kThreads)
        Counts c{};
        if ((int)threadIdx.x < P) c = y.wk.counts[threadIdx.x];
        int v[8] = {c.low, c.low_equal, c.high, c.high_equal, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 + i] = (int)threadIdx.x < y.p ? v[i] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) v[i] += __shfl_xor(v[i], d);
        if (lane == 0) {
            sums[w][0] = Counts{v[0], v[1], v[2], v[3]};
            sums[w][1] = Counts{v[4], v[5], v[6], v[7]};
        }
        __syncthreads();
        Counts all{}, before{};
        for (int i = 0; i < kWaves; ++i) {
            add(all, sums[i][0]);
            add(before, sums[i][1]);
        }
        if (y.p == 0 && threadIdx.x == 0) y.wk.state[2] = movers_of(all, want);
        if (y.j0 < y.j1) {
            add(before, y.wk.waves[y.p * kWaves + w]);
            const int64_t run = rows / kWaves, j0 = y.j0 + w * run;
            Listing to{holes_of(before, (int)(j0 < y.low ? j0 : y.low), want), movers_of(before, want),
                       before.low_equal + before.high_equal};
            for (int64_t j = j0; j < j0 + run && j < y.j1; j += 128) {
                const int64_t i = j + lane;
                const float v0 = i < y.j1 ? y.wr[i] : 0.f, v1 = i + 64 < y.j1 ? y.wr[i + 64] : 0.f;
                const int base = y.g.a << ps, back = (y.g.used - y.g.b) << ps;
                to.rows(y.wk, v0, i < y.j1 ? key_of(v0) : 0, (int)i, y.low, last, want, base, back, lane);
                to.rows(y.wk, v1, i + 64 < y.j1 ? key_of(v1) : 0, (int)i + 64, y.low, last, want, base, back, lane);
            }
        }
    }
    copy_weights(x, y.n, y.g, y.p * rows, (y.p + 1) * rows < cap ? (y.p + 1) * rows : cap);
    if (y.p == 0) {
        write_table(x, y.n, y.g, y.wk.hold);
        if (threadIdx.x == 0) x.lens_out[y.n] = y.g.E ? y.g.len - (y.g.E << ps) : x.lens[y.n];
    }
}

// Moves rows, 16 bytes a thread at a time, four under way; a destination is never
// a source. The last workgroup of a sequence closes up the weights behind the pages.
__global__ __launch_bounds__(256) void mla_evict_move_kernel(MlaEvictArgs x, int per, uint32_t inverse) {
    __shared__ int64_t page_to[kMove], page_from[kMove];
    __shared__ int row_to[kMove], row_from[kMove];
    const int n = (int)(blockIdx.x / (unsigned)(per + 1)), c = (int)(blockIdx.x % (unsigned)(per + 1)), tid = threadIdx.x;
    const int ps = x.page_shift;
    const Work wk = work_of(x, n);
    const int E = wk.state[1], moves = wk.state[2];
    if (!E) return;
    if (c == per) {
        const Range g(x, wk.state[0]);
        const float* from = x.w_in + n * capacity(x);
        float* to = x.w_out + n * capacity(x);
        const int gone = E << ps;
        constexpr int kRows = 16;
        for (int64_t j0 = (int64_t)g.b << ps; j0 < g.len; j0 += 256 * kRows) {
            float v[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t j = j0 + 256 * i + tid;
                v[i] = j < g.len ? from[j] : 0.f;
            }
            __syncthreads();                                // in place, rows go to where others were read
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t j = j0 + 256 * i + tid;
                if (j < g.len) to[j - gone] = v[i];
            }
        }
        __syncthreads();
        for (int j = g.len - gone + tid; j < g.len; j += 256) to[j] = 0.f;
        return;
    }
    const int32_t* table = x.table_out + (int64_t)n * x.max_pages;
    float* weights = x.w_out + n * capacity(x);
    const int mask = (1 << ps) - 1;
    const int64_t row_bytes = 16 * (int64_t)(x.codes + x.rope) + x.scale_bytes, plane = (16 * (int64_t)x.codes) << ps;
    for (int64_t m0 = (int64_t)c * kMove; m0 < moves; m0 += (int64_t)per * kMove) {
        const int rows = moves - m0 < kMove ? (int)(moves - m0) : kMove, all = rows * x.units;
        __syncthreads();
        if (tid < rows) {
            const int d = wk.dst[m0 + tid], s = wk.src[m0 + tid];
            page_to[tid] = table[d >> ps] * (row_bytes << ps);
            page_from[tid] = table[s >> ps] * (row_bytes << ps);
            row_to[tid] = d & mask;
            row_from[tid] = s & mask;
            weights[d] = wk.val[m0 + tid];
        }
        __syncthreads();
        for (int i0 = tid; i0 < all; i0 += 1024) {
            u32x4 v[4];
            char* to[4];
            int small[4];                                   // 8 bytes (scales of 256 channels)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + 256 * q;
                if (i >= all) continue;
                const int m = (int)((uint32_t)i * inverse >> 24), u = i - m * x.units;      // i / units
                const bool code = u < x.codes, scale = x.scale_bytes && u == x.codes;
                const int step = code ? 16 * x.codes : scale ? x.scale_bytes : 16 * x.rope;
                const int64_t at = code ? 16 * u
                                        : scale ? plane
                                                : plane + ((int64_t)x.scale_bytes << ps) + 16 * (u - x.codes - (x.scale_bytes ? 1 : 0));
                const char* const from = x.cache + page_from[m] + at + (int64_t)row_from[m] * step;
                to[q] = x.cache + page_to[m] + at + (int64_t)row_to[m] * step;
                small[q] = scale && x.scale_bytes == 8;
                if (small[q]) {
                    const uint2 y = *reinterpret_cast<const uint2*>(from);
                    v[q] = u32x4{y.x, y.y, 0, 0};
                } else {
                    v[q] = *reinterpret_cast<const u32x4*>(from);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (i0 + 256 * q >= all) continue;
                if (small[q]) *reinterpret_cast<uint2*>(to[q]) = make_uint2(v[q][0], v[q][1]);
                else *reinterpret_cast<u32x4*>(to[q]) = v[q];
            }
        }
    }
}

}  // namespace

// The lists of moves: rows that stay of the pages that go are no more than these
// pages hold, nor than the others have room: half of the rows.
size_t mla_evict_workspace(int32_t Nb, int32_t page_shift, int32_t max_pages) {
    return 4 * (size_t)Nb * (size_t)words_a_sequence((int64_t)max_pages << page_shift, max_pages);
}
int64_t mla_evict_workgroups(int32_t Nb, int32_t page_shift, int32_t max_pages) {
    const int64_t cap = (int64_t)max_pages << page_shift, P = (cap + kPart - 1) / kPart;
    return Nb * (cap <= kOne ? 1 : P < kMost ? P : kMost);
}

hipError_t launch_mla_evict(const MlaEvictArgs& a, hipStream_t s) {
    const int64_t cap = capacity(a);
    if (const int P = parts_of(cap)) {
        const dim3 grid((unsigned)(a.Nb * P));
        mla_evict_begin_kernel<<<dim3((unsigned)a.Nb), kThreads, 0, s>>>(a);
        for (int pass = 0; pass < kPasses; ++pass) mla_evict_bins_kernel<<<grid, kThreads, 0, s>>>(a, pass);
        mla_evict_count_kernel<<<grid, kThreads, 0, s>>>(a);
        mla_evict_list_kernel<<<grid, kThreads, 0, s>>>(a);
    } else {
        mla_evict_plan_kernel<<<dim3((unsigned)a.Nb), kThreads, 0, s>>>(a);
    }
    if (const hipError_t e = hipGetLastError()) return e;
    int64_t per = (cap / 2 + kMove - 1) / kMove;        // workgroups a sequence: as many as may have work, 2048 in all
    const int64_t share = a.Nb < 2048 ? 2048 / a.Nb : 1;
    if (per > share) per = share;
    const uint32_t inverse = ((1u << 24) + a.units - 1) / a.units;       // exact for all i < kMove * units, units < 724
    mla_evict_move_kernel<<<dim3((unsigned)(a.Nb * (per + 1))), 256, 0, s>>>(a, (int)per, inverse);
    return hipGetLastError();
}

}  // namespace kda
