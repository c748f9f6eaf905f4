// Eviction of cached rows by their gathered weights (include/kda_mla_cache.h has
// the rule). One kernel decides: a workgroup a sequence selects the rows that
// stay by their weights' bits, eleven at a time from the top (a radix select),
// lists what moves where, and writes the page table, length and weights. A
// second one moves the rows: only those that stay of the pages that go, never
// more than half of the rows looked at.
#include "launchers.hpp"
#include "mla_common.hpp"

namespace kda {
namespace {

using namespace mla;

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 2048;

// Larger weights have larger keys; NaN the largest; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (!(w == w)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

__global__ __launch_bounds__(kThreads) void mla_evict_plan_kernel(MlaEvictArgs x, int most) {
    __shared__ int bins[kBins];
    __shared__ int part[kWaves][2];
    __shared__ uint32_t found[2];
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, w = tid >> 6, ps = x.page_shift;
    const int cap = x.max_pages << ps, len = x.lens[n] < 0 ? 0 : x.lens[n];
    const int32_t* table = x.table + (int64_t)n * x.max_pages;
    const float* win = x.w_in + (int64_t)n * cap;
    float* wout = x.w_out + (int64_t)n * cap;
    // pages a .. b - 1 may go, E of them do, of `used`
    const int a = (int)(((int64_t)x.first + (1 << ps) - 1) >> ps), b = (len > x.recent ? len - x.recent : 0) >> ps;
    int E = len > x.keep ? (len - x.keep) >> ps : 0;
    if (E > b - a) E = b - a;
    const int used = (int)(((int64_t)len + (1 << ps) - 1) >> ps);
    bool fault = len > cap;
    if (!fault && E > 0)
        for (int p = a + tid; p < b; p += kThreads) fault |= table[p] < 0 || table[p] >= x.n_pages;
    fault = __syncthreads_or(fault);
    if (fault && tid == 0) atomicAdd(x.status, 1u);
    if (fault || E <= 0) {
        if (x.table_out != x.table)
            for (int p = tid; p < x.max_pages; p += kThreads) x.table_out[(int64_t)n * x.max_pages + p] = table[p];
        if (wout != win)
            for (int j = tid; j < cap; j += kThreads) wout[j] = win[j];
        if (tid == 0) {
            x.lens_out[n] = x.lens[n];
            x.moves[n] = 0;
        }
        return;
    }
    const int R = (b - a) << ps, low = (b - a - E) << ps;         // rows looked at; of the pages that stay, and that many stay
    const float* wr = win + ((int64_t)a << ps);
    int32_t* dst = x.moves + ((x.Nb + 3) & ~3) + (int64_t)n * 2 * most;
    int32_t* src = dst + most;
    int moves = 0;
    if (low > 0) {
        // the low-th largest key
        uint32_t prefix = 0;
        int want = low;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
            __syncthreads();
            for (int j = tid; j < R; j += kThreads) {
                const uint32_t k = key_of(wr[j]);
                if (pass == 0 || k >> (shift + width) == prefix) atomicAdd(&bins[k >> shift & ((1 << width) - 1)], 1);
            }
            __syncthreads();
            // counts from the top: thread t has bins 2 t and 2 t + 1
            const int c0 = bins[2 * tid], c1 = bins[2 * tid + 1];
            int s = c0 + c1;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_down(s, d);
                s += lane + d < 64 ? v : 0;
            }
            if (lane == 0) part[w][0] = s;
            __syncthreads();
            for (int v = w + 1; v < kWaves; ++v) s += part[v][0];
            // s: rows in this thread's bins and above
            const int above1 = s - c0 - c1, above0 = s - c0;
            if (above1 < want && above1 + c1 >= want) {
                found[0] = 2 * tid + 1;
                found[1] = above1;
            }
            if (above0 < want && above0 + c0 >= want) {
                found[0] = 2 * tid;
                found[1] = above0;
            }
            __syncthreads();
            prefix = prefix << width | found[0];
            want -= (int)found[1];
            __syncthreads();
        }
        // stays: a key above prefix, or equal and one of the first `want` of these. A wave takes a run of rows.
        const int run = (R + kWaves * 64 - 1) / (kWaves * 64) * 64, j0 = w * run, j1 = j0 + run < R ? j0 + run : R;
        int eq = 0;
        for (int j = j0 + lane; j < j1; j += 64) eq += key_of(wr[j]) == prefix;
        eq = wave_sum(eq);
        if (lane == 0) part[w][0] = eq;
        __syncthreads();
        int eq0 = 0;
        for (int v = 0; v < w; ++v) eq0 += part[v][0];
        __syncthreads();
        const uint64_t under = (1ull << lane) - 1;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {                    // count, then write
            int holes = 0, movers = 0, ties = eq0;
            if (pass == 1)
                for (int v = 0; v < w; ++v) {
                    holes += part[v][0];
                    movers += part[v][1];
                }
            for (int i = j0; i < j1; i += 64) {
                const int j = i + lane;
                const uint32_t k = j < j1 ? key_of(wr[j]) : 0;
                const bool same = j < j1 && k == prefix;
                const uint64_t sm = __ballot(same);
                const bool stays = j < j1 && (k > prefix || (same && ties + __popcll(sm & under) < want));
                ties += __popcll(sm);
                const bool hole = j < j1 && j < low && !stays, mover = stays && j >= low;
                const uint64_t hm = __ballot(hole), mm = __ballot(mover);
                if (pass == 1) {
                    const int base = a << ps;
                    if (hole) dst[holes + __popcll(hm & under)] = base + j;
                    if (mover) src[movers + __popcll(mm & under)] = base + j;
                }
                holes += __popcll(hm);
                movers += __popcll(mm);
            }
            if (pass == 0) {
                if (lane == 0) {
                    part[w][0] = holes;
                    part[w][1] = movers;
                }
                __syncthreads();
                for (int v = 0; v < kWaves; ++v) moves += part[v][1];
            }
        }
        __syncthreads();
    }
    // weights: everything in place first, then the holes, then the rows that close up
    const int stay = (b - E) << ps, next = b << ps, gone = E << ps;
    if (wout != win) {
        for (int j = tid; j < stay; j += kThreads) wout[j] = win[j];
        for (int j = len + tid; j < cap; j += kThreads) wout[j] = win[j];
        __syncthreads();
    }
    for (int i = tid; i < moves; i += kThreads) wout[dst[i]] = win[src[i]];
    __syncthreads();
    for (int j0 = next; j0 < len; j0 += kThreads) {
        const float v = j0 + tid < len ? win[j0 + tid] : 0.f;
        __syncthreads();
        if (j0 + tid < len) wout[j0 + tid - gone] = v;
    }
    __syncthreads();
    for (int j = len - gone + tid; j < len; j += kThreads) wout[j] = 0.f;
    // the page table: pages from b on close up, the emptied ones come behind them
    int32_t* tout = x.table_out + (int64_t)n * x.max_pages;
    if (x.table_out != x.table) {
        for (int p = tid; p < x.max_pages; p += kThreads)
            tout[p] = p < b - E || p >= used ? table[p] : p < used - E ? table[p + E] : table[p - (used - b)];
    } else {
        // in place, by way of the workspace
        int32_t* hold = x.moves + ((x.Nb + 3) & ~3) + (int64_t)x.Nb * 2 * most + (int64_t)n * x.max_pages;
        for (int p = b - E + tid; p < used; p += kThreads) hold[p] = table[p];
        __syncthreads();
        for (int p = b - E + tid; p < used; p += kThreads) tout[p] = p < used - E ? hold[p + E] : hold[p - (used - b)];
    }
    // where the sources lie under the new table
    for (int i = tid; i < moves; i += kThreads) src[i] += (used - b) << ps;
    if (tid == 0) {
        x.lens_out[n] = len - gone;
        x.moves[n] = moves;
    }
}

// Moves rows, 16 bytes a thread. A destination is never a source.
__global__ __launch_bounds__(256) void mla_evict_move_kernel(MlaEvictArgs x, int most, int per) {
    const int n = blockIdx.x / per, ps = x.page_shift;
    const int32_t* dst = x.moves + ((x.Nb + 3) & ~3) + (int64_t)n * 2 * most;
    const int32_t* src = dst + most;
    const int32_t* table = x.table_out + (int64_t)n * x.max_pages;
    const int64_t units = (int64_t)x.moves[n] * x.units, mask = (1 << ps) - 1;
    const int64_t row_bytes = 16 * (int64_t)(x.codes + x.rope) + x.scale_bytes;
    for (int64_t i = (int64_t)(blockIdx.x % per) * 256 + threadIdx.x; i < units; i += (int64_t)per * 256) {
        const int64_t m = i / x.units;
        const int u = (int)(i % x.units);
        const int64_t d = dst[m], s = src[m];
        char* const to = x.cache + table[d >> ps] * (row_bytes << ps);
        const char* const from = x.cache + table[s >> ps] * (row_bytes << ps);
        if (u < x.codes) {
            *reinterpret_cast<u32x4*>(to + (d & mask) * (16 * x.codes) + 16 * u) =
                *reinterpret_cast<const u32x4*>(from + (s & mask) * (16 * x.codes) + 16 * u);
            continue;
        }
        const int64_t plane = (16 * (int64_t)x.codes) << ps;
        if (x.scale_bytes && u == x.codes) {
            for (int j = 0; j < x.scale_bytes; j += 8)
                *reinterpret_cast<uint2*>(to + plane + (d & mask) * x.scale_bytes + j) =
                    *reinterpret_cast<const uint2*>(from + plane + (s & mask) * x.scale_bytes + j);
            continue;
        }
        const int64_t at = plane + ((int64_t)x.scale_bytes << ps);
        const int v = u - x.codes - (x.scale_bytes ? 1 : 0);
        *reinterpret_cast<u32x4*>(to + at + (d & mask) * (16 * x.rope) + 16 * v) =
            *reinterpret_cast<const u32x4*>(from + at + (s & mask) * (16 * x.rope) + 16 * v);
    }
}

}  // namespace

// Rows that stay of the pages that go are no more than these pages hold, nor
// than the others have room: half of the rows.
int64_t mla_evict_moves(int32_t page_shift, int32_t max_pages) { return ((int64_t)max_pages << page_shift) / 2; }

hipError_t launch_mla_evict(const MlaEvictArgs& a, hipStream_t s) {
    const int64_t most = mla_evict_moves(a.page_shift, a.max_pages);
    mla_evict_plan_kernel<<<dim3((unsigned)a.Nb), kThreads, 0, s>>>(a, (int)most);
    if (const hipError_t e = hipGetLastError()) return e;
    int64_t per = (most * a.units + 255) / 256;           // workgroups a sequence: as many as may have work, 2048 in all
    const int64_t share = a.Nb < 2048 ? 2048 / a.Nb : 1;
    if (per > share) per = share;
    if (per < 1) per = 1;
    mla_evict_move_kernel<<<dim3((unsigned)(a.Nb * per)), 256, 0, s>>>(a, (int)most, (int)per);
    return hipGetLastError();
}

}  // namespace kda
