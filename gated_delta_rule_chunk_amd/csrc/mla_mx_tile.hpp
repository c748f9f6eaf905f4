// Tiles of 64 rows of a 4-bit cache in LDS, and the scores of bf16 queries against
// them on the scaled matrix instructions.
#pragma once

#include "mla_mx.hpp"
#include "mla_step.hpp"

namespace kda {
namespace {

constexpr int kRows = 64, kWaves = 8;    // of a tile, of a workgroup

// Where the parts of a tile as it lies in memory come to in LDS: codes, shared
// parts, scale bytes, each in four quarters of 16 rows. A row of codes is 16 or 8
// chunks of 16 bytes, one of the shared part 8; chunk c lies at c ^ swz(r), that of codes
// at c ^ swz(r) ^ swz_quarter(quarter).
// The scores' operand reads take, of 16 lanes that LDS serves at a time, 8 rows of
// chunk c and 8 other rows of chunk c ^ 4, c ^ 2 (codes) or c ^ 1 (shared part):
// rows 0-3 and 12-15, and 4-11; the outputs' transposing reads 8 bytes of chunk c of
// four rows in each quarter. Under these permutations each takes every bank once.
template <int DC, int DR> struct RawTile {
    static constexpr int NB = DC / 32;
    static constexpr int kCodes = 16 * DC / 2, kRope = 16 * DR * 2;                // bytes of 16 rows
    static constexpr int kRopeAt = 4 * kCodes, kScalesAt = kRopeAt + 4 * kRope, kBytes = kScalesAt + 4 * 256;
    static __device__ __forceinline__ int swz_codes(int r) {
        if constexpr (NB == 16) return (r & 7) << 1 | ((r >> 3 ^ r >> 2) & 1);
        else return (r >> 1 & 3) << 1 | ((r >> 3 ^ r >> 2) & 1);
    }
    static __device__ __forceinline__ int swz_quarter(int q) { return (q & 1) | (q >> 1) << (NB == 16 ? 3 : 2); }
    static __device__ __forceinline__ int swz_rope(int r) { return r >> 1 & 7; }
    static __device__ __forceinline__ int codes(int r, int c) {
        return r * (DC / 2) + ((c ^ swz_codes(r & 15) ^ swz_quarter(r >> 4)) << 4);
    }
    static __device__ __forceinline__ int rope(int r, int c) { return kRopeAt + r * (DR * 2) + ((c ^ swz_rope(r & 15)) << 4); }
    static __device__ __forceinline__ int scales(int r) { return kScalesAt + (r >> 4) * 256 + (r & 15) * NB; }
};

// Sends the tile of rows k0 .. k0 + 63 of a sequence (of `rows`) on its way to LDS
// by eight waves (this one w); returns which of its quarters of 16 rows exist. Rows past the
// sequence and of missing pages are zeros there: their weights are 0, but what
// these multiply has to be finite. pages: the page numbers from pbase on, one a
// lane, exist: which of them do. Two waves load a quarter: of its instructions of
// 1 KB every other one, the first its scale bytes too. Not waited for.
template <int DC, int DR>
__device__ __forceinline__ int mx_fetch(char* to, const char* cache, int64_t page_bytes, int pages, uint64_t exist, int pbase,
                                        int ps, int k0, int rows, int w, int lane) {
    using Raw = RawTile<DC, DR>;
    constexpr int NB = DC / 32;
    const int quarter = w & 3, j0 = w >> 2;
    int have = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) have |= (int)(exist >> (((k0 + 16 * q) >> ps) - pbase) & 1) << q;
    const int kq = k0 + 16 * quarter, row = kq & ((1 << ps) - 1);
    // (a missing page's address is not used)
    const char* const page = cache +
                             __builtin_amdgcn_readlane(pages, (kq >> ps) - pbase) * page_bytes;
    const char* const from_codes = page + (int64_t)row * (DC / 2);
    const char* const from_scales = page + (((int64_t)DC / 2) << ps) + row * NB;
    const char* const from_rope = page + (((int64_t)DC / 2 + NB) << ps) + (int64_t)row * (DR * 2);
    int ln = lane;
    asm volatile("" : "+v"(ln));                          // offsets are formed here, not kept in registers
    const int rc = (1024 / (DC / 2)) * j0 + ln / NB, off = rc * (DC / 2) + (((ln % NB) ^ Raw::swz_codes(rc) ^ Raw::swz_quarter(quarter)) << 4);
    const int rr = 8 * j0 + ln / 8, off_rope = rr * 128 + (((ln % 8) ^ Raw::swz_rope(rr)) << 4);
    char* const to_codes = to + quarter * Raw::kCodes + j0 * 1024;
    char* const to_rope = to + Raw::kRopeAt + quarter * Raw::kRope + j0 * 1024;
    char* const to_scales = to + Raw::kScalesAt + quarter * 256;
    if (have == 15 && k0 + kRows <= rows) {
        load_lds16s(from_codes, off, to_codes);
        // 8 rows on: the permutations differ in one bit
        if constexpr (NB == 16) load_lds16s(from_codes, (off ^ 16) + 2048, to_codes + 2048);
        if constexpr (DR > 0) load_lds16s(from_rope, off_rope, to_rope);
        if (j0 == 0 && (NB == 16 || ln < 32)) load_lds4s(from_scales, 4 * ln, to_scales);
        return have;
    }
    const int left = have >> quarter & 1 ? rows - kq : 0; // rows of the quarter to be read
    auto copy = [&](char* at, const char* from, bool there) {
        *reinterpret_cast<u32x4*>(at + 16 * ln) = there ? *reinterpret_cast<const u32x4*>(from) : u32x4{0, 0, 0, 0};
    };
    copy(to_codes, from_codes + off, rc < left);
    if constexpr (NB == 16) copy(to_codes + 2048, from_codes + (off ^ 16) + 2048, rc + 8 < left);
    if constexpr (DR > 0) copy(to_rope, from_rope + off_rope, rr < left);
    if (j0 == 0 && (NB == 16 || ln < 32))
        *reinterpret_cast<uint32_t*>(to_scales + 4 * ln) =
            ln / (NB / 4) < left ? *reinterpret_cast<const uint32_t*>(from_scales + 4 * ln) : 0u;
    return have;
}

// Scores of 16 rows of queries against NG groups of 16 keys of a tile, from key0
// on: lane l holds row l % 16 and keys 4 (l / 16) .. + 3 of each. A step's operands
// are read under the one before. (The results are not waited for: settle.)
template <int DC, int DR, int NG>
__device__ __forceinline__ void mx_scores(const char* buf, int key0, int lane, const MxQuery16 (&qm)[DC / 128], uint32_t qs,
                                          const bf16x8 (&qf)[DR ? DR / 32 : 1], f32x4 (&sc)[NG]) {
    using Raw = RawTile<DC, DR>;
    constexpr int NM = DC / 128, NS = DR / 32;
    int ln = lane;
    asm volatile("" : "+v"(ln));                          // LDS addresses are formed here, not kept over the loop
    const int g = ln >> 4, n = ln & 15, r0 = key0 + n;
    uint32_t ks[NG];
    u32x4 x[2][NG];
    auto read = [&](int i) {
#pragma unroll
        for (int h = 0; h < NG; ++h) x[i & 1][h] = *reinterpret_cast<const u32x4*>(buf + Raw::codes(r0 + 16 * h, NM * g + i));
    };
#pragma unroll
    for (int h = 0; h < NG; ++h) {
        sc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (NM == 4) ks[h] = *reinterpret_cast<const uint32_t*>(buf + Raw::scales(r0 + 16 * h) + 4 * g);
        else ks[h] = *reinterpret_cast<const uint16_t*>(buf + Raw::scales(r0 + 16 * h) + 2 * g);
    }
    read(0);
    bf16x8 y[NG];
    auto rope = [&](int s) {
#pragma unroll
        for (int h = 0; h < NG; ++h) y[h] = *reinterpret_cast<const bf16x8*>(buf + Raw::rope(r0 + 16 * h, 4 * s + g));
    };
    auto step = [&](auto I) {
        constexpr int i = I.value;
        if constexpr (i + 1 < NM) read(i + 1);
        else if constexpr (NS > 0) rope(0);
#pragma unroll
        for (int h = 0; h < NG; ++h) sc[h] = mma_mx16<i>(x[i & 1][h], qm[i].hi, sc[h], ks[h], qs);
#pragma unroll
        for (int h = 0; h < NG; ++h)
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
        for (int h = 0; h < NG; ++h) sc[h] = mma16(y[h], qf[s], sc[h]);
        if (s + 1 < NS) rope(s + 1);
    }
    // (sends the products on their way here: the compiler would move them behind what follows)
#pragma unroll
    for (int h = 0; h < NG; ++h) asm volatile("" : "+v"(sc[h]));
}

}  // namespace
}  // namespace kda
