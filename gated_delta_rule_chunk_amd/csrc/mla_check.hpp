// Argument checks shared by the C entries of the latent-attention calls.
#pragma once

#include <math.h>
#include <stdarg.h>

#include "../../include/kda_mla.h"
#include "launchers.hpp"

namespace {

kda_status fail(kda_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    kda::set_error(fmt, ap);
    va_end(ap);
    return st;
}

bool aligned(const void* p) { return ((uintptr_t)p & 15) == 0; }

struct Ranges {     // inputs and outputs that may not be the same memory
    const char* fn;
    kda_status st = KDA_OK;
    void apart(const char* name, const void* out, const char* what, const void* in) {
        if (st == KDA_OK && out && out == in) st = fail(KDA_ERR_INVALID_ARG, "%s: %s must not alias %s", fn, name, what);
    }
};

kda_status check_type(const char* fn, kda_dtype dtype) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_UNSUPPORTED, "%s: dtype %d is not KDA_F32 or KDA_BF16", fn, (int)dtype);
    return KDA_OK;
}
kda_status check_scale(const char* fn, float scale) {
    if (!(scale > 0.f) || !isfinite(scale))
        return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite and > 0 (got %g)", fn, (double)scale);
    return KDA_OK;
}
// Strides of a tensor that need not be contiguous: no check of the extent is
// possible, only of what the kernels' 16-byte accesses need.
bool stride_ok(int64_t s, kda_dtype dtype) { return s >= 0 && s * (dtype == KDA_BF16 ? 2 : 4) % 16 == 0; }

// A launch counts its threads in 32 bits: so many workgroups of 256.
constexpr int64_t kMaxGrid = 0xffffffffll / 256;

kda_status check_cache(const char* fn, const void* cache, const int32_t* table, const int32_t* lens, int32_t n_pages,
                       int32_t page_size, int32_t max_pages, int32_t Dc, int32_t Dr, kda_dtype dtype, int32_t& shift) {
    if (kda_status st = check_type(fn, dtype)) return st;
    if ((Dc != 256 && Dc != 512) || (Dr != 0 && Dr != 64))
        return fail(KDA_ERR_UNSUPPORTED, "%s: Dc=%d, Dr=%d; supported are Dc 256, 512 and Dr 0, 64", fn, Dc, Dr);
    if (page_size < 16 || page_size > (1 << 24) || (page_size & (page_size - 1)))
        return fail(KDA_ERR_UNSUPPORTED, "%s: page_size=%d; a power of two from 16 to 2^24 is needed", fn, page_size);
    if (n_pages < 1 || max_pages < 1)
        return fail(KDA_ERR_INVALID_ARG, "%s: need n_pages >= 1 and max_pages >= 1 (got %d, %d)", fn, n_pages, max_pages);
    if (!cache || !table || !lens)
        return fail(KDA_ERR_INVALID_ARG, "%s: cache, page_table and the lengths must be non-NULL", fn);
    if (!aligned(cache)) return fail(KDA_ERR_INVALID_ARG, "%s: cache must be 16-byte aligned", fn);
    shift = 0;
    while ((1 << shift) < page_size) ++shift;
    if ((int64_t)max_pages * page_size > ((int64_t)1 << 30))
        return fail(KDA_ERR_UNSUPPORTED, "%s: max_pages * page_size = %lld; at most 2^30 rows a sequence", fn,
                    (long long)max_pages * page_size);
    return KDA_OK;
}

kda_status finish(const char* fn, hipError_t e) {
    return e == hipSuccess ? KDA_OK : fail(KDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
}

bool step_sizes_ok(int32_t Nb, int32_t Tq, int32_t H) {
    return Nb >= 0 && Tq >= 0 && H >= 1 && (int64_t)Tq * H <= (1 << 20) && (int64_t)Nb * Tq * H <= ((int64_t)1 << 30);
}

// A cache write's arguments; fills a on success. none: there is nothing to write.
kda_status check_append(const char* fn, const void* latent, int64_t latent_row, int64_t latent_batch, const void* k_rope,
                        int64_t k_rope_row, int64_t k_rope_batch, void* cache, const int32_t* page_table,
                        const int32_t* cache_lens, const int32_t* cu_seqlens, int32_t n_pages, int32_t page_size,
                        int32_t max_pages, int32_t B, int32_t T, int32_t Dc, int32_t Dr, int32_t N, kda_dtype dtype,
                        kda::MlaAppendArgs& a, bool& none) {
    if (B < 0 || T < 0 || N < 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: need B >= 0, T >= 0, N >= 0 (got %d, %d, %d)", fn, B, T, N);
    if (cu_seqlens ? (B != 1 || N < 1) : N != B)
        return fail(KDA_ERR_INVALID_ARG, "%s: packed tokens (cu_seqlens) need B == 1 and N >= 1, others N == B (B=%d, N=%d)",
                    fn, B, N);
    none = (int64_t)B * T == 0;
    if (none) return KDA_OK;
    if (kda_status st = check_cache(fn, cache, page_table, cache_lens, n_pages, page_size, max_pages, Dc, Dr, dtype,
                                    a.page_shift))
        return st;
    // a thread for each 16 bytes of a token (the 4-bit write has the same limit, though its grid would hold more)
    if ((int64_t)B * T > kMaxGrid * 256 / ((Dc + Dr) * (dtype == KDA_BF16 ? 2 : 4) / 16))
        return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: B * T = %lld", fn, (long long)B * T);
    if (!latent || (Dr == 0) != (k_rope == nullptr))
        return fail(KDA_ERR_INVALID_ARG, "%s: latent must be non-NULL, k_rope NULL if and only if Dr = 0", fn);
    if (!stride_ok(latent_row, dtype) || !stride_ok(latent_batch, dtype) ||
        (Dr && (!stride_ok(k_rope_row, dtype) || !stride_ok(k_rope_batch, dtype))) || !aligned(latent) ||
        !aligned(k_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: latent and k_rope must be 16-byte aligned, strides included", fn);
    if (latent == cache || k_rope == cache) return fail(KDA_ERR_INVALID_ARG, "%s: cache must not alias an input", fn);
    a.latent = latent; a.lat_row = latent_row; a.lat_batch = latent_batch;
    a.kr = k_rope; a.kr_row = k_rope_row; a.kr_batch = k_rope_batch;
    a.cache = cache; a.table = page_table; a.lens = cache_lens; a.cu = cu_seqlens;
    a.n_pages = n_pages; a.max_pages = max_pages; a.B = B; a.T = T; a.Dc = Dc; a.Dr = Dr; a.N = N;
    a.bf16 = dtype == KDA_BF16;
    return KDA_OK;
}

// The queries, cache and sizes of a call over cached rows; fills a on success.
kda_status check_step(const char* fn, const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                      const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                      const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                      int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                      kda_dtype dtype, kda::MlaStepArgs& a) {
    if (kda_status st = check_cache(fn, cache, page_table, seq_lens, n_pages, page_size, max_pages, Dc, Dr, dtype,
                                    a.page_shift))
        return st;
    if (kda_status st = check_scale(fn, scale)) return st;
    if (!q_latent || (Dr == 0) != (q_rope == nullptr))
        return fail(KDA_ERR_INVALID_ARG, "%s: q_latent must be non-NULL, q_rope NULL if and only if Dr = 0", fn);
    // the kernels count the cache's 32-row tiles in 31 bits
    if ((int64_t)Nb * (((int64_t)max_pages * page_size + 31) / 32) > ((int64_t)1 << 30))
        return fail(KDA_ERR_UNSUPPORTED, "%s: Nb * max_pages * page_size too large", fn);
    const int64_t st[] = {q_latent_n, q_latent_t, q_latent_h, q_rope_n, q_rope_t, q_rope_h};
    for (int i = 0; i < (Dr ? 6 : 3); ++i)
        if (!stride_ok(st[i], dtype))
            return fail(KDA_ERR_INVALID_ARG, "%s: strides of q_latent and q_rope must be multiples of 16 bytes", fn);
    if (!aligned(q_latent) || !aligned(q_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: q_latent and q_rope must be 16-byte aligned", fn);
    a.ql = q_latent; a.ql_b = q_latent_n; a.ql_t = q_latent_t; a.ql_h = q_latent_h;
    a.qr = q_rope; a.qr_b = q_rope_n; a.qr_t = q_rope_t; a.qr_h = q_rope_h;
    a.cache = cache; a.table = page_table; a.lens = seq_lens;
    a.n_pages = n_pages; a.max_pages = max_pages; a.Nb = Nb; a.Tq = Tq; a.H = H; a.Dc = Dc; a.Dr = Dr;
    a.scale = scale; a.bf16 = dtype == KDA_BF16;
    return KDA_OK;
}

// The word that counts cache rows which do not exist; looked up last, as it needs a device.
kda_status set_status(const char* fn, unsigned int*& status) {
    status = kda::device_status_word();
    if (!status) return fail(KDA_ERR_HIP, "%s: the device status word is not accessible", fn);
    status += 2;
    return KDA_OK;
}

// Output and workspace of a decode call. plan: the split, its workspace in bytes.
kda_status check_step_outputs(const char* fn, kda::MlaStepArgs& a, size_t (*plan)(kda::MlaStepArgs&), void* workspace,
                              size_t workspace_bytes, void* o, float* lse) {
    if (!o || !aligned(o)) return fail(KDA_ERR_INVALID_ARG, "%s: q_latent, q_rope and o must be 16-byte aligned, o non-NULL", fn);
    Ranges r{fn};
    r.apart("o", o, "q_latent", a.ql);
    r.apart("o", o, "q_rope", a.qr);
    r.apart("o", o, "cache", a.cache);
    r.apart("workspace", workspace, "cache", a.cache);
    r.apart("workspace", workspace, "o", o);
    if (r.st != KDA_OK) return r.st;
    a.o = o;
    a.lse = lse;
    a.part = static_cast<float*>(workspace);
    const size_t need = plan(a);
    const int64_t joins = (int64_t)a.Nb * ((a.Tq * a.H + a.join_rows - 1) / a.join_rows);   // workgroups of the second kernel
    if (joins > kMaxGrid) return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: Nb = %d", fn, a.Nb);
    if (!workspace || workspace_bytes < need || !aligned(workspace))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn,
                    workspace ? workspace_bytes : 0, need);
    return KDA_OK;
}

// The split of a decode call of these sizes, for its workspace; 0 for sizes out of range.
size_t step_workspace(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size, int32_t max_pages,
                      kda_dtype dtype, size_t (*plan)(kda::MlaStepArgs&)) {
    if (!step_sizes_ok(Nb, Tq, H) || (int64_t)Nb * Tq == 0 || (Dc != 256 && Dc != 512) || page_size < 16 ||
        page_size > (1 << 24) || (page_size & (page_size - 1)) || max_pages < 1 ||
        (int64_t)max_pages * page_size > ((int64_t)1 << 30))
        return 0;
    kda::MlaStepArgs a{};
    a.Nb = Nb; a.Tq = Tq; a.H = H; a.Dc = Dc; a.max_pages = max_pages; a.bf16 = dtype == KDA_BF16;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    return plan(a);
}

const char* const kStepSizes = "%s: need Nb >= 0, Tq >= 0, H >= 1, Tq * H <= 2^20, Nb * Tq * H <= 2^30 (got %d, %d, %d)";

}  // namespace
