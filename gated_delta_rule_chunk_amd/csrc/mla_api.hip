// C ABI of the latent-attention calls: argument checks, workspaces, errors.
#include <math.h>
#include <stdarg.h>

#include "../../include/kda_mla.h"
#include "launchers.hpp"
#include "mla_common.hpp"

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

// The expanded kernels take a workgroup per head and tile of 128 rows (small
// launches of 32 rows: far from the limit) of a side's queries or keys.
kda_status check_tiles(const char* fn, const int32_t* cu, int32_t B, int32_t N, int32_t T, int32_t H) {
    if (kda::mla::tile_slots(cu, B, N, T, 128) > kMaxGrid / H)
        return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: over %lld tiles of 128 rows, heads counted", fn,
                    (long long)kMaxGrid);
    return KDA_OK;
}

// Checks shared by the forward and the backward; fills a on success.
kda_status check_expanded(const char* fn, const void* q, const void* kv, const void* k_rope, int64_t kr_row,
                          int64_t kr_batch, const int32_t* cuq, const int32_t* cuk, int32_t B, int32_t Tq, int32_t Tk,
                          int32_t H, int32_t Dn, int32_t Dr, int32_t N, int32_t causal, float scale, kda_dtype dtype,
                          int32_t zero_rest, kda::MlaArgs& a) {
    if (B < 1 || Tq < 0 || Tk < 0 || H < 1 || N < 1)
        return fail(KDA_ERR_INVALID_ARG, "%s: need B >= 1, Tq >= 0, Tk >= 0, H >= 1, N >= 1 (got %d, %d, %d, %d, %d)",
                    fn, B, Tq, Tk, H, N);
    if (kda_status st = check_type(fn, dtype)) return st;
    if ((Dn != 64 && Dn != 128) || (Dr != 0 && Dr != 64))
        return fail(KDA_ERR_UNSUPPORTED, "%s: Dn=%d, Dr=%d; supported are Dn 64, 128 and Dr 0, 64", fn, Dn, Dr);
    if ((cuq == nullptr) != (cuk == nullptr))
        return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens_q and cu_seqlens_k come together", fn);
    if (cuq && B != 1)
        return fail(KDA_ERR_INVALID_ARG, "%s: packed sequences (cu_seqlens) need B == 1, got B=%d", fn, B);
    if (!cuq && N != B) return fail(KDA_ERR_INVALID_ARG, "%s: without cu_seqlens N must equal B (N=%d, B=%d)", fn, N, B);
    if (causal != 0 && causal != 1) return fail(KDA_ERR_INVALID_ARG, "%s: causal must be 0 or 1, got %d", fn, causal);
    if (kda_status st = check_scale(fn, scale)) return st;
    if (Tq > 0 && !q) return fail(KDA_ERR_INVALID_ARG, "%s: q must be non-NULL when Tq > 0", fn);
    if (Tk > 0 && !kv) return fail(KDA_ERR_INVALID_ARG, "%s: kv must be non-NULL when Tk > 0", fn);
    if (Dr == 0 ? k_rope != nullptr : (Tk > 0 && !k_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: k_rope must be NULL if and only if Dr = 0", fn);
    if (Dr && (!stride_ok(kr_row, dtype) || !stride_ok(kr_batch, dtype)))
        return fail(KDA_ERR_INVALID_ARG, "%s: k_rope strides must be multiples of 16 bytes (got %lld, %lld elements)", fn,
                    (long long)kr_row, (long long)kr_batch);
    if (!aligned(q) || !aligned(kv) || !aligned(k_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: q, kv and k_rope must be 16-byte aligned", fn);
    if (kda_status st = check_tiles(fn, cuq, B, N, Tq, H)) return st;
    // the kernels hold the bytes of a tile's 64 rows in 31 bits
    if (H > 4096 || (Dr && kr_row > (1 << 22)))
        return fail(KDA_ERR_UNSUPPORTED, "%s: H=%d, k_rope row stride %lld; at most 4096 and 2^22 elements", fn, H,
                    (long long)kr_row);
    a.q = q; a.kv = kv; a.kr = k_rope; a.kr_row = kr_row; a.kr_batch = kr_batch; a.cuq = cuq; a.cuk = cuk;
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H; a.Dn = Dn; a.Dr = Dr; a.N = N;
    a.causal = causal != 0; a.bf16 = dtype == KDA_BF16; a.zero_rest = zero_rest != 0; a.scale = scale;
    return KDA_OK;
}

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

}  // namespace

extern "C" {

kda_status kda_mla_fwd(const void* q, const void* kv, const void* k_rope, int64_t k_rope_row, int64_t k_rope_batch,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t B, int32_t Tq, int32_t Tk,
                       int32_t H, int32_t Dn, int32_t Dr, int32_t N, int32_t causal, float scale, kda_dtype dtype,
                       int32_t zero_rest, void* o, float* lse, void* stream) {
    const char* fn = "kda_mla_fwd";
    kda::clear_error();
    kda::MlaArgs a{};
    if (kda_status st = check_expanded(fn, q, kv, k_rope, k_rope_row, k_rope_batch, cu_seqlens_q, cu_seqlens_k, B, Tq,
                                       Tk, H, Dn, Dr, N, causal, scale, dtype, zero_rest, a))
        return st;
    if (Tq == 0) return KDA_OK;
    if (!o || !aligned(o)) return fail(KDA_ERR_INVALID_ARG, "%s: o must be non-NULL and 16-byte aligned", fn);
    Ranges r{fn};
    r.apart("o", o, "q", q);
    r.apart("o", o, "kv", kv);
    r.apart("o", o, "k_rope", k_rope);
    if (r.st != KDA_OK) return r.st;
    a.o = o;
    a.lse = lse;
    return finish(fn, kda::launch_mla_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_bwd_workspace_bytes(int32_t B, int32_t Tq, int32_t Tk, int32_t H, int32_t Dr) {
    if (B < 1 || Tq < 0 || Tk < 0 || H < 1 || (Dr != 0 && Dr != 64)) return 0;
    // enough for any call: packed sequences have no fewer tiles and bf16 no more
    // parts than dense float32 ones
    kda::MlaArgs a{};
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.H = H; a.Dn = 128; a.Dr = Dr; a.N = B;
    return kda::mla_bwd_plan(a);
}

kda_status kda_mla_bwd(const void* q, const void* kv, const void* k_rope, int64_t k_rope_row, int64_t k_rope_batch,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, const void* o, const float* lse,
                       const void* d_o, int32_t B, int32_t Tq, int32_t Tk, int32_t H, int32_t Dn, int32_t Dr,
                       int32_t N, int32_t causal, float scale, kda_dtype dtype, int32_t zero_rest, void* workspace,
                       size_t workspace_bytes, void* dq, void* dkv, void* dk_rope, void* stream) {
    const char* fn = "kda_mla_bwd";
    kda::clear_error();
    kda::MlaArgs a{};
    if (kda_status st = check_expanded(fn, q, kv, k_rope, k_rope_row, k_rope_batch, cu_seqlens_q, cu_seqlens_k, B, Tq,
                                       Tk, H, Dn, Dr, N, causal, scale, dtype, zero_rest, a))
        return st;
    if (kda_status st = check_tiles(fn, cu_seqlens_k, B, N, Tk, H)) return st;
    if (Dr && (int64_t)B * Tk > kMaxGrid * 256 / 16)      // the sum of dk_rope: a thread for each 4 of its columns
        return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: B * Tk = %lld", fn, (long long)B * Tk);
    if (Tq == 0 && Tk == 0) return KDA_OK;
    if (Tq > 0 && (!o || !lse || !d_o || !dq))
        return fail(KDA_ERR_INVALID_ARG, "%s: o, lse, d_o and dq must be non-NULL when Tq > 0", fn);
    if (Tk > 0 && !dkv) return fail(KDA_ERR_INVALID_ARG, "%s: dkv must be non-NULL when Tk > 0", fn);
    if (Dr == 0 ? dk_rope != nullptr : (Tk > 0 && !dk_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: dk_rope must be NULL if and only if Dr = 0", fn);
    const size_t need = kda_mla_bwd_workspace_bytes(B, Tq, Tk, H, Dr);
    if (need && (!workspace || workspace_bytes < need))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace ? workspace_bytes : 0,
                    need);
    if (!aligned(o) || !aligned(d_o) || !aligned(dq) || !aligned(dkv) || !aligned(dk_rope) || !aligned(workspace))
        return fail(KDA_ERR_INVALID_ARG, "%s: every tensor and the workspace must be 16-byte aligned", fn);
    Ranges r{fn};
    const void* outs[] = {dq, dkv, dk_rope, workspace};
    const char* names[] = {"dq", "dkv", "dk_rope", "workspace"};
    for (int i = 0; i < 4; ++i) {
        r.apart(names[i], outs[i], "q", q);
        r.apart(names[i], outs[i], "kv", kv);
        r.apart(names[i], outs[i], "k_rope", k_rope);
        r.apart(names[i], outs[i], "o", o);
        r.apart(names[i], outs[i], "lse", lse);
        r.apart(names[i], outs[i], "d_o", d_o);
        for (int j = 0; j < i; ++j) r.apart(names[i], outs[i], names[j], outs[j]);
    }
    if (r.st != KDA_OK) return r.st;
    a.o = const_cast<void*>(o);
    a.lse = const_cast<float*>(lse);
    a.d_o = d_o; a.dq = dq; a.dkv = dkv; a.dkr = dk_rope;
    a.delta = static_cast<float*>(workspace);
    kda::mla_bwd_plan(a);
    return finish(fn, kda::launch_mla_bwd(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_mla_cache_append(const void* latent, int64_t latent_row, int64_t latent_batch, const void* k_rope,
                                int64_t k_rope_row, int64_t k_rope_batch, void* cache, const int32_t* page_table,
                                const int32_t* cache_lens, const int32_t* cu_seqlens, int32_t n_pages,
                                int32_t page_size, int32_t max_pages, int32_t B, int32_t T, int32_t Dc, int32_t Dr,
                                int32_t N, kda_dtype dtype, void* stream) {
    const char* fn = "kda_mla_cache_append";
    kda::clear_error();
    if (B < 0 || T < 0 || N < 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: need B >= 0, T >= 0, N >= 0 (got %d, %d, %d)", fn, B, T, N);
    if (cu_seqlens ? (B != 1 || N < 1) : N != B)
        return fail(KDA_ERR_INVALID_ARG, "%s: packed tokens (cu_seqlens) need B == 1 and N >= 1, others N == B (B=%d, N=%d)",
                    fn, B, N);
    if ((int64_t)B * T == 0) return KDA_OK;
    kda::MlaAppendArgs a{};
    if (kda_status st = check_cache(fn, cache, page_table, cache_lens, n_pages, page_size, max_pages, Dc, Dr, dtype,
                                    a.page_shift))
        return st;
    // a thread for each 16 bytes of a token
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
    a.status = kda::device_status_word();
    if (!a.status) return fail(KDA_ERR_HIP, "%s: the device status word is not accessible", fn);
    a.status += 2;
    return finish(fn, kda::launch_mla_append(a, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_step_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size,
                                    int32_t max_pages, kda_dtype dtype) {
    if (!step_sizes_ok(Nb, Tq, H) || (int64_t)Nb * Tq == 0 || (Dc != 256 && Dc != 512) || page_size < 16 ||
        page_size > (1 << 24) || (page_size & (page_size - 1)) || max_pages < 1 ||
        (int64_t)max_pages * page_size > ((int64_t)1 << 30))
        return 0;
    kda::MlaStepArgs a{};
    a.Nb = Nb; a.Tq = Tq; a.H = H; a.Dc = Dc; a.max_pages = max_pages; a.bf16 = dtype == KDA_BF16;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    return kda::mla_step_plan(a);
}

kda_status kda_mla_step(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                        const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                        const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                        int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                        kda_dtype dtype, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream) {
    const char* fn = "kda_mla_step";
    kda::clear_error();
    if (!step_sizes_ok(Nb, Tq, H))
        return fail(KDA_ERR_INVALID_ARG,
                    "%s: need Nb >= 0, Tq >= 0, H >= 1, Tq * H <= 2^20, Nb * Tq * H <= 2^30 (got %d, %d, %d)", fn, Nb,
                    Tq, H);
    if ((int64_t)Nb * Tq == 0) return KDA_OK;
    kda::MlaStepArgs a{};
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
    if (!o || !aligned(o) || !aligned(q_latent) || !aligned(q_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: q_latent, q_rope and o must be 16-byte aligned, o non-NULL", fn);
    Ranges r{fn};
    r.apart("o", o, "q_latent", q_latent);
    r.apart("o", o, "q_rope", q_rope);
    r.apart("o", o, "cache", cache);
    r.apart("workspace", workspace, "cache", cache);
    r.apart("workspace", workspace, "o", o);
    if (r.st != KDA_OK) return r.st;
    a.ql = q_latent; a.ql_b = q_latent_n; a.ql_t = q_latent_t; a.ql_h = q_latent_h;
    a.qr = q_rope; a.qr_b = q_rope_n; a.qr_t = q_rope_t; a.qr_h = q_rope_h;
    a.cache = cache; a.table = page_table; a.lens = seq_lens; a.o = o; a.lse = lse;
    a.part = static_cast<float*>(workspace);
    a.n_pages = n_pages; a.max_pages = max_pages; a.Nb = Nb; a.Tq = Tq; a.H = H; a.Dc = Dc; a.Dr = Dr;
    a.scale = scale; a.bf16 = dtype == KDA_BF16;
    const size_t need = kda::mla_step_plan(a);
    const int64_t joins = (int64_t)Nb * ((Tq * H + a.join_rows - 1) / a.join_rows);     // workgroups of the second kernel
    if (joins > kMaxGrid) return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: Nb = %d", fn, Nb);
    if (!workspace || workspace_bytes < need || !aligned(workspace))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn,
                    workspace ? workspace_bytes : 0, need);
    a.status = kda::device_status_word();
    if (!a.status) return fail(KDA_ERR_HIP, "%s: the device status word is not accessible", fn);
    a.status += 2;
    return finish(fn, kda::launch_mla_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
