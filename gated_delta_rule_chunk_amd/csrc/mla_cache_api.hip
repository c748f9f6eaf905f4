// C ABI of include/kda_mla_cache.h: argument checks, workspaces, errors.
#include "../../include/kda_mla_cache.h"
#include "mla_check.hpp"
#include "mla_mx.hpp"

namespace {

// the cache's form: 0 rows of dtype, 1 latents in 4 bits
kda_status check_form(const char* fn, int32_t form) {
    if (form != 0 && form != 1) return fail(KDA_ERR_INVALID_ARG, "%s: form must be 0 or 1, got %d", fn, form);
    return KDA_OK;
}

int shift_of(int32_t page_size) {
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    return shift;
}

}  // namespace

extern "C" {

size_t kda_mla_mx_row_bytes(int32_t Dc, int32_t Dr, kda_dtype dtype) {
    if ((Dc != 256 && Dc != 512) || (Dr != 0 && Dr != 64) || (dtype != KDA_F32 && dtype != KDA_BF16)) return 0;
    return (size_t)kda::mla::mx_row_bytes(Dc, Dr, dtype == KDA_BF16 ? 2 : 4);
}

kda_status kda_mla_cache_append_mx(const void* latent, int64_t latent_row, int64_t latent_batch, const void* k_rope,
                                   int64_t k_rope_row, int64_t k_rope_batch, void* cache, const int32_t* page_table,
                                   const int32_t* cache_lens, const int32_t* cu_seqlens, int32_t n_pages,
                                   int32_t page_size, int32_t max_pages, int32_t B, int32_t T, int32_t Dc, int32_t Dr,
                                   int32_t N, kda_dtype dtype, void* stream) {
    const char* fn = "kda_mla_cache_append_mx";
    kda::clear_error();
    kda::MlaAppendArgs a{};
    bool none;
    if (kda_status st = check_append(fn, latent, latent_row, latent_batch, k_rope, k_rope_row, k_rope_batch, cache,
                                     page_table, cache_lens, cu_seqlens, n_pages, page_size, max_pages, B, T, Dc, Dr, N,
                                     dtype, a, none))
        return st;
    if (none) return KDA_OK;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_append_mx(a, static_cast<hipStream_t>(stream)));
}

kda_status kda_mla_cache_read_mx(const void* cache, const int32_t* page_table, const int32_t* starts,
                                 const int32_t* cu_seqlens, int32_t n_pages, int32_t page_size, int32_t max_pages,
                                 int32_t T, int32_t Dc, int32_t Dr, int32_t N, kda_dtype dtype, int32_t zero_rest,
                                 void* latent, void* k_rope, void* stream) {
    const char* fn = "kda_mla_cache_read_mx";
    kda::clear_error();
    if (T < 0 || N < 1) return fail(KDA_ERR_INVALID_ARG, "%s: need T >= 0 and N >= 1 (got %d, %d)", fn, T, N);
    if (T == 0) return KDA_OK;
    kda::MlaReadArgs a{};
    if (kda_status st = check_cache(fn, cache, page_table, cu_seqlens, n_pages, page_size, max_pages, Dc, Dr, dtype,
                                    a.page_shift))
        return st;
    if ((int64_t)T > kMaxGrid * 256 / (Dc / 8 + 16))             // as the header has it; the grid would hold more, 16 rows a workgroup
        return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: T = %d", fn, T);
    if (!latent || (Dr == 0) != (k_rope == nullptr))
        return fail(KDA_ERR_INVALID_ARG, "%s: latent must be non-NULL, k_rope NULL if and only if Dr = 0", fn);
    if (!aligned(latent) || !aligned(k_rope))
        return fail(KDA_ERR_INVALID_ARG, "%s: latent and k_rope must be 16-byte aligned", fn);
    Ranges r{fn};
    r.apart("latent", latent, "cache", cache);
    r.apart("k_rope", k_rope, "cache", cache);
    r.apart("k_rope", k_rope, "latent", latent);
    if (r.st != KDA_OK) return r.st;
    a.cache = cache; a.table = page_table; a.starts = starts; a.cu = cu_seqlens; a.latent = latent; a.rope = k_rope;
    a.n_pages = n_pages; a.max_pages = max_pages; a.T = T; a.Dc = Dc; a.Dr = Dr; a.N = N;
    a.bf16 = dtype == KDA_BF16; a.zero_rest = zero_rest != 0;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_read_mx(a, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_step_mx_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size,
                                       int32_t max_pages, kda_dtype dtype) {
    return step_workspace(Nb, Tq, H, Dc, page_size, max_pages, dtype, kda::mla_step_mx_plan);
}

kda_status kda_mla_step_mx(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                           const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                           const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                           int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                           kda_dtype dtype, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream) {
    const char* fn = "kda_mla_step_mx";
    kda::clear_error();
    if (!step_sizes_ok(Nb, Tq, H)) return fail(KDA_ERR_INVALID_ARG, kStepSizes, fn, Nb, Tq, H);
    if ((int64_t)Nb * Tq == 0) return KDA_OK;
    kda::MlaStepArgs a{};
    if (kda_status st = check_step(fn, q_latent, q_latent_n, q_latent_t, q_latent_h, q_rope, q_rope_n, q_rope_t, q_rope_h,
                                   cache, page_table, seq_lens, n_pages, page_size, max_pages, Nb, Tq, H, Dc, Dr, scale,
                                   dtype, a))
        return st;
    if (kda_status st = check_step_outputs(fn, a, kda::mla_step_mx_plan, workspace, workspace_bytes, o, lse)) return st;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_step_mx(a, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_weigh_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, kda_dtype dtype,
                                     int32_t form) {
    if (!step_sizes_ok(Nb, Tq, H) || (Dc != 256 && Dc != 512) || (Dr != 0 && Dr != 64)) return 0;
    kda::MlaWeighArgs x{};
    x.s.Nb = Nb; x.s.Tq = Tq; x.s.H = H; x.s.Dc = Dc; x.s.Dr = Dr; x.s.bf16 = dtype == KDA_BF16; x.mx = form == 1;
    return kda::mla_weigh_workspace(x);
}

kda_status kda_mla_weigh(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                         const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                         const int32_t* page_table, const int32_t* seq_lens, const float* lse, const float* weights,
                         int32_t fresh, float decay, int32_t n_pages, int32_t page_size, int32_t max_pages, int32_t Nb,
                         int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale, kda_dtype dtype, int32_t form,
                         void* workspace, size_t workspace_bytes, float* weights_out, void* stream) {
    const char* fn = "kda_mla_weigh";
    kda::clear_error();
    if (!step_sizes_ok(Nb, Tq, H)) return fail(KDA_ERR_INVALID_ARG, kStepSizes, fn, Nb, Tq, H);
    if ((int64_t)Nb * Tq == 0) return KDA_OK;
    kda::MlaWeighArgs x{};
    if (kda_status st = check_step(fn, q_latent, q_latent_n, q_latent_t, q_latent_h, q_rope, q_rope_n, q_rope_t, q_rope_h,
                                   cache, page_table, seq_lens, n_pages, page_size, max_pages, Nb, Tq, H, Dc, Dr, scale,
                                   dtype, x.s))
        return st;
    if (kda_status st = check_form(fn, form)) return st;
    if (fresh < 0) return fail(KDA_ERR_INVALID_ARG, "%s: fresh must be >= 0, got %d", fn, fresh);
    if (!(decay >= 0.f && decay <= 1.f))
        return fail(KDA_ERR_INVALID_ARG, "%s: decay must be in [0, 1], got %g", fn, (double)decay);
    if (!lse || !weights || !weights_out)
        return fail(KDA_ERR_INVALID_ARG, "%s: lse, weights and weights_out must be non-NULL", fn);
    Ranges r{fn};
    r.apart("weights_out", weights_out, "q_latent", q_latent);
    r.apart("weights_out", weights_out, "q_rope", q_rope);
    r.apart("weights_out", weights_out, "cache", cache);
    r.apart("weights_out", weights_out, "lse", lse);
    if (r.st != KDA_OK) return r.st;
    const size_t need = kda_mla_weigh_workspace_bytes(Nb, Tq, H, Dc, Dr, dtype, form);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace)))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn,
                    workspace ? workspace_bytes : 0, need);
    if (need) {
        r.apart("workspace", workspace, "cache", cache);
        r.apart("workspace", workspace, "weights_out", weights_out);
        r.apart("workspace", workspace, "q_latent", q_latent);
        r.apart("workspace", workspace, "q_rope", q_rope);
        r.apart("workspace", workspace, "lse", lse);
        r.apart("workspace", workspace, "weights", weights);
        if (r.st != KDA_OK) return r.st;
    }
    x.split = static_cast<char*>(workspace);
    x.lse = lse; x.w_in = weights; x.w_out = weights_out; x.fresh = fresh; x.decay = decay; x.mx = form == 1;
    if (kda_status st = set_status(fn, x.s.status)) return st;
    return finish(fn, kda::launch_mla_weigh(x, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_evict_workspace_bytes(int32_t Nb, int32_t page_size, int32_t max_pages) {
    if (Nb < 1 || Nb >= (1 << 22) || page_size < 16 || page_size > (1 << 24) || (page_size & (page_size - 1)) ||
        max_pages < 1 || (int64_t)max_pages * page_size > ((int64_t)1 << 30))
        return 0;
    return kda::mla_evict_workspace(Nb, shift_of(page_size), max_pages);
}

kda_status kda_mla_evict(void* cache, const int32_t* page_table, const int32_t* seq_lens, const float* weights,
                         int32_t keep, int32_t first, int32_t recent, int32_t n_pages, int32_t page_size,
                         int32_t max_pages, int32_t Nb, int32_t Dc, int32_t Dr, kda_dtype dtype, int32_t form,
                         void* workspace, size_t workspace_bytes, int32_t* page_table_out, int32_t* seq_lens_out,
                         float* weights_out, void* stream) {
    const char* fn = "kda_mla_evict";
    kda::clear_error();
    if (Nb < 0 || Nb >= (1 << 22)) return fail(KDA_ERR_INVALID_ARG, "%s: need 0 <= Nb < 2^22, got %d", fn, Nb);
    if (Nb == 0) return KDA_OK;
    kda::MlaEvictArgs a{};
    if (kda_status st = check_cache(fn, cache, page_table, seq_lens, n_pages, page_size, max_pages, Dc, Dr, dtype,
                                    a.page_shift))
        return st;
    if (kda_status st = check_form(fn, form)) return st;
    if (keep < 0 || first < 0 || recent < 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: keep, first and recent must be >= 0 (got %d, %d, %d)", fn, keep, first,
                    recent);
    if (!weights || !page_table_out || !seq_lens_out || !weights_out)
        return fail(KDA_ERR_INVALID_ARG, "%s: weights and the three outputs must be non-NULL", fn);
    if (kda::mla_evict_workgroups(Nb, a.page_shift, max_pages) >= (1 << 22))
        return fail(KDA_ERR_UNSUPPORTED, "%s: problem too large: Nb = %d sequences of up to %lld rows", fn, Nb,
                    (long long)max_pages * page_size);
    const size_t need = kda::mla_evict_workspace(Nb, a.page_shift, max_pages);
    if (!workspace || workspace_bytes < need || !aligned(workspace))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", fn,
                    workspace ? workspace_bytes : 0, need);
    Ranges r{fn};
    const void* outs[] = {page_table_out, seq_lens_out, weights_out, workspace};
    const void* ins[] = {page_table, seq_lens, weights, nullptr};
    const char* names[] = {"page_table_out", "seq_lens_out", "weights_out", "workspace"};
    const char* in_names[] = {"page_table", "seq_lens", "weights", ""};
    for (int i = 0; i < 4; ++i) {
        r.apart(names[i], outs[i], "cache", cache);
        for (int j = 0; j < 3; ++j)
            if (j != i) r.apart(names[i], outs[i], in_names[j], ins[j]);
        for (int j = 0; j < i; ++j) r.apart(names[i], outs[i], names[j], outs[j]);
    }
    if (r.st != KDA_OK) return r.st;
    const int es = dtype == KDA_BF16 ? 2 : 4;
    a.cache = static_cast<char*>(cache); a.table = page_table; a.lens = seq_lens; a.w_in = weights;
    a.table_out = page_table_out; a.lens_out = seq_lens_out; a.w_out = weights_out;
    a.work = static_cast<int32_t*>(workspace);
    a.n_pages = n_pages; a.max_pages = max_pages; a.Nb = Nb; a.keep = keep; a.first = first; a.recent = recent;
    a.codes = form ? Dc / 32 : (Dc + Dr) * es / 16;
    a.scale_bytes = form ? Dc / 32 : 0;
    a.rope = form ? Dr * es / 16 : 0;
    a.units = a.codes + (form ? 1 : 0) + a.rope;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_evict(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
