// C ABI of the latent-attention calls: argument checks, workspaces, errors.
#include "mla_check.hpp"
#include "mla_common.hpp"

namespace {

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
    kda::MlaAppendArgs a{};
    bool none;
    if (kda_status st = check_append(fn, latent, latent_row, latent_batch, k_rope, k_rope_row, k_rope_batch, cache,
                                     page_table, cache_lens, cu_seqlens, n_pages, page_size, max_pages, B, T, Dc, Dr, N,
                                     dtype, a, none))
        return st;
    if (none) return KDA_OK;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_append(a, static_cast<hipStream_t>(stream)));
}

size_t kda_mla_step_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size,
                                    int32_t max_pages, kda_dtype dtype) {
    return step_workspace(Nb, Tq, H, Dc, page_size, max_pages, dtype, kda::mla_step_plan);
}

kda_status kda_mla_step(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                        const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                        const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                        int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                        kda_dtype dtype, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream) {
    const char* fn = "kda_mla_step";
    kda::clear_error();
    if (!step_sizes_ok(Nb, Tq, H)) return fail(KDA_ERR_INVALID_ARG, kStepSizes, fn, Nb, Tq, H);
    if ((int64_t)Nb * Tq == 0) return KDA_OK;
    kda::MlaStepArgs a{};
    if (kda_status st = check_step(fn, q_latent, q_latent_n, q_latent_t, q_latent_h, q_rope, q_rope_n, q_rope_t, q_rope_h,
                                   cache, page_table, seq_lens, n_pages, page_size, max_pages, Nb, Tq, H, Dc, Dr, scale,
                                   dtype, a))
        return st;
    if (kda_status st = check_step_outputs(fn, a, kda::mla_step_plan, workspace, workspace_bytes, o, lse)) return st;
    if (kda_status st = set_status(fn, a.status)) return st;
    return finish(fn, kda::launch_mla_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
