/*
 * kda_mla.h — latent attention in libkda.so (see kda.h for the library's
 * conventions, status codes and error messages, which hold here too).
 *
 * Latent attention is the softmax attention of the layers that stand between
 * the KDA layers of the K3 backbone (24 of its 93: hysenlabs "kimi-k3-mlx",
 * section "Attention is 93 layers split between KDA and a NoPE gated MLA";
 * 96 heads, key-value latent 512). A token's keys and values all come from
 * one latent c of Dc channels; a key may have Dr more channels r that the
 * heads share. For query row i and key row j of one sequence
 *     s_ij = scale * (q_i[0:Dn] . k_j + q_i[Dn:Dn+Dr] . r_j)
 *     o_i  = sum_j softmax_j(s_ij) v_j,      lse_i = log sum_j exp(s_ij)
 * over the keys that i sees. Expanded form (kda_mla_fwd, kda_mla_bwd): k and v
 * are per head, up-projected from c by the caller; for prompts and training.
 * Absorbed form (kda_mla_step): the caller multiplies the up-projection of the
 * keys into the query and the output, and the queries meet the cached latents
 * themselves; for generated tokens. The projections are outside the library.
 *
 * A row that sees no key has o = 0 and lse = -inf. Forward: a NaN or an infinity
 * in a row of k or r reaches only rows that see it; in a row of v, and in the
 * latent part of a cache row, which is both, it may reach every row of its
 * sequence (a hidden key's weight is an exact 0, and 0 * NaN is NaN). Backward:
 * it may reach every gradient of its sequence. Other sequences are not
 * touched. Cache rows past a sequence's length are never read.
 *
 * dtype: KDA_BF16 runs on the bf16 matrix cores, scores, softmax statistics
 * and sums in float32, probabilities and score gradients rounded to bf16 once
 * as operands of the second product (relative to the norm of the result, an
 * error of about 0.0017 each, next to the 0.0017 of the result's own rounding).
 * The rounding of o stays out of the backward, but for dq of rows (in blocks of
 * 128 of which one sees over 128 keys) with nearly all their weight on one key:
 * up to 0.006 of the norm.
 * KDA_F32 runs on the float32 matrix cores.
 *
 * Preconditions that are not checked: finite inputs; cu_seqlens starting at 0
 * and non-decreasing. Offsets are clipped to the tensor, so that a wrong one
 * gives wrong results but no access outside it. They may end before T: rows
 * behind the last sequence are then not read, and are left as they were or,
 * with zero_rest, written as zeros (lse as -inf).
 */
#ifndef KDA_MLA_H
#define KDA_MLA_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Expanded forward.
 *
 *   q       [B,Tq,H,Dn+Dr] dtype: each head's own part, then the part that meets r
 *   kv      [B,Tk,H,2*Dn]  dtype: each head's key, then its value (Dv = Dn)
 *   k_rope  [B,Tk,Dr]      dtype, the key part shared by the heads: rows
 *           k_rope_row elements apart, batches k_rope_batch, channels
 *           contiguous (a slice of a projection's output will do); NULL if
 *           and only if Dr = 0. Both strides multiples of 16 bytes.
 *   cu_seqlens_q, cu_seqlens_k  [N+1] int32 offsets of N packed sequences in
 *           q and in kv (B must be 1), both or neither; NULL: N must equal B
 *           and row b is sequence b. Zero-length sequences are allowed.
 *   causal  0: every row sees all keys of its sequence. 1: the last query is
 *           aligned with the last key: of Lq queries and Lk keys, row i sees
 *           the keys j <= i + Lk - Lq (Lk > Lq: the queries continue a prefix;
 *           Lk < Lq: the first rows see nothing).
 *   scale   finite and > 0
 *   zero_rest  see above (packed calls only; ignored otherwise)
 *   o       [B,Tq,H,Dn] dtype;  lse [B,H,Tq] float32, or NULL
 * Neither may alias an input. Every tensor pointer is 16-byte aligned.
 * Supported: Dn in {64, 128}, Dr in {0, 64}, KDA_BF16 and KDA_F32, H <= 4096,
 * k_rope_row <= 2^22. A launch holds 2^24 - 1 workgroups: more tiles of 128
 * query rows of a sequence times H are refused (packed: Tq / 128 + N + 1 tiles);
 * in the backward, of key rows too, and, with Dr > 0, B * Tk past 2^28 - 16.
 * Tq = 0 is a no-op; with Tk = 0, kv and k_rope may be NULL.
 */
kda_status kda_mla_fwd(const void* q, const void* kv, const void* k_rope, int64_t k_rope_row, int64_t k_rope_batch,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t B, int32_t Tq, int32_t Tk,
                       int32_t H, int32_t Dn, int32_t Dr, int32_t N, int32_t causal, float scale, kda_dtype dtype,
                       int32_t zero_rest, void* o, float* lse, void* stream);

/*
 * Backward of kda_mla_fwd: the gradients of sum(d_o * o).
 *
 *   q, kv, k_rope, cu_seqlens, sizes, causal, scale, dtype  as in the forward
 *   o, lse     what the forward returned;  d_o [B,Tq,H,Dn] dtype
 *   workspace  at least kda_mla_bwd_workspace_bytes(...) bytes of device
 *              memory, 16-byte aligned; contents on entry do not matter. Mostly
 *              the heads' shares of dk_rope, 4 * B * H * Tk * Dr bytes (96 heads:
 *              24 KB a key); small calls up to four times that and as many
 *              float32 gradients, for any dtype
 *   dq [B,Tq,H,Dn+Dr], dkv [B,Tk,H,2*Dn], dk_rope [B,Tk,Dr] (contiguous; NULL
 *              if and only if Dr = 0) dtype. Sums are float32, rounded to
 *              dtype at the end; the sum of dk_rope over the heads is float32
 *              too. The same inputs give the same bits (no atomic sums).
 * Every row of every sequence is written (zeros where it takes no part).
 */
size_t kda_mla_bwd_workspace_bytes(int32_t B, int32_t Tq, int32_t Tk, int32_t H, int32_t Dr);
kda_status kda_mla_bwd(const void* q, const void* kv, const void* k_rope, int64_t k_rope_row, int64_t k_rope_batch,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, const void* o, const float* lse,
                       const void* d_o, int32_t B, int32_t Tq, int32_t Tk, int32_t H, int32_t Dn, int32_t Dr,
                       int32_t N, int32_t causal, float scale, kda_dtype dtype, int32_t zero_rest, void* workspace,
                       size_t workspace_bytes, void* dq, void* dkv, void* dk_rope, void* stream);

/*
 * The cache: n_pages pages of page_size rows of Dc + Dr elements (latent, then
 * shared key part), [n_pages,page_size,Dc+Dr] dtype, 16-byte aligned. Row p of
 * sequence n lies in page page_table[n][p / page_size] at p % page_size;
 * page_table is [Nb,max_pages] int32, entries past a sequence's length are not
 * read. page_size is a power of two, 16 to 2^24; max_pages * page_size is at
 * most 2^30. Pages may be shared by sequences (a common prefix) as long as
 * nobody writes to them.
 *
 * A page_table entry outside [0, n_pages) for a row within the length, or a
 * length past max_pages * page_size, is a fault of the caller that only the
 * device can see: such rows are skipped (not read, hidden from the softmax;
 * not written), and the next kda_device_check returns KDA_ERR_DEVICE.
 *
 * kda_mla_cache_append writes new tokens behind the cached ones.
 *   latent [B,T,Dc], k_rope [B,T,Dr] (NULL if and only if Dr = 0) dtype, rows
 *          and batches *_row and *_batch elements apart, channels contiguous,
 *          strides multiples of 16 bytes
 *   cache_lens [N] int32: each sequence's length before the call (not
 *          changed); negative: a padding row, nothing is written for it
 *   cu_seqlens [N+1]: packed new tokens (B = 1), tokens behind the last
 *          sequence are not written; or NULL: N = B, T new tokens each
 * Two tokens of one call must not land in the same cache row (sequences that
 * share the page they grow into): which one stays is then not defined.
 * B * T = 0 is a no-op. Dc in {256, 512}, Dr in {0, 64}. B * T tokens of over
 * 2^32 - 256 16-byte chunks together are refused.
 */
kda_status kda_mla_cache_append(const void* latent, int64_t latent_row, int64_t latent_batch, const void* k_rope,
                                int64_t k_rope_row, int64_t k_rope_batch, void* cache, const int32_t* page_table,
                                const int32_t* cache_lens, const int32_t* cu_seqlens, int32_t n_pages,
                                int32_t page_size, int32_t max_pages, int32_t B, int32_t T, int32_t Dc, int32_t Dr,
                                int32_t N, kda_dtype dtype, void* stream);

/*
 * Absorbed attention of Tq new tokens per sequence over the cache, which holds
 * them already (kda_mla_cache_append first): of seq_lens[n] rows, token t sees
 * the first seq_lens[n] - Tq + t + 1. seq_lens[n] <= 0 is a padding row.
 *
 *   q_latent [Nb,Tq,H,Dc], q_rope [Nb,Tq,H,Dr] (NULL if and only if Dr = 0)
 *            dtype, each with its own strides over sequences (_n), tokens (_t)
 *            and heads (_h) in elements, multiples of 16 bytes, channels
 *            contiguous (a head-major product's output, or a slice)
 *   workspace  at least kda_mla_step_workspace_bytes(...) bytes, 16-byte
 *            aligned; calls that may run at the same time need their own. It
 *            grows with Tq * H past 1024 rows (64 float32 results a row: 13 GB at
 *            1024 tokens of 96 heads, Dc = 512): this call is for few new tokens,
 *            the expanded form for many
 *   o        [Nb,Tq,H,Dc] dtype, in latent space;  lse [Nb,Tq,H] float32 or NULL
 * scale finite and > 0 (the expanded head's, 1 / sqrt(Dn + Dr), not Dc's).
 * Nb * Tq = 0 is a no-op. Dc in {256, 512}, Dr in {0, 64}. At most: Tq * H
 * 2^20, Nb * Tq * H 2^30, Nb 2^24 - 1.
 */
size_t kda_mla_step_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size,
                                    int32_t max_pages, kda_dtype dtype);
kda_status kda_mla_step(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                        const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                        const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                        int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                        kda_dtype dtype, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_MLA_H */
