/*
 * kda_mla_cache.h — a smaller cache for the latent attention of kda_mla.h:
 * latents held in 4 bits, the attention weight that cached rows have gathered,
 * and the eviction of those that gathered least (see kda.h for the library's
 * conventions, status codes and error messages, which hold here too, and
 * kda_mla.h for the paged cache, its page table, and what is not checked).
 *
 * The 4-bit cache (OCP microscaling format MXFP4). 32 consecutive channels of
 * a latent share a scale 2^e; each is held as a 4-bit code of a multiple of it:
 * codes 0 to 7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6, bit 3 is the sign. The
 * scale is a byte e + 127. e is the smallest with max|c| <= 7 * 2^e, at most 125,
 * so that no rounding is off by more than 2^e, or in blocks of more than 7 * 2^125
 * by 2 * 2^e; values are rounded to the nearest multiple, ties to the even code,
 * past 6 to 6. A block whose largest magnitude is below 2^-100 is held as zeros
 * (codes and scale byte 0); a block with a NaN or an infinity as NaN (scale byte
 * 255). The key part r that the heads share keeps its dtype: its scores are the
 * sensitive ones, and it is a ninth of a row's channels.
 * A page of page_size rows is, in this order,
 *     page_size * Dc / 2   bytes of codes (channel 2 i in the low half of byte i)
 *     page_size * Dc / 32  scale bytes
 *     page_size * Dr       elements of dtype
 * each of them row by row: kda_mla_mx_row_bytes(Dc, Dr, dtype) bytes a row (400
 * for Dc = 512, Dr = 64, KDA_BF16, where a row of kda_mla.h's cache has 1152).
 * What it gives is room: with many heads, where products bound the attention, a
 * step over one sequence takes as long as over kda_mla.h's cache or a little
 * longer; batches, and few heads, gain time too.
 * The cache is 16-byte aligned. Dc in {256, 512}, Dr in {0, 64}, page_size a
 * power of two from 16 to 2^24, max_pages * page_size at most 2^30.
 */
#ifndef KDA_MLA_CACHE_H
#define KDA_MLA_CACHE_H

#include "kda_mla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a row of the 4-bit cache; 0 for sizes that are not supported. */
size_t kda_mla_mx_row_bytes(int32_t Dc, int32_t Dr, kda_dtype dtype);

/*
 * kda_mla_cache_append for the 4-bit cache: rounds new rows as above and writes
 * them behind the cached ones. Arguments and errors as there; latent and k_rope
 * are dtype.
 */
kda_status kda_mla_cache_append_mx(const void* latent, int64_t latent_row, int64_t latent_batch, const void* k_rope,
                                   int64_t k_rope_row, int64_t k_rope_batch, void* cache, const int32_t* page_table,
                                   const int32_t* cache_lens, const int32_t* cu_seqlens, int32_t n_pages,
                                   int32_t page_size, int32_t max_pages, int32_t B, int32_t T, int32_t Dc, int32_t Dr,
                                   int32_t N, kda_dtype dtype, void* stream);

/*
 * Reads rows of the 4-bit cache back, packed: of sequence n the rows
 * starts[n] .. starts[n] + cu_seqlens[n+1] - cu_seqlens[n] - 1, to rows
 * cu_seqlens[n] .. of the outputs (a cached prefix that the expanded form is to
 * attend to, say).
 *   starts      [N] int32, or NULL: from row 0
 *   cu_seqlens  [N+1] int32 offsets into the outputs, clipped to [0, T]
 *   latent [T,Dc], k_rope [T,Dr] (NULL if and only if Dr = 0)  dtype, contiguous,
 *               16-byte aligned: exact for latents (a 4-bit value times a power of
 *               two is a bf16 number)
 *   zero_rest   as in kda_mla.h, for rows behind the last sequence
 * Rows past the page table, before row 0 or in pages that do not exist are
 * written as zeros and reported by kda_device_check. T = 0 is a no-op;
 * T * (Dc / 8 + 16) past 2^32 - 256 is refused.
 */
kda_status kda_mla_cache_read_mx(const void* cache, const int32_t* page_table, const int32_t* starts,
                                 const int32_t* cu_seqlens, int32_t n_pages, int32_t page_size, int32_t max_pages,
                                 int32_t T, int32_t Dc, int32_t Dr, int32_t N, kda_dtype dtype, int32_t zero_rest,
                                 void* latent, void* k_rope, void* stream);

/*
 * kda_mla_step over the 4-bit cache. Arguments, rules and errors as there.
 * The scores of KDA_BF16 run on the scaled matrix instructions with the 4-bit
 * codes as they stand; a query of bf16 is two 8-bit floats (e4m3) there, whose
 * sum is the query itself except for channels below 2^-13 of the largest of
 * their 32, which are off by at most 2^-21 of that; where the largest is below
 * 2^-111, any of them by at most 2^-132. Of the outputs, the product of a
 * weight (before the division by their sum) and a block's 2^e below 2^-126 may
 * count as 0: 6 * 2^-126 a row at most. KDA_F32 runs on the float32 matrix
 * cores. A NaN block reaches the sequences that hold it and no others.
 */
size_t kda_mla_step_mx_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t page_size,
                                       int32_t max_pages, kda_dtype dtype);
kda_status kda_mla_step_mx(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                           const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                           const int32_t* page_table, const int32_t* seq_lens, int32_t n_pages, int32_t page_size,
                           int32_t max_pages, int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale,
                           kda_dtype dtype, void* workspace, size_t workspace_bytes, void* o, float* lse, void* stream);

/*
 * The attention weight that cached rows gather: for row j of sequence n
 *     weights_out[n][j] = decay * weights[n][j] + sum_{t,h} exp(s_thj - lse[n][t][h])
 * over the tokens t that see row j, s as in kda_mla_step of the same arguments
 * and lse its result. (With the weights of one decode step or of a prompt's last
 * tokens, rows that attention has no use for stay low.)
 *
 *   q_latent, q_rope, cache, page_table, seq_lens, sizes, scale, dtype
 *              as in kda_mla_step; form 0: cache as in kda_mla.h, 1: 4-bit, whose
 *              scores are those of kda_mla_step_mx
 *   lse        [Nb,Tq,H] float32
 *   weights, weights_out  [Nb, max_pages * page_size] float32, the same memory
 *              (in place) or apart. Rows from seq_lens[n] on are neither read nor
 *              written.
 *   fresh      the last `fresh` rows of each sequence have no weight yet: theirs
 *              is not read and counts as 0. (Tq after a decode step; a prompt's
 *              rows, or more, after a prefill.) >= 0
 *   decay      in [0, 1]; 1 sums all steps, less forgets, 0 starts anew (and reads
 *              no weight)
 *   workspace  at least kda_mla_weigh_workspace_bytes(...) bytes, 16-byte aligned;
 *              calls that may run at the same time need their own. NULL where that
 *              is 0: it is not for KDA_BF16 over the 4-bit cache with Tq * H > 128
 *              (18 KB for 16 of these rows, Dc = 512, Dr = 64)
 * Sums are float32, in an order that the sizes decide: the same inputs give the
 * same bits. Rows in missing pages get no new weight and are reported as in
 * kda_mla_step. Limits as in kda_mla_step. Nb * Tq = 0 is a no-op: nothing is
 * written.
 */
size_t kda_mla_weigh_workspace_bytes(int32_t Nb, int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, kda_dtype dtype,
                                     int32_t form);
kda_status kda_mla_weigh(const void* q_latent, int64_t q_latent_n, int64_t q_latent_t, int64_t q_latent_h,
                         const void* q_rope, int64_t q_rope_n, int64_t q_rope_t, int64_t q_rope_h, const void* cache,
                         const int32_t* page_table, const int32_t* seq_lens, const float* lse, const float* weights,
                         int32_t fresh, float decay, int32_t n_pages, int32_t page_size, int32_t max_pages, int32_t Nb,
                         int32_t Tq, int32_t H, int32_t Dc, int32_t Dr, float scale, kda_dtype dtype, int32_t form,
                         void* workspace, size_t workspace_bytes, float* weights_out, void* stream);

/*
 * Evicts rows by whole pages. With ps = page_size, of a sequence of L rows
 *     a = ceil(first / ps)  pages at the front and those from
 *     b = floor(max(L - recent, 0) / ps)  on (the last `recent` rows) stay;
 *     E = min(floor((L - keep) / ps), b - a) pages go (none if E <= 0):
 * of the rows of pages a .. b-1, the E * ps of least weight are dropped (of
 * equal ones the later first; NaN counts as the largest). What stays of the last
 * E of these pages moves, in order, into the rows dropped from the others, in
 * order; the pages behind close up, and the E emptied pages come behind them in
 * the page table, where appended rows will use them (or the caller takes them). So the
 * sequence has L - E * ps rows, and only rows that must move do. Attention over a
 * cache does not depend on the order of its rows; the order of the rows from b on,
 * by which later calls know the recent ones, is kept.
 *
 *   cache       written in place; pages a .. b-1 must not be shared by sequences
 *   page_table, page_table_out  [Nb,max_pages] int32
 *   seq_lens, seq_lens_out      [Nb] int32; <= 0: padding row
 *   weights, weights_out        [Nb, max_pages * page_size] float32: weights of
 *               moved rows move with them; rows from the new length to the old
 *               become 0
 *               Each pair the same memory (in place) or apart; what does not
 *               change is copied then.
 *   keep, first, recent  >= 0
 *   form, Dc, Dr, dtype  the cache's rows, as above
 *   workspace   at least kda_mla_evict_workspace_bytes(...) bytes, 16-byte aligned;
 *               calls that may run at the same time need their own
 * A sequence longer than its page table, or with a page among a .. b-1 that does
 * not exist, stays as it is and is reported by kda_device_check. Nb = 0 is a
 * no-op. Nb below 2^22; with page tables of R > 16384 rows,
 * Nb * min(ceil(R / 2048), 1024) too.
 */
size_t kda_mla_evict_workspace_bytes(int32_t Nb, int32_t page_size, int32_t max_pages);
kda_status kda_mla_evict(void* cache, const int32_t* page_table, const int32_t* seq_lens, const float* weights,
                         int32_t keep, int32_t first, int32_t recent, int32_t n_pages, int32_t page_size,
                         int32_t max_pages, int32_t Nb, int32_t Dc, int32_t Dr, kda_dtype dtype, int32_t form,
                         void* workspace, size_t workspace_bytes, int32_t* page_table_out, int32_t* seq_lens_out,
                         float* weights_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_MLA_CACHE_H */
