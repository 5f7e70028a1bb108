/*
 * flexq_serve.h -- C ABI of the operators a decoding step runs around the quantized
 * linear layers of flexq.h (same library, same conventions: device pointers owned by
 * the caller, a hipStream_t passed as void*, every argument checked on the host before
 * anything is enqueued, flexq_status returned):
 *
 *   flexq_pack_w4, flexq_gemv_w4     products of a few activation rows with 4-bit
 *                                    group-scaled weights (a drafting model's layers)
 *   flexq_block_tables               block tables and slot maps of a paged cache from
 *                                    request lengths
 *   flexq_kv_cache_write             new keys and values into the paged cache
 *   flexq_tree_attention             attention of drafted tokens over the paged cache
 *   flexq_kv4_cache_write, flexq_kv4_cache_read, flexq_kv4_attention
 *                                    the same over a paged cache of 4-bit codes, with an
 *                                    optional sliding window whose first tokens stay visible
 *   flexq_lora_add                   low-rank adapters of many requests at once, added to a
 *                                    shared projection's output
 *
 * Element type: `dtype` says whether 16-bit tensors hold IEEE half (FLEXQ_FP16) or
 * bfloat16 (FLEXQ_BF16).  Lengths, tables and slot maps are int32.  A step's lengths
 * live on the GPU: the calls take only upper bounds from the host, so one captured
 * HIP graph serves steps of different lengths.
 *
 * 4-bit weights (w4), 0.5 byte per code, laid out in the order the MFMA fragments
 * take them: 16-row tiles, then 128-deep k-blocks; in a tile and k-block 64 lanes of
 * four dwords.  Dword j of lane l holds the codes of row l % 16 at
 * k = 32 j + 8 (l / 16) + c, c = 0 .. 7, code c as q + 8 (q in [-7, 7]; -8 decodes but
 * is never produced) at bits 4 (c / 2) + 16 (c % 2).  The dword of row n, column k is
 *   ((n / 16) * (K / 128) + k / 128) * 256 + ((k % 32) / 8 * 16 + n % 16) * 4
 *     + (k % 128) / 32.
 * s_w is fp16 [K/group][N], group-major.
 *
 * Paged cache: num_pages pages of page_size tokens (16, 32, 64, 128 or 256), a page's
 * tokens in blocks of 16; element d of key head h of the token at slot
 * s = page * page_size + r lives at
 *   keys    ((page * Hkv + h) * (page_size / 16) + r / 16) * 16 D
 *             + (d / 32) * 512 + (r % 16) * 32 + d % 32
 *   values  the same block offset + d * 16 + r % 16
 * (keys in 32-wide slices of D, values with the token innermost: each is the order an
 * MFMA fragment takes, so the attention stages whole cache lines in LDS as they are).
 * As torch tensors: keys [pages][Hkv][page_size/16][D/32][16][32], values
 * [pages][Hkv][page_size/16][D][16].  D is 64, 96, 128 or 256.
 * block_table[b][i] is the page of request b's tokens i * page_size ...
 *
 * 4-bit cache: pages, slots and tables as above, (D + 8) bytes a token and head instead of
 * 4 D.  A row x[0 .. D) of a token and head is held as x = b + s c:
 *   b = fp16(min x);  s = fp16((max x - min x) / 15);
 *   c = clamp(rint((x - b) / s), 0, 15), 0 where s = 0
 *   (IEEE binary32 before the roundings to fp16, which are to nearest, ties to even, as rint)
 * for fp16 and bfloat16 rows alike.  A row with a NaN, or whose b or s is not finite, has NaN for
 * both and so reads as NaN.  Of the token at slot page * page_size + r, with block =
 * (page * Hkv + h) * (page_size / 16) + r / 16,
 *   keys    code of d at dword block * 2 D + (r % 16) * (D / 8) + d / 8,
 *           bits 4 (d % 8 / 2) + 16 (d % 2) ..
 *   values  code of d in dword block * 2 D + (r % 16 / 8) * D + d / 2 * 2 + r % 8 / 4,
 *           byte 0, 2, 1, 3 for r % 4 = 0 .. 3, bits 4 (d % 2) .. of it
 *   scales  fp16 at block * 64 + r % 16: s of the key, + 16 its b, + 32 s of the value, + 48 its b
 * (keys in the order a score's MFMA takes, values with tokens in bytes that can be written alone).
 * As torch tensors: k_codes int32 [pages][Hkv][page_size/16][16][D/8], v_codes int32
 * [pages][Hkv][page_size/16][2][D/2][2], scales fp16 [pages][Hkv][page_size/16][4][16].
 */
#ifndef FLEXQ_SERVE_H
#define FLEXQ_SERVE_H

#include "flexq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FLEXQ_FP16 = 0, FLEXQ_BF16 = 1 } flexq_dtype;

/* Bytes of w4 for an N x K weight: N * K / 2.  Returns 0 for N <= 0, K <= 0 or K not a
   multiple of 128. */
size_t flexq_packed_w4_bytes(int64_t N, int64_t K);

/* 4-bit weight group quantization and packing: per row n and group of `group_size`
   consecutive k,
     amax = max |w|;  s16 = fp16(amax / 7);  q = clamp(rint(w / float(s16)), -7, 7),
     q = 0 where s16 = 0  (IEEE binary32 division, round half to even)
     w     [N][K] of dtype, 16-byte aligned               (input)
     w4    flexq_packed_w4_bytes(N, K), 16-byte aligned    (output)
     s_w   [K/group_size][N] fp16 bits, 2-byte aligned      (output)
   group_size is 32, 64 or 128.  N == 0 is a no-op.  Errors: INVALID_VALUE (null,
   N < 0, K <= 0, dtype, overlap), UNSUPPORTED (group_size, K % 128, N % 16,
   N > 2^24, K > 2^22, N * K / group_size >= 2^29, alignment). */
flexq_status flexq_pack_w4(const uint16_t* w, int32_t dtype, int64_t N, int64_t K,
                           int32_t group_size, uint32_t* w4, uint16_t* s_w_fp16, void* stream);

/* Y[m][n] = sum_g s_w[g][n] * sum_{k in g} x[m][k] * q[n][k]: products and sums in fp32
   (a product of a 16-bit activation and a 4-bit code is exact in it), rounded once to
   dtype.  For few rows: weights are streamed once per 64 rows.
     x     [M][K] of dtype, rows x_stride elements apart, 16-byte aligned rows
     w4, s_w_fp16 as flexq_pack_w4 writes them; s_w_fp16 8-byte aligned
     y     [M][N] of dtype, 8-byte aligned (output)
     workspace  flexq_gemv_w4_workspace_bytes(M, N, K) bytes, 16-byte aligned (NULL where
           that is 0), overwritten; not to be used by other work until this call's kernels
           have run
   The result does not depend on the order in which workgroups run.  M == 0 or N == 0 is
   a no-op.  Errors: INVALID_VALUE (null, negative size, dtype, x_stride < K with M > 1,
   workspace too small, overlap), UNSUPPORTED (as flexq_pack_w4, x_stride % 8,
   x_stride > 2^24, M > 1,048,560, alignment). */
flexq_status flexq_gemv_w4(const uint16_t* x, int32_t dtype, int64_t x_stride,
                           const uint32_t* w4, const uint16_t* s_w_fp16, int64_t M, int64_t N,
                           int64_t K, int32_t group_size, void* workspace,
                           size_t workspace_bytes, uint16_t* y, void* stream);

/* Bytes of workspace flexq_gemv_w4 needs on the current device: 0 up to 4 rows of moderate
   length and for weights of many rows, else fp32 sums of slices of K.  0 for a size that it
   refuses or that makes it a no-op. */
size_t flexq_gemv_w4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* Block tables and slot maps of a step.  Request b holds ctx_lens[b] tokens in the
   pages block_table[b][0 .. have_b - 1], have_b = ceil(ctx_lens[b] / page_size), and
   gets new_lens[b] more.  With add_b = ceil((ctx_lens[b] + new_lens[b]) / page_size) -
   have_b and off_b the sum of add over the requests before b, head = *free_head
   (0 where free_head is NULL):
     block_table[b][have_b + j] = free_pages[head + off_b + j],  0 <= j < add_b
     cu_new[b] = sum of new_lens before b;  cu_new[B] = their total
     slot_map[cu_new[b] + i] = block_table[b][p / page_size] * page_size + p % page_size,
                               p = ctx_lens[b] + i,  0 <= i < new_lens[b]
     slot_map[t] = -1 for cu_new[B] <= t < max_tokens
     counts = {cu_new[B], sum of add, head + sum of add}  (the last: the next step's head)
   Where the free list or a table row ends too soon, the table gets -1 (or nothing past
   its row) and such tokens the slot -1, as tokens do whose slot int32 does not hold; tokens
   past max_tokens get no slot.  The caller
   sees it in counts.  A negative length counts as 0.  Other table entries are kept.
     ctx_lens, new_lens int32[B]       free_pages int32[num_free]     free_head int32[1]
     block_table int32[B][max_blocks]  (in, out)
     slot_map int32[max_tokens], cu_new int32[B + 1], counts int32[3]  (out)
   All 4-byte aligned.  page_size is a power of two from 1 to 65536.  B == 0 still
   writes slot_map, cu_new and counts.  The sums must stay below 2^31 (no access is out
   of range if they do not).  Errors: INVALID_VALUE (null, negative size, page_size not
   positive, an output overlapping another argument), UNSUPPORTED (page_size not such a
   power, B > 4096, max_blocks or max_tokens or num_free above 2^30, alignment). */
flexq_status flexq_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t B,
                                const int32_t* free_pages, int64_t num_free,
                                const int32_t* free_head, int32_t page_size,
                                int32_t* block_table, int64_t max_blocks, int64_t max_tokens,
                                int32_t* slot_map, int32_t* cu_new, int32_t* counts,
                                void* stream);

/* Keys and values of T tokens into the paged cache: token t's go to slot slot_map[t];
   a slot outside [0, num_pages * page_size) (such as -1) drops the token.  Two tokens
   with one slot leave either's value.  A copy of 16-bit elements of either dtype.
     k, v      element (t, h, d) at t * stride_t + h * stride_h + d (strides in
               elements, the tensors' own; that of an axis of length one plays no
               part), 16-byte aligned rows
     slot_map  int32[T]      k_cache, v_cache  the layouts above, 16-byte aligned
   T == 0 is a no-op.  Errors: INVALID_VALUE (null, negative size, negative stride, a
   cache overlapping another argument), UNSUPPORTED (D, page_size, strides % 8, Hkv >
   65535, T * Hkv * D >= 2^34, num_pages * Hkv * page_size / 16 >= 2^31, alignment). */
flexq_status flexq_kv_cache_write(const uint16_t* k, int64_t k_stride_t, int64_t k_stride_h,
                                  const uint16_t* v, int64_t v_stride_t, int64_t v_stride_h,
                                  const int32_t* slot_map, int64_t T, int64_t Hkv, int64_t D,
                                  int64_t num_pages, int32_t page_size, uint16_t* k_cache,
                                  uint16_t* v_cache, void* stream);

/* Attention of drafted tokens over the paged cache.  The drafted tokens of request b
   are the rows cu_new[b] .. cu_new[b + 1] - 1 of q, and their keys and values are
   already in the cache behind the request's ctx_lens[b] others.  Token t (in its request)
   attends every one of the ctx_lens[b] tokens, and drafted token j where bit j % 32 of
   tree_mask[cu_new[b] + t][j / 32] is set; without a tree_mask, where j <= t (a chain; one
   token alone is ordinary decoding).  For head h with key head h / (H / Hkv):
     s_j = scale * (q . k_j);  out = sum_j softmax(s)_j v_j;  lse = ln sum_j exp(s_j)
   over the attended j; a row that attends nothing gives out = 0, lse = -inf.  Scores,
   statistics and sums are fp32; the probabilities enter the product with the values as
   the sum of two 16-bit parts, within 2^-17 of themselves or, for fp16, 2^-34 of the row's
   largest, whichever is more; out is rounded once.
   What masked places, unused slots and pages hold does not matter, NaN and infinities
   included; an infinite value of an attended key gives an infinity of its sign.  Tokens on
   a page outside [0, num_pages) are left out.
     q          element (t, h, d) at t * q_stride_t + h * q_stride_h + d, t < T (the
                stride of an axis of length one plays no part)
     tree_mask  int32[T][mask_words] or NULL; bits past mask_words are 0
     out        [T][H][D] of dtype, 16-byte aligned     lse  fp32[T][H] or NULL
     max_new    no request has more drafted tokens (further ones are not computed); the
                work and the workspace are laid out for that many rows a request
     workspace  flexq_tree_attention_workspace_bytes(B, max_new, H, Hkv, D) bytes, 16-byte
                aligned, overwritten; not to be used by other work until this call's
                kernels have run
   Rows of out and lse past cu_new[B] are not written.  The result does not depend on
   the order in which workgroups run.  B == 0, T == 0 or max_new == 0 is a no-op.
   Errors: INVALID_VALUE (null, negative size or stride, no page, dtype, H % Hkv, scale
   not finite, max_new > 32 * mask_words with a tree_mask, workspace too small, an output or
   the workspace overlapping another argument), UNSUPPORTED (D, page_size, q strides %
   8, H > 4096, B > 4096, T > 2^24, max_new > 65536, max_blocks * page_size > 2^24,
   num_pages * Hkv * page_size / 16 >= 2^31, alignment). */
flexq_status flexq_tree_attention(const uint16_t* q, int32_t dtype, int64_t q_stride_t,
                                  int64_t q_stride_h, const uint16_t* k_cache,
                                  const uint16_t* v_cache, int64_t num_pages, int32_t page_size,
                                  const int32_t* block_table, int64_t max_blocks,
                                  const int32_t* ctx_lens, const int32_t* cu_new, int64_t B,
                                  int64_t T, int64_t max_new, int64_t H, int64_t Hkv, int64_t D,
                                  const int32_t* tree_mask, int64_t mask_words, float scale,
                                  void* workspace, size_t workspace_bytes, uint16_t* out,
                                  float* lse, void* stream);

/* Bytes of workspace flexq_tree_attention needs on the current device.  0 for a size
   that it refuses or that makes it a no-op. */
size_t flexq_tree_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                            int64_t D);

/* Keys and values of T tokens into the 4-bit cache: token t's go to slot slot_map[t]; a
   slot outside [0, num_pages * page_size) (such as -1) drops the token.  No other token's place
   is written, also where two calls write neighbouring slots at once.  The slots of a call
   should differ: of two tokens with one slot that slot holds a mixture afterwards.
     k, v      of dtype, as in flexq_kv_cache_write       slot_map  int32[T]
     k_codes, v_codes, scales  the layouts above, 16-byte aligned (output)
   T == 0 is a no-op.  Errors: as flexq_kv_cache_write, and INVALID_VALUE for dtype. */
flexq_status flexq_kv4_cache_write(const uint16_t* k, int64_t k_stride_t, int64_t k_stride_h,
                                   const uint16_t* v, int64_t v_stride_t, int64_t v_stride_h,
                                   int32_t dtype, const int32_t* slot_map, int64_t T, int64_t Hkv,
                                   int64_t D, int64_t num_pages, int32_t page_size,
                                   uint32_t* k_codes, uint32_t* v_codes, uint16_t* scales,
                                   void* stream);

/* The tokens at slots slot_map[0 .. T) of the 4-bit cache as rows of dtype, b + s c rounded
   once: what attention over the cache sees of them.  A slot outside the cache reads as 0.  (The
   last code of a row that reaches fp16's largest value may stand for more, infinite in fp16.)
     k, v      [T][Hkv][D] of dtype, 16-byte aligned (output)
   T == 0 is a no-op.  Errors: INVALID_VALUE (null, negative size, dtype, overlap), UNSUPPORTED
   (D, page_size, sizes as flexq_kv_cache_write, alignment). */
flexq_status flexq_kv4_cache_read(const uint32_t* k_codes, const uint32_t* v_codes,
                                  const uint16_t* scales, const int32_t* slot_map, int64_t T,
                                  int64_t Hkv, int64_t D, int64_t num_pages, int32_t page_size,
                                  int32_t dtype, uint16_t* k, uint16_t* v, void* stream);

/* Attention of drafted tokens over the 4-bit cache: flexq_tree_attention's with the keys and
   values that the codes stand for, b + s c.
   window  0, or how many positions a token sees, itself among them: of the context token t (in
           its request) attends the keys from ctx_lens[b] + n_t - window on, n_t the
           request's drafted tokens that it attends (t + 1 in a chain), and of a chain's
           drafted tokens those from there on too; a tree's bits hold whatever the window.
   sinks   with a window, the first `sinks` tokens of the request stay visible; without one it
           plays no part.
   Keys before every window of the request's tokens (behind the sinks) are not read.  Scores,
   statistics and sums are fp32; the queries enter whole down to 2^-24 of a row's largest, and
   below within 2^-34 of it; probabilities times the values' scales enter their product as two
   fp16 parts, within 2^-22 of themselves or 2^-35 of the row's largest, whichever is more (a scale
   of 0 counting as 2^-60); out is rounded once.  What masked places, unused slots and pages hold
   does not matter.  A row that attends a NaN key or value is NaN.
   All else (arguments, masks, rows that attend nothing, rows past cu_new[B], workspace, limits,
   errors) as flexq_tree_attention, with the workspace of the function below; INVALID_VALUE also
   for a negative window or negative sinks. */
flexq_status flexq_kv4_attention(const uint16_t* q, int32_t dtype, int64_t q_stride_t,
                                 int64_t q_stride_h, const uint32_t* k_codes,
                                 const uint32_t* v_codes, const uint16_t* scales,
                                 int64_t num_pages, int32_t page_size, const int32_t* block_table,
                                 int64_t max_blocks, const int32_t* ctx_lens,
                                 const int32_t* cu_new, int64_t B, int64_t T, int64_t max_new,
                                 int64_t H, int64_t Hkv, int64_t D, const int32_t* tree_mask,
                                 int64_t mask_words, int64_t window, int64_t sinks, float scale,
                                 void* workspace, size_t workspace_bytes, uint16_t* out,
                                 float* lse, void* stream);

/* Bytes of workspace flexq_kv4_attention needs on the current device.  0 for a size that it
   refuses or that makes it a no-op. */
size_t flexq_kv4_attention_workspace_bytes(int64_t B, int64_t max_new, int64_t H, int64_t Hkv,
                                           int64_t D);

/* Low-rank adapters beside a projection shared by many requests:
     out[t] = y[t] + scales[i] * B_i (A_i x[t]),  i = adapters[t]
   with the first ranks[i] rows of A_i and columns of B_i (ranks between 0 and R; what A and B
   hold past them does not matter).  A token whose adapter is outside [0, L) (such as -1) has
   out[t] = y[t].  Both products sum in fp32; A x enters the second one as two 16-bit parts, within
   2^-17 of itself (fp16: 2^-22, or 2^-39 of the token's largest, whichever is more); the sum
   with y is rounded once to dtype.
     x         [T][K], y and out [T][N] of dtype, rows their stride apart, 16-byte aligned rows;
               out may be y itself, with the same stride
     adapters  int32[T], in any order       ranks  int32[L] or NULL (all R)
     a         [L][R][K], b [L][N][R] of dtype, 16-byte aligned
     scales    fp32[L] or NULL (all 1)
     workspace  flexq_lora_add_workspace_bytes(T, N, K, R, L) bytes, 16-byte aligned (NULL
               where that is 0), overwritten; not to be used by other work until this call's
               kernels have run
   Adapters are read once per 64 consecutive tokens.  The result does not depend on the order
   in which workgroups run.  T == 0 or N == 0 is a no-op.  Errors: INVALID_VALUE (null, negative
   size, dtype, a stride less than a row with T > 1, workspace too small, an output or the
   workspace overlapping another argument), UNSUPPORTED (K % 128, N % 16, R % 8, R > 256, K > 2^22,
   N > 2^24, L > 2^20, T > 4,194,240, strides % 8, alignment). */
flexq_status flexq_lora_add(const uint16_t* x, int32_t dtype, int64_t x_stride, const uint16_t* y,
                            int64_t y_stride, const int32_t* adapters, const uint16_t* a,
                            const uint16_t* b, const int32_t* ranks, const float* scales,
                            int64_t T, int64_t N, int64_t K, int64_t R, int64_t L,
                            void* workspace, size_t workspace_bytes, uint16_t* out,
                            int64_t out_stride, void* stream);

/* Bytes of workspace flexq_lora_add needs on the current device: fp32 sums of slices of K.  0 for
   a size that it refuses or that makes it a no-op. */
size_t flexq_lora_add_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L);

#ifdef __cplusplus
}
#endif
#endif /* FLEXQ_SERVE_H */
