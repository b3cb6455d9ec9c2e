/*
 * qoq_attn.h -- C ABI of the attention operators of libqoq.so (sm_100a)
 *
 * What stands between the QKV projection and the output projection of a
 * transformer block, around the W4A8 layer of qoq.h:
 *   - rotary positions;
 *   - a paged key/value cache in 4 or 8 bits, quantised as it is written,
 *     and read back;
 *   - attention of new tokens (one per sequence, or chunks) over that cache;
 *   - causal attention of whole prompts, before anything is quantised.
 * The KV4 cache of qoq.h takes its scales per channel over all tokens of a
 * sequence, so it is filled once; this one takes them per token and head,
 * so it grows token by token.
 *
 * Sources, by page title: "QServe Guide: W4A8KV4 Quantization for LLM
 * Serving", The Architecture, subsection 3 (a 4-bit KV cache beside the
 * layer). The pages name neither paging nor rotary positions; the formulas
 * below are this library's definitions.
 *
 * Conventions (those of qoq.h, and):
 *   - FP16 activations as uint16_t bits. A matrix of heads is [T][H][d]:
 *     row t starts at x + t * ld (elements), head h at + h * d, so q, k and
 *     v may be column ranges of one projection output. ld >= H * d, a
 *     multiple of 8.
 *   - d is 64 or 128 (rotary alone: any multiple of 16 up to 512).
 *   - Query head h attends with KV head h / (Hq / Hkv); Hq is a multiple of
 *     Hkv, Hq / Hkv <= 64, Hq <= 1024.
 *   - 16-byte aligned pointers (index arrays: 4-byte). T <= 2^21 rows,
 *     B <= 65536, pages >= 1, table_pages * page_size <= 2^24.
 *   - Infinities and NaN in the rows are not hidden: a cached row with one
 *     stands for d NaN, and a row of q with one, or one that sees a key with
 *     a NaN or a value with either, gives outputs that are not finite (of a
 *     prompt's values: in their channel).
 *     Tokens that a row does not see (later new tokens of its own sequence
 *     apart) do not reach it, whatever they hold.
 *   - T, B == 0 are valid empty problems: QOQ_OK, nothing launched.
 *   - Index arrays are read on the device and checked there: an index that
 *     points outside its array skips the access, as said below.
 *   - Waits inside the kernels are bounded; one that runs out is reported by
 *     qoq_device_error, and the call's outputs are then unspecified.
 *
 * One description of a batch serves every call:
 *   cu      int32 [B + 1]  sequence b's new tokens are rows cu[b] ..
 *                          cu[b+1] - 1 (n_b rows, maybe none); rows outside
 *                          cu[0] .. cu[B] belong to no sequence, and no call
 *                          writes their outputs.
 *                          It does not decrease and stays within 0 .. T;
 *                          a sequence with rows beyond T is not attended.
 *   kv_len  int32 [B]      tokens of sequence b in the cache, its new ones
 *                          included: new token i has position
 *                          kv_len[b] - n_b + i.
 *   table   int32 [B][table_pages]  page number of the tokens p * page_size
 *                          .. of sequence b. A number outside 0 .. pages - 1
 *                          is an absent page (dropped or not allocated):
 *                          nothing is written to it, it reads as zeros, and
 *                          attention does not see its tokens. Positions
 *                          below 0 or from table_pages * page_size on are
 *                          absent too.
 */
#ifndef QOQ_ATTN_H
#define QOQ_ATTN_H

#include "qoq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rotary positions: for i < rot / 2, a = pos[t] * freq[i],
 *     y1 = amplitude * (x1 * cos a - x2 * sin a)
 *     y2 = amplitude * (x1 * sin a + x2 * cos a)
 * on channels (x1, x2) = (i, i + rot/2), or (2i, 2i + 1) when interleaved
 * is 1; channels from rot on are copied. The angle and the rotation are
 * computed in FP64 and rounded to FP16 once, so far positions lose nothing.
 *   pos     device int32 [T];  freq device float64 [rot/2], radians per
 *           position (scaled for long contexts by the caller).
 *   rot     a multiple of 16, 0 <= rot <= d.
 *   y       may be x itself with the same ld. */
QOQ_API int qattn_rotary(const uint16_t *x, int64_t ldx, const int32_t *pos, const double *freq, int T, int H,
                         int d, int rot, int interleaved, float amplitude, uint16_t *y, int64_t ldy,
                         void *stream);

/* The cache. Per (page, KV head, token) one row of d codes of `bits` bits
 * (4 or 8) for the key and one for the value, and FP16 (s, m) of each:
 *     k_codes, v_codes  uint8 [pages][Hkv][page_size][d * bits / 8];
 *                       4 bits: byte j holds channel 2j (low nibble) and
 *                       2j + 1 (high nibble)
 *     k_par, v_par      uint16 [pages][Hkv][page_size][2]
 * page_size is 16, 32, 64 or 128. A row x is kept as
 *     m = min x,  s = fp16_towards_zero((max x - min x) / (2^bits - 1)),
 *     c = min(round((x - m) / s), 2^bits - 1)   (0 when s is 0),
 * in FP32 with IEEE division, half to even; c stands for s * c + m. Rounding
 * s down keeps every value within the row's range, so none overflows.
 *
 * Appends the new tokens of a batch: rows of k and v [T][Hkv][d] go to
 * their positions' pages. With rot > 0 the keys are rotated by their
 * positions first (rounded to FP16 as by qattn_rotary, then quantised: the
 * same bits as the two calls), and when q is given, its rows are rotated
 * into q_out (which may be q itself with the same ld). The pages that
 * receive tokens must not repeat within a batch. */
QOQ_API int qattn_cache_append(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const uint16_t *q,
                               int64_t ldq, uint16_t *q_out, int64_t ldqo, int T, int Hq, int Hkv, int d,
                               const double *freq, int rot, int interleaved, float amplitude, int bits,
                               int page_size, int pages, uint8_t *k_codes, uint8_t *v_codes, uint16_t *k_par,
                               uint16_t *v_par, const int32_t *table, int table_pages, const int32_t *cu,
                               const int32_t *kv_len, int B, void *stream);

/* Reads the last n_b = cu[b+1] - cu[b] cached tokens of each sequence back:
 * K, V [T][Hkv][d] FP16, dense, fp16(s * c + m); zeros for absent pages. */
QOQ_API int qattn_cache_read(const uint8_t *k_codes, const uint8_t *v_codes, const uint16_t *k_par,
                             const uint16_t *v_par, int bits, int page_size, int pages, int Hkv, int d,
                             const int32_t *table, int table_pages, const int32_t *cu, const int32_t *kv_len,
                             int B, int T, uint16_t *K, uint16_t *V, void *stream);

/* Bytes of scratch qattn_paged_attention needs; 0 for an invalid or empty
 * shape. */
QOQ_API size_t qattn_paged_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int d, int table_pages,
                                                     int page_size, int max_new);

/* Attention of the new tokens over the cache (which holds them already):
 * row i of sequence b sees positions j <= kv_len[b] - n_b + i, and
 *     out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
 * with k, v the values the cache stands for. A row that sees nothing gets
 * zeros. Sums and the softmax's statistics are FP32, weights are rounded to
 * FP16, and so is the output. Scores are products of q with the cached codes,
 * without a rounding in between, for up to 32 rows per sequence and KV head
 * (n_b * Hq / Hkv); with more, keys and values may be rounded to FP16 first,
 * to what qattn_cache_read gives: half a step, as of any FP16 key. Weights
 * below 2^-30 of a row's largest may count as nothing.
 *   max_new    an upper bound of every n_b that the caller knows (T when it
 *              knows none). It only chooses kernels: rows beyond it are
 *              computed all the same. A decode step without it takes kernels
 *              for 16 rows instead of 8, and launches those for chunks.
 *   out        [T][Hq][d] FP16, row stride ldo.
 * The call's rows times its longest context are limited: (T * Hq / 256 +
 * min(T, B) * Hkv) * (table_pages * page_size / 128 + 2) < 2^31 (a table
 * wider than the contexts need counts in full).
 *   workspace  any contents; calls that may run at the same time need one
 *              each. */
QOQ_API int qattn_paged_attention(const uint16_t *q, int64_t ldq, int T, int Hq, int Hkv, int d,
                                  const uint8_t *k_codes, const uint8_t *v_codes, const uint16_t *k_par,
                                  const uint16_t *v_par, int bits, int page_size, int pages,
                                  const int32_t *table, int table_pages, const int32_t *cu,
                                  const int32_t *kv_len, int B, int max_new, float scale, uint16_t *out,
                                  int64_t ldo, void *workspace, size_t workspace_bytes, void *stream);

/* Causal attention of whole prompts, packed one after another: row i of
 * sequence b sees rows 0 .. i of the same sequence. No cache is involved.
 *   q [T][Hq][d], k, v [T][Hkv][d], out [T][Hq][d], each with its ld. */
QOQ_API int qattn_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk,
                                   const uint16_t *v, int64_t ldv, int T, int Hq, int Hkv, int d,
                                   const int32_t *cu, int B, float scale, uint16_t *out, int64_t ldo,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QOQ_ATTN_H */
