/*
 * hh_kv.h -- C ABI of libhh.so, the KV-cache operators: a cache kept in 4 bits,
 * decode attention over it, and eviction by accumulated attention weight.
 *
 * "The economics of hybrid attention" (table in "What a token of context
 * costs") prices a cached token of the 16 attention layers in three formats:
 * 64 KiB in f16, 34 KiB in q8_0, 18 KiB in q4_0.  hh.h serves the first two;
 * this header adds the third, and the means to bound the cache's growth.
 *
 * The conventions of hh.h hold (device pointers, 16-byte aligned, contiguous;
 * arguments checked before anything is enqueued; no device allocation; status
 * codes and hh_last_error()).  All offsets are 64-bit.
 *
 * The q4_0 format.  Every 32 consecutive elements x_0 .. x_31 of a cached row
 * (one head of one token) form a block: with m the element of largest
 * magnitude (the first one on ties),
 *     s   = fp16(m / -8), saturated to +-65504;
 *     c_i = clamp(rint(x_i / s) + 8, 0, 15)   (8 where s = 0),
 * and element i stands for s (c_i - 8).  A block that holds an infinity or a
 * NaN gets s = NaN: whatever attends it reads NaN, as with the bf16 cache.
 * Two arrays, as for q8_0:
 *     values [B, T_cache, H_kv, d/2]  uint8  byte j of a row: element 2j in
 *                                     its low half, 2j + 1 in its high half
 *     scales [B, T_cache, H_kv, d/32] fp16 bit patterns
 * 0.5625 bytes an element: 18 KiB a token in the page's layout.  The layout is
 * this library's own: caches that other programs keep under the same name pair
 * other elements in a byte and cannot be exchanged with these.
 *
 * Accumulated weights.  acc [B, H_kv, T_cache] fp32 holds, for every cached
 * position of every kv head, the attention weight it has drawn: each decode
 * step adds the sum of softmax weights over the query heads of the group (a
 * prompt's own queries add nothing).  A serving loop runs  append -> decode
 * (accumulating) -> ...  and, when a cache is full,  kv_evict_select ->
 * kv_compact,  after which cache_len is min(cache_len, n_keep).
 */
#ifndef HH_KV_H_
#define HH_KV_H_

#include "hh.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kv_append_q4_0 -- quantise the keys and values of new tokens into a q4_0
 * cache: one token per sequence in a decode step, or a whole prompt.
 *
 * cache_len counts the tokens that each sequence holds AFTER the call: its
 * n_new[b] new tokens are the last ones, so token i (0 <= i < n_new[b]) of
 * sequence b goes to position cache_len[b] - n_new[b] + i.  The same cache_len
 * then serves the step's decode.  Tokens whose position lies outside
 * [0, T_cache) are dropped.  All other positions are left as they were.
 *
 *   k, v               [B, n, H_kv, d]          bf16
 *   k_values, v_values [B, T_cache, H_kv, d/2]  uint8  written
 *   k_scales, v_scales [B, T_cache, H_kv, d/32] fp16   written
 *   cache_len          [B] int32, nullable (all = T_cache)
 *   n_new              [B] int32, nullable (all = n); clamped to [0, n]
 *   k_held, v_held     [B, n, H_kv, d] bf16, both or neither: written with the
 *                      values that the cache now stands for, rounded to bf16,
 *                      for the tokens that were stored (a prompt's attention
 *                      over them sees what later decode steps will read);
 *                      they overlap neither k, v nor each other
 * Supported: d = 128 or 256, B, n, T_cache >= 0.
 */
HH_API int kv_append_q4_0(const hh_bf16 *k, const hh_bf16 *v, uint8_t *k_values, uint16_t *k_scales,
                          uint8_t *v_values, uint16_t *v_scales, const int32_t *cache_len, const int32_t *n_new,
                          hh_bf16 *k_held, hh_bf16 *v_held, int B, int n, int T_cache, int H_kv, int d,
                          hh_stream stream);

/*
 * gqa_attn_decode_q4_0 -- gqa_attn_decode over a q4_0 cache, optionally
 * accumulating the attention weights.  Positions at and past cache_len[b] are
 * neither read into the result nor written, whatever they hold.
 *
 *   q, gate, o         [B, H_q, d]              bf16  (gate nullable; o written)
 *   k_values, v_values [B, T_cache, H_kv, d/2]  uint8
 *   k_scales, v_scales [B, T_cache, H_kv, d/32] fp16
 *   cache_len          as for gqa_attn_decode
 *   acc_out            [B, H_kv, T_cache] fp32, nullable: position j < cache_len[b]
 *                      becomes acc_in[b, hk, j] + sum over the group's query
 *                      heads of their softmax weight of j (before the gate)
 *   acc_in             as acc_out, nullable (zeros); may equal acc_out (in place)
 *   workspace          gqa_attn_decode_q4_0_workspace_size(...) bytes, 256-byte
 *                      aligned; contents on entry are ignored
 * Supported: d = 128 or 256, H_q % H_kv == 0, H_q / H_kv <= 16, B >= 0.
 * Sums are fp32; weights are rounded to fp16, and once more with V's scale.  A
 * logit is good to 2^-21 of scale x (sum over the blocks of 8 s sum |q|).  What a
 * block's small values give is good to 2^-24 of the largest value that the block
 * holds in the cache, and to 2^-20 of it where 131,072 keys of vanishing weight
 * add up.
 */
HH_API size_t gqa_attn_decode_q4_0_workspace_size(int B, int H_q, int H_kv, int d, int T_cache, int with_acc);
HH_API int gqa_attn_decode_q4_0(const hh_bf16 *q, const uint8_t *k_values, const uint16_t *k_scales,
                                const uint8_t *v_values, const uint16_t *v_scales, const int32_t *cache_len,
                                const hh_bf16 *gate, hh_bf16 *o, const float *acc_in, float *acc_out,
                                void *workspace, size_t ws_bytes, int B, int T_cache, int H_q, int H_kv, int d,
                                float scale, hh_stream stream);

/*
 * gqa_attn_decode_acc, gqa_attn_decode_q8_0_acc -- gqa_attn_decode and
 * gqa_attn_decode_q8_0 with acc_in / acc_out as above (acc_out not NULL) and a
 * workspace of gqa_attn_decode_acc_workspace_size(B, H_q, d, T_cache) bytes
 * (the logits of the step, 4 bytes per query head and position, and the
 * partial outputs).  The q8_0 form takes queries and V scales of any size, where
 * gqa_attn_decode_q8_0 has the limits of fp16 (hh.h).
 */
HH_API size_t gqa_attn_decode_acc_workspace_size(int B, int H_q, int d, int T_cache);
HH_API int gqa_attn_decode_acc(const hh_bf16 *q, const hh_bf16 *k_cache, const hh_bf16 *v_cache,
                               const int32_t *cache_len, const hh_bf16 *gate, hh_bf16 *o, const float *acc_in,
                               float *acc_out, void *workspace, size_t ws_bytes, int B, int T_cache, int H_q,
                               int H_kv, int d, float scale, hh_stream stream);
HH_API int gqa_attn_decode_q8_0_acc(const hh_bf16 *q, const int8_t *k_values, const uint16_t *k_scales,
                                    const int8_t *v_values, const uint16_t *v_scales, const int32_t *cache_len,
                                    const hh_bf16 *gate, hh_bf16 *o, const float *acc_in, float *acc_out,
                                    void *workspace, size_t ws_bytes, int B, int T_cache, int H_q, int H_kv, int d,
                                    float scale, hh_stream stream);

/*
 * kv_evict_select -- which positions of each (sequence, kv head) stay when its
 * cache is cut to n_keep positions: the last n_recent ones, and of the others
 * those with the largest accumulated weight.  On equal weights the lower
 * position stays; +0 and -0 are equal; a NaN counts as larger than any number.
 *
 *   acc       [B, H_kv, T_cache] fp32
 *   cache_len [B] int32, nullable (all = T_cache); clamped to [0, T_cache]
 *   keep      [B, H_kv, n_keep] int32, written: the min(cache_len[b], n_keep)
 *             positions that stay, ascending, then -1
 * Supported: 0 <= n_recent <= n_keep, B, T_cache, H_kv >= 0 (nothing to do
 * where a size is 0).
 */
HH_API int kv_evict_select(const float *acc, const int32_t *cache_len, int32_t *keep, int B, int T_cache, int H_kv,
                           int n_keep, int n_recent, hh_stream stream);

/*
 * kv_compact -- move the positions that stay to the front of a cache:
 *     dst[b, i, h] = src[b, keep[b, h, i], h]     for every array of the cache,
 *     acc_dst[b, h, i] = acc_src[b, h, keep[b, h, i]],
 * for i < n_keep; entries of keep outside [0, T_src) move nothing.  Positions
 * of the arrays with no entry keep what they held; acc_dst becomes 0 there, up
 * to T_dst, so that tokens appended later start from 0.
 * An array may be compacted in place (dst[a] == src[a], T_dst == T_src); its
 * keep rows must then ascend, as kv_evict_select writes them (entry i is moved
 * from a position >= i).  Otherwise dst and src must not overlap; no
 * array overlaps another one, the weights or keep.
 *
 *   keep      [B, H_kv, n_keep] int32
 *   src, dst  HOST arrays of n_arrays device pointers: the cache's arrays,
 *             [B, T_src, H_kv, row_bytes[a]] and [B, T_dst, H_kv, row_bytes[a]]
 *             bytes (bf16 rows: 2 d; q8_0: d and d/16; q4_0: d/2 and d/16)
 *   row_bytes HOST array, multiples of 8 up to 4096
 *   acc_src, acc_dst  [B, H_kv, T_src], [B, H_kv, T_dst] fp32, both or neither
 * Supported: 0 <= n_arrays <= 8, T_dst >= n_keep, T_src >= 1.
 */
HH_API int kv_compact(const int32_t *keep, const void *const *src, void *const *dst, const int32_t *row_bytes,
                      int n_arrays, const float *acc_src, float *acc_dst, int B, int T_src, int T_dst, int H_kv,
                      int n_keep, hh_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* HH_KV_H_ */
