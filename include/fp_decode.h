/*
 * fp_decode.h -- what follows a prefill: rotary positions, the paged key/value
 * cache (quantised as it is written, and read back), and the attention of
 * drafted tokens over that cache.
 *
 * A decode step is fp_rope_apply on the new tokens' q and k, fp_kv_write of
 * their k and v, fp_tree_attn over the cache (one new token per sequence is
 * the plain step, a tree of drafted tokens the speculative one).  A new prefill
 * over a cached prefix is fp_kv_read into the packed head-major layout that
 * fp_sparse_attn and fp_varlen_* take.
 *
 * Conventions.  Tensors of tokens are indexed [head][token][element] and given
 * as a pointer with two strides in elements: element i of head h of token t is
 * at ptr + t*tok + h*head + i (the elements of a head are contiguous).  So
 * head-major tensors have tok = d, head = T*d, and the rows of a fused
 * projection tok = row length, head = d.  Rows must start on 16-byte
 * boundaries (pointer and strides), unless stated.  Query head h reads KV head
 * h / (Hq/Hkv).  All pointers are of the current device; all calls are
 * asynchronous on `stream` (a cudaStream_t, NULL = legacy default stream),
 * allocate nothing on the device and may be captured into a CUDA graph (a
 * library call made before on the same device has done the set-up).  The
 * caller keeps every buffer alive until the stream has passed the call; a
 * captured call reads its tables anew at every replay.
 *
 * Errors: FP_OK or an FP_ERR_* code of fp_sparse.h; argument errors are found
 * on the host before any launch.  Tables that live on the device (slots, block
 * tables, lengths) are checked by the kernels: an entry outside its range is
 * never followed, and sets FP_ERR_RANGE in the sticky word that
 * fp_get_device_error() reads.
 */
#ifndef FP_DECODE_H
#define FP_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "fp_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types: tensors are bf16, fp16 or fp32; caches bf16, fp16, int8, e4m3. */
enum { FP_DT_BF16 = 0, FP_DT_F16 = 1, FP_DT_F32 = 2, FP_DT_INT8 = 3, FP_DT_E4M3 = 4 };

/* ---- Rotary positions --------------------------------------------------- */

/* Which elements make a pair: i with i + rot/2, or 2i with 2i + 1. */
enum { FP_ROPE_HALF = 0, FP_ROPE_INTERLEAVED = 1 };

/* How the frequencies f_i = theta^(-2i/rot), i < rot/2, are changed for
 * contexts longer than the original length `orig_len` by `factor`:
 *   NONE    not at all
 *   LINEAR  f_i / factor
 *   BASE    theta replaced by theta * factor^(rot/(rot-2))
 *   BANDS   by the turns n_i = orig_len f_i / (2 pi) that pair i makes within
 *           the original length: kept from n_i >= high, divided by factor to
 *           n_i <= low, between them f_i (w + (1-w)/factor), w = (n_i-low)/(high-low)
 *   RAMP    by the index (the YaRN method): c(n) = rot ln(orig_len/(2 pi n)) /
 *           (2 ln theta), a = max(floor(c(high)), 0), b = min(ceil(c(low)), rot-1),
 *           u_i = clamp((i-a)/max(b-a, 0.001), 0, 1), f_i (1-u_i) + f_i u_i/factor */
enum { FP_ROPE_NONE = 0, FP_ROPE_LINEAR = 1, FP_ROPE_BASE = 2, FP_ROPE_BANDS = 3, FP_ROPE_RAMP = 4 };

/* Opaque: the frequencies of one model's rotary embedding (host memory only). */
typedef struct fp_rope fp_rope;

/* Makes the frequencies.  d: elements of a head, even, 2..512; rot: the first
 * rot of them are rotated, even, 2..min(d, 256), the rest is passed through;
 * layout, scaling as above; theta > 1; factor > 0; orig_len, low, high are
 * read by BANDS (orig_len > 0, 0 < low < high) and RAMP (orig_len > 0,
 * 0 < low < high) only; BASE needs rot > 2.  amplitude (> 0) multiplies the
 * rotated elements (the attention factor of RAMP; 1 otherwise).  *out receives
 * the handle (NULL on error).  No CUDA call. */
int fp_rope_create(int d, int rot, int layout, double theta, int scaling, double factor, double orig_len, double low,
                   double high, double amplitude, fp_rope **out);
void fp_rope_free(fp_rope *r);

/* Copies the rot/2 frequencies (radians per position) to HOST freqs. */
int fp_rope_freqs(const fp_rope *r, double *freqs);

/* Rotates q and k: for the pair (a, b) of frequency f_i of token t, with
 * x = pos[t] f_i and m the amplitude,
 *   a' = m (a cos x - b sin x),  b' = m (b cos x + a sin x),
 * and with inverse != 0 by -x, which is the transpose: the gradient of the
 * inputs from the gradient of the outputs.  The angle is formed exactly in
 * 64-bit fixed point (any int32 position, negative ones too), sine, cosine and
 * products in fp32, one rounding to the output.
 * q_in, q_out [Hq][T][d], k_in, k_out [Hkv][T][d] with strides, of type dtype
 * (FP_DT_BF16, _F16 or _F32); aligned to their element type (16-byte aligned
 * rows take the fast path); an output may be its input itself (same pointer and
 * strides), any other overlap is the caller's error.  Hq or Hkv may be 0 (its
 * pointers are then not looked at).  pos: device int32[T], 4-byte aligned.
 * T = 0 is a no-op. */
int fp_rope_apply(const fp_rope *r, const void *q_in, int64_t q_in_tok, int64_t q_in_head, const void *k_in,
                  int64_t k_in_tok, int64_t k_in_head, void *q_out, int64_t q_out_tok, int64_t q_out_head,
                  void *k_out, int64_t k_out_tok, int64_t k_out_head, int dtype, int T, int Hq, int Hkv,
                  const int32_t *pos, int inverse, void *stream);

/* ---- Paged key/value cache ---------------------------------------------- */

/* Opaque: a view of caller-owned pools (host memory only). */
typedef struct fp_kv fp_kv;

/* Describes a cache of `pages` pages of `page` tokens (16, 32, 64 or 128) for
 * Hkv KV heads of d (64 or 128) elements:
 *   k_pool, v_pool   device [pages][Hkv][page][d] of type dtype
 *                    (FP_DT_BF16, _F16, _INT8, _E4M3), 16-byte aligned
 *   k_scale, v_scale device fp32 [pages][Hkv][page], 16-byte aligned, for int8
 *                    and e4m3; NULL for bf16 and fp16
 * Token `off` of page `p` is slot p*page + off.  pages*Hkv*page < 2^31.  The
 * pools stay the caller's.  A view belongs to the device that is current here;
 * calls with another current device return FP_ERR_ARG.  *out receives the
 * handle (NULL on error). */
int fp_kv_create(void *k_pool, void *v_pool, float *k_scale, float *v_scale, int dtype, int64_t pages, int page,
                 int Hkv, int d, fp_kv **out);
void fp_kv_free(fp_kv *kv);

/* Writes T tokens' k and v [Hkv][T][d] (strides as above; dtype FP_DT_BF16,
 * _F16 or _F32) to the slots slots[t] (device int64[T], 8-byte aligned); a
 * negative slot skips its token (padding), one past the cache is not written
 * and sets FP_ERR_RANGE.  The slots of one call must differ: of two tokens with
 * the same slot, whose codes and whose scale the slot then holds is not
 * specified.  Each (token, head) row is quantised by itself:
 *   scale = M / c,  code = round(c x / M),  M = max|x|,
 *   c = 127 and rounding half to even for int8, c = 448 and the conversion's
 *   rounding half to even for e4m3;
 * code 0 and scale 0 for a row of zeros.  A row with an infinity or a NaN gets
 * scale NaN and code 0, so that it reads back as NaN.  bf16 and fp16 caches
 * hold the rows rounded to their type.  k or v may be NULL to write the other
 * alone.  T = 0 is a no-op. */
int fp_kv_write(const fp_kv *kv, const void *k, int64_t k_tok, int64_t k_head, const void *v, int64_t v_tok,
                int64_t v_head, int dtype, int T, const int64_t *slots, void *stream);

/* Reads cached tokens back, code*scale rounded to dtype (FP_DT_BF16, _F16 or
 * _F32), packed: rows cu[s] .. cu[s+1]-1 of k and v [Hkv][T][d] receive the
 * tokens first[s], first[s]+1, .. of sequence s.
 *   block_table  device int32[nseq][max_pages]: the pages of a sequence in order
 *   cu           device int32[nseq+1], cu[0] = 0, non-decreasing
 *   first        device int32[nseq] or NULL for 0 (4-byte aligned, all three)
 * T is the number of rows of the outputs; rows behind cu[nseq] are left as they
 * were, and so are rows whose position or page is out of range (FP_ERR_RANGE).
 * k or v may be NULL to read the other alone.  T = 0 or nseq = 0 is a no-op. */
int fp_kv_read(const fp_kv *kv, const int32_t *block_table, int max_pages, const int32_t *cu, const int32_t *first,
               int nseq, int T, void *k, int64_t k_tok, int64_t k_head, void *v, int64_t v_tok, int64_t v_head,
               int dtype, void *stream);

/* ---- Attention of drafted tokens over the cache ------------------------- */

/* Bytes of device workspace that fp_tree_attn needs for these sizes on the
 * current device (0 for sizes that it does not take): nseq sequences of at most
 * max_q new tokens; it also serves calls with a smaller max_q or fewer query heads.  The contents need not be set, and are not kept between
 * calls; calls that may run at the same time, captured graphs among them, need
 * a workspace each. */
size_t fp_tree_attn_workspace(int nseq, int max_q, int Hq, int Hkv, int d);

/* Attention of the new tokens of nseq sequences over their cached tokens.
 * Sequence s has n = cu_q[s+1] - cu_q[s] new tokens, the rows cu_q[s] .. of q
 * and out, and kv_len[s] cached tokens, the last n of which are the new ones
 * (written before this call).  New token i sees every cached token p <
 * kv_len[s] - n, and new token j when bit j of its mask is set (without mask:
 * when j <= i):
 *   out[h][i] = sum_p softmax_p(scale q_i . k_p) v_p,
 *   lse[h][i] = ln sum_p exp(scale q_i . k_p)     (lse may be NULL)
 * with fp32 scores, sums and accumulation, and probabilities rounded to the
 * 16-bit type of the matrix product: to bf16 over bf16 caches (off by at most
 * 2^-8 of each), elsewhere to fp16, over int8 and e4m3 times V's scale (2^-11
 * of each or 2^-26 of the row's largest, whichever is larger; V's scales
 * from 2^-80 to 2^80).  Probabilities below 2^-80 of the row's largest may count
 * as 0.  A token that sees nothing gets out 0 and
 * lse -inf.  Values that are not visible have no effect, NaN and infinities
 * included.
 *   q, out       [Hq][T][d] with strides, dtype FP_DT_BF16 or FP_DT_F16; over a
 *                bf16 or fp16 cache the cache's type
 *   block_table  device int32[nseq][max_pages] (max_pages*page <= 2^30), kv_len
 *                device int32[nseq], cu_q device int32[nseq+1] (cu_q[0] = 0, non-decreasing,
 *                cu_q[nseq] <= T), 4-byte aligned
 *   mask         device uint64[T][ceil(max_q/64)] or NULL, 8-byte aligned
 *   lse          device fp32 [Hq][T]
 *   work         workspace, 16-byte aligned, of at least fp_tree_attn_workspace
 *                bytes (work_bytes)
 * scale > 0; 1 <= max_q <= 256; n <= max_q; kv_len[s] >= n.  A sequence that breaks one of
 * the last two, or whose length passes max_pages*page, is left out (its rows of
 * out and lse stay as they were) and sets FP_ERR_RANGE, as does a page outside
 * the cache (its tokens are then unspecified).  Rows behind cu_q[nseq] stay as
 * they were. */
int fp_tree_attn(const fp_kv *kv, const void *q, int64_t q_tok, int64_t q_head, int dtype, int T, int Hq,
                 const int32_t *block_table, int max_pages, const int32_t *kv_len, const int32_t *cu_q, int nseq,
                 int max_q, const uint64_t *mask, float scale, void *out, int64_t o_tok, int64_t o_head, float *lse,
                 void *work, size_t work_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP_DECODE_H */
