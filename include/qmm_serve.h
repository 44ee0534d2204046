/*
 * qmm_serve.h -- C ABI of what one step of a batch of requests adds to the quantized
 * projections (qmm.h) and the token mixers (qmm_mix.h):
 *   qmm_lora          low-rank adapters of many requests beside a shared projection
 *   qmm_kv8_append    keys and values into a paged 8-bit cache, rotated on the way
 *   qmm_kv8_attn      attention over that cache, with a window and first tokens that stay visible
 *   qmm_spec_verify   drafted tokens against the target's probabilities
 * The pages serve adapters beside their 4-bit weights, look drafts up in the prompt or take
 * them from a draft head, and hold keys and values in compressed form ("Sanctum-MLX", the
 * server section; the saragossa README, speculation and cache formats).
 *
 * Conventions are those of qmm.h: device pointers owned by the caller, an explicit stream,
 * a status code, arguments validated before anything is enqueued, nothing allocated, kept
 * or synchronised, row-major contiguous arrays, inputs assumed finite.  Every call can be
 * captured in a graph.  A workspace belongs to one call at a time: calls that may run at
 * the same time (two streams, two captured graphs) need a workspace each.  The same call
 * gives the same bits every time.
 */
#ifndef QMM_SERVE_H
#define QMM_SERVE_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache of keys and values in 8 bits: n_pages pages of page_size token slots for each
 * of n_kv_heads heads.  The 16 keys 16j .. 16j+15 of a sequence are a block; the keys of a
 * block and head share one fp32 scale, and so do its values: x = scale * c, c in -127 .. 127.
 *   k_codes [n_pages][n_kv_heads][page_size][head_dim] int8
 *   v_codes [n_pages][n_kv_heads][page_size/8][head_dim][8] int8: the codes of eight
 *           neighbouring slots side by side, the order of the product with the probabilities
 *   k_scale, v_scale [n_pages][n_kv_heads][page_size/16] fp32
 * head_dim 64, 128 or 256; page_size a power of two from 16 to 4096; n_pages * page_size
 * below 2^31.  All arrays 16-byte aligned.
 */
typedef struct qmm_kv8_cache {
  int8_t* k_codes;
  float* k_scale;
  int8_t* v_codes;
  float* v_scale;
  int64_t n_pages, page_size, n_kv_heads, head_dim;
} qmm_kv8_cache;

/*
 * qmm_kv8_append -- the new tokens of B sequences into the cache.
 *   k, v [T][n_kv_heads][head_dim] in in_dtype (QMM_OUT_BF16 or QMM_OUT_F32: as the
 *     projections leave them).  q_start, kv_lens, page_table, max_q and B as qmm_kv8_attn
 *     takes them: token j of the n of a sequence becomes its key p = kv_len - n + j.  A token
 *     with p < 0, without a page or past max_q stores nothing.  No two sequences
 *     append to the same block.
 *   cos_sin != NULL: keys (and q) are rotated first, as qmm_kv4_append does it, by the row
 *     positions[token] (int32 [T]; NULL: p) of cos_sin fp32 [max_pos][rot_dim], clamped to
 *     [0, max_pos); rot_dim even, 2 .. head_dim.
 *   cos_sin == NULL: k is stored as it is, q and positions must be NULL.
 *   q (nullable) [T][n_q_heads][head_dim] in in_dtype -> q_out the same shape in bf16, for all
 *     tokens of the sequences up to max_q.
 *   k_held, v_held (nullable) bf16 [T][n_kv_heads][head_dim]: the values that the cache now
 *     stands for; rows of tokens that store nothing are left as they were.
 * Quantization (fp32, each operation rounded): x clamped to +-57344; need = (largest |x| of the
 * call's tokens in the block and head) * (1/127).  A block whose first key is among them begins
 * anew: scale = need.  Otherwise it holds earlier keys: its scale stays if need is not above it,
 * else it becomes the larger of need and 1.25 scale, and the codes of the earlier keys
 * become rint(c * (old scale / new scale)).  c = rint(x * (1/scale)) clamped to +-127 (0 where the
 * scale is not above 2^-127).  A scale that grows, grows by a quarter: so the roundings of a key whose block
 * fills token by token add up to 2.5 steps at most.  Slots of a block behind its last key hold any codes.
 * T and max_q up to 2^24, B up to 65535, B * (max_q / 16 + 2) up to 2^26 - 4.
 */
int qmm_kv8_append(const qmm_kv8_cache* cache, const void* k, const void* v, int64_t T, int in_dtype,
                   const int32_t* q_start, const int32_t* kv_lens, const int32_t* page_table, int64_t B,
                   int64_t max_pages, int64_t max_q, const int32_t* positions, const float* cos_sin,
                   int64_t max_pos, int64_t rot_dim, const void* q, int64_t n_q_heads, uint16_t* q_out,
                   uint16_t* k_held, uint16_t* v_held, hipStream_t stream);

/*
 * qmm_kv8_attn -- softmax(scale * q K^T) V over the cache, for B sequences.
 *   q [T][n_q_heads][head_dim] bf16, out the same shape in bf16; n_q_heads a multiple of
 *     n_kv_heads, head a reading KV head a / (n_q_heads / n_kv_heads).
 *   q_start int32 [B+1]: sequence b's queries are rows q_start[b] .. q_start[b+1]-1 of q
 *     (ascending; q_start[B] <= T; rows from q_start[B] on are left as they were).
 *     NULL: one query a sequence, T = B.
 *   kv_lens int32 [B]: keys of sequence b, its new tokens' (appended before) among them;
 *     clamped to [0, max_pages * page_size].
 *   page_table int32 [B][max_pages]: page of keys t of the sequence at entry t / page_size.
 *     An entry outside [0, n_pages) is "no page": its keys are not seen.  max_pages * page_size
 *     up to 2^31 - 65536.
 *   max_q: no sequence has more queries; rows of a sequence past max_q are left as they were.  How a call is cut
 *     follows from it, so give prompts and sequences of few queries calls of their own (63 single tokens beside a prompt of
 *     512, 40 / 8 heads x 128: 723 us in one call, 176 in two).
 *     n_kv_heads times the blocks of 128 rows in max_q * n_q_heads / n_kv_heads up to 65535.
 *     T and max_q up to 2^24, B up to 65535.
 *   causal = 1: query j of n (0-based) of a sequence stands at p = kv_len - n + j and sees
 *     keys t <= p, with window > 0 only t > p - window and t < sinks (sinks > 0 needs a window).
 *   causal = 0 (window must be 0): every query sees all keys.
 *   What is stored for keys that no query sees does not matter (pages behind a window may have
 *   been given away while the table still names them).
 *   A query that sees no key gives zeros.  scale > 0 and finite; |q| and the scales of keys below 2^100, q . k
 *   and scale * q . k below 2^126.
 *   gate (nullable) [T][n_q_heads][head_dim] bf16: out is multiplied by 1 / (1 + exp(-gate)).
 * Scores, sums, maxima and the softmax are fp32, from exact codes and queries (of a query row,
 * values below 2^-24 of its largest lose digits).  A key's weight times its values' scale is rounded to
 * fp16: 2^-11 of it; where it is small, 2^-39 of the largest scale for few queries (up to 16 rows = max_q x heads of
 * a group), 2^-36 of the row's largest such product for prompts (more than 256 rows), between them one of the two.
 * At the ends of the range: few queries are off by 2^-140 at least; prompts take value scales below 2^-80 of the largest
 * one that any of a sequence's queries sees as that, so that values of such blocks beside much larger ones are off
 * by up to 127 * 2^-80 of the largest scale, and value scales are up to 2^88 (qmm_kv8_append's are below 2^9).
 * workspace: 256-byte aligned, at least qmm_kv8_attn_workspace_bytes of the same T, B, max_q,
 * heads, max_kv = max_pages * page_size, window and sinks (0 for sizes out of range; always > 0
 * otherwise).
 */
size_t qmm_kv8_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t n_q_heads, int64_t n_kv_heads,
                                    int64_t head_dim, int64_t max_kv, int64_t window, int64_t sinks);
int qmm_kv8_attn(const uint16_t* q, int64_t T, const int32_t* q_start, const int32_t* kv_lens,
                 const int32_t* page_table, int64_t B, int64_t max_pages, int64_t max_q,
                 const qmm_kv8_cache* cache, int64_t n_q_heads, float scale, int causal, int64_t window,
                 int64_t sinks, const uint16_t* gate, void* workspace, size_t workspace_bytes, uint16_t* out,
                 hipStream_t stream);

/*
 * qmm_spec_verify -- drafted tokens of B sequences against the target's probabilities.
 *   draft int32 [D], draft_start int32 [B+1]: sequence b drafted tokens draft_start[b] ..
 *     draft_start[b+1]-1 (ascending, draft_start[B] <= D; at most max_draft of them count).
 *   target [D+B][V], in prob_dtype (QMM_OUT_BF16 or QMM_OUT_F32): with a = draft_start[b] + b, row
 *     a + j is p_j, the target's probabilities of the token behind the sequence's first j drafts, j = 0 .. n.
 *   draft_probs (nullable) [D][V] in prob_dtype: row of draft j is q_j, which it was drawn from.
 *     NULL: drafts that were looked up, q_j = 1 at the draft.
 *   u fp32 [D+B] in [0, 1): u[a + j] decides draft j, u[a + n] the new token.
 *   Draft j (d = draft[j]) is kept while u q_j(d) < p_j(d); one outside [0, V) never is.  The new
 *   token is drawn with the weights w = max(p_j - q_j, 0) of the first draft j that is not kept (where
 *   they are all 0: p_j), of p_n if all are: the least v with w(v) > 0 and w(0) + .. + w(v) >
 *   u[a + n] (w(0) + .. + w(V-1)), or the last v with w(v) > 0 if there is none; -1 if
 *   there is no w(v) > 0.  So kept and new tokens are distributed as the target's.
 *   Weights that are negative or NaN count as 0.  Products, differences and sums are 64-bit.
 *   tokens int32 [B][max_draft+1]: the kept drafts, the new token, then -1.
 *   accepted int32 [B]: how many drafts were kept.
 * V up to 2^24, B up to 65535, D up to 2^24, max_draft 0 .. 65535.  draft may be NULL where D = 0.
 * workspace: 256-byte aligned, at least qmm_spec_verify_workspace_bytes(B, V) bytes (0 for sizes out
 * of range; always > 0 otherwise).
 */
size_t qmm_spec_verify_workspace_bytes(int64_t B, int64_t V);
int qmm_spec_verify(const int32_t* draft, int64_t D, const int32_t* draft_start, int64_t B, int64_t max_draft,
                    const void* target, const void* draft_probs, int64_t V, int prob_dtype, const float* u,
                    int32_t* tokens, int32_t* accepted, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/*
 * qmm_lora -- y_p[t] = base_p[t] + scales[i] B_{i,p} (A_{i,p} x[t]), i = ids[t], for the n_parts
 * (1 .. 3) outputs p of one projection of x (Q, K and V of a fused one, say).
 *   x bf16 [T][K], K a multiple of 64 up to QMM_MAX_K.
 *   a bf16 [n_adapters][n_parts * rank][K]; b bf16 [n_adapters][rows_0 + .. ][rank]: the parts'
 *     rows one after the other.  rank 8, 16, 32, 64 or 128 (smaller ones padded with zeros).
 *   ids int32 [T]: a token's adapter; one outside [0, n_adapters) means none: y_p[t] = base_p[t].
 *   scales fp32 [n_adapters], NULL: 1.
 *   part_rows int64 [n_parts], base and y: pointers [n_parts]; these three arrays are host memory.
 *     base_p [T][rows_p] in base_dtype, y_p the same shape in out_dtype (QMM_OUT_BF16 or
 *     QMM_OUT_F32).  base NULL, or base_p = y_p (both dtypes the same): y is updated in place.
 *   Tokens of one adapter that stand side by side (a request's prompt) share its weights' reads.
 * Sums are fp32; A x is taken on as three bf16 pieces (24 bits), so y is rounded once.
 * T up to 2^24, the sum of rows up to 2^24, n_adapters up to 65535, (T / 32 + 17) * (rows / 256 + 3)
 * below 2^24.
 * workspace: 256-byte aligned, at least qmm_lora_workspace_bytes of the same sizes (0 for sizes
 * out of range; always > 0 otherwise).
 */
size_t qmm_lora_workspace_bytes(int64_t T, int64_t K, int64_t rank, int64_t n_parts);
int qmm_lora(const uint16_t* x, int64_t T, int64_t K, const uint16_t* a, const uint16_t* b, int64_t n_adapters,
             int64_t rank, const int32_t* ids, const float* scales, int64_t n_parts, const int64_t* part_rows,
             const void* const* base, int base_dtype, void* const* y, int out_dtype, void* workspace,
             size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_SERVE_H */
