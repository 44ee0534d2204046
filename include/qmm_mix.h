/*
 * qmm_mix.h -- C ABI of the token mixers next to the quantized projections (qmm.h): what
 * runs between the fused QKV projection and the output projection of a hybrid decoder.
 *   qmm_kv4_append   keys and values into a paged 4-bit cache, rotated on the way
 *   qmm_kv4_attn     attention over that cache, for single tokens and for prompts
 *   qmm_gdn          the gated delta rule, for single tokens and for prompts
 * The pages name all three as kernels of their own: the 4-bit KV compression and the
 * attention that dequantizes in registers with an online softmax in fp32, and the gated
 * delta net's fused scan ("Sanctum-MLX", the six optimisations and the model section:
 * 16 full-attention and 48 linear-attention layers).
 *
 * Conventions are those of qmm.h: device pointers owned by the caller, an explicit stream,
 * a status code, arguments validated before anything is enqueued, nothing allocated, kept
 * or synchronised, row-major contiguous arrays, inputs assumed finite.  Every call can be
 * captured in a graph.  A workspace belongs to one call at a time: calls that may run at
 * the same time (two streams, two captured graphs) need a workspace each.
 */
#ifndef QMM_MIX_H
#define QMM_MIX_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache of keys and values in 4 bits: n_pages pages of page_size token slots for
 * each of n_kv_heads heads.  Slot s is place s % page_size of page s / page_size.
 * The head_dim values of a slot's key (or value) are affine in groups of 64, as the
 * library's weights: x = scale * c + bias, c in 0..15, with fp16 scale and bias.
 *   k_codes [n_pages][n_kv_heads][page_size][head_dim/8] uint32, eight codes a word, the
 *           first in the lowest bits.  The word of dims 8w .. 8w+7 stands at place
 *           16(w/16) + 4((w%8)/2) + 2((w%16)/8) + w%2 of its row (head_dim 64: at place w):
 *           a lane's 16 bytes then hold codes of two whole groups, in the order in which
 *           the matrix instructions take them.
 *   v_codes [n_pages][n_kv_heads][page_size/8][head_dim/4][8] uint16: four codes (dims
 *           4u .. 4u+3, the first in the lowest bits) of eight neighbouring slots side by
 *           side, which is the order the product with the probabilities takes.
 *   k_meta, v_meta [n_pages][n_kv_heads][page_size][head_dim/64] uint32: the fp16 scale in
 *           the low half, the fp16 bias in the high half.
 * 4.5 bits per value.  head_dim 64, 128 or 256; page_size a power of two from 16 to 4096;
 * n_pages * page_size below 2^31.  All arrays 16-byte aligned.
 */
typedef struct qmm_kv4_cache {
  uint32_t* k_codes;
  uint32_t* k_meta;
  uint16_t* v_codes;
  uint32_t* v_meta;
  int64_t n_pages, page_size, n_kv_heads, head_dim;
} qmm_kv4_cache;

/*
 * qmm_kv4_append -- T new tokens' keys and values into the cache.
 *   k, v [T][n_kv_heads][head_dim] in in_dtype (QMM_OUT_BF16 or QMM_OUT_F32: as the
 *     projections leave them); slots int32 [T]: the token's slot; a slot outside
 *     [0, n_pages * page_size) stores nothing (a padded row).  Slots in range must be
 *     distinct: two tokens of one call with the same slot leave a mixture there.
 *   cos_sin != NULL: keys (and q) are rotated first, as qmm_fused_qkv_rope does it:
 *     for i < rot_dim/2 the dims (i, i + rot_dim/2), values (a, b), become
 *     (a*c - b*s, b*c + a*s), c = cos_sin[p][i], s = cos_sin[p][rot_dim/2 + i],
 *     p = positions[token] clamped to [0, max_pos); the dims from rot_dim on pass through.
 *     positions int32 [T], cos_sin fp32 [max_pos][rot_dim], rot_dim even, 2 .. head_dim.
 *   cos_sin == NULL: k is stored as it is (already rotated), and q must be NULL.
 *   q (nullable) [T][n_q_heads][head_dim] in in_dtype -> q_out the same shape in bf16.
 *   k_held, v_held (nullable) bf16 [T][n_kv_heads][head_dim]: the values that the cache
 *     now stands for, for callers that also use the new tokens' keys and values in dense form.
 * Quantization of a group of 64 (fp32, each operation rounded): x clamped to +-57344;
 * scale = fp16((max - min) * (1/15)), bias = fp16(min), c = rint((x - bias) * (1/scale))
 * clamped to 0..15 (c = 0 where the scale is 0).
 */
int qmm_kv4_append(const qmm_kv4_cache* cache, const void* k, const void* v, int64_t T, int in_dtype,
                   const int32_t* slots, const int32_t* positions, const float* cos_sin, int64_t max_pos,
                   int64_t rot_dim, const void* q, int64_t n_q_heads, uint16_t* q_out, uint16_t* k_held,
                   uint16_t* v_held, hipStream_t stream);

/*
 * qmm_kv4_attn -- softmax(scale * q K^T) V over the cache, for B sequences.
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
 *   max_q: no sequence has more queries; rows of a sequence past max_q are left as they were.
 *     n_kv_heads times the blocks of 128 rows in max_q * n_q_heads / n_kv_heads up to 65535 (40 / 8
 *     heads: 209689 queries).  T and max_q up to 2^24, B up to 65535.
 *   causal = 1: query j of n (0-based) of a sequence stands at p = kv_len - n + j and sees
 *     keys t <= p, with window > 0 only t > p - window.  causal = 0 (window must be 0):
 *     every query sees all keys.
 *   A query that sees no key gives zeros.  scale > 0 and finite; |q| below 2^100 and q . k
 *   below 2^126, and for prompts scale * |q| * log2(e) below 65504 (larger ones are taken as that).
 *   gate (nullable) [T][n_q_heads][head_dim] bf16: out is multiplied by
 *     1 / (1 + exp(-gate)) (the output gate that qmm_fused_qkv_rope writes).
 * Sums, maxima and the softmax are fp32.  Rounded to fp16 (2^-11 of the value) are, for few queries
 * (up to 128 rows = queries x heads of a group, 64 at head_dim 256), the probabilities and the
 * probabilities times scale, with keys and queries exact; for prompts the scaled queries, the dequantized
 * keys and values (values of a magnitude above 65504 do not occur in a cache that qmm_kv4_append
 * wrote) and the probabilities.  Below fp16's normal range such a value is off by an absolute amount: a
 * prompt's scaled query and, of the row's largest, its probability by up to 2^-25, the few queries'
 * probability by 2^-28.  The same call gives the same bits every time.
 * workspace: 256-byte aligned, at least qmm_kv4_attn_workspace_bytes of the same T, B, max_q,
 * heads and max_kv = max_pages * page_size (0 for sizes out of range; always > 0 otherwise).
 */
size_t qmm_kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t n_q_heads, int64_t n_kv_heads,
                                    int64_t head_dim, int64_t max_kv);
int qmm_kv4_attn(const uint16_t* q, int64_t T, const int32_t* q_start, const int32_t* kv_lens,
                 const int32_t* page_table, int64_t B, int64_t max_pages, int64_t max_q,
                 const qmm_kv4_cache* cache, int64_t n_q_heads, float scale, int causal, int64_t window,
                 const uint16_t* gate, void* workspace, size_t workspace_bytes, uint16_t* out, hipStream_t stream);

/*
 * qmm_gdn -- the gated delta rule ("Sanctum-MLX", the gated delta net's recurrence): per
 * sequence and value head, with a state S of Dk x Dv and, per token,
 *   S <- exp(g) S;   S <- S + k (beta (v - S^T k))^T;   y = S^T (scale q).
 *   q, k [T][Hk][Dk] bf16, v [T][Hv][Dv] bf16, g and beta fp32 [T][Hv] (g the natural
 *     logarithm of the decay, <= 0; -infinity forgets all before the token), y [T][Hv][Dv] bf16 or fp32 per out_dtype; Hv a multiple of Hk,
 *     value head a reading key head a / (Hv / Hk).
 *   l2norm = 1: q and k are divided by sqrt(sum of squares + 1e-6) first.
 *   seq_start int32 [B+1] as q_start above (rows behind the last sequence are left as they
 *     were), NULL: one token a sequence, T = B.  max_len: no sequence is longer.  A longer
 *     one is cut there.
 *   state_in, state_out fp32 [n_slots][Hv][Dv][Dk] (the layout the pages give):
 *     state_out == state_in updates in place; otherwise they must not overlap.  Sequence b
 *     reads and writes slot state_slots[b] (NULL: slot b).  A slot outside [0, n_slots):
 *     the sequence starts from zeros and its last state is not kept.  Slots in range must
 *     be distinct.  A sequence without tokens copies its state (T = 0: q, k, v, g, beta and y may be NULL).
 *   Dk and Dv 64 or 128.  T and max_len up to 2^24, B up to 65535, Hv up to 1024, and with max_len
 *   above 16 B * Hv (rounded up to 8) * Dv below 2^28.
 * The state and all sums are fp32.  Sequences of up to 16 tokens (max_len) run token by
 * token; longer ones in chunks of 64 tokens on the matrix cores with each fp32 factor as
 * a sum of three bf16 values (two where only a bf16 y reads it).  Inputs are finite: in a
 * chunk an infinite v or q would reach the outputs of earlier tokens of the chunk too.
 * The same call gives the same bits every time.
 * workspace: 256-byte aligned, at least qmm_gdn_workspace_bytes of the same sizes (0 for sizes
 * out of range; always > 0 otherwise).
 */
size_t qmm_gdn_workspace_bytes(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv);
int qmm_gdn(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* g, const float* beta, int64_t T,
            const int32_t* seq_start, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
            float scale, int l2norm, const float* state_in, float* state_out, const int32_t* state_slots,
            int64_t n_slots, void* workspace, size_t workspace_bytes, void* y, int out_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_MIX_H */
