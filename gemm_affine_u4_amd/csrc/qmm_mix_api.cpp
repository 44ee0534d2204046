// C ABI of the token mixers (declared and documented in include/qmm_mix.h): validate, then
// enqueue.  Nothing here allocates, synchronises or keeps state.
#include "qmm_mix.h"

#include <cmath>

#include "mix_internal.h"
#include "qmm_validate.h"

using qmm::Range;

namespace {

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxI32 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSeqs = 65535;  // a grid dimension
// Keys of a page table: the kernels number keys in 32 bits and look up to 64 steps of 256 ahead.
constexpr int64_t kMaxKeys = (int64_t(1) << 31) - (1 << 16);

bool hd_ok(int64_t hd) { return hd == 64 || hd == 128 || hd == 256; }

struct CacheBytes {
  uint64_t codes, meta;
};
CacheBytes cache_bytes(const qmm_kv4_cache& c) {
  const uint64_t rows = uint64_t(c.n_pages) * uint64_t(c.n_kv_heads) * uint64_t(c.page_size);
  return {rows * uint64_t(c.head_dim) / 2, rows * uint64_t(c.head_dim / 64) * 4};
}

int check_cache(const qmm_kv4_cache* c, qmm::Kv4* out) {
  if (!c || !c->k_codes || !c->k_meta || !c->v_codes || !c->v_meta) return QMM_ERR_NULL;
  if (!hd_ok(c->head_dim) || c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads || c->page_size < 16 ||
      c->page_size > 4096 || (c->page_size & (c->page_size - 1)) || c->n_pages < 1 || c->n_pages > kMaxI32 ||
      c->n_pages * c->page_size > kMaxI32)
    return QMM_ERR_SHAPE;
  if (!qmm::aligned(c->k_codes, 16) || !qmm::aligned(c->k_meta, 16) || !qmm::aligned(c->v_codes, 16) ||
      !qmm::aligned(c->v_meta, 16))
    return QMM_ERR_ALIGN;
  int shift = 4;
  while ((int64_t(1) << shift) < c->page_size) ++shift;
  *out = {c->k_codes, c->k_meta, c->v_codes, c->v_meta, int32_t(c->n_pages), shift, int32_t(c->n_kv_heads),
          int32_t(c->head_dim)};
  return QMM_OK;
}

bool gdn_dim_ok(int64_t d) { return d == 64 || d == 128; }
bool gdn_sizes_ok(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv) {
  if (T < 0 || T > kMaxTokens || B < 1 || B > kMaxSeqs || max_len < 1 || max_len > kMaxTokens || Hk < 1 || Hv < Hk ||
      Hv > kMaxHeads || Hv % Hk || !gdn_dim_ok(Dk) || !gdn_dim_ok(Dv))
    return false;
  return qmm::gdn_launches(B, max_len, Hv, Dv);
}
bool attn_sizes_ok(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv) {
  if (T < 0 || T > kMaxTokens || B < 1 || B > kMaxSeqs || max_q < 1 || max_q > kMaxTokens || n_kv < 1 ||
      n_kv > kMaxHeads || n_q < n_kv || n_q > kMaxHeads || n_q % n_kv || !hd_ok(hd) || max_kv < 1 || max_kv > kMaxKeys)
    return false;
  const int64_t rows = max_q * (n_q / n_kv), block = qmm::kv4_attn_rows(rows, hd);
  return (rows + block - 1) / block * n_kv <= 65535;  // a grid dimension
}

}  // namespace

extern "C" {

int qmm_kv4_append(const qmm_kv4_cache* cache, const void* k, const void* v, int64_t T, int in_dtype,
                   const int32_t* slots, const int32_t* positions, const float* cos_sin, int64_t max_pos,
                   int64_t rot_dim, const void* q, int64_t n_q_heads, uint16_t* q_out, uint16_t* k_held,
                   uint16_t* v_held, hipStream_t stream) {
  qmm::Kv4AppendArgs a = {};
  if (int st = check_cache(cache, &a.c)) return st;
  if (!k || !v || !slots || (cos_sin && !positions) || (q && (!q_out || !cos_sin))) return QMM_ERR_NULL;
  if (in_dtype != QMM_OUT_BF16 && in_dtype != QMM_OUT_F32) return QMM_ERR_ENUM;
  const int64_t hd = cache->head_dim, n_kv = cache->n_kv_heads;
  if (T < 0 || T > kMaxTokens || (q && (n_q_heads < 1 || n_q_heads > kMaxHeads)) ||
      (cos_sin && (rot_dim < 2 || rot_dim % 2 || rot_dim > hd || max_pos < 1 || max_pos > kMaxI32)))
    return QMM_ERR_SHAPE;
  const size_t e = in_dtype == QMM_OUT_F32 ? 4 : 2;
  if (!qmm::aligned(k, 16) || !qmm::aligned(v, 16) || !qmm::aligned(slots, 4) || !qmm::aligned(positions, 4) ||
      !qmm::aligned(cos_sin, 4) || !qmm::aligned(q, 16) || (q && !qmm::aligned(q_out, 16)) ||
      !qmm::aligned(k_held, 16) || !qmm::aligned(v_held, 16))
    return QMM_ERR_ALIGN;
  const uint64_t kvn = uint64_t(T * n_kv * hd), qn = q ? uint64_t(T * n_q_heads * hd) : 0;
  const CacheBytes cb = cache_bytes(*cache);
  const Range outs[] = {{cache->k_codes, cb.codes}, {cache->v_codes, cb.codes}, {cache->k_meta, cb.meta},
                        {cache->v_meta, cb.meta},   {q ? q_out : nullptr, qn * 2},
                        {k_held, k_held ? kvn * 2 : 0}, {v_held, v_held ? kvn * 2 : 0}};
  const Range ins[] = {{k, kvn * e}, {v, kvn * e}, {q, qn * e}, {slots, uint64_t(T) * 4},
                       {cos_sin ? positions : nullptr, uint64_t(T) * 4},
                       {cos_sin, cos_sin ? uint64_t(max_pos) * uint64_t(rot_dim) * 4 : 0}};
  if (qmm::any_alias(outs, 7, ins, 6)) return QMM_ERR_ALIAS;
  if (T == 0) return QMM_OK;
  a.k = k;
  a.v = v;
  a.q = q;
  a.slots = slots;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_out = q_out;
  a.k_held = k_held;
  a.v_held = v_held;
  a.T = T;
  a.max_pos = int32_t(max_pos);
  a.rot = cos_sin ? int32_t(rot_dim) : 0;
  a.n_q = q ? int32_t(n_q_heads) : 0;
  a.f32_in = in_dtype == QMM_OUT_F32;
  return qmm::launch_kv4_append(a, stream);
}

size_t qmm_kv4_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t n_q_heads, int64_t n_kv_heads,
                                    int64_t head_dim, int64_t max_kv) {
  if (!attn_sizes_ok(T, B, max_q, n_q_heads, n_kv_heads, head_dim, max_kv)) return 0;
  return size_t(qmm::kv4_attn_workspace(T, B, max_q, n_q_heads, n_kv_heads, head_dim, max_kv));
}

int qmm_kv4_attn(const uint16_t* q, int64_t T, const int32_t* q_start, const int32_t* kv_lens,
                 const int32_t* page_table, int64_t B, int64_t max_pages, int64_t max_q,
                 const qmm_kv4_cache* cache, int64_t n_q_heads, float scale, int causal, int64_t window,
                 const uint16_t* gate, void* workspace, size_t workspace_bytes, uint16_t* out, hipStream_t stream) {
  qmm::Kv4AttnArgs a = {};
  if (int st = check_cache(cache, &a.c)) return st;
  if (!q || !kv_lens || !page_table || !workspace || !out) return QMM_ERR_NULL;
  const int64_t hd = cache->head_dim;
  if (causal != 0 && causal != 1) return QMM_ERR_ENUM;
  if (max_pages < 1 || max_pages > kMaxKeys / cache->page_size ||
      !attn_sizes_ok(T, B, max_q, n_q_heads, cache->n_kv_heads, hd, max_pages * cache->page_size) ||
      (!q_start && (T != B || max_q != 1)) || window < 0 || (window > 0 && !causal) || !(scale > 0.f) ||
      !std::isfinite(scale))
    return QMM_ERR_SHAPE;
  const uint64_t need = qmm::kv4_attn_workspace(T, B, max_q, n_q_heads, cache->n_kv_heads, hd,
                                                max_pages * cache->page_size);
  if (workspace_bytes < need) return QMM_ERR_SHAPE;
  if (!qmm::aligned(q, 16) || !qmm::aligned(out, 16) || !qmm::aligned(gate, 16) || !qmm::aligned(workspace, 256) ||
      !qmm::aligned(q_start, 4) || !qmm::aligned(kv_lens, 4) || !qmm::aligned(page_table, 4))
    return QMM_ERR_ALIGN;
  const uint64_t qn = uint64_t(T * n_q_heads * hd) * 2;
  const CacheBytes cb = cache_bytes(*cache);
  const Range outs[] = {{out, qn}, {workspace, need}};
  const Range ins[] = {{q, qn}, {gate, gate ? qn : 0}, {q_start, q_start ? uint64_t(B + 1) * 4 : 0},
                       {kv_lens, uint64_t(B) * 4}, {page_table, uint64_t(B) * uint64_t(max_pages) * 4},
                       {cache->k_codes, cb.codes}, {cache->v_codes, cb.codes}, {cache->k_meta, cb.meta},
                       {cache->v_meta, cb.meta}};
  if (qmm::any_alias(outs, 2, ins, 9)) return QMM_ERR_ALIAS;
  if (T == 0) return QMM_OK;
  a.q = q;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.table = page_table;
  a.gate = gate;
  a.out = out;
  a.ws = workspace;
  a.T = T;
  a.window = window;
  a.B = int32_t(B);
  a.max_pages = int32_t(max_pages);
  a.max_q = int32_t(max_q);
  a.n_q = int32_t(n_q_heads);
  a.causal = causal;
  a.scale = scale;
  return qmm::launch_kv4_attn(a, stream);
}

size_t qmm_gdn_workspace_bytes(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv) {
  if (!gdn_sizes_ok(T, B, max_len, Hk, Hv, Dk, Dv)) return 0;
  return size_t(qmm::gdn_workspace(T, B, max_len, Hk, Hv, Dk, Dv));
}

int qmm_gdn(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* g, const float* beta, int64_t T,
            const int32_t* seq_start, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv,
            float scale, int l2norm, const float* state_in, float* state_out, const int32_t* state_slots,
            int64_t n_slots, void* workspace, size_t workspace_bytes, void* y, int out_dtype, hipStream_t stream) {
  if ((T != 0 && (!q || !k || !v || !g || !beta || !y)) || !state_in || !state_out || !workspace) return QMM_ERR_NULL;
  if ((out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) || (l2norm != 0 && l2norm != 1)) return QMM_ERR_ENUM;
  if (!gdn_sizes_ok(T, B, max_len, Hk, Hv, Dk, Dv) || (!seq_start && (T != B || max_len != 1)) || n_slots < 1 ||
      n_slots > kMaxI32 || (!state_slots && n_slots < B) || !std::isfinite(scale))
    return QMM_ERR_SHAPE;
  const uint64_t need = qmm::gdn_workspace(T, B, max_len, Hk, Hv, Dk, Dv);
  if (workspace_bytes < need) return QMM_ERR_SHAPE;
  const size_t e = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (!qmm::aligned(q, 16) || !qmm::aligned(k, 16) || !qmm::aligned(v, 16) || !qmm::aligned(g, 4) ||
      !qmm::aligned(beta, 4) || !qmm::aligned(state_in, 16) || !qmm::aligned(state_out, 16) || !qmm::aligned(y, 16) ||
      !qmm::aligned(workspace, 256) || !qmm::aligned(seq_start, 4) || !qmm::aligned(state_slots, 4))
    return QMM_ERR_ALIGN;
  const uint64_t sb = uint64_t(n_slots) * uint64_t(Hv * Dk * Dv) * 4;
  const bool in_place = state_in == state_out;
  const Range outs[] = {{y, uint64_t(T * Hv * Dv) * e}, {workspace, need}, {state_out, sb}};
  const Range ins[] = {{q, uint64_t(T * Hk * Dk) * 2}, {k, uint64_t(T * Hk * Dk) * 2}, {v, uint64_t(T * Hv * Dv) * 2},
                       {g, uint64_t(T * Hv) * 4}, {beta, uint64_t(T * Hv) * 4},
                       {seq_start, seq_start ? uint64_t(B + 1) * 4 : 0},
                       {state_slots, state_slots ? uint64_t(B) * 4 : 0}, {in_place ? nullptr : state_in, sb}};
  if (qmm::any_alias(outs, 3, ins, 8)) return QMM_ERR_ALIAS;
  qmm::GdnArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.seq_start = seq_start;
  a.state_in = state_in;
  a.state_out = state_out;
  a.slots = state_slots;
  a.y = y;
  a.ws = workspace;
  a.T = T;
  a.B = int32_t(B);
  a.max_len = int32_t(max_len);
  a.Hk = int32_t(Hk);
  a.Hv = int32_t(Hv);
  a.n_slots = int32_t(n_slots);
  a.l2norm = l2norm;
  a.f32_out = out_dtype == QMM_OUT_F32;
  a.Dk = int32_t(Dk);
  a.Dv = int32_t(Dv);
  a.scale = scale;
  return qmm::launch_gdn(a, stream);
}

}  // extern "C"
