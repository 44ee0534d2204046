// C ABI of a serving step (declared and documented in include/qmm_serve.h): validate, then
// enqueue.  Nothing here allocates, synchronises or keeps state.
#include "qmm_serve.h"

#include <cmath>

#include "qmm_validate.h"
#include "serve_internal.h"

using qmm::Range;

namespace {

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxI32 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxSeqs = 65535;  // a grid dimension
// Keys of a page table: the kernels number keys in 32 bits and look up some tiles ahead.
constexpr int64_t kMaxKeys = (int64_t(1) << 31) - (1 << 16);

// Blocks of 16 keys that an append may meet: a wave each, four in a workgroup, of a launch of less than 2^32 threads.
constexpr int64_t kMaxBlocks = (int64_t(1) << 26) - 4;

bool type_ok(int t) { return t == QMM_OUT_BF16 || t == QMM_OUT_F32; }
size_t type_bytes(int t) { return t == QMM_OUT_F32 ? 4 : 2; }
bool hd_ok(int64_t hd) { return hd == 64 || hd == 128 || hd == 256; }

struct CacheBytes {
  uint64_t codes, scales;
};
CacheBytes cache_bytes(const qmm_kv8_cache& c) {
  const uint64_t rows = uint64_t(c.n_pages) * uint64_t(c.n_kv_heads) * uint64_t(c.page_size);
  return {rows * uint64_t(c.head_dim), rows / 16 * 4};
}

int check_cache(const qmm_kv8_cache* c, qmm::Kv8* out) {
  if (!c || !c->k_codes || !c->k_scale || !c->v_codes || !c->v_scale) return QMM_ERR_NULL;
  if (!hd_ok(c->head_dim) || c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads || c->page_size < 16 ||
      c->page_size > 4096 || (c->page_size & (c->page_size - 1)) || c->n_pages < 1 || c->n_pages > kMaxI32 ||
      c->n_pages * c->page_size > kMaxI32)
    return QMM_ERR_SHAPE;
  if (!qmm::aligned(c->k_codes, 16) || !qmm::aligned(c->k_scale, 16) || !qmm::aligned(c->v_codes, 16) ||
      !qmm::aligned(c->v_scale, 16))
    return QMM_ERR_ALIGN;
  int shift = 4;
  while ((int64_t(1) << shift) < c->page_size) ++shift;
  *out = {c->k_codes, c->k_scale, c->v_codes, c->v_scale, int32_t(c->n_pages), shift, int32_t(c->n_kv_heads),
          int32_t(c->head_dim)};
  return QMM_OK;
}

bool batch_ok(int64_t T, int64_t B, int64_t max_q) {
  return T >= 0 && T <= kMaxTokens && B >= 1 && B <= kMaxSeqs && max_q >= 1 && max_q <= kMaxTokens;
}
bool attn_sizes_ok(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv,
                   int64_t window, int64_t sinks) {
  if (!batch_ok(T, B, max_q) || n_kv < 1 || n_kv > kMaxHeads || n_q < n_kv || n_q > kMaxHeads || n_q % n_kv ||
      !hd_ok(hd) || max_kv < 1 || max_kv > kMaxKeys || window < 0 || sinks < 0 || (sinks > 0 && window == 0))
    return false;
  return (max_q * (n_q / n_kv) + 127) / 128 * n_kv <= 65535;  // a grid dimension
}

// Windows and first keys beyond any table are as good as that.
int64_t within_keys(int64_t x) { return x < kMaxI32 ? x : kMaxI32; }

bool lora_sizes_ok(int64_t T, int64_t K, int64_t rank, int64_t n_parts) {
  return T >= 0 && T <= kMaxTokens && qmm::k_ok(K) && n_parts >= 1 && n_parts <= 3 &&
         (rank == 8 || rank == 16 || rank == 32 || rank == 64 || rank == 128);
}

}  // namespace

extern "C" {

int qmm_kv8_append(const qmm_kv8_cache* cache, const void* k, const void* v, int64_t T, int in_dtype,
                   const int32_t* q_start, const int32_t* kv_lens, const int32_t* page_table, int64_t B,
                   int64_t max_pages, int64_t max_q, const int32_t* positions, const float* cos_sin,
                   int64_t max_pos, int64_t rot_dim, const void* q, int64_t n_q_heads, uint16_t* q_out,
                   uint16_t* k_held, uint16_t* v_held, hipStream_t stream) {
  qmm::Kv8AppendArgs a = {};
  if (int st = check_cache(cache, &a.c)) return st;
  if (!k || !v || !kv_lens || !page_table || (!cos_sin && (q || positions)) || (q && !q_out)) return QMM_ERR_NULL;
  if (!type_ok(in_dtype)) return QMM_ERR_ENUM;
  const int64_t hd = cache->head_dim, n_kv = cache->n_kv_heads;
  if (!batch_ok(T, B, max_q) || (!q_start && (T != B || max_q != 1)) || B * (max_q / 16 + 2) > kMaxBlocks ||
      max_pages < 1 || max_pages > kMaxKeys / cache->page_size || (q && (n_q_heads < 1 || n_q_heads > kMaxHeads)) ||
      (cos_sin && (rot_dim < 2 || rot_dim % 2 || rot_dim > hd || max_pos < 1 || max_pos > kMaxI32)))
    return QMM_ERR_SHAPE;
  if (!qmm::aligned(k, 16) || !qmm::aligned(v, 16) || !qmm::aligned(q_start, 4) || !qmm::aligned(kv_lens, 4) ||
      !qmm::aligned(page_table, 4) || !qmm::aligned(positions, 4) || !qmm::aligned(cos_sin, 4) ||
      !qmm::aligned(q, 16) || (q && !qmm::aligned(q_out, 16)) || !qmm::aligned(k_held, 16) ||
      !qmm::aligned(v_held, 16))
    return QMM_ERR_ALIGN;
  const size_t e = type_bytes(in_dtype);
  const uint64_t kvn = uint64_t(T * n_kv * hd), qn = q ? uint64_t(T * n_q_heads * hd) : 0;
  const CacheBytes cb = cache_bytes(*cache);
  const Range outs[] = {{cache->k_codes, cb.codes}, {cache->v_codes, cb.codes}, {cache->k_scale, cb.scales},
                        {cache->v_scale, cb.scales}, {q ? q_out : nullptr, qn * 2},
                        {k_held, k_held ? kvn * 2 : 0}, {v_held, v_held ? kvn * 2 : 0}};
  const Range ins[] = {{k, kvn * e}, {v, kvn * e}, {q, qn * e}, {q_start, q_start ? uint64_t(B + 1) * 4 : 0},
                       {kv_lens, uint64_t(B) * 4}, {page_table, uint64_t(B) * uint64_t(max_pages) * 4},
                       {positions, positions ? uint64_t(T) * 4 : 0},
                       {cos_sin, cos_sin ? uint64_t(max_pos) * uint64_t(rot_dim) * 4 : 0}};
  if (qmm::any_alias(outs, 7, ins, 8)) return QMM_ERR_ALIAS;
  if (T == 0) return QMM_OK;
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.table = page_table;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_out = q_out;
  a.k_held = k_held;
  a.v_held = v_held;
  a.T = T;
  a.B = int32_t(B);
  a.max_pages = int32_t(max_pages);
  a.max_q = int32_t(max_q);
  a.max_pos = cos_sin ? int32_t(max_pos) : 0;
  a.rot = cos_sin ? int32_t(rot_dim) : 0;
  a.n_q = q ? int32_t(n_q_heads) : 0;
  a.f32_in = in_dtype == QMM_OUT_F32;
  return qmm::launch_kv8_append(a, stream);
}

size_t qmm_kv8_attn_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t n_q_heads, int64_t n_kv_heads,
                                    int64_t head_dim, int64_t max_kv, int64_t window, int64_t sinks) {
  if (!attn_sizes_ok(T, B, max_q, n_q_heads, n_kv_heads, head_dim, max_kv, window, sinks)) return 0;
  return size_t(qmm::kv8_attn_workspace(T, B, max_q, n_q_heads, n_kv_heads, head_dim, max_kv, within_keys(window),
                                        within_keys(sinks)));
}

int qmm_kv8_attn(const uint16_t* q, int64_t T, const int32_t* q_start, const int32_t* kv_lens,
                 const int32_t* page_table, int64_t B, int64_t max_pages, int64_t max_q,
                 const qmm_kv8_cache* cache, int64_t n_q_heads, float scale, int causal, int64_t window,
                 int64_t sinks, const uint16_t* gate, void* workspace, size_t workspace_bytes, uint16_t* out,
                 hipStream_t stream) {
  qmm::Kv8AttnArgs a = {};
  if (int st = check_cache(cache, &a.c)) return st;
  if (!q || !kv_lens || !page_table || !workspace || !out) return QMM_ERR_NULL;
  if (causal != 0 && causal != 1) return QMM_ERR_ENUM;
  const int64_t hd = cache->head_dim;
  if (max_pages < 1 || max_pages > kMaxKeys / cache->page_size ||
      !attn_sizes_ok(T, B, max_q, n_q_heads, cache->n_kv_heads, hd, max_pages * cache->page_size, window, sinks) ||
      (!q_start && (T != B || max_q != 1)) || (window > 0 && !causal) || !(scale > 0.f) || !std::isfinite(scale))
    return QMM_ERR_SHAPE;
  window = within_keys(window), sinks = within_keys(sinks);
  const uint64_t need = qmm::kv8_attn_workspace(T, B, max_q, n_q_heads, cache->n_kv_heads, hd,
                                                max_pages * cache->page_size, window, sinks);
  if (workspace_bytes < need) return QMM_ERR_SHAPE;
  if (!qmm::aligned(q, 16) || !qmm::aligned(out, 16) || !qmm::aligned(gate, 16) || !qmm::aligned(workspace, 256) ||
      !qmm::aligned(q_start, 4) || !qmm::aligned(kv_lens, 4) || !qmm::aligned(page_table, 4))
    return QMM_ERR_ALIGN;
  const uint64_t qn = uint64_t(T * n_q_heads * hd) * 2;
  const CacheBytes cb = cache_bytes(*cache);
  const Range outs[] = {{out, qn}, {workspace, need}};
  const Range ins[] = {{q, qn}, {gate, gate ? qn : 0}, {q_start, q_start ? uint64_t(B + 1) * 4 : 0},
                       {kv_lens, uint64_t(B) * 4}, {page_table, uint64_t(B) * uint64_t(max_pages) * 4},
                       {cache->k_codes, cb.codes}, {cache->v_codes, cb.codes}, {cache->k_scale, cb.scales},
                       {cache->v_scale, cb.scales}};
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
  a.sinks = sinks;
  a.B = int32_t(B);
  a.max_pages = int32_t(max_pages);
  a.max_q = int32_t(max_q);
  a.n_q = int32_t(n_q_heads);
  a.causal = causal;
  a.scale = scale;
  return qmm::launch_kv8_attn(a, stream);
}

size_t qmm_spec_verify_workspace_bytes(int64_t B, int64_t V) {
  if (B < 1 || B > kMaxSeqs || V < 1 || V > kMaxTokens) return 0;
  return size_t(qmm::verify_workspace(B, V));
}

int qmm_spec_verify(const int32_t* draft, int64_t D, const int32_t* draft_start, int64_t B, int64_t max_draft,
                    const void* target, const void* draft_probs, int64_t V, int prob_dtype, const float* u,
                    int32_t* tokens, int32_t* accepted, void* workspace, size_t workspace_bytes,
                    hipStream_t stream) {
  if ((!draft && D != 0) || !draft_start || !target || !u || !tokens || !accepted || !workspace) return QMM_ERR_NULL;
  if (!type_ok(prob_dtype)) return QMM_ERR_ENUM;
  if (B < 1 || B > kMaxSeqs || V < 1 || V > kMaxTokens || D < 0 || D > kMaxTokens || max_draft < 0 ||
      max_draft > 65535)
    return QMM_ERR_SHAPE;
  const uint64_t need = qmm::verify_workspace(B, V), e = type_bytes(prob_dtype);
  if (workspace_bytes < need) return QMM_ERR_SHAPE;
  if (!qmm::aligned(draft, 4) || !qmm::aligned(draft_start, 4) || !qmm::aligned(target, e) ||
      !qmm::aligned(draft_probs, e) || !qmm::aligned(u, 4) || !qmm::aligned(tokens, 4) ||
      !qmm::aligned(accepted, 4) || !qmm::aligned(workspace, 256))
    return QMM_ERR_ALIGN;
  const Range outs[] = {{tokens, uint64_t(B) * uint64_t(max_draft + 1) * 4}, {accepted, uint64_t(B) * 4},
                        {workspace, need}};
  const Range ins[] = {{draft, uint64_t(D) * 4}, {draft_start, uint64_t(B + 1) * 4},
                       {target, uint64_t(D + B) * uint64_t(V) * e},
                       {draft_probs, draft_probs ? uint64_t(D) * uint64_t(V) * e : 0}, {u, uint64_t(D + B) * 4}};
  if (qmm::any_alias(outs, 3, ins, 5)) return QMM_ERR_ALIAS;
  qmm::VerifyArgs a = {};
  a.draft = draft;
  a.start = draft_start;
  a.p = target;
  a.q = draft_probs;
  a.u = u;
  a.tokens = tokens;
  a.accepted = accepted;
  a.ws = static_cast<double*>(workspace);
  a.D = D;
  a.V = V;
  a.B = int32_t(B);
  a.max_draft = int32_t(max_draft);
  a.f32 = prob_dtype == QMM_OUT_F32;
  return qmm::launch_verify(a, stream);
}

size_t qmm_lora_workspace_bytes(int64_t T, int64_t K, int64_t rank, int64_t n_parts) {
  if (!lora_sizes_ok(T, K, rank, n_parts)) return 0;
  return size_t(qmm::lora_workspace(T, K, rank, n_parts));
}

int qmm_lora(const uint16_t* x, int64_t T, int64_t K, const uint16_t* a, const uint16_t* b, int64_t n_adapters,
             int64_t rank, const int32_t* ids, const float* scales, int64_t n_parts, const int64_t* part_rows,
             const void* const* base, int base_dtype, void* const* y, int out_dtype, void* workspace,
             size_t workspace_bytes, hipStream_t stream) {
  if (!x || !a || !b || !ids || !part_rows || !y || !workspace) return QMM_ERR_NULL;
  if (!type_ok(out_dtype) || (base && !type_ok(base_dtype))) return QMM_ERR_ENUM;
  if (!lora_sizes_ok(T, K, rank, n_parts) || n_adapters < 1 || n_adapters > 65535) return QMM_ERR_SHAPE;
  const uint64_t need = qmm::lora_workspace(T, K, rank, n_parts);
  if (workspace_bytes < need) return QMM_ERR_SHAPE;
  if (!qmm::aligned(x, 16) || !qmm::aligned(a, 16) || !qmm::aligned(b, 16) || !qmm::aligned(ids, 4) ||
      !qmm::aligned(scales, 4) || !qmm::aligned(workspace, 256))
    return QMM_ERR_ALIGN;
  qmm::LoraArgs g = {};
  Range outs[4] = {{workspace, need}};
  Range ins[8] = {};
  int64_t rows = 0;
  for (int64_t p = 0; p < n_parts; ++p) {
    if (!y[p] || (base && !base[p])) return QMM_ERR_NULL;
    if (part_rows[p] < 1 || part_rows[p] > kMaxTokens) return QMM_ERR_SHAPE;
    rows += part_rows[p];
    const void* from = base ? base[p] : y[p];
    const size_t bt = type_bytes(base ? base_dtype : out_dtype), ot = type_bytes(out_dtype);
    if (!qmm::aligned(from, bt) || !qmm::aligned(y[p], ot)) return QMM_ERR_ALIGN;
    const uint64_t n = uint64_t(T) * uint64_t(part_rows[p]);
    const bool in_place = from == y[p] && bt == ot;
    outs[1 + p] = {y[p], n * ot};
    ins[5 + p] = {in_place ? nullptr : from, n * bt};
    g.base[p] = from;
    g.y[p] = y[p];
    g.rows[p] = int32_t(part_rows[p]);
  }
  if (rows > kMaxTokens || !qmm::lora_launches(T, g.rows)) return QMM_ERR_SHAPE;
  const uint64_t ra = uint64_t(n_adapters) * uint64_t(rank) * 2;
  ins[0] = {x, uint64_t(T) * uint64_t(K) * 2};
  ins[1] = {a, ra * uint64_t(n_parts) * uint64_t(K)};
  ins[2] = {b, ra * uint64_t(rows)};
  ins[3] = {ids, uint64_t(T) * 4};
  ins[4] = {scales, scales ? uint64_t(n_adapters) * 4 : 0};
  if (qmm::any_alias(outs, 4, ins, 8)) return QMM_ERR_ALIAS;
  if (T == 0) return QMM_OK;
  g.x = x;
  g.a = a;
  g.b = b;
  g.ids = ids;
  g.scales = scales;
  g.ws = static_cast<float*>(workspace);
  g.T = T;
  g.K = int32_t(K);
  g.rank = int32_t(rank);
  g.n_parts = int32_t(n_parts);
  g.n_adapters = int32_t(n_adapters);
  g.base_f32 = (base ? base_dtype : out_dtype) == QMM_OUT_F32;
  g.out_f32 = out_dtype == QMM_OUT_F32;
  return qmm::launch_lora(g, stream);
}

}  // extern "C"
