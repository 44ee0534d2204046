// Host-side launch interface between the token mixers' C ABI (qmm_mix_api.cpp) and their
// kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace qmm {

// The paged 4-bit cache as the kernels take it (layout: include/qmm_mix.h).
struct Kv4 {
  uint32_t* k_codes;
  uint32_t* k_meta;
  uint16_t* v_codes;
  uint32_t* v_meta;
  int32_t n_pages, page_shift, n_kv, hd;
};

struct Kv4AppendArgs {
  Kv4 c;
  const void* k;
  const void* v;
  const void* q;  // nullable
  const int32_t* slots;
  const int32_t* positions;
  const float* cos_sin;  // nullable: no rotation
  uint16_t* q_out;
  uint16_t* k_held;  // nullable
  uint16_t* v_held;  // nullable
  int64_t T;
  int32_t max_pos, rot, n_q, f32_in;
};
int launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s);

struct Kv4AttnArgs {
  Kv4 c;
  const uint16_t* q;
  const int32_t* q_start;  // nullable: one query a sequence
  const int32_t* kv_lens;
  const int32_t* table;
  const uint16_t* gate;  // nullable
  uint16_t* out;
  void* ws;
  int64_t T, window;
  int32_t B, max_pages, max_q, n_q, causal;
  float scale;
};
// (Query, head) rows of a block, of a call with `rows` of them per sequence and KV head.
int64_t kv4_attn_rows(int64_t rows, int64_t hd);
// Bytes of workspace of a call's launch shape.
uint64_t kv4_attn_workspace(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd,
                            int64_t max_kv);
int launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s);

struct GdnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* g;
  const float* beta;
  const int32_t* seq_start;  // nullable: one token a sequence
  const float* state_in;
  float* state_out;
  const int32_t* slots;  // nullable: slot b
  void* y;
  void* ws;
  int64_t T;
  int32_t B, max_len, Hk, Hv, n_slots, l2norm, f32_out, Dk, Dv;
  float scale;
};
// Whether a launch can hold a call's threads (2^32 along a grid's dimension).
bool gdn_launches(int64_t B, int64_t max_len, int64_t Hv, int64_t Dv);
uint64_t gdn_workspace(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv);
int launch_gdn(const GdnArgs& a, hipStream_t s);

}  // namespace qmm
