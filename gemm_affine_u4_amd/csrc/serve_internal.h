// Host-side launch interface between the serving step's C ABI (qmm_serve_api.cpp) and its
// kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace qmm {

// The paged 8-bit cache as the kernels take it (layout: include/qmm_serve.h).
struct Kv8 {
  int8_t* k_codes;
  float* k_scale;
  int8_t* v_codes;
  float* v_scale;
  int32_t n_pages, page_shift, n_kv, hd;
};

struct Kv8AppendArgs {
  Kv8 c;
  const void* k;
  const void* v;
  const void* q;  // nullable
  const int32_t* q_start;  // nullable: one token a sequence
  const int32_t* kv_lens;
  const int32_t* table;
  const int32_t* positions;  // nullable: the key's place
  const float* cos_sin;      // nullable: no rotation
  uint16_t* q_out;
  uint16_t* k_held;  // nullable
  uint16_t* v_held;  // nullable
  int64_t T;
  int32_t B, max_pages, max_q, max_pos, rot, n_q, f32_in;
};
int launch_kv8_append(const Kv8AppendArgs& a, hipStream_t s);

struct Kv8AttnArgs {
  Kv8 c;
  const uint16_t* q;
  const int32_t* q_start;  // nullable: one query a sequence
  const int32_t* kv_lens;
  const int32_t* table;
  const uint16_t* gate;  // nullable
  uint16_t* out;
  void* ws;
  int64_t T, window, sinks;
  int32_t B, max_pages, max_q, n_q, causal;
  float scale;
};
uint64_t kv8_attn_workspace(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd,
                            int64_t max_kv, int64_t window, int64_t sinks);
int launch_kv8_attn(const Kv8AttnArgs& a, hipStream_t s);

struct VerifyArgs {
  const int32_t* draft;
  const int32_t* start;
  const void* p;
  const void* q;  // nullable: looked-up drafts
  const float* u;
  int32_t* tokens;
  int32_t* accepted;
  double* ws;
  int64_t D, V;
  int32_t B, max_draft, f32;
};
uint64_t verify_workspace(int64_t B, int64_t V);
int launch_verify(const VerifyArgs& a, hipStream_t s);

struct LoraArgs {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* ids;
  const float* scales;  // nullable: 1
  float* ws;
  const void* base[3];
  void* y[3];
  int32_t rows[3];  // 0: no such part
  int64_t T;
  int32_t K, rank, n_parts, n_adapters, base_f32, out_f32;
};
// Whether a launch can hold a call's threads (2^32 along a grid's dimension).
bool lora_launches(int64_t T, const int32_t (&rows)[3]);
uint64_t lora_workspace(int64_t T, int64_t K, int64_t rank, int64_t n_parts);
int launch_lora(const LoraArgs& a, hipStream_t s);

}  // namespace qmm
