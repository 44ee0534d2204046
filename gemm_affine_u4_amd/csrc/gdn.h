// What the gated delta rule's kernels share.
#pragma once
#include <hip/hip_runtime.h>

#include "kv4_device.h"
#include "mix_internal.h"
#include "qmm_device.h"

namespace qmm {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr float kGdnEps = 1e-6f;
// Calls of up to this max_len run token by token, longer ones in chunks.  Measured at 16 tokens
// against 17, 32 heads x 128: one sequence 11.8 against 12.7 us, 16 of them 43 against 58, 64 of
// them 132 against 210; at 24 one sequence would take 16 us by tokens.
constexpr int kGdnStepLen = 16;
uint64_t gdn_chunk_workspace(int64_t T, int64_t B, int64_t Hk, int64_t Hv, int64_t Dk);
int launch_gdn_chunk(const GdnArgs& a, hipStream_t s);

struct GdnSeq {
  int t0, len, slot;
};
// Sequence b: its tokens (held inside [0, T] whatever seq_start says) and its state's slot.
__device__ __forceinline__ GdnSeq gdn_seq(const GdnArgs& g, int b) {
  int64_t a = b, e = int64_t(b) + 1;
  if (g.seq_start) {
    a = g.seq_start[b], e = g.seq_start[b + 1];
    a = a < 0 ? 0 : a > g.T ? g.T : a;
    e = e < a ? a : e > g.T ? g.T : e;
  }
  GdnSeq s;
  s.t0 = int(a);
  s.len = int(e - a) < g.max_len ? int(e - a) : g.max_len;
  s.slot = g.slots ? g.slots[b] : b;
  return s;
}

// Sum over the lane's row of 16 (all of them active).
__device__ __forceinline__ float sum16_lanes(float x) {
  x += dpp_mov<kQuadXor1>(x);
  x += dpp_mov<kQuadXor2>(x);
  x += dpp_mov<kHalfMirror>(x);
  return x + dpp_mov<kRowMirror>(x);
}

__device__ __forceinline__ void gdn_store(const GdnArgs& g, int64_t at, float y) {
  if (g.f32_out) static_cast<float*>(g.y)[at] = y;
  else static_cast<uint16_t*>(g.y)[at] = f32_to_bf16_bits(y);
}

}  // namespace qmm
