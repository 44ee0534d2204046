// What the attention kernels over the paged 4-bit cache share: a sequence's place in the
// call, the keys that a block's rows can see, their split over blocks, and the store.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "mix_internal.h"
#include "qmm_device.h"

namespace qmm {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <int N, class F, int I = 0>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, F, I + 1>(static_cast<F&&>(f));
  }
}

// x of lane LN of the lane's row of 16 (DPP row_newbcast).
template <int LN>
__device__ __forceinline__ float row_bcast(float x) {
  return __uint_as_float(
      uint32_t(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(x)), 0x150 + LN, 0xf, 0xf, true)));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

struct AttnSeq {
  int q0, q_len, kv_len;
  int first;  // position of query 0 (negative where there are more queries than keys)
};
// Sequence b: its rows of q (held inside [0, T] whatever q_start says) and its keys.
__device__ __forceinline__ AttnSeq attn_seq(const Kv4AttnArgs& g, int b) {
  AttnSeq s;
  int64_t a = b, e = int64_t(b) + 1;
  if (g.q_start) {
    a = g.q_start[b], e = g.q_start[b + 1];
    a = a < 0 ? 0 : a > g.T ? g.T : a;
    e = e < a ? a : e > g.T ? g.T : e;
  }
  s.q0 = int(a);
  s.q_len = int(e - a) < g.max_q ? int(e - a) : g.max_q;
  const int64_t most = int64_t(g.max_pages) << g.c.page_shift;
  const int64_t n = g.kv_lens[b];
  s.kv_len = int(n < 0 ? 0 : n > most ? most : n);
  s.first = s.kv_len - int(e - a);
  return s;
}

struct AttnSpan {
  int lo, hi;  // in tiles of 32 keys
};
// Keys that queries j0 .. j1 of a sequence can see.
__device__ __forceinline__ AttnSpan attn_span(const Kv4AttnArgs& g, const AttnSeq& s, int j0, int j1) {
  int64_t lo = 0, hi = s.kv_len;
  if (g.causal) {
    const int64_t p0 = s.first;
    hi = p0 + j1 + 1;
    if (g.window > 0 && p0 + j0 - g.window + 1 > 0) lo = p0 + j0 - g.window + 1;
  }
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  return {int(lo >> 5), int((hi + 31) >> 5)};
}

constexpr int kSplitKeys = 128;  // a split has at least this many keys
struct AttnSplit {
  int count, begin, end;  // splits of the span; this split's tiles
};
__device__ __forceinline__ AttnSplit attn_split(const AttnSpan& sp, int nsplit_max, int split) {
  const int tiles = sp.hi - sp.lo;
  int c = (tiles * 32 + kSplitKeys - 1) / kSplitKeys;
  c = c > nsplit_max ? nsplit_max : c < 1 ? 1 : c;
  const int per = (tiles + c - 1) / c;
  if (per > 0) c = (tiles + per - 1) / per;
  AttnSplit r;
  r.count = c < 1 ? 1 : c;
  r.begin = sp.lo + split * per;
  r.end = r.begin + per < sp.hi ? r.begin + per : sp.hi;
  return r;
}
int attn_nsplit(int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t max_kv);
int launch_kv4_decode(const Kv4AttnArgs& a, hipStream_t s);

// Four neighbouring outputs: the weighted sum over its weight, times the gate's sigmoid.
__device__ __forceinline__ void attn_store4(const Kv4AttnArgs& g, int64_t at, float4 o, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (g.gate) {
    const uint2 w = *reinterpret_cast<const uint2*>(g.gate + at);
    const float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= __builtin_amdgcn_rcpf(1.f + exp2_hw(-1.4426950408889634f * x[i]));
  }
  *reinterpret_cast<uint2*>(g.out + at) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

}  // namespace qmm
