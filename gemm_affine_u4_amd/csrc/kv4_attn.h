// What the attention kernels over the paged caches share (the split and the plan: 4 bits only): a sequence's place in the
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
template <class Args>
__device__ __forceinline__ AttnSeq attn_seq(const Args& g, int b) {
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

// The sequence of rank b by falling number of keys (b becomes its index), up to 64 of them, one a
// lane.  Blocks start in that order, so that the last ones to end are short: 64 single tokens on
// 100 to 16000 keys 134 -> 126 us, five prompts on 2480 to 6695 keys 458 -> 400.  It costs a block
// ~1.5 us at 64 sequences, so tables of up to 2048 keys keep the order given (64 single tokens on
// 500 keys each 12 us, ordered 14).  More than 64 run in the order given, and do not even out by
// themselves: 66 such tokens in any order 133 us, given longest first 114; 200 of them 362 and 296.
template <class Args>
__device__ __forceinline__ AttnSeq attn_longest_first(const Args& g, int& b, int lane) {
  const int n = int(gridDim.z);
  if (n == 1 || n > 64 || (int64_t(g.max_pages) << g.c.page_shift) <= 2048) return attn_seq(g, b);
  const AttnSeq s = attn_seq(g, lane < n ? lane : 0);
  // one number for length and place, all different (lengths from 2^25 on count as that)
  const uint32_t len = uint32_t(s.kv_len < (1 << 25) ? s.kv_len : (1 << 25) - 1);
  const uint32_t key = lane < n ? len << 6 | uint32_t(63 - lane) : 0u;
  int before = lane < n ? 0 : 64;
  for (int j = 0; j < n; j += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) before += uint32_t(__builtin_amdgcn_readlane(int(key), j + k)) > key;
  }
  b = __ffsll(static_cast<unsigned long long>(__ballot(before == b))) - 1;
  return {__builtin_amdgcn_readlane(s.q0, b), __builtin_amdgcn_readlane(s.q_len, b),
          __builtin_amdgcn_readlane(s.kv_len, b), __builtin_amdgcn_readlane(s.first, b)};
}

// How a call is cut: a function of its sizes alone (host), the same for its workspace.
struct AttnPlan {
  int rows;     // (query, head) rows of a block: 16 (kv4_decode.hip) or kAttnRows (kv4_prefill.hip)
  int waves;    // of a block
  int shift;    // log2 of the keys of a tile
  int nsplit;   // at most this many splits of a block's keys ...
  int keys;     // ... of at least this many keys
};
constexpr int kAttnRows = 128;
AttnPlan attn_plan(int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv);

struct AttnSplit {
  int count, begin, end;  // splits of the block's keys; this split's tiles
};
// The tiles of keys that rows row0 .. row0 + rows - 1 of a sequence can see, cut evenly.
__device__ __forceinline__ AttnSplit attn_split(const Kv4AttnArgs& g, const AttnSeq& s, int row0, int rows, int group,
                                                const AttnPlan& p, int split) {
  int64_t lo = 0, hi = s.kv_len;
  if (g.causal) {
    hi = int64_t(s.first) + (row0 + rows - 1) / group + 1;
    const int64_t w = int64_t(s.first) + row0 / group - g.window + 1;
    if (g.window > 0 && w > 0) lo = w;
  }
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  const int t0 = int(lo >> p.shift), t1 = int((hi + (1 << p.shift) - 1) >> p.shift), tiles = t1 - t0;
  const int least = p.keys >> p.shift;
  int c = (tiles + least - 1) / least;
  c = c > p.nsplit ? p.nsplit : c < 1 ? 1 : c;
  const int per = (tiles + c - 1) / c;
  AttnSplit r;
  r.count = per > 0 ? (tiles + per - 1) / per : 1;
  r.begin = t0 + split * per;
  r.end = r.begin + per < t1 ? r.begin + per : t1;
  return r;
}
int launch_kv4_decode(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s);
int launch_kv4_prefill(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s);
int launch_kv4_join(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s);

// Four neighbouring outputs: the weighted sum over its weight, times the gate's sigmoid.
template <class Args>
__device__ __forceinline__ void attn_store4(const Args& g, int64_t at, float4 o, float l) {
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
