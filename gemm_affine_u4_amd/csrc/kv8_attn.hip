// Attention over the paged 8-bit cache (qmm_kv8_attn; include/qmm_serve.h): a wave a query and head,
// 64 keys at a time with the running maximum and sum of the softmax.
#include <hip/hip_runtime.h>

#include "kv4_attn.h"
#include "qmm_device.h"
#include "qmm_internal.h"
#include "serve_internal.h"

namespace qmm {
namespace {

template <int HD>
__global__ __launch_bounds__(64) void kv8_attn_kernel(Kv8AttnArgs g, int group) {
  const int lane = threadIdx.x, b = blockIdx.z, head = blockIdx.y, kvh = head / group;
  const AttnSeq sq = attn_seq(g, b);
  const int j = blockIdx.x;
  if (j >= sq.q_len) return;
  const int64_t row = (int64_t(sq.q0) + j) * g.n_q + head;
  __shared__ float s_q[HD], s_p[64];
  for (int d = lane; d < HD; d += 64) s_q[d] = bf16_bits_to_f32(g.q[row * HD + d]);
  __syncthreads();
  int lo = 0, hi = sq.kv_len;
  if (g.causal) {
    const int64_t p = int64_t(sq.first) + j;
    hi = p < 0 ? 0 : int(p) + 1;
    if (g.window > 0 && p - g.window + 1 > 0) lo = int(p - g.window + 1);
  }
  const int32_t* table = g.table + int64_t(b) * g.max_pages;
  constexpr int V = HD / 64;
  float m = -1e30f, l = 0.f, o[V] = {};
  for (int t0 = 0; t0 < hi; t0 += 64) {
    if (t0 + 64 <= lo && t0 >= g.sinks) continue;
    const int t = t0 + lane, shift = g.c.page_shift;
    const int page = t < sq.kv_len ? table[t >> shift] : -1;
    const bool there = uint32_t(page) < uint32_t(g.c.n_pages);
    const int64_t slot = ((int64_t(there ? page : 0) * g.c.n_kv + kvh) << shift) + (t & ((1 << shift) - 1));
    float s = -INFINITY, vs = 0.f;
    if (there && t < hi && (t >= lo || t < g.sinks)) {
      float x = 0.f;
      for (int d = 0; d < HD; ++d) x = fmaf(s_q[d], float(g.c.k_codes[slot * HD + d]), x);
      s = x * g.c.k_scale[slot >> 4] * g.scale;
      vs = g.c.v_scale[slot >> 4];
    }
    float mn = s;
    for (int w = 32; w; w >>= 1) mn = fmaxf(mn, __shfl_xor(mn, w));
    mn = fmaxf(m, mn);
    const float f = expf(m - mn), p = s > -INFINITY ? expf(s - mn) : 0.f;
    float sum = p;
    for (int w = 32; w; w >>= 1) sum += __shfl_xor(sum, w);
    l = l * f + sum;
    m = mn;
    s_p[lane] = p * vs;
    __syncthreads();
    for (int i = 0; i < V; ++i) o[i] *= f;
    for (int k = 0; k < 64; ++k) {
      const int64_t at = __shfl(slot, k);
      const float w = s_p[k];
      if (w == 0.f) continue;
      for (int i = 0; i < V; ++i) o[i] = fmaf(w, float(g.c.v_codes[(at >> 3) * 8 * HD + (lane + 64 * i) * 8 + (at & 7)]), o[i]);
    }
    __syncthreads();
  }
  for (int i = 0; i < V; ++i) {
    const int64_t at = row * HD + lane + 64 * i;
    float v = l > 0.f ? o[i] / l : 0.f;
    if (g.gate) v /= 1.f + expf(-bf16_bits_to_f32(g.gate[at]));
    g.out[at] = f32_to_bf16_bits(v);
  }
}

}  // namespace

uint64_t kv8_attn_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
  return 256;
}

int launch_kv8_attn(const Kv8AttnArgs& a, hipStream_t s) {
  const dim3 grid(uint32_t(a.max_q), uint32_t(a.n_q), uint32_t(a.B));
  const int group = a.n_q / a.c.n_kv;
  if (a.c.hd == 64) kv8_attn_kernel<64><<<grid, 64, 0, s>>>(a, group);
  else if (a.c.hd == 128) kv8_attn_kernel<128><<<grid, 64, 0, s>>>(a, group);
  else kv8_attn_kernel<256><<<grid, 64, 0, s>>>(a, group);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace qmm
