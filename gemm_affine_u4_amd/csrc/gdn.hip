// The gated delta rule token by token (qmm_gdn's serving form; see include/qmm_mix.h).
//
// Mathematics, per value head with the state's row S[v][:] over the Dk key dims:
//   S <- e^g S;  d = beta (v - S.k);  S <- S + d k;  y = S.q  =  (e^g S).q + d (k.q),
// so both products of a row are taken before its update and meet in one reduction.
// Bound: HBM for a batch's single tokens (the state is read and written once), latency for
// one sequence.
// Split: rows of the state are independent given k and q, so a wave takes 4 rows at a time,
// 16 lanes to a row (each lane 8 of 128 dims, in two 16-byte pieces), RR times over in
// registers: RR = 4 for a batch (8 KB of state in flight per wave), 1 where the call would
// otherwise leave compute units idle.  The dims of a row meet by DPP.
//
// Measured: one token of 32 heads x 128 x 128: 3.6 us (launch); 96 tokens of as many sequences of
// 48 heads: 109 us, 5.6 TB/s of state.
#include <hip/hip_runtime.h>

#include "gdn.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

// A batch's state is read and written past the caches, which it would only sweep
// (96 states of 48 heads x 128 x 128, 604 MB in and out: 119 -> 109 us); one sequence's stays in them.
template <int RR>
__device__ __forceinline__ f32x4_t load_state(const float* p) {
  const f32x4_t* at = reinterpret_cast<const f32x4_t*>(p);
  if constexpr (RR > 1) return __builtin_nontemporal_load(at);
  else return *at;
}
template <int RR>
__device__ __forceinline__ void store_state(float* p, f32x4_t x) {
  f32x4_t* at = reinterpret_cast<f32x4_t*>(p);
  if constexpr (RR > 1) __builtin_nontemporal_store(x, at);
  else *at = x;
}

template <int DK, int RR>
__global__ __launch_bounds__(256) void gdn_step_kernel(GdnArgs g) {
  constexpr int P = DK / 64;  // 16-byte pieces of a lane
  const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15;
  const int hv = blockIdx.y, b = blockIdx.z, hk = hv / (g.Hv / g.Hk);
  const int r0 = int(blockIdx.x) * 16 * RR + (tid >> 6) * 4 * RR + (lane >> 4);  // + 4 rr
  const GdnSeq sq = gdn_seq(g, b);
  const bool kept = uint32_t(sq.slot) < uint32_t(g.n_slots);
  if (sq.len == 0 && (!kept || g.state_in == g.state_out)) return;

  const int64_t base = ((int64_t(kept ? sq.slot : 0) * g.Hv + hv) * g.Dv + r0) * DK + i16 * 4;
  f32x4_t s[RR][P];
#pragma unroll
  for (int r = 0; r < RR; ++r) {
#pragma unroll
    for (int p = 0; p < P; ++p)
      s[r][p] = kept ? load_state<RR>(g.state_in + base + int64_t(4 * r) * DK + 64 * p) : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  for (int t = 0; t < sq.len; ++t) {
    const int64_t tok = int64_t(sq.t0) + t;
    float k[P][4], q[P][4];
    const uint16_t* kp = g.k + (tok * g.Hk + hk) * DK + i16 * 4;
    const uint16_t* qp = g.q + (tok * g.Hk + hk) * DK + i16 * 4;
    float v[RR];
#pragma unroll
    for (int r = 0; r < RR; ++r) v[r] = bf16_bits_to_f32(g.v[(tok * g.Hv + hv) * g.Dv + r0 + 4 * r]);
    const float decay = expf(g.g[tok * g.Hv + hv]), beta = g.beta[tok * g.Hv + hv];
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint2 a = *reinterpret_cast<const uint2*>(kp + 64 * p), c = *reinterpret_cast<const uint2*>(qp + 64 * p);
      k[p][0] = bf16_lo(a.x), k[p][1] = bf16_hi(a.x), k[p][2] = bf16_lo(a.y), k[p][3] = bf16_hi(a.y);
      q[p][0] = bf16_lo(c.x), q[p][1] = bf16_hi(c.x), q[p][2] = bf16_lo(c.y), q[p][3] = bf16_hi(c.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kk = fmaf(k[p][i], k[p][i], kk);
        qq = fmaf(q[p][i], q[p][i], qq);
        kq = fmaf(k[p][i], q[p][i], kq);
      }
    }
    float rk = 1.f, rq = g.scale;
    if (g.l2norm) {
      rk = 1.f / sqrtf(sum16_lanes(kk) + kGdnEps);
      rq *= 1.f / sqrtf(sum16_lanes(qq) + kGdnEps);
    }
    kq = sum16_lanes(kq) * rk * rq;
#pragma unroll
    for (int r = 0; r < RR; ++r) {
      float dk = 0.f, dq = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[r][p][i] *= decay;
          dk = fmaf(s[r][p][i], k[p][i], dk);
          dq = fmaf(s[r][p][i], q[p][i], dq);
        }
      }
      dk = sum16_lanes(dk) * rk;
      dq = sum16_lanes(dq) * rq;
      const float d = (v[r] - dk) * beta, dr = d * rk;
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[r][p][i] = fmaf(dr, k[p][i], s[r][p][i]);
      }
      if (i16 == 0) gdn_store(g, (tok * g.Hv + hv) * g.Dv + r0 + 4 * r, fmaf(d, kq, dq));
    }
  }
  if (kept) {
#pragma unroll
    for (int r = 0; r < RR; ++r) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        store_state<RR>(g.state_out + base + int64_t(4 * r) * DK + 64 * p, s[r][p]);
    }
  }
}

template <int DK>
int launch_step(const GdnArgs& a, hipStream_t s) {
  // 64 rows per block where that still gives every compute unit two blocks
  if (int64_t(a.B) * a.Hv * (a.Dv / 64) >= 2 * int64_t(device_cus()))
    gdn_step_kernel<DK, 4><<<dim3(uint32_t(a.Dv / 64), uint32_t(a.Hv), uint32_t(a.B)), 256, 0, s>>>(a);
  else
    gdn_step_kernel<DK, 1><<<dim3(uint32_t(a.Dv / 16), uint32_t(a.Hv), uint32_t(a.B)), 256, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

bool gdn_launches(int64_t B, int64_t max_len, int64_t Hv, int64_t Dv) {
  return max_len <= kGdnStepLen || (B * Hv + 7) / 8 * 8 * (Dv / 32) * 512 < (int64_t(1) << 32);  // the walk's grid
}

uint64_t gdn_workspace(int64_t T, int64_t B, int64_t max_len, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv) {
  return max_len <= kGdnStepLen ? 256 : gdn_chunk_workspace(T, B, Hk, Hv, Dk);
}

int launch_gdn(const GdnArgs& a, hipStream_t s) {
  if (a.max_len > kGdnStepLen) return launch_gdn_chunk(a, s);
  return a.Dk == 64 ? launch_step<64>(a, s) : launch_step<128>(a, s);
}

}  // namespace qmm
