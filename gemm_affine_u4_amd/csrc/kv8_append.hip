// Keys and values of new tokens into the paged 8-bit cache, rotated on the way
// (qmm_kv8_append; layout and arithmetic: include/qmm_serve.h).
//
// Mathematics: per block of 16 keys and head one scale, as qmm_serve.h gives it.  Every fp32
// operation is rounded by itself (no contraction), so codes and scales are functions of the
// inputs that a caller can reproduce bit for bit.
// Bound: HBM (the inputs once, q_out, held values, a byte per cached value), and the launch
// and two round trips to memory for a decode batch.
// Split: a wave takes one block of 16 keys of one head at a time (an item: a query, key or value
// head), with all its values in registers between the largest magnitude and the codes.  For queries
// and keys hd/8 lanes share a token, each with the 4 + 4 dims of four rotation pairs, so that a
// pair needs one load of each value and of its angle; a wave's items follow each other over the
// heads, and the angles stay in registers.  For values a lane holds two dims of eight neighbouring
// keys, which are its 16 bytes of codes.
#include <hip/hip_runtime.h>

#include "kv4_attn.h"
#include "qmm_device.h"
#include "qmm_internal.h"
#include "serve_internal.h"

namespace qmm {
namespace {

constexpr int kBlock = 16;  // keys that share a scale
constexpr float kLimit = 57344.0f;

template <bool F32>
__device__ __forceinline__ void load4(const void* p, int64_t at, float* x) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  }
}
template <bool F32>
__device__ __forceinline__ void load2(const void* p, int64_t at, float* x) {
  if constexpr (F32) {
    const float2 a = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
    x[0] = a.x, x[1] = a.y;
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + at);
    x[0] = bf16_lo(w), x[1] = bf16_hi(w);
  }
}
template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void store4_bf16(uint16_t* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}

__device__ __forceinline__ float clamped(float x) { return fminf(fmaxf(x, -kLimit), kLimit); }
__device__ __forceinline__ float max_wave(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}

// A block's scale: `most` the new keys' largest magnitude, `old` its scale so far (0 where it begins).
struct Scale {
  float s, inv, ratio;  // ratio: of the earlier keys' codes, 1 where they stay
};
__device__ __forceinline__ Scale block_scale(float most, float old, bool begins) {
#pragma clang fp contract(off)
  const float need = most * (1.0f / 127.0f);
  Scale r;
  r.s = begins ? need : need <= old ? old : fmaxf(need, old * 1.25f);
  r.ratio = !begins && r.s != old ? old / r.s : 1.f;
  r.inv = r.s > 0.f ? 1.0f / r.s : 0.f;
  return r;
}
__device__ __forceinline__ float code_of(float x, float inv) {
#pragma clang fp contract(off)
  return fminf(fmaxf(__builtin_rintf(x * inv), -127.f), 127.f);
}
__device__ __forceinline__ uint32_t byte_of(float c) { return uint32_t(int(c)) & 255u; }
__device__ __forceinline__ uint32_t recode(uint32_t byte, float ratio) {
#pragma clang fp contract(off)
  return byte_of(__builtin_rintf(float(int8_t(byte)) * ratio));
}

// VEC: rot a multiple of 8, a lane's dims are two runs of 4 that pair up; otherwise 8 neighbours.
template <int HD, bool F32, bool VEC>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8AppendArgs g, int blocks, int groups, int per_wave) {
  constexpr int LPT = HD / 8, PPT = 64 / LPT, PASSES = kBlock / PPT;  // lanes of a token, tokens of a pass
  const int lane = threadIdx.x & 63;
  const int64_t wid = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = wid / groups;  // (sequence, block)
  const int b = int(unit / blocks);
  if (b >= g.B) return;
  const AttnSeq sq = attn_seq(g, b);
  const int64_t k0 = ((int64_t(sq.first) >> 4) + unit % blocks) * kBlock;  // the block's first key (it may lie below 0)
  const int64_t end = int64_t(sq.first) + sq.q_len;
  const int lo = int(sq.first > k0 ? sq.first - k0 : 0), hi = int(end < k0 + kBlock ? end - k0 : kBlock);
  if (lo >= hi) return;
  const int64_t row0 = sq.q0 + (k0 - sq.first);  // token row of place 0 of the block
  const int items = g.n_q + 2 * g.c.n_kv, u0 = int(wid % groups) * per_wave;
  const int u1 = u0 + per_wave < items ? u0 + per_wave : items;

  // keys below 0 do not occur in a block that starts at 0 or later
  int page = -1;
  if (k0 >= 0) page = g.table[int64_t(b) * g.max_pages + (k0 >> g.c.page_shift)];
  const bool kept = uint32_t(page) < uint32_t(g.c.n_pages);
  const int place0 = int(k0 & ((1 << g.c.page_shift) - 1));

  const int li = lane % LPT, sub = lane / LPT;
  const int half = g.rot >> 1, pairs = g.rot >> 3;
  const bool paired = VEC && li < pairs;
  const int da = !VEC ? 8 * li : paired ? 4 * li : g.rot + 8 * (li - pairs);
  const int db = paired ? half + 4 * li : da + 4;

  // angles of the lane's pairs, for each pass's token (keys and queries)
  float c[PASSES][VEC ? 4 : 1], s[PASSES][VEC ? 4 : 1];
  int64_t angle[PASSES];
  if (u0 < g.n_q + g.c.n_kv && g.rot) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int i = p * PPT + sub;
      angle[p] = 0;
      if (i < lo || i >= hi) continue;
      int64_t pos = g.positions ? g.positions[row0 + i] : k0 + i;
      pos = pos < 0 ? 0 : pos >= g.max_pos ? g.max_pos - 1 : pos;
      angle[p] = pos * g.rot;
      if constexpr (VEC) {
        if (paired) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[p][e] = g.cos_sin[angle[p] + 4 * li + e];
            s[p][e] = g.cos_sin[angle[p] + half + 4 * li + e];
          }
        }
      }
    }
  }
  // a pass's token of a head, rotated: the lane's dims da .. da + 3, db .. db + 3
  auto turned = [&](const void* src, int64_t at, int p, float (&x)[8]) {
#pragma clang fp contract(off)
    load4<F32>(src, at + da, x);
    load4<F32>(src, at + db, x + 4);
    if constexpr (VEC) {
      if (paired) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[e], o = x[4 + e];
          const float ac = a * c[p][e], os = o * s[p][e], oc = o * c[p][e], as = a * s[p][e];
          x[e] = ac - os;
          x[4 + e] = oc + as;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = da + e;
        if (d < g.rot) {
          const int j = d < half ? d : d - half;
          const float cc = g.cos_sin[angle[p] + j], ss = g.cos_sin[angle[p] + half + j];
          const float o = load1<F32>(src, at + (d < half ? d + half : j));
          const float xc = x[e] * cc, os = o * ss;
          x[e] = d < half ? xc - os : xc + os;
        }
      }
    }
  };

  for (int u = u0; u < u1; ++u) {
    if (u < g.n_q) {  // query head: rotate and round
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = p * PPT + sub;
        if (i < lo || i >= hi) continue;
        const int64_t at = ((row0 + i) * g.n_q + u) * HD;
        float x[8];
        turned(g.q, at, p, x);
        store4_bf16(g.q_out + at + da, x);
        store4_bf16(g.q_out + at + db, x + 4);
      }
      continue;
    }
    if (!kept) return;
    const bool is_v = u >= g.n_q + g.c.n_kv;
    const int head = u - g.n_q - (is_v ? g.c.n_kv : 0);
    const int64_t base = ((int64_t(page) * g.c.n_kv + head) << g.c.page_shift) + place0;  // the block's first slot
    float* scale = (is_v ? g.c.v_scale : g.c.k_scale) + (base >> 4);
    const float old = lo > 0 ? *scale : 0.f;
    float most = 0.f;
    if (!is_v) {
      float x[PASSES][8];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = p * PPT + sub;
        if (i < lo || i >= hi) continue;
        turned(g.k, ((row0 + i) * g.c.n_kv + head) * HD, p, x[p]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[p][e] = clamped(x[p][e]);
          most = fmaxf(most, fabsf(x[p][e]));
        }
      }
      const Scale sc = block_scale(max_wave(most), old, lo == 0);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int i = p * PPT + sub;
        uint32_t* ca = reinterpret_cast<uint32_t*>(g.c.k_codes + (base + i) * HD + da);
        uint32_t* cb = reinterpret_cast<uint32_t*>(g.c.k_codes + (base + i) * HD + db);
        if (i < lo) {
          if (sc.ratio == 1.f) continue;
          const uint32_t oa = *ca, ob = *cb;
          uint32_t wa = 0, wb = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            wa |= recode(oa >> (8 * e), sc.ratio) << (8 * e);
            wb |= recode(ob >> (8 * e), sc.ratio) << (8 * e);
          }
          *ca = wa, *cb = wb;
        } else if (i < hi) {
          float held[8];
          uint32_t wa = 0, wb = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = code_of(x[p][e], sc.inv), o = code_of(x[p][4 + e], sc.inv);
            wa |= byte_of(a) << (8 * e);
            wb |= byte_of(o) << (8 * e);
            held[e] = a * sc.s;
            held[4 + e] = o * sc.s;
          }
          *ca = wa, *cb = wb;
          if (g.k_held) {
            uint16_t* h = g.k_held + ((row0 + i) * g.c.n_kv + head) * HD;
            store4_bf16(h + da, held);
            store4_bf16(h + db, held + 4);
          }
        }
      }
      if (lane == 0 && (lo == 0 || sc.s != old)) *scale = sc.s;
    } else {
      constexpr int NU = HD / 64;  // a lane's units: two dims of eight keys
      float x[NU][8][2];
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        const int n = lane + 64 * j, d = 2 * (n % (HD / 2)), i0 = 8 * (n / (HD / 2));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[j][e][0] = x[j][e][1] = 0.f;
          if (i0 + e < lo || i0 + e >= hi) continue;
          load2<F32>(g.v, ((row0 + i0 + e) * g.c.n_kv + head) * HD + d, x[j][e]);
          x[j][e][0] = clamped(x[j][e][0]);
          x[j][e][1] = clamped(x[j][e][1]);
          most = fmaxf(most, fmaxf(fabsf(x[j][e][0]), fabsf(x[j][e][1])));
        }
      }
      const Scale sc = block_scale(max_wave(most), old, lo == 0);
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        const int n = lane + 64 * j, d = 2 * (n % (HD / 2)), i0 = 8 * (n / (HD / 2));
        if (i0 >= hi || (i0 + 8 <= lo && sc.ratio == 1.f)) continue;
        u32x4_t* at = reinterpret_cast<u32x4_t*>(g.c.v_codes + (base + i0) * HD + d * 8);
        u32x4_t w = {0, 0, 0, 0};
        if (i0 < lo) w = *at;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int word = 2 * k + e / 4, sh = 8 * (e % 4);
            const float cv = code_of(x[j][e][k], sc.inv);
            uint32_t byte = byte_of(cv);
            if (i0 + e < lo) byte = sc.ratio == 1.f ? (w[word] >> sh) & 255u : recode(w[word] >> sh, sc.ratio);
            w[word] = (w[word] & ~(255u << sh)) | (byte << sh);
            x[j][e][k] = cv * sc.s;
          }
          if (g.v_held && i0 + e >= lo && i0 + e < hi)
            *reinterpret_cast<uint32_t*>(g.v_held + ((row0 + i0 + e) * g.c.n_kv + head) * HD + d) =
                pack_bf16x2(x[j][e][0], x[j][e][1]);
        }
        *at = w;
      }
      if (lane == 0 && (lo == 0 || sc.s != old)) *scale = sc.s;
    }
  }
}

template <int HD, bool F32>
int launch_hd(const Kv8AppendArgs& a, hipStream_t s) {
  const int64_t blocks = (int64_t(a.max_q) + 14) / kBlock + 1;  // of a sequence, the first one begun anywhere
  const int items = a.n_q + 2 * a.c.n_kv;
  // One item a wave up to 16 waves for each compute unit, then several, whose angles are read once.
  const int64_t fill = int64_t(device_cus()) * 16 / (a.B * blocks);
  const int want = int(fill < 1 ? 1 : fill < items ? fill : items);
  const int per = (items + want - 1) / want, groups = (items + per - 1) / per;
  const int64_t wgs = (a.B * blocks * groups + 3) / 4;
  if (a.rot % 8 == 0)
    kv8_append_kernel<HD, F32, true><<<dim3(uint32_t(wgs)), 256, 0, s>>>(a, int(blocks), groups, per);
  else
    kv8_append_kernel<HD, F32, false><<<dim3(uint32_t(wgs)), 256, 0, s>>>(a, int(blocks), groups, per);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

int launch_kv8_append(const Kv8AppendArgs& a, hipStream_t s) {
  if (a.c.hd == 64) return a.f32_in ? launch_hd<64, true>(a, s) : launch_hd<64, false>(a, s);
  if (a.c.hd == 128) return a.f32_in ? launch_hd<128, true>(a, s) : launch_hd<128, false>(a, s);
  return a.f32_in ? launch_hd<256, true>(a, s) : launch_hd<256, false>(a, s);
}

}  // namespace qmm
