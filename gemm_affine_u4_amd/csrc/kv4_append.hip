// Keys and values of new tokens into the paged 4-bit cache, rotated on the way
// (qmm_kv4_append; layout and arithmetic: include/qmm_mix.h).
//
// Mathematics: per group of 64 dims the affine code of qmm_mix.h.  Every fp32 operation is
// rounded by itself (no contraction), so the codes are a function of the inputs that a
// caller can reproduce bit for bit.
// Bound: HBM (the inputs once, q_out, the held values and 4.5 bits per cached value), and
// the launch for a decode batch.
// Split: a lane holds 8 dims of one head (16 bytes of bf16), so a head takes hd/8 lanes, a
// group of 64 exactly 8 lanes (its extremes meet by DPP), a key word one lane.  A wave
// keeps one token: its lanes' cos and sin (the same dims for every head) are read once and
// stay in registers over the token's heads; small calls take one step of heads per wave.
//
// Measured, 40/8 heads x 128: 16 tokens 3.7 us; 8192 tokens 56 us (4.4 TB/s; 40 us where inputs are
// in the last-level cache).  1021 fp32 tokens of 24/4 heads x 256: 10.9 us, 4.7 TB/s.  q is
// written through the caches: the attention that follows reads it.
#include <hip/hip_runtime.h>

#include "kv4_device.h"
#include "mix_internal.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr float kLimit = 57344.0f;

// 8 consecutive values from element offset `at` of a bf16 or fp32 array.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float (&x)[8]) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = w;
}

// The lane's share of a token's rotation: where its dims' partners are, and their angles.
struct Turn {
  int32_t partner;  // dim of the partner of the lane's first dim (vector form), or -1: pass through
  float c[8], s[8];  // out = x * c + partner * s (s carries its sign)
};

// x of the lane's 8 dims (d0 .. d0+7) of the head at element offset `row`, rotated.
template <int HD, bool F32, bool VEC>
__device__ __forceinline__ void turned8(const void* p, int64_t row, int d0, int half, const Turn& t, float (&x)[8]) {
#pragma clang fp contract(off)
  load8<F32>(p, row + d0, x);
  if constexpr (VEC) {  // rot/2 a multiple of 8: the partners of 8 dims are 8 neighbours
    if (t.partner >= 0) {
      float o[8];
      load8<F32>(p, row + t.partner, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[i] * t.c[i], b = o[i] * t.s[i];
        x[i] = a + b;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = d0 + i;
      if (d < 2 * half) {
        const float o = load1<F32>(p, row + (d < half ? d + half : d - half));
        const float a = x[i] * t.c[i], b = o * t.s[i];
        x[i] = a + b;
      }
    }
  }
}

template <int HD, bool F32, bool VEC>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4AppendArgs g, int units, int q_units, int per_wave,
                                                         int waves_per_token) {
  constexpr int LPH = HD / 8;       // lanes of a head
  constexpr int HPW = 64 / LPH;     // heads of a wave's step
  const int lane = threadIdx.x & 63;
  const int64_t wid = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tok = wid / waves_per_token;
  if (tok >= g.T) return;
  const int u0 = int(wid % waves_per_token) * per_wave;
  const int u1 = u0 + per_wave < units ? u0 + per_wave : units;
  const int d0 = (lane % LPH) * 8, hsub = lane / LPH;
  const int half = g.rot >> 1;

  Turn t;
  t.partner = -1;
  if (g.cos_sin) {
    int pos = g.positions[tok];
    pos = pos < 0 ? 0 : pos >= g.max_pos ? g.max_pos - 1 : pos;
    const float* cs = g.cos_sin + int64_t(pos) * g.rot;
    if constexpr (VEC) {
      if (d0 < g.rot) {
        const bool first = d0 < half;
        t.partner = first ? d0 + half : d0 - half;
        const int i0 = first ? d0 : d0 - half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t.c[i] = cs[i0 + i];
          const float s = cs[half + i0 + i];
          t.s[i] = first ? -s : s;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        t.c[i] = t.s[i] = 0.f;
        if (d < g.rot) {
          const bool first = d < half;
          const int j = first ? d : d - half;
          t.c[i] = cs[j];
          t.s[i] = first ? -cs[half + j] : cs[half + j];
        }
      }
    }
  }
  const int turn_half = g.cos_sin ? half : 0;

  const int slot = g.slots[tok];
  const bool kept = slot >= 0 && uint32_t(slot) < (uint32_t(g.c.n_pages) << g.c.page_shift);
  const int64_t page = slot >> g.c.page_shift;
  const int place = slot & ((1 << g.c.page_shift) - 1);

  for (int u = u0; u < u1; ++u) {
    if (u < q_units) {  // query heads: rotate and round
      const int head = u * HPW + hsub;
      if (head < g.n_q) {
        float x[8];
        const int64_t row = (tok * g.n_q + head) * HD;
        turned8<HD, F32, VEC>(g.q, row, d0, turn_half, t, x);
        store8_bf16(g.q_out + row + d0, x);
      }
      continue;
    }
    // key heads, then value heads.  Lanes past the last head redo it and store nothing:
    // all lanes take part in the group's extremes.
    const int idx0 = (u - q_units) * HPW + hsub;
    const bool live = idx0 < 2 * g.c.n_kv;
    const int idx = live ? idx0 : 2 * g.c.n_kv - 1;
    const bool is_v = idx >= g.c.n_kv;
    const int head = is_v ? idx - g.c.n_kv : idx;
    const int64_t row = (tok * g.c.n_kv + head) * HD;
    float x[8];
    if (is_v) load8<F32>(g.v, row + d0, x);
    else turned8<HD, F32, VEC>(g.k, row, d0, turn_half, t, x);

    float lo, hi;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kLimit), kLimit);
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
    lo = min8_lanes(lo), hi = max8_lanes(hi);

    uint32_t word = 0;
    uint32_t meta;
    float held[8];
    {
#pragma clang fp contract(off)
      float step = (hi - lo) * (1.0f / 15.0f);
      asm volatile("" : "+v"(step));  // rounded to fp32 before fp16: no product straight into fp16
      const _Float16 sh = static_cast<_Float16>(step);
      const _Float16 bh = static_cast<_Float16>(lo);
      const float s = static_cast<float>(sh), b = static_cast<float>(bh);
      const float inv = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = x[i] - b;
        const float c = fminf(fmaxf(__builtin_rintf(d * inv), 0.f), 15.f);
        word |= uint32_t(c) << (4 * i);
        held[i] = s * c + b;  // s * c is exact, so this is one rounding either way
      }
      meta = uint32_t(__builtin_bit_cast(uint16_t, sh)) | (uint32_t(__builtin_bit_cast(uint16_t, bh)) << 16);
    }
    if (live && kept) {
      const int64_t base = (page * g.c.n_kv + head) << g.c.page_shift;  // first row of (page, head)
      const int64_t r = base + place;
      const int w = d0 >> 3;
      if (is_v) {
        uint16_t* v = g.c.v_codes + ((base >> 3) + (place >> 3)) * (HD / 4 * 8) + (place & 7);
        v[(2 * w) * 8] = uint16_t(word);
        v[(2 * w + 1) * 8] = uint16_t(word >> 16);
        if ((w & 7) == 0) g.c.v_meta[r * (HD / 64) + (w >> 3)] = meta;
      } else {
        g.c.k_codes[r * LPH + k_word_place<HD>(w)] = word;
        if ((w & 7) == 0) g.c.k_meta[r * (HD / 64) + (w >> 3)] = meta;
      }
    }
    if (live) {
      uint16_t* h = is_v ? g.v_held : g.k_held;
      if (h) store8_bf16(h + row + d0, held);
    }
  }
}

template <int HD, bool F32>
int launch_hd(const Kv4AppendArgs& a, hipStream_t s) {
  constexpr int HPW = 512 / HD;
  const int q_units = a.q ? (a.n_q + HPW - 1) / HPW : 0;
  const int units = q_units + (2 * a.c.n_kv + HPW - 1) / HPW;
  // One step of heads per wave up to 16 waves for each compute unit, then several: the lane's 16
  // angles are then read once for them (8192 tokens, 14 steps: one wave 56 us, a wave a step 74; 1024
  // tokens: 4 waves a token 9.4 us, 1 wave 13.3).
  const int64_t fill = a.T ? int64_t(device_cus()) * 16 / a.T : 1;
  const int want = int(fill < 1 ? 1 : fill < units ? fill : units);
  const int per = (units + want - 1) / want, wpt = (units + per - 1) / per;
  const int64_t blocks = (a.T * wpt + 3) / 4;
  if (a.rot % 16 == 0)
    kv4_append_kernel<HD, F32, true><<<dim3(uint32_t(blocks)), 256, 0, s>>>(a, units, q_units, per, wpt);
  else
    kv4_append_kernel<HD, F32, false><<<dim3(uint32_t(blocks)), 256, 0, s>>>(a, units, q_units, per, wpt);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

int launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s) {
  if (a.c.hd == 64) return a.f32_in ? launch_hd<64, true>(a, s) : launch_hd<64, false>(a, s);
  if (a.c.hd == 128) return a.f32_in ? launch_hd<128, true>(a, s) : launch_hd<128, false>(a, s);
  return a.f32_in ? launch_hd<256, true>(a, s) : launch_hd<256, false>(a, s);
}

}  // namespace qmm
