// Keys and values of new tokens into the paged 8-bit cache, rotated on the way
// (qmm_kv8_append; layout and arithmetic: include/qmm_serve.h).
//
// Mathematics: per block of 16 keys and head one scale, as qmm_serve.h gives it.  Every fp32
// operation is rounded by itself (no contraction), so codes and scales are functions of the
// inputs that a caller can reproduce bit for bit.
// Bound: HBM (the inputs once, q_out, held values, a byte per cached value), and the launch
// and two round trips to memory for a decode batch.
// Split: a wave takes one block of 16 keys of one head at a time (an item: a query, key or value
// head), with all its values in registers between the largest magnitude and the codes, and the next
// item's loads under way.  For queries and keys hd/16 lanes share a token, each with the 8 + 8 dims of
// eight rotation pairs, so that a pair needs one load of each value and of its angle; a wave's items
// follow each other over the heads, and the angles stay in registers.  For values a lane holds 4 dims
// (2 of 64) of eight neighbouring keys, which are its 32 bytes of codes.
// Measured (40 query and 8 KV heads of 128): 16 single tokens 5.1 us, 64 of them 7.1, prompts of 256 MB in and out 57 us
// (4.4 TB/s); 24 and 4 heads of 256, fp32, 92 MB at odd places: 31 us, as nothing of the next head is under way there.  With
// rotated dims that are no multiple of 16 pairs are turned one by one, at 256 dims out of scratch (104 registers): the
// same chunks with 56 dims rotated 148 us, of bf16 209 (64 dims 22).
#include <hip/hip_runtime.h>

#include "kv4_attn.h"
#include "qmm_device.h"
#include "qmm_internal.h"
#include "serve_internal.h"

namespace qmm {
namespace {

constexpr int kBlock = 16;  // keys that share a scale
constexpr float kLimit = 57344.0f;

// N neighbouring values of an fp32 or bf16 array, as loaded: `at` values on from `p`, which all lanes share (a block's
// rows lie within 2^24 values).
template <bool F32, int N>
struct Raw {
  static constexpr int kWords = F32 ? N : N / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p, uint32_t at) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p + at * (F32 ? 4u : 2u));
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(from + i);
        w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
      }
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *from;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    else return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};
template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void store8_bf16(uint16_t* p, const float* x) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = w;
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
  r.inv = r.s > 0x1p-127f ? 1.0f / r.s : 0.f;  // finite
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

// VEC: rot a multiple of 16, a lane's dims are two runs of 8 that pair up; otherwise 16 neighbours.
template <int HD, bool F32, bool VEC>
__global__ __launch_bounds__(256, HD == 256 && VEC ? 3 : 2) void kv8_append_kernel(Kv8AppendArgs g, int blocks,
                                                                                   int groups, int per_wave) {
  constexpr int LPT = HD / 16, PPT = 64 / LPT, PASSES = kBlock / PPT;  // lanes of a token, tokens of a pass
  const int lane = threadIdx.x & 63;
  const uint32_t wid = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t unit = wid / uint32_t(groups);  // (sequence, block)
  const int b = int(unit / uint32_t(blocks));
  if (b >= g.B) return;
  const AttnSeq sq = attn_seq(g, b);
  // the block's first key (it may lie below 0)
  const int64_t k0 = ((int64_t(sq.first) >> 4) + unit % uint32_t(blocks)) * kBlock;
  const int64_t end = int64_t(sq.first) + sq.q_len;
  const int lo = int(sq.first > k0 ? sq.first - k0 : 0), hi = int(end < k0 + kBlock ? end - k0 : kBlock);
  if (lo >= hi) return;
  const int64_t row0 = sq.q0 + (k0 - sq.first);  // token row of place 0 of the block
  const int n_k = g.n_q + g.c.n_kv, items = n_k + g.c.n_kv, u0 = int(wid % uint32_t(groups)) * per_wave;
  int u1 = u0 + per_wave < items ? u0 + per_wave : items;

  // keys below 0 do not occur in a block that starts at 0 or later
  int page = -1;
  if (k0 >= 0) page = g.table[int64_t(b) * g.max_pages + (k0 >> g.c.page_shift)];
  const bool kept = uint32_t(page) < uint32_t(g.c.n_pages);
  const int place0 = int(k0 & ((1 << g.c.page_shift) - 1));
  if (!kept) u1 = u1 < g.n_q ? u1 : g.n_q;
  auto slot_of = [&](int head) { return ((int64_t(page) * g.c.n_kv + head) << g.c.page_shift) + place0; };

  constexpr int kSize = F32 ? 4 : 2;

  // ---- queries and keys
  const int li = lane % LPT, sub = lane / LPT;
  const int half = g.rot >> 1, pairs = g.rot >> 4;
  const bool paired = VEC && li < pairs;
  const int da = !VEC ? 16 * li : paired ? 8 * li : g.rot + 16 * (li - pairs);
  const int db = paired ? half + 8 * li : da + 8;
  auto live = [&](int p) { return p * PPT + sub >= lo && p * PPT + sub < hi; };
  // A block's values stay in registers where they fit with the next item's loads under way, and the angles.  Of 256 dims, or
  // where pairs are taken one by one, no loads are under way, angles are read for every head, and keys (not queries or
  // values) are read and turned twice: for the scale, then for the codes.
  constexpr bool HELD = HD < 256 && VEC;
  using Run = Raw<F32, 8>;
  const int u_k = u1 < n_k ? u1 : n_k;
  if (u0 < u_k) {
    auto heads_of = [&](int u) { return u < g.n_q ? g.n_q : g.c.n_kv; };
    auto first_of = [&](int u) { return (row0 * heads_of(u) + (u < g.n_q ? u : u - g.n_q)) * HD; };
    auto offset = [&](int u, int p) { return uint32_t(p * PPT + sub) * uint32_t(heads_of(u) * HD); };
    auto fetch = [&](int u, int p, Run& a, Run& o) {
      const char* from = static_cast<const char*>(u < g.n_q ? g.q : g.k) + first_of(u) * kSize;
      a.load(from, offset(u, p) + da);
      o.load(from, offset(u, p) + db);
    };
    int place[PASSES];  // in the table of angles, of each pass's token
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      place[p] = 0;
      if (!g.rot || !live(p)) continue;
      const int64_t pos = g.positions ? g.positions[row0 + p * PPT + sub] : k0 + p * PPT + sub;
      place[p] = pos < 0 ? 0 : pos >= g.max_pos ? g.max_pos - 1 : int(pos);
    }
    auto angle_of = [&](int p) { return int64_t(place[p]) * g.rot; };
    using Angles = Raw<true, 8>;
    auto angles = [&](int64_t at, Angles& c, Angles& s) {
      const float* cs = g.cos_sin + at + 8 * li;
#pragma unroll
      for (int e = 0; e < 8; ++e) c.w[e] = __float_as_uint(cs[e]), s.w[e] = __float_as_uint(cs[half + e]);
    };
    auto widen = [&](const Run& a, const Run& o, float (&x)[16]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = a.at(e), x[8 + e] = o.at(e);
    };
    auto turn = [&](float (&x)[16], const Angles& c, const Angles& s) {
#pragma clang fp contract(off)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[e], o = x[8 + e], cc = c.at(e), ss = s.at(e);
        const float ac = a * cc, os = o * ss, oc = o * cc, as = a * ss;
        x[e] = ac - os;
        x[8 + e] = oc + as;
      }
    };
    // a pass's token, turned, from memory
    auto turned = [&](int u, int p, float (&x)[16]) {
#pragma clang fp contract(off)
      Run a, o;
      fetch(u, p, a, o);
      widen(a, o, x);
      if (!g.rot) return;
      const int64_t angle = angle_of(p);
      if constexpr (VEC) {
        if (paired) {
          Angles c, s;
          angles(angle, c, s);
          turn(x, c, s);
        }
      } else {
        const void* src = u < g.n_q ? g.q : g.k;
        const int64_t at = first_of(u) + offset(u, p);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int d = da + e;
          if (d < g.rot) {
            const int j = d < half ? d : d - half;
            const float cc = g.cos_sin[angle + j], ss = g.cos_sin[angle + half + j];
            const float o = load1<F32>(src, at + (d < half ? d + half : j));
            const float xc = x[e] * cc, os = o * ss;
            x[e] = d < half ? xc - os : xc + os;
          }
        }
      }
    };
    auto put_q = [&](int u, int p, const float (&x)[16]) {
      uint16_t* to = g.q_out + first_of(u);
      store8_bf16(to + (offset(u, p) + da), x);
      store8_bf16(to + (offset(u, p) + db), x + 8);
    };
    auto largest = [&](const float (&x)[16], float most) {
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(clamped(x[e])));
      return most;
    };
    auto codes_at = [&](int64_t base, int p, int d) {
      return reinterpret_cast<uint2*>(g.c.k_codes + base * HD + uint32_t((p * PPT + sub) * HD + d));
    };
    auto put_k = [&](int u, int p, int64_t base, const float (&x)[16], const Scale& sc) {
      uint32_t w[4] = {0, 0, 0, 0};
      float held[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float cv = code_of(clamped(x[e]), sc.inv);
        w[e / 4] |= byte_of(cv) << (8 * (e % 4));
        held[e] = cv * sc.s;
      }
      *codes_at(base, p, da) = uint2{w[0], w[1]};
      *codes_at(base, p, db) = uint2{w[2], w[3]};
      if (g.k_held) {
        uint16_t* to = g.k_held + first_of(u);
        store8_bf16(to + (offset(u, p) + da), held);
        store8_bf16(to + (offset(u, p) + db), held + 8);
      }
    };
    auto recode_k = [&](int p, int64_t base, float ratio) {  // a key that was there before
      const uint2 oa = *codes_at(base, p, da), ob = *codes_at(base, p, db);
      const uint32_t o[4] = {oa.x, oa.y, ob.x, ob.y};
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e / 4] |= recode(o[e / 4] >> (8 * (e % 4)), ratio) << (8 * (e % 4));
      *codes_at(base, p, da) = uint2{w[0], w[1]};
      *codes_at(base, p, db) = uint2{w[2], w[3]};
    };
    auto scale_at = [&](int u) { return g.c.k_scale + (slot_of(u - g.n_q) >> 4); };
    auto settle = [&](int u, float most) {  // the block's scale; the keys that were there before follow it
      float* at = scale_at(u);
      const float old = lo > 0 ? *at : 0.f;
      const Scale sc = block_scale(max_wave(most), old, lo == 0);
      if (sc.ratio != 1.f) {
        const int64_t base = slot_of(u - g.n_q);
        for (int p = 0; p < PASSES; ++p)
          if (p * PPT + sub < lo) recode_k(p, base, sc.ratio);
      }
      if (lane == 0 && (lo == 0 || sc.s != old)) *at = sc.s;
      return sc;
    };
    if constexpr (HELD) {
      Run xa[PASSES], xb[PASSES];
      Angles c[PASSES], s[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (live(p)) {
          fetch(u0, p, xa[p], xb[p]);
          if (paired) angles(angle_of(p), c[p], s[p]);
        }
      for (int u = u0; u < u_k; ++u) {
        Run na[PASSES], nb[PASSES];
        if (u + 1 < u_k) {
#pragma unroll
          for (int p = 0; p < PASSES; ++p)
            if (live(p)) fetch(u + 1, p, na[p], nb[p]);
        }
        float x[PASSES][16], most = 0.f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          if (live(p)) {
            widen(xa[p], xb[p], x[p]);
            if (paired) turn(x[p], c[p], s[p]);
            if (u < g.n_q) put_q(u, p, x[p]);
            else most = largest(x[p], most);
          }
        if (u >= g.n_q) {
          const Scale sc = settle(u, most);
#pragma unroll
          for (int p = 0; p < PASSES; ++p)
            if (live(p)) put_k(u, p, slot_of(u - g.n_q), x[p], sc);
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) xa[p] = na[p], xb[p] = nb[p];
      }
    } else {
      for (int u = u0; u < u_k; ++u) {
        float most = 0.f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          if (live(p)) {
            float x[16];
            turned(u, p, x);
            if (u < g.n_q) put_q(u, p, x);
            else most = largest(x, most);
          }
        if (u >= g.n_q) {
          const Scale sc = settle(u, most);
#pragma unroll
          for (int p = 0; p < PASSES; ++p)
            if (live(p)) {
              float x[16];
              turned(u, p, x);
              put_k(u, p, slot_of(u - g.n_q), x, sc);
            }
        }
      }
    }
  }

  // ---- values
  constexpr int DV = HD == 64 ? 2 : 4, NU = HD * 2 / DV / 64;  // dims of a lane's unit, units: HD / DV for each of two octets
  using Few = Raw<F32, DV>;
  auto unit_dim = [&](int j) { return DV * ((lane + 64 * j) % (HD / DV)); };
  auto unit_key = [&](int j) { return 8 * ((lane + 64 * j) / (HD / DV)); };
  auto fetch_v = [&](int u, Few (&x)[NU][8]) {
    const char* from = static_cast<const char*>(g.v) + (row0 * g.c.n_kv + (u - n_k)) * HD * kSize;
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = unit_key(j) + e;
        if (i >= lo && i < hi) x[j][e].load(from, uint32_t(i) * uint32_t(g.c.n_kv * HD) + unit_dim(j));
        else
#pragma unroll
          for (int k = 0; k < Few::kWords; ++k) x[j][e].w[k] = 0;
      }
  };
  const int u_v = u0 > n_k ? u0 : n_k;
  if (u_v >= u1) return;
  auto item_v = [&](int u, const Few (&xv)[NU][8]) __attribute__((always_inline)) {
    const int head = u - n_k;
    const int64_t base = slot_of(head);
    float* scale = g.c.v_scale + (base >> 4);
    const float old = lo > 0 ? *scale : 0.f;
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int k = 0; k < DV; ++k) most = fmaxf(most, fabsf(clamped(xv[j][e].at(k))));
    const Scale sc = block_scale(max_wave(most), old, lo == 0);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int d = unit_dim(j), i0 = unit_key(j);
      if (i0 >= hi || (i0 + 8 <= lo && sc.ratio == 1.f)) continue;
      u32x4_t* at = reinterpret_cast<u32x4_t*>(g.c.v_codes + base * HD + uint32_t(i0 * HD + d * 8));
      uint32_t w[2 * DV];
#pragma unroll
      for (int k = 0; k < DV / 2; ++k) {
        u32x4_t o = {0, 0, 0, 0};
        if (i0 < lo) o = at[k];
        w[4 * k] = o[0], w[4 * k + 1] = o[1], w[4 * k + 2] = o[2], w[4 * k + 3] = o[3];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float held[DV];
        const bool mine = i0 + e >= lo && i0 + e < hi;
#pragma unroll
        for (int k = 0; k < DV; ++k) {
          const int word = 2 * k + e / 4, sh = 8 * (e % 4);
          const float cv = code_of(clamped(xv[j][e].at(k)), sc.inv);
          uint32_t byte = byte_of(cv);
          if (i0 + e < lo) byte = sc.ratio == 1.f ? (w[word] >> sh) & 255u : recode(w[word] >> sh, sc.ratio);
          w[word] = (w[word] & ~(255u << sh)) | (byte << sh);
          held[k] = cv * sc.s;
        }
        if (g.v_held && mine) {
          uint16_t* to = g.v_held + (row0 * g.c.n_kv + head) * HD + (uint32_t(i0 + e) * uint32_t(g.c.n_kv * HD) + d);
          if constexpr (DV == 4)
            *reinterpret_cast<uint2*>(to) = uint2{pack_bf16x2(held[0], held[1]), pack_bf16x2(held[2], held[3])};
          else *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(held[0], held[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k < DV / 2; ++k) at[k] = u32x4_t{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
    }
    if (lane == 0 && (lo == 0 || sc.s != old)) *scale = sc.s;
  };
  Few xv[HD < 256 ? NU : 1][8];
  if constexpr (HD < 256) fetch_v(u_v, xv);
  for (int u = u_v; u < u1; ++u) {
    Few nv[NU][8];
    if constexpr (HD < 256) {
      if (u + 1 < u1) fetch_v(u + 1, nv);
      item_v(u, xv);
#pragma unroll
      for (int j = 0; j < NU; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) xv[j][e] = nv[j][e];
    } else {
      fetch_v(u, nv);
      item_v(u, nv);
    }
  }
}

template <int HD, bool F32>
int launch_hd(const Kv8AppendArgs& a, hipStream_t s) {
  const int64_t blocks = (int64_t(a.max_q) + 14) / kBlock + 1;  // of a sequence, the first one begun anywhere
  const int items = a.n_q + 2 * a.c.n_kv;
  // One item a wave up to 48 waves for each compute unit, then several, whose angles are read once (8192 tokens, 56
  // items a block: 3 a wave 58 us, 8 of them 68).
  const int64_t met = a.T / kBlock + a.B;  // blocks that tokens meet, about
  const int64_t fill = int64_t(device_cus()) * 48 / met;
  // (and a grid's workgroups fit where max_q is far above what sequences have)
  const int64_t fits = ((int64_t(1) << 26) - 4) / (a.B * blocks), most = fits < items ? fits : items;
  const int want = int(fill < 1 || most < 1 ? 1 : fill < most ? fill : most);
  const int per = (items + want - 1) / want, groups = (items + per - 1) / per;
  const int64_t wgs = (a.B * blocks * groups + 3) / 4;
  if (a.rot % 16 == 0)
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
