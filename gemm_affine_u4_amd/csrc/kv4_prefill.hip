// Attention of prompts over the paged 4-bit cache (qmm_kv4_attn's prompt form).
//
// Mathematics: that of kv4_decode.hip, but a key tile serves many queries here, so its codes are
// dequantized once per block: fp16(s c + b), one rounding (2^-11 of the value, an eighth of
// the output's), into LDS.  Scores, maxima and sums are fp32, probabilities fp16.
//
// Bound: the matrix cores beside the softmax's exponentials; LDS reads of the shared tile
// come next.
//
// Split.  A block of NW waves takes 32 NW (query, head) rows of one KV head (the heads of a
// group share the tile) and walks the keys 64 at a time; a wave keeps 32 rows: their queries
// as operands and their output in registers.  Keys and dims are the rows of the products, as
// in kv4_decode.hip, so a lane's scores are its share of the next operand.  Of tile i + 1 the
// codes are in registers while tile i is multiplied; they are dequantized into the other LDS
// buffer between the two products.  One barrier a tile.
#include <hip/hip_runtime.h>

#include "kv4_attn.h"
#include "kv4_device.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kKeys = 64;
constexpr float kFloor = -1e30f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // a row's reference maximum may lag by 2^8: p stays below fp16's range

__device__ __forceinline__ f16x2_t h2(uint32_t x) { return __builtin_bit_cast(f16x2_t, x); }
__device__ __forceinline__ uint32_t u32(f16x2_t x) { return __builtin_bit_cast(uint32_t, x); }

// The codes at bits 4j and 4j + 16 of w as fp16 numbers (exact).
template <int J>
__device__ __forceinline__ f16x2_t code_pair(uint32_t w, uint32_t magic) {
  const uint32_t x = J >= 2 ? w >> 8 : w;
  if constexpr (J & 1) {  // 1024 + 16 c
    const f16x2_t v = h2((x & 0x00F000F0u) | magic);
    return v * f16x2_t{(_Float16)0.0625f, (_Float16)0.0625f} - f16x2_t{(_Float16)64.f, (_Float16)64.f};
  } else {  // 1024 + c
    return h2((x & 0x000F000Fu) | magic) - f16x2_t{(_Float16)1024.f, (_Float16)1024.f};
  }
}

// LDS address (in fp16) of 16-byte chunk `c` of key row `t`, and of token chunk `c` of dim row `d`.
template <int HD>
__device__ __forceinline__ int k_at(int t, int c) {
  constexpr int M = HD / 8 - 1 < 15 ? HD / 8 - 1 : 15;
  if constexpr (HD == 64) return t * HD + ((c ^ ((t >> 1) & M)) << 3);
  return t * HD + ((c ^ (t & M)) << 3);
}
__device__ __forceinline__ int v_at(int d, int c) { return d * kKeys + ((c ^ ((d >> 1) & 7)) << 3); }

template <int HD, int NW>
struct Units {
  static constexpr int kEach = HD / 32;  // wave loads of a tile's key codes; as many of its value codes
  static constexpr int kPer = 2 * kEach >= NW ? 2 * kEach / NW : 1;
};

template <int HD, int NW>
__global__ __launch_bounds__(NW * 64, HD == 256 && NW == 4 ? 1 : 2) void kv4_prefill_kernel(Kv4AttnArgs g, int group, AttnPlan plan, int tiles) {
  constexpr int NG = HD / 64, KE = Units<HD, NW>::kEach, PER = Units<HD, NW>::kPer, ROWS = 32 * NW;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x, b = blockIdx.z;
  const int kvh = blockIdx.y % g.c.n_kv, rt = tiles - 1 - int(blockIdx.y) / g.c.n_kv;  // longest rows first

  const AttnSeq sq = attn_seq(g, b);
  const int row0 = rt * ROWS, rows = sq.q_len * group - row0;
  if (rows <= 0) return;
  const AttnSplit pl = attn_split(g, sq, row0, rows < ROWS ? rows : ROWS, group, plan, split);
  if (split >= pl.count) return;

  __shared__ __attribute__((aligned(16))) _Float16 s_k[2][kKeys * HD], s_v[2][HD * kKeys];

  // the lane's row
  const int r = wave * 32 + n;
  const bool row_ok = r < rows;
  const int cj = (row0 + r) / group, ch = kvh * group + (row0 + r) % group;
  const int64_t qrow = (int64_t(sq.q0) + cj) * g.n_q + ch;
  int c_lo = 0, c_hi = sq.kv_len;
  if (row_ok && g.causal) {
    const int64_t p = int64_t(sq.first) + cj;
    c_hi = p < 0 ? 0 : int(p) + 1;
    c_lo = g.window > 0 && p - g.window + 1 > 0 ? int(p - g.window + 1) : 0;
  }
  int u_lo = c_lo, u_hi = c_hi;  // keys that all rows of the wave see
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    u_lo = max(u_lo, __shfl_xor(u_lo, o));
    u_hi = min(u_hi, __shfl_xor(u_hi, o));
  }
  u_lo = __builtin_amdgcn_readfirstlane(u_lo);
  u_hi = __builtin_amdgcn_readfirstlane(u_hi);

  // q: operand e takes chunks 2e + hh, in the order of the codes of a word: 0 4 1 5 2 6 3 7
  f16x8_t qf[HD / 16];
  float qs;
  {
    float mx = 0.f;
    u32x4_t raw[HD / 16];
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) {
      raw[e] = u32x4_t{0, 0, 0, 0};
      if (row_ok) raw[e] = *reinterpret_cast<const u32x4_t*>(g.q + qrow * HD + 16 * e + 8 * hh);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(raw[e][i])), fabsf(bf16_hi(raw[e][i]))));
    }
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const int ex = mx > 0.f ? int((__float_as_uint(mx) >> 23) & 255) - 127 : 0;
    const int sh = 8 - ex;  // largest in [2^8, 2^9): bf16 values stay exact, sums stay far from fp32's ends
    qs = g.scale * kLog2e * ldexpf(1.f, -sh);
#pragma unroll
    for (int e = 0; e < HD / 16; ++e) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = ldexpf(bf16_lo(raw[e][i]), sh);
        x[2 * i + 1] = ldexpf(bf16_hi(raw[e][i]), sh);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[e][2 * i] = static_cast<_Float16>(x[i]);
        qf[e][2 * i + 1] = static_cast<_Float16>(x[i + 4]);
      }
    }
  }

  const int psh = g.c.page_shift, pmask = (1 << psh) - 1;
  const int32_t* __restrict__ table = g.table + int64_t(b) * g.max_pages;
  const int last_key = sq.kv_len > 0 ? sq.kv_len - 1 : 0;
  auto page_of = [&](int t) { return table[(t < last_key ? t : last_key) >> psh]; };
  auto page_ok = [&](int id) { return uint32_t(id) < uint32_t(g.c.n_pages); };
  auto slot_row = [&](int id, int t) {  // row of key t of this head in its (checked) page
    return ((int64_t(page_ok(id) ? id : 0) * g.c.n_kv + kvh) << psh) + (t & pmask);
  };

  // wave load u: keys (u < KE) or values; a lane's key of the tile, first of 8 for values
  struct Codes {
    u32x4_t w;
    uint32_t m0, m1;
  };
  auto unit = [&](int i) { return wave + NW * i; };
  auto key_of = [&](int u) {
    if (u < KE) return HD == 64 ? u * 32 + (lane >> 1) : HD == 128 ? u * 16 + (lane >> 2) : u * 8 + (lane >> 3);
    const int v = u - KE;
    return 8 * (HD == 64 ? v * 4 + (lane >> 4) : HD == 128 ? v * 2 + (lane >> 5) : v);
  };
  auto chunk_of = [&]() { return lane & (HD / 32 - 1); };     // 16-byte piece of a key's row
  auto quad_of = [&]() { return lane & (HD / 4 - 1); };        // dims 4 quad .. +3 of a value
  auto load = [&](int u, int t0, int id, Codes& x) {
    if (2 * KE < NW && u >= 2 * KE) return;
    const int t = t0 + key_of(u);
    const int64_t row = slot_row(id, t);
    if (u < KE) {
      const int c = chunk_of();
      x.w = *reinterpret_cast<const u32x4_t*>(g.c.k_codes + row * (HD / 8) + 4 * c);
      const int p = HD == 64 ? 0 : 2 * (c >> 2);
      const bool ok = page_ok(id) && t < sq.kv_len;
      x.m0 = g.c.k_meta[row * NG + p];
      x.m1 = HD == 64 ? x.m0 : g.c.k_meta[row * NG + p + 1];
      x.m0 = ok ? x.m0 : 0u;
      x.m1 = ok ? x.m1 : 0u;
    } else {
      const int q = quad_of();
      x.w = *reinterpret_cast<const u32x4_t*>(g.c.v_codes + (row >> 3) * (HD * 2) + q * 8);
      x.m0 = g.c.v_meta[(row + (lane & 7)) * NG + (q >> 4)];  // key t + lane % 8
      x.m0 = page_ok(id) && t + (lane & 7) < sq.kv_len ? x.m0 : 0u;
    }
  };
  const uint32_t magic = in_vgpr(0x64006400u);
  auto unpack = [&](int u, const Codes& x, int buf) {
    if (2 * KE < NW && u >= 2 * KE) return;
    if (u < KE) {
      const int t = key_of(u), c = chunk_of();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x2_t sb = h2(HD == 64 || j < 2 ? x.m0 : x.m1);
        const f16x2_t s = {sb[0], sb[0]}, bb = {sb[1], sb[1]};
        u32x4_t o;
        static_for<4>([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          o[i] = u32(__builtin_elementwise_fma(code_pair<i>(x.w[j], magic), s, bb));
        });
        // the word's place among the row's chunks (its dims)
        const int w = HD == 64 ? 4 * c + j : 16 * (c >> 2) + 8 * (j >> 1) + 2 * (c & 3) + (j & 1);
        *reinterpret_cast<u32x4_t*>(&s_k[buf][k_at<HD>(t, w)]) = o;
      }
    } else {
      const int tb = key_of(u) >> 3, q = quad_of();
      f16x2_t s[4], bb[4];
      static_for<4>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const uint32_t a = __float_as_uint(row_bcast<2 * i>(__uint_as_float(x.m0)));
        const uint32_t c = __float_as_uint(row_bcast<2 * i + 1>(__uint_as_float(x.m0)));
        s[i] = h2(__builtin_amdgcn_perm(c, a, 0x05040100u));
        bb[i] = h2(__builtin_amdgcn_perm(c, a, 0x07060302u));
      });
      static_for<4>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = u32(__builtin_elementwise_fma(code_pair<j>(x.w[i], magic), s[i], bb[i]));
        *reinterpret_cast<u32x4_t*>(&s_v[buf][v_at(4 * q + j, tb)]) = o;
      });
    }
  };

  constexpr int OT = HD / 32;
  f32x16_t acc[OT];
#pragma unroll
  for (int i = 0; i < OT; ++i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
  }
  float m = kFloor, l = 0.f;

  Codes x[PER];
  int id[PER], idm = 0;
  uint64_t ok0 = 0, ok1 = 0, ok2 = 0;  // keys there are, of this tile and the next two
  const int t_begin = pl.begin * kKeys, t_end = pl.end * kKeys;
  auto ids = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) id[i] = page_of(t0 + key_of(unit(i)));
    idm = page_of(t0 + lane);
  };
  auto issue = [&](int t0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load(unit(i), t0, id[i], x[i]);
    return __ballot(page_ok(idm) && t0 + lane < sq.kv_len);
  };
  // rows 8a + 4h + e of a product's 32 are keys 16 (a / 2) + 8h + 4 (a % 2) + e, so that a lane's
  // eight scores of 16 keys are neighbours
  const int krow = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);

  if (t_begin < t_end) {
    ids(t_begin);
    ok0 = issue(t_begin);
    ids(t_begin + kKeys);
#pragma unroll
    for (int i = 0; i < PER; ++i) unpack(unit(i), x[i], 0);
    if (t_begin + kKeys < t_end) {
      ok1 = issue(t_begin + kKeys);
      ids(t_begin + 2 * kKeys);
    }
    __syncthreads();
  }
  int buf = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += kKeys, buf ^= 1) {
    const bool more = t0 + kKeys < t_end;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int tb = t0 + 32 * a;
      f32x16_t sc;
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[e] = 0.f;
#pragma unroll
      for (int e = 0; e < HD / 16; ++e) {
        const f16x8_t kf = *reinterpret_cast<const f16x8_t*>(&s_k[buf][k_at<HD>(32 * a + krow, 2 * e + hh)]);
        sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[e], sc, 0, 0, 0);
      }
      if (a == 0 && more) {
#pragma unroll
        for (int i = 0; i < PER; ++i) unpack(unit(i), x[i], buf ^ 1);
        if (t0 + 2 * kKeys < t_end) {
          ok2 = issue(t0 + 2 * kKeys);
          ids(t0 + 3 * kKeys);
        }
      }
      const uint32_t okb = uint32_t(ok0 >> (32 * a));
      if (tb < u_lo || tb + 32 > u_hi || okb != 0xFFFFFFFFu) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = 16 * (e >> 3) + 8 * hh + (e & 7);
          const bool see = ((okb >> k) & 1) && tb + k >= c_lo && tb + k < c_hi;
          sc[e] = see ? sc[e] : -INFINITY;
        }
      }
      float mx = sc[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[e]);
      if (__any(mx * qs > fmaf(m, qs, kSlack))) {
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx), fac = exp2_hw((m - mn) * qs);
        m = mn;
        l *= fac;
#pragma unroll
        for (int i = 0; i < OT; ++i) acc[i] *= fac;
      }
      const float off = m == kFloor ? 0.f : -m * qs;
      f16x8_t p[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = exp2_hw(fmaf(sc[e], qs, off));
        l += v;
        p[e >> 3][e & 7] = static_cast<_Float16>(v);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          const f16x8_t vf = *reinterpret_cast<const f16x8_t*>(&s_v[buf][v_at(32 * i + n, 4 * a + 2 * s + hh)]);
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[s], acc[i], 0, 0, 0);
        }
      }
    }
    ok0 = ok1, ok1 = ok2;
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  const int64_t R0 = g.T * g.n_q;
  float* po = static_cast<float*>(g.ws);
#pragma unroll
  for (int i = 0; i < OT; ++i) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 o = {acc[i][4 * a], acc[i][4 * a + 1], acc[i][4 * a + 2], acc[i][4 * a + 3]};
      const int d = 32 * i + 8 * a + 4 * hh;
      if (pl.count == 1) attn_store4(g, qrow * HD + d, o, l);
      else *reinterpret_cast<float4*>(po + (split * R0 + qrow) * HD + d) = o;
    }
  }
  if (pl.count > 1 && hh == 0) {
    float* pm = po + plan.nsplit * R0 * HD;
    pm[(split * R0 + qrow) * 2] = m * qs;
    pm[(split * R0 + qrow) * 2 + 1] = l;
  }
}

template <int HD, int NW>
int launch(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv, tiles = int((int64_t(a.max_q) * group + p.rows - 1) / p.rows);
  kv4_prefill_kernel<HD, NW>
      <<<dim3(uint32_t(p.nsplit), uint32_t(a.c.n_kv * tiles), uint32_t(a.B)), NW * 64, 0, s>>>(a, group, p, tiles);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

template <int HD>
int launch_hd(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  return p.rows == 256 ? launch<HD, 8>(a, p, s) : launch<HD, 4>(a, p, s);
}

}  // namespace

int launch_kv4_prefill(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.hd == 64) return launch_hd<64>(a, p, s);
  if (a.c.hd == 128) return launch_hd<128>(a, p, s);
  return launch_hd<256>(a, p, s);
}

}  // namespace qmm
