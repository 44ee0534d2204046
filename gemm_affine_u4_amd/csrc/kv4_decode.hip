// Attention of few queries over the paged 4-bit cache (qmm_kv4_attn's serving form).
//
// Mathematics.  For a key t with group scales s, biases b and codes c the score is
//   q.k_t = sum_g s_g (q_g . c_g) + b_g sum(q_g),
// so the codes enter the matrix product exactly and each group's scale and bias are two
// fp32 multiply-adds on the product.  The output is
//   sum_t p_t v_t = sum_t (p_t s_t) c_t + sum_t p_t b_t,
// with p_t s_t rounded to fp16 and the weights p in the sums' products likewise (2^-11 of p_t s_t
// and p_t; below 2^-28 of a wave's largest p and s, 2^-39 of those; below 2^-17 of the largest p,
// 2^-28 of it); the rest is fp32.
// Key codes enter as normal fp16 numbers.  Value codes stay masked in place, the fp16 numbers
// c 2^-24 (or, in the next four bits, 16 c 2^-24): subnormals, half an instruction a code and no
// conversion.  The matrix cores line up a product's eight neighbouring terms by their exponents, and
// a subnormal's is not its own: terms below 2^-14 of the largest possible one are cut off (as a
// probe shows).  For values that is 2^-14 of the largest weight times scale among eight keys,
// an eighth of that weight's own rounding; queries, though, may span any range, and with codes in
// place scores of 2^18 had no digits left for differences of 1.  (Conversion, differences before
// products and the lift of the value scales, below, together: 64 sequences 123 against 120 us, 131071
// keys 34.6 against 33.7, 16 x 12 queries on 2000 keys 28.6 against 26.3.)
//
// Measured: 64 sequences of 100 to 16000 keys, 40/8 heads x 128: 123 us, 5.6 TB/s of cache; one of 131071
// keys, 24/4 heads x 256: 34.6 us, 4.4 TB/s; one of 517 keys: 8.5 us.
//
// Bound: the cache's bytes (HBM) for long contexts, launch and latency for short ones.
//
// Split.  A block of 4 or 8 waves takes one KV head's up to 16 (query, head) rows and a range of
// keys; its waves take 32 keys at a time and keep an online softmax of their own (maximum,
// sum and output in registers, no barrier), joined once at the end.  Keys are the rows of
// the first product (S^T = K Q^T) and dims the rows of the second (O^T = V^T P^T), so a lane
// that gets the scores of keys 8h .. 8h+7 of its column holds exactly the probabilities
// that the second product wants from it: nothing crosses lanes between the two.  A lane's
// share of the scales is one word per group pair, read once and broadcast along the row
// (DPP row_newbcast).  Sums of weights and of weights times biases, and of biases times query
// sums, are products of their own with the matrix cores.
#include <hip/hip_runtime.h>

#include <utility>

#include "kv4_attn.h"
#include "kv4_device.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kTile = 32;  // keys of a wave's step
constexpr float kFloor = -1e30f;  // maximum of a row that has seen no key yet
constexpr float kLog2e = 1.4426950408889634f;
// Calls of up to this many rows per KV head run here.  Against the prompts' kernel: 16 sequences of
// 2000 keys x 8 heads x 128: 60 rows 29 against 33 us, 90 rows 38 against 36, 125 rows 48 against 40; one
// of 8000 keys: 50 rows 18 against 22, 125 rows 24 against 24; four of 1000 keys x 2 heads x 64: 126
// rows 10 against 18; four of 8000 keys x 4 heads x 256: 48 rows 32 against 36, 60 rows 35 against 37.
// So batches of 128 dims would cross at about 90 rows (40 sequences of 700 keys, 125 rows: 54 against 32); it stands
// where single sequences and 64 dims still gain.
constexpr int64_t decode_rows(int64_t hd) { return hd == 256 ? 64 : 128; }

template <int HD>
struct Buf {
  static constexpr int NG = HD / 64, NKL = HD == 256 ? 2 : 1, R = NG > 1 ? NG / 2 : 1;
  u32x4_t k[2][NKL];  // key codes of the two 16-key tiles
  u32x4_t v[NG];      // value codes: 8 keys x 4 dims of each group
  uint32_t kb[2][NG];  // the scales of the lane's two rows of the first product (their biases)
  uint32_t km[R], vm[R];
};

// Lane (of its row of 16) and register that hold the meta word of key tk (0..7), group g.
template <int NG>
constexpr int meta_lane(int tk, int g) { return (tk * NG + g) / (NG > 1 ? NG / 2 : 1); }
template <int NG>
constexpr int meta_reg(int tk, int g) { return (tk * NG + g) % (NG > 1 ? NG / 2 : 1); }

__device__ __forceinline__ float half_lo(uint32_t w) {
  return float(__builtin_bit_cast(_Float16, uint16_t(w)));
}

// x of the lane N places on in the row of 16 (DPP row_shl; zero past its end).
template <int N>
__device__ __forceinline__ uint32_t row_next(uint32_t x) {
  if constexpr (N == 0) return x;
  else return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x100 + N, 0xf, 0xf, true));
}

// The four operands (dims 4n + 0..3 of the 16 rows n) of 8 keys' value codes: nibbles in place.
__device__ __forceinline__ f16x8_t nib_operand(const u32x4_t& w, int j) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = j >= 2 ? w[i] >> 8 : w[i];
    r[i] = x & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
  }
  return __builtin_bit_cast(f16x8_t, r);
}
// The operand of one key word: its codes as normal fp16 numbers, in the order 0 2 1 3 4 6 5 7.  The byte c is the
// fp8 (e4m3) number c 2^-9, subnormal or not, so its conversion, times 512, gives the code exactly.
__device__ __forceinline__ f16x8_t key_operand(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.f, false));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.f, true));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.f, true));
  return __builtin_bit_cast(f16x8_t, r);
}
__device__ __forceinline__ f32x4_t mma16(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <int HD, bool PG32, int NW>
__global__ __launch_bounds__(NW * 64, 2) void kv4_decode_kernel(Kv4AttnArgs g, int group, AttnPlan plan) {
  using B = Buf<HD>;
  constexpr int NG = B::NG, NKL = B::NKL, R = B::R;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x;
  int b = blockIdx.z;
  const int kvh = blockIdx.y % g.c.n_kv, rt = blockIdx.y / g.c.n_kv;

  const AttnSeq sq = attn_longest_first(g, b, lane);
  const int row0 = rt * 16, rows = sq.q_len * group - row0;
  if (rows <= 0) return;
  const AttnSplit pl = attn_split(g, sq, row0, rows < 16 ? rows : 16, group, plan, split);
  if (split >= pl.count) return;

  // Pages, a window of 64 of the wave's tiles at a time: lane i holds the page of its i-th
  // tile from the window's first on (and of its second half, where pages are of 16).
  const int psh = g.c.page_shift, pmask = (1 << psh) - 1;
  const int32_t* __restrict__ table = g.table + int64_t(b) * g.max_pages;
  const int last_key = sq.kv_len > 0 ? sq.kv_len - 1 : 0;
  constexpr int kStride = NW * kTile;
  const int t_end = pl.end * kTile;
  int t = (pl.begin + wave) * kTile, window = t;
  int pages0 = 0, pages1 = 0;          // 0 where there is no page,
  uint64_t there0 = 0, there1 = 0;     // its bit clear then
  auto enter = [&](int t0) {
    window = t0;
    const int k = t0 + lane * kStride;
    // checked here, so that the wait for the entries stays in this rare branch
    const int id0 = table[(k < last_key ? k : last_key) >> psh];
    there0 = __ballot(uint32_t(id0) < uint32_t(g.c.n_pages));
    pages0 = uint32_t(id0) < uint32_t(g.c.n_pages) ? id0 : 0;
    if constexpr (!PG32) {
      const int id1 = table[(k + 16 < last_key ? k + 16 : last_key) >> psh];
      there1 = __ballot(uint32_t(id1) < uint32_t(g.c.n_pages));
      pages1 = uint32_t(id1) < uint32_t(g.c.n_pages) ? id1 : 0;
    }
  };
  enter(t);

  // rows (token slots of this head) of the tile's two halves, and whether their page exists
  struct Where {
    int64_t r0, r1;
    bool ok0, ok1;
  };
  auto where = [&](int t0) {
    Where w;
    const int i = (t0 - window) / kStride;
    w.ok0 = (there0 >> i) & 1;
    w.r0 = ((int64_t(__builtin_amdgcn_readlane(pages0, i)) * g.c.n_kv + kvh) << psh) + (t0 & pmask);
    if constexpr (PG32) {
      w.ok1 = w.ok0;
      w.r1 = w.r0 + 16;
    } else {
      w.ok1 = (there1 >> i) & 1;
      w.r1 = ((int64_t(__builtin_amdgcn_readlane(pages1, i)) * g.c.n_kv + kvh) << psh) + ((t0 + 16) & pmask);
    }
    return w;
  };
  const int krow = 8 * ((n >> 2) & 1) + (n & 3);  // + 4u: the lane's key within its half (n / 8)
  auto load = [&](const Where& w, B& x) {
    const int64_t rk = PG32 ? w.r0 + 8 * (n >> 2) + (n & 3) : (n < 8 ? w.r0 : w.r1) + krow;
    const int64_t rv = PG32 ? w.r0 + 8 * hg : (hg < 2 ? w.r0 : w.r1) + 8 * (hg & 1);
    const uint32_t* kp = g.c.k_codes + rk * (HD / 8);
    const uint32_t* kb = g.c.k_meta + rk * NG;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int p = 0; p < NKL; ++p) {
        if constexpr (HD == 64) {
          const uint2 v = *reinterpret_cast<const uint2*>(kp + 4 * u * (HD / 8) + 2 * hg);
          x.k[u][p] = u32x4_t{v.x, v.y, 0, 0};
        } else {
          x.k[u][p] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(kp + 4 * u * (HD / 8) + 16 * p + 4 * hg));
        }
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) x.kb[u][i] = kb[4 * u * NG + i];
    }
    const int moff = NG == 1 ? (n & 7) : n * R;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      x.km[i] = g.c.k_meta[rv * NG + moff + i];
      x.vm[i] = g.c.v_meta[rv * NG + moff + i];
    }
    const uint16_t* vp = g.c.v_codes + (rv >> 3) * (HD * 2) + n * 8;
#pragma unroll
    for (int i = 0; i < NG; ++i) x.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(vp + i * 128));
  };

  // Behind its last tile a wave loads that one again: were the loads conditional, the wait for
  // a tile's own would have to wait for the next one's too.
  const int t_last = t + (t < t_end ? (t_end - 1 - t) / kStride * kStride : 0);
  auto ahead = [&](int t0, Where& w, B& x) {
    const int tc = t0 < t_last ? t0 : t_last;
    if (tc - window >= 64 * kStride) enter(tc);
    w = where(tc);
    load(w, x);
  };
  B x0, x1;
  Where w0, w1;
  ahead(t, w0, x0);  // under way while the queries are laid out

  // the lane's column: one (query, head) row
  const bool col_ok = n < rows;
  const int cj = (row0 + n) / group, ch = kvh * group + (row0 + n) % group;
  const int64_t qrow = (int64_t(sq.q0) + cj) * g.n_q + ch;
  int c_lo = 0, c_hi = sq.kv_len;
  if (col_ok && g.causal) {
    const int64_t p = int64_t(sq.first) + cj;
    c_hi = p < 0 ? 0 : int(p) + 1;
    c_lo = g.window > 0 && p - g.window + 1 > 0 ? int(p - g.window + 1) : 0;
  }

  // q as operands: fp16 scaled by a power of two so that the row's largest is in
  // [2^7, 2^8) (bf16 values stay exact, 64 of them add up within fp16); and the groups' sums, in
  // two fp16 pieces (22 bits), against the biases
  f16x8_t qf[NG][2], xf;
  float qs;
  {
    float x[NG][2][8], xs[NG], mx = 0.f;
#pragma unroll
    for (int e = 0; e < NG * 2; ++e) {
      const int p = HD == 64 ? 0 : e / 4, j = HD == 64 ? e : e % 4;
      const int gi = HD == 64 ? 0 : 2 * p + (j >> 1);
      const int w = k_word_of<HD>(p, hg, j);
      u32x4_t v = {0, 0, 0, 0};
      if (col_ok) v = *reinterpret_cast<const u32x4_t*>(g.q + qrow * HD + 8 * w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[gi][j & 1][2 * i] = bf16_lo(v[i]);
        x[gi][j & 1][2 * i + 1] = bf16_hi(v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += x[i][j >> 3][j & 7], mx = fmaxf(mx, fabsf(x[i][j >> 3][j & 7]));
      s += __shfl_xor(s, 16);
      xs[i] = s + __shfl_xor(s, 32);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const int ex = mx > 0.f ? int((__float_as_uint(mx) >> 23) & 255) - 127 : 0;
    const int sh = 7 - ex;  // in [-120, 134]
    qs = fminf(g.scale * kLog2e * ldexpf(1.f, -sh), 3e38f);  // finite: it meets differences of 0
#pragma unroll
    for (int i = 0; i < 8; ++i) xf[i] = static_cast<_Float16>(0.f);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      // the products' k places i and NG + i of the first lane group
      const float y = hg == 0 ? ldexpf(xs[i], sh) : 0.f;
      xf[i] = static_cast<_Float16>(y);
      xf[NG + i] = static_cast<_Float16>(y - static_cast<float>(xf[i]));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // operand order: codes (0, 2), (1, 3), (4, 6), (5, 7)
          const int d = 4 * (e >> 1) + (e & 1);
          qf[i][j][2 * e] = static_cast<_Float16>(ldexpf(x[i][j][d], sh));
          qf[i][j][2 * e + 1] = static_cast<_Float16>(ldexpf(x[i][j][d + 2], sh));
        }
      }
    }
  }

  // wave-uniform: tiles wholly inside [u_lo, u_hi) need no mask
  int u_lo = c_lo, u_hi = c_hi;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    u_lo = max(u_lo, __shfl_xor(u_lo, o));
    u_hi = min(u_hi, __shfl_xor(u_hi, o));
  }
  u_lo = __builtin_amdgcn_readfirstlane(u_lo);
  u_hi = __builtin_amdgcn_readfirstlane(u_hi);

  // output, and in a lane's rows of two more products: the weights' sum, and (rows 0, 1 of
  // bacc[i], lane group 0) sums of weight times bias of group i, R + i
  f32x4_t acc[NG][4], bacc[R], lacc = {0.f, 0.f, 0.f, 0.f};
  float m = kFloor;
  // Value scales are lifted by a power of two that brings the largest one met so far into
  // [2^11, 2^12): all of them are below vtop, a power of two too.  acc is in these units.
  float vtop = 0x1p-23f, lift = 0x1p35f;
#pragma unroll
  for (int i = 0; i < R; ++i) bacc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NG; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  f16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = static_cast<_Float16>(1.f);

  auto step = [&](const B& x, int t0, const Where& w) {
    const bool masked = t0 < u_lo || t0 + kTile > u_hi || !w.ok0 || !w.ok1;
    float sk[R], sv[R], top = 0.f;
    uint32_t vm[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      sk[i] = half_lo(x.km[i]);
      vm[i] = x.vm[i];
      // keys that are not there may have any scale, NaN among them
      if (masked) {
        const int tk = t0 + 8 * hg + (NG == 1 ? (n & 7) : n * R / NG);
        vm[i] = (hg < 2 ? w.ok0 : w.ok1) && tk < sq.kv_len ? vm[i] : 0u;
      }
      sv[i] = half_lo(vm[i]);
      top = fmaxf(top, sv[i]);
    }
    float sc[8];
    static_for<2>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      // sum_g b_g sum(q_g): biases in k places g and NG + g
      u32x4_t bw = {0, 0, 0, 0};
      if constexpr (NG == 1) {
        bw[0] = __builtin_amdgcn_perm(x.kb[u][0], x.kb[u][0], 0x07060706u);
      } else if constexpr (NG == 2) {
        bw[0] = bw[1] = __builtin_amdgcn_perm(x.kb[u][1], x.kb[u][0], 0x07060302u);
      } else {
        bw[0] = bw[2] = __builtin_amdgcn_perm(x.kb[u][1], x.kb[u][0], 0x07060302u);
        bw[1] = bw[3] = __builtin_amdgcn_perm(x.kb[u][NG - 1], x.kb[u][NG - 2], 0x07060302u);
      }
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      const f32x4_t bias = mma16(__builtin_bit_cast(f16x8_t, bw), xf, zero);
      f32x4_t d[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) d[i] = zero;
#pragma unroll
      for (int e = 0; e < NG * 2; ++e) {
        const int p = HD == 64 ? 0 : e / 4, j = HD == 64 ? e : e % 4;
        const int gi = HD == 64 ? 0 : 2 * p + (j >> 1);
        d[gi] = mma16(key_operand(x.k[u][p][j]), qf[gi][j & 1], d[gi]);
      }
      static_for<4>([&](auto ic) {
        constexpr int i = decltype(ic)::value, tk = 4 * u + i;
        float s = bias[i];
        static_for<NG>([&](auto gc) {
          constexpr int gi = decltype(gc)::value;
          s = fmaf(row_bcast<meta_lane<NG>(tk, gi)>(sk[meta_reg<NG>(tk, gi)]), d[gi][i], s);
        });
        sc[tk] = s;
      });
    });
    uint32_t vis = 0xFF;
    if (masked) {
      const int tb = t0 + 8 * hg;
      const bool ok = hg < 2 ? w.ok0 : w.ok1;
      vis = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool see = ok && tb + i >= c_lo && tb + i < c_hi;
        vis |= see ? 1u << i : 0u;
        sc[i] = see ? sc[i] : -INFINITY;
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
    if (__any(mx > m || top >= vtop)) {
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m, mx);
      const float fac = exp2_hw((m - mn) * qs);
      m = mn;
      float vfac = fac;
      if (__any(top >= vtop)) {  // larger value scales than the wave has met
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const uint32_t e = __builtin_amdgcn_readfirstlane(__float_as_uint(top) >> 23);
        lift = __uint_as_float((265 - e) << 23);
        vfac *= vtop * lift * 0x1p-12f;
        vtop = __uint_as_float((e + 1) << 23);
      }
      lacc *= fac;
#pragma unroll
      for (int i = 0; i < R; ++i) bacc[i] *= fac;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] *= vfac;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) sv[i] *= lift;
    // probabilities times 8 (p <= 1 and lifted scales below 2^12 keep p s within fp16).  The difference
    // comes first: rounded products of scores of 2^20 and more would be off by a factor of their own.
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = exp2_hw(fmaf(sc[i] - m, qs, 3.f));
    if (masked) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = (vis >> i) & 1 ? p[i] : 0.f;
    }
    f16x8_t ps[NG], pf;
    static_for<8>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      pf[i] = static_cast<_Float16>(p[i]);
      static_for<NG>([&](auto gc) {
        constexpr int gi = decltype(gc)::value;
        ps[gi][i] = static_cast<_Float16>(p[i] * row_bcast<meta_lane<NG>(i, gi)>(sv[meta_reg<NG>(i, gi)]));
      });
    });
    lacc = mma16(ones, pf, lacc);
    // biases: row n of the operand from the lanes n, n + 16 / 8, .. that hold its group's keys
    constexpr int kHop = NG == 1 ? 1 : 2;
    static_for<R>([&](auto rc) {
      constexpr int r = decltype(rc)::value;
      u32x4_t bw;
      static_for<4>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        bw[i] = __builtin_amdgcn_perm(row_next<(2 * i + 1) * kHop>(vm[r]), row_next<2 * i * kHop>(vm[r]), 0x07060302u);
      });
      bacc[r] = mma16(__builtin_bit_cast(f16x8_t, bw), pf, bacc[r]);
    });
#pragma unroll
    for (int i = 0; i < NG; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mma16(nib_operand(x.v[i], j), ps[i], acc[i][j]);
    }
  };

  // the wave's tiles, the next one's loads under way while one is computed
  if (t < t_end) {
    for (;;) {
      ahead(t + kStride, w1, x1);
      step(x0, t, w0);
      if ((t += kStride) > t_last) break;
      ahead(t + kStride, w0, x0);
      step(x1, t, w1);
      if ((t += kStride) > t_last) break;
    }
  }

  // join the waves.  Rows 0 and 1 of bacc are in lane group 0: group i's sum for the column
  const float l = lacc[0];
  float bias[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    // group i: register i % R, row i / R of the operand
    bias[i] = __shfl(bacc[i % R][NG == 1 ? 0 : i / R], n);
  }
  __shared__ float s_o[NW][16][HD];
  __shared__ float s_m[NW][16], s_l[NW][16], s_qs[16];
  if (hg == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
    if (wave == 0) s_qs[n] = qs;
  }
  __syncthreads();
  float mm = kFloor;
#pragma unroll
  for (int i = 0; i < NW; ++i) mm = fmaxf(mm, s_m[i][n]);
  if (col_ok) {
    const float fac = exp2_hw((m - mm) * qs), even = vtop * 4096.f, odd = vtop * 256.f;  // 2^24 / lift, 2^20 / lift
#pragma unroll
    for (int i = 0; i < NG; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float4 o;
        o.x = fmaf(acc[i][0][r], even, bias[i]) * fac;
        o.y = fmaf(acc[i][1][r], odd, bias[i]) * fac;
        o.z = fmaf(acc[i][2][r], even, bias[i]) * fac;
        o.w = fmaf(acc[i][3][r], odd, bias[i]) * fac;
        *reinterpret_cast<float4*>(&s_o[wave][n][64 * i + 16 * hg + 4 * r]) = o;
      }
    }
  }
  __syncthreads();
  const int cols = rows < 16 ? rows : 16;
  constexpr int Q = HD / 4;  // float4s of a row
  for (int e = tid; e < cols * Q; e += NW * 64) {
    const int c = e / Q, d = (e % Q) * 4;
    float cm = kFloor, cl = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) cm = fmaxf(cm, s_m[i][c]);
    const float cqs = s_qs[c];
    float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      cl = fmaf(s_l[i][c], exp2_hw((s_m[i][c] - cm) * cqs), cl);
      const float4 v = *reinterpret_cast<const float4*>(&s_o[i][c][d]);
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    const int j = (row0 + c) / group, h = kvh * group + (row0 + c) % group;
    const int64_t row = (int64_t(sq.q0) + j) * g.n_q + h;
    if (pl.count == 1) {
      attn_store4(g, row * HD + d, o, cl);
    } else {
      const int64_t R0 = g.T * g.n_q, at = split * R0 + row;
      float* po = static_cast<float*>(g.ws);
      *reinterpret_cast<float4*>(po + at * HD + d) = o;
      if (d == 0) {
        float* pm = po + plan.nsplit * R0 * HD;
        pm[at * 2] = cm;  // as it is: the join scales differences, as the waves do
        pm[at * 2 + 1] = cl;
        if (split == 0) pm[plan.nsplit * R0 * 2 + row] = cqs;
      }
    }
  }
}

// Joins the splits of one (query, head) row: 4 waves over the splits, lanes over the dims.
template <int HD>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttnArgs g, int group, AttnPlan plan) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.z, kvh = blockIdx.y, rr = blockIdx.x;
  const AttnSeq sq = attn_seq(g, b);
  if (rr >= sq.q_len * group) return;
  const int row0 = rr / plan.rows * plan.rows, rows = sq.q_len * group - row0;
  const int count = attn_split(g, sq, row0, rows < plan.rows ? rows : plan.rows, group, plan, 0).count;
  if (count == 1) return;
  const int64_t row = (int64_t(sq.q0) + rr / group) * g.n_q + kvh * group + rr % group, R0 = g.T * g.n_q;
  const float* po = static_cast<const float*>(g.ws);
  const float* pm = po + plan.nsplit * R0 * HD;
  const float qs = plan.rows == 16 ? pm[plan.nsplit * R0 * 2 + row] : 1.f;  // prompts' maxima are powers of two
  float mm = -INFINITY;
  for (int s = lane; s < count; s += 64) mm = fmaxf(mm, pm[(s * R0 + row) * 2]);
#pragma unroll
  for (int o = 32; o; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
  constexpr int V = HD / 64;
  float acc[V], l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int s = wave; s < count; s += 4) {
    const int64_t at = s * R0 + row;
    const float f = exp2_hw((pm[at * 2] - mm) * qs);
    l = fmaf(pm[at * 2 + 1], f, l);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(po[at * HD + lane * V + i], f, acc[i]);
  }
  __shared__ float s_a[4][HD], s_l[4];
#pragma unroll
  for (int i = 0; i < V; ++i) s_a[wave][lane * V + i] = acc[i];
  if (lane == 0) s_l[wave] = l;
  __syncthreads();
  if (tid < HD / 4) {
    float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&s_a[i][tid * 4]);
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    attn_store4(g, row * HD + tid * 4, o, s_l[0] + s_l[1] + s_l[2] + s_l[3]);
  }
}

// The same for many rows or few splits: HD / 4 lanes a row.
template <int HD>
__global__ __launch_bounds__(256) void kv4_join_rows_kernel(Kv4AttnArgs g, int group, AttnPlan plan) {
  constexpr int LPR = HD / 4, RPB = 256 / LPR;  // lanes of a row, rows of a block (all of one row block)
  const int b = blockIdx.z, kvh = blockIdx.y, rr = int(blockIdx.x) * RPB + int(threadIdx.x) / LPR;
  const int d = (threadIdx.x % LPR) * 4;
  const AttnSeq sq = attn_seq(g, b);
  if (rr >= sq.q_len * group) return;
  const int row0 = rr / plan.rows * plan.rows, rows = sq.q_len * group - row0;
  const int count = attn_split(g, sq, row0, rows < plan.rows ? rows : plan.rows, group, plan, 0).count;
  if (count == 1) return;
  const int64_t row = (int64_t(sq.q0) + rr / group) * g.n_q + kvh * group + rr % group, R0 = g.T * g.n_q;
  const float* po = static_cast<const float*>(g.ws);
  const float* pm = po + plan.nsplit * R0 * HD;
  const float qs = plan.rows == 16 ? pm[plan.nsplit * R0 * 2 + row] : 1.f;
  float mm = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int s = 0; s < count; ++s) mm = fmaxf(mm, pm[(s * R0 + row) * 2]);
  float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < count; ++s) {
    const int64_t at = s * R0 + row;
    const float f = exp2_hw((pm[at * 2] - mm) * qs);
    const float4 v = *reinterpret_cast<const float4*>(po + at * HD + d);
    l = fmaf(pm[at * 2 + 1], f, l);
    o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
  }
  attn_store4(g, row * HD + d, o, l);
}

template <int HD>
int launch_hd(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv;
  const int64_t rts = (int64_t(a.max_q) * group + 15) / 16;
  const dim3 grid(uint32_t(p.nsplit), uint32_t(a.c.n_kv * rts), uint32_t(a.B));
  if (p.waves == 8) {
    if (a.c.page_shift >= 5) kv4_decode_kernel<HD, true, 8><<<grid, 512, 0, s>>>(a, group, p);
    else kv4_decode_kernel<HD, false, 8><<<grid, 512, 0, s>>>(a, group, p);
  } else {
    if (a.c.page_shift >= 5) kv4_decode_kernel<HD, true, 4><<<grid, 256, 0, s>>>(a, group, p);
    else kv4_decode_kernel<HD, false, 4><<<grid, 256, 0, s>>>(a, group, p);
  }
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

template <int HD>
int join_hd(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv;
  const uint32_t rows = uint32_t(a.max_q * group), rpb = 1024 / HD;
  // few splits: HD / 4 lanes a row go through them one by one (16 sequences of 4096 keys: 22.7
  // against 23.9 us); at 16 splits the waves of a row are faster (2000 keys: 10.0 against 12.0)
  if (p.rows == 16 && p.nsplit > 8)
    kv4_join_kernel<HD><<<dim3(rows, uint32_t(a.c.n_kv), uint32_t(a.B)), 256, 0, s>>>(a, group, p);
  else
    kv4_join_rows_kernel<HD><<<dim3((rows + rpb - 1) / rpb, uint32_t(a.c.n_kv), uint32_t(a.B)), 256, 0, s>>>(a, group, p);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

int64_t kv4_attn_rows(int64_t rows, int64_t hd) { return rows <= decode_rows(hd) ? 16 : kAttnRows; }

// Few queries: one block per compute unit for few long sequences (131071 keys x 4 heads: 64
// splits 36 us, 128 splits 40 us: a block's fixed part is ~6 us), and up to 4 for many, whose
// lengths may differ (64 sequences of 100 to 16000 keys x 8 heads, before they were ordered: 141 us in 4, 156 in 2).
// Splits of at least 1024 keys, and down to 128 while half of the units would idle (one
// sequence of 4096 keys x 8 heads: 10.3 against 14.1 us; four of 2000: 10.9 against 15.4).  None up to
// 768 keys or two splits, where the second launch costs more (517 keys: 8.3 against 10.0 us;
// 16 sequences of 2000 keys, 12 queries each: 29 against 50).  8 waves a block
// where that leaves half of the units idle (517 keys x 8 heads: 8.3 against 8.8 us).
// Prompts: as many splits of 512 keys as leave one block to a unit (512 queries on 8000 keys,
// 24/4 heads x 256: 165 us, unsplit 289), or up to 128 dims, where a unit holds two, as many of
// 2048 keys as leave two (40/8 heads x 128: 115 us, one 160; with shorter splits of many blocks
// the join costs more: 4 x 200 queries on 2000 keys 62 against 54 us).
AttnPlan attn_plan(int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv) {
  const int64_t rows = max_q * (n_q / n_kv), cus = device_cus();
  AttnPlan p;
  p.rows = int(kv4_attn_rows(rows, hd));
  const int64_t blocks = B * n_kv * ((rows + p.rows - 1) / p.rows);
  int64_t ns;
  if (p.rows == 16) {
    p.shift = 5, p.keys = 1024;
    while (p.keys > 128 && blocks * ((max_kv + p.keys - 1) / p.keys) <= cus / 2) p.keys /= 2;
    ns = 8 * cus / blocks < 4 ? 8 * cus / blocks : 4;
    if (ns < cus / blocks) ns = cus / blocks;
    if (max_kv <= 768 || max_kv <= 2 * p.keys) ns = 1;
  } else {
    p.shift = 6, p.keys = 512;
    ns = cus / blocks;
    if (hd < 256) {
      const int64_t two = 2 * cus / blocks, longs = (max_kv + 2047) / 2048;
      if ((two < longs ? two : longs) > ns) ns = two, p.keys = 2048;
    }
  }
  const int64_t most = (max_kv + p.keys - 1) / p.keys;
  ns = ns > most ? most : ns;
  p.nsplit = int(ns > 256 ? 256 : ns < 1 ? 1 : ns);
  p.waves = p.rows == 16 && blocks * p.nsplit <= cus / 2 ? 8 : 4;
  return p;
}

int launch_kv4_decode(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.hd == 64) return launch_hd<64>(a, p, s);
  if (a.c.hd == 128) return launch_hd<128>(a, p, s);
  return launch_hd<256>(a, p, s);
}

int launch_kv4_join(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.hd == 64) return join_hd<64>(a, p, s);
  if (a.c.hd == 128) return join_hd<128>(a, p, s);
  return join_hd<256>(a, p, s);
}

uint64_t kv4_attn_workspace(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd,
                            int64_t max_kv) {
  const uint64_t ns = uint64_t(attn_plan(B, max_q, n_q, n_kv, hd, max_kv).nsplit);
  // of a row: each split's output, maximum and sum; the factor of its scores
  return ns > 1 && T > 0 ? uint64_t(T) * uint64_t(n_q) * (ns * uint64_t(hd + 2) + 1) * 4 : 256;
}

int launch_kv4_attn(const Kv4AttnArgs& a, hipStream_t s) {
  const AttnPlan p = attn_plan(a.B, a.max_q, a.n_q, a.c.n_kv, a.c.hd, int64_t(a.max_pages) << a.c.page_shift);
  const int st = p.rows == 16 ? launch_kv4_decode(a, p, s) : launch_kv4_prefill(a, p, s);
  return st || p.nsplit == 1 ? st : launch_kv4_join(a, p, s);
}

}  // namespace qmm
