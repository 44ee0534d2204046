// Attention of few queries over the paged 8-bit cache (qmm_kv8_attn's serving form).
//
// Mathematics.  With the scales s_k, s_v of a key's block, the score is s_k (q . c_k) and the output
// sum_t (p_t s_v) c_v / sum_t p_t: codes enter both matrix products exactly (as fp16 numbers), queries
// exactly (bf16 values times a power of two).  Weights times scales are rounded to fp16
// (2^-11; with the scales lifted by a power of two that brings a wave's largest one so far to 2^11, below
// 2^-28 of the largest weight and scale by 2^-39 of it); the rest is fp32.
//
// Bound: the cache's bytes (HBM) for long contexts, launch and latency for short ones.
//
// Split.  A block of 4 or 8 waves takes one KV head's up to 16 (query, head) rows and a range of
// keys; its waves take 32 keys at a time and keep an online softmax of their own (maximum,
// sum and output in registers, no barrier), joined once at the end.  Keys are the rows of
// the first product (S^T = K Q^T) and dims the rows of the second (O^T = V^T P^T), so a lane
// that gets the scores of keys 8h .. 8h+7 of its column holds exactly the weights that the
// second product wants from it: nothing crosses lanes between the two, and its eight keys
// share their scales.
// Measured (40 query and 8 KV heads of 128): 64 contexts of 100 to 16000 keys 174 us (5.6 TB/s), one of 517 keys
// 9.7 us, most of it the chain from the table over keys and values to the join.  At 256 dims 6 to 8 registers spill (28 to 36
// bytes of scratch): 24 and 4 heads, 64 contexts of 100 to 16000 keys 194 us (4.9 TB/s).
#include <hip/hip_runtime.h>

#include "kv8_attn.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kTile = 32;         // keys of a wave's step
constexpr float kFloor = -1e38f;  // maximum of a row that has seen no key yet
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ f32x4_t mma16(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <int HD>
struct Buf {
  static constexpr int NK = HD / 64, NV = HD / 32;
  u32x4_t k[2][NK];  // key codes of the two 16-key products: 16 dims each
  u32x4_t v[NV];     // value codes: 8 keys x 2 dims of each 32
  float ks, vs;      // scales of the lane's keys (lane group's eight)
};

// A tile of codes, read once where a call's rows are one tile, so that it takes no cache from others; of several
// row tiles' blocks, which run side by side, the later ones find it in the cache (64 sequences of 4000
// keys, 4 heads x 128: 48 rows 133 -> 90 us; one row tile the other way, 64 long contexts: 184 -> 174 us).
template <bool ONCE>
__device__ __forceinline__ u32x4_t load_codes(const int8_t* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  else return *reinterpret_cast<const u32x4_t*>(p);
}

template <int HD, bool PG32, int NW, bool ONCE>
__global__ __launch_bounds__(NW * 64, 2) void kv8_decode_kernel(Kv8AttnArgs g, int group, Attn8Plan plan) {
  using B = Buf<HD>;
  constexpr int NK = B::NK, NV = B::NV;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = attn8_split(plan);
  int b = blockIdx.z;
  const int kvh = blockIdx.x, rt = blockIdx.y / plan.nsplit;

  const AttnSeq sq = attn_longest_first(g, b, lane);
  const int row0 = rt * 16, rows = sq.q_len * group - row0;
  if (rows <= 0) return;
  const Attn8Tiles pl = attn8_tiles(g, sq, row0, rows < 16 ? rows : 16, group, plan, split);
  if (split >= pl.count) return;

  // Pages, a window of 64 of the wave's tiles at a time: lane i holds the page of its i-th
  // tile from the window's first on (and of its second half, where pages are of 16).
  const int psh = g.c.page_shift, pmask = (1 << psh) - 1;
  const int32_t* __restrict__ table = g.table + int64_t(b) * g.max_pages;
  const int last_key = sq.kv_len > 0 ? sq.kv_len - 1 : 0;
  int t = pl.begin + wave, window = t;  // tiles by number
  int pages0 = 0, pages1 = 0;           // 0 where there is no page,
  uint64_t there0 = 0, there1 = 0;      // its bit clear then
  auto enter = [&](int v) {
    window = v;
    const int64_t key = int64_t(pl.at(v + lane * NW)) * kTile;
    const int k = int(key < last_key ? key : last_key), k1 = int(key + 16 < last_key ? key + 16 : last_key);
    // checked here, so that the wait for the entries stays in this rare branch
    const int id0 = table[k >> psh];
    there0 = __ballot(uint32_t(id0) < uint32_t(g.c.n_pages));
    pages0 = uint32_t(id0) < uint32_t(g.c.n_pages) ? id0 : 0;
    if constexpr (!PG32) {
      const int id1 = table[k1 >> psh];
      there1 = __ballot(uint32_t(id1) < uint32_t(g.c.n_pages));
      pages1 = uint32_t(id1) < uint32_t(g.c.n_pages) ? id1 : 0;
    }
  };
  enter(t);

  // a tile's first key, the rows (token slots of this head) of its two halves, and whether their page exists
  struct Where {
    int64_t r0, r1;
    int key;
    bool ok0, ok1;
  };
  auto where = [&](int v) {
    Where w;
    const int i = (v - window) / NW;
    w.key = pl.at(v) * kTile;
    w.ok0 = (there0 >> i) & 1;
    w.r0 = ((int64_t(__builtin_amdgcn_readlane(pages0, i)) * g.c.n_kv + kvh) << psh) + (w.key & pmask);
    if constexpr (PG32) {
      w.ok1 = w.ok0;
      w.r1 = w.r0 + 16;
    } else {
      w.ok1 = (there1 >> i) & 1;
      w.r1 = ((int64_t(__builtin_amdgcn_readlane(pages1, i)) * g.c.n_kv + kvh) << psh) + ((w.key + 16) & pmask);
    }
    return w;
  };
  auto load = [&](const Where& w, B& x) {
    // the lane's key of product u: 8 (n / 4) + 4u + n % 4
    const int64_t rk = (n < 8 ? w.r0 : w.r1) + 8 * ((n >> 2) & 1) + (n & 3);
    const int64_t rv = (hg < 2 ? w.r0 : w.r1) + 8 * (hg & 1);
    const int8_t* kp = g.c.k_codes + rk * HD + 16 * hg;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int p = 0; p < NK; ++p) x.k[u][p] = load_codes<ONCE>(kp + 4 * u * HD + 64 * p);
    x.ks = g.c.k_scale[rv >> 4];
    x.vs = g.c.v_scale[rv >> 4];
    const int8_t* vp = g.c.v_codes + rv * HD + 16 * n;
#pragma unroll
    for (int i = 0; i < NV; ++i) x.v[i] = load_codes<ONCE>(vp + i * 256);
  };

  // Behind its last tile a wave loads that one again: were the loads conditional, the wait for
  // a tile's own would have to wait for the next one's too.
  const int t_last = t + (t < pl.end ? (pl.end - 1 - t) / NW * NW : 0);
  auto ahead = [&](int v, Where& w, B& x) {
    const int tc = v < t_last ? v : t_last;
    if (tc - window >= 64 * NW) enter(tc);
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
  if (g.causal) {  // columns without a row see what the last row does
    const int64_t p = int64_t(sq.first) + (row0 + (col_ok ? n : rows - 1)) / group;
    c_hi = p < 0 ? 0 : int(p) + 1;
    c_lo = g.window > 0 && p - g.window + 1 > 0 ? int(p - g.window + 1) : 0;
  }
  const int sinks = int(g.sinks < sq.kv_len ? g.sinks : sq.kv_len);

  // q as operands: fp16 scaled by a power of two so that the row's largest is in [2^7, 2^8) (a
  // code's product stays below 2^15); bf16 values stay exact down to 2^-24 of that
  f16x8_t qf[NK][2];
  float qs;
  {
    u32x4_t raw[NK][2];
    float mx = 0.f;
#pragma unroll
    for (int p = 0; p < NK; ++p)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        raw[p][e] = u32x4_t{0, 0, 0, 0};
        if (col_ok) raw[p][e] = *reinterpret_cast<const u32x4_t*>(g.q + qrow * HD + 64 * p + 16 * hg + 8 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(raw[p][e][i])), fabsf(bf16_hi(raw[p][e][i]))));
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const int ex = mx > 0.f ? int((__float_as_uint(mx) >> 23) & 255) - 127 : 0;
    const int sh = 7 - ex;  // in [-120, 134]
    qs = fminf(g.scale * kLog2e * ldexpf(1.f, -sh), 3e38f);  // finite: it meets differences of 0
#pragma unroll
    for (int p = 0; p < NK; ++p)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qf[p][e][2 * i] = static_cast<_Float16>(ldexpf(bf16_lo(raw[p][e][i]), sh));
          qf[p][e][2 * i + 1] = static_cast<_Float16>(ldexpf(bf16_hi(raw[p][e][i]), sh));
        }
  }

  // wave-uniform: tiles wholly inside [u_lo, u_hi) or the first keys need no mask
  int u_lo = c_lo, u_hi = c_hi;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    u_lo = max(u_lo, __shfl_xor(u_lo, o));
    u_hi = min(u_hi, __shfl_xor(u_hi, o));
  }
  u_lo = __builtin_amdgcn_readfirstlane(u_lo);
  u_hi = __builtin_amdgcn_readfirstlane(u_hi);

  f32x4_t acc[NV][2];  // in units of 1 / lift
  float m = kFloor, l = 0.f;
  // All value scales met so far are below vtop, a power of two; lift brings that to 2^12 (fp32 ends there: where all scales
  // are below 2^-100, weights times scales are off by up to 2^-140).
  float vtop = 0x1p-100f, lift = 0x1p112f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto step = [&](const B& x, const Where& w) {
    const bool masked = w.key + kTile > u_hi || (w.key < u_lo && w.key + kTile > sinks) || !w.ok0 || !w.ok1;
    const int tb = w.key + 8 * hg;
    float vs = x.vs;
    float sc[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < NK; ++p) {
        d = mma16(code_operand(x.k[u][p][0], x.k[u][p][1]), qf[p][0], d);
        d = mma16(code_operand(x.k[u][p][2], x.k[u][p][3]), qf[p][1], d);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[4 * u + i] = x.ks * d[i];
    }
    uint32_t vis = 0xFF;
    if (masked) {
      const bool ok = hg < 2 ? w.ok0 : w.ok1;
      vis = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool see = ok && (tb + i >= c_lo || tb + i < sinks) && tb + i < c_hi;
        vis |= see ? 1u << i : 0u;
        sc[i] = see ? sc[i] : -INFINITY;
      }
      if (!vis) vs = 0.f;  // keys that are not there, or not seen any more, may have any scale, NaN among them
    }
    float mx = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
    if (__any(mx > m || vs >= vtop)) {
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m, mx);
      const float fac = exp2_hw((m - mn) * qs);
      m = mn;
      float vfac = fac;
      if (__any(vs >= vtop)) {  // larger value scales than the wave has met
        float top = vs;
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        const uint32_t e = __builtin_amdgcn_readfirstlane(__float_as_uint(top) >> 23);
        lift = __uint_as_float((265 - e) << 23);
        vfac *= vtop * lift * 0x1p-12f;
        vtop = __uint_as_float((e + 1) << 23);
      }
      l *= fac;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] *= vfac;
    }
    vs *= lift;
    // weights times 8 (p <= 1 and lifted scales below 2^12 keep p s within fp16).  The difference comes
    // first: rounded products of scores of 2^20 and more would be off by a factor of their own.
    f16x8_t pf;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float p0 = exp2_hw(fmaf(sc[i] - m, qs, 3.f)), p1 = exp2_hw(fmaf(sc[i + 1] - m, qs, 3.f));
      if (masked) {
        p0 = (vis >> i) & 1 ? p0 : 0.f;
        p1 = (vis >> (i + 1)) & 1 ? p1 : 0.f;
      }
      l += p0;
      l += p1;
      const f16x2_t h = half_pair(p0 * vs, p1 * vs);
      pf[i] = h[0], pf[i + 1] = h[1];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mma16(code_operand(x.v[i][2 * j], x.v[i][2 * j + 1]), pf, acc[i][j]);
  };

  // the wave's tiles, the next one's loads under way while one is computed
  if (t < pl.end) {
    for (;;) {
      ahead(t + NW, w1, x1);
      step(x0, w0);
      if ((t += NW) > t_last) break;
      ahead(t + NW, w0, x0);
      step(x1, w1);
      if ((t += NW) > t_last) break;
    }
  }

  // join the waves
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  __shared__ __attribute__((aligned(16))) float s_o[NW][16][HD + 4];
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
    const float fac = exp2_hw((m - mm) * qs), unit = vtop * 0x1p-12f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // rows 4h + e are dims 8h + 2e + j
        o[2 * e] = acc[i][0][e] * unit * fac;
        o[2 * e + 1] = acc[i][1][e] * unit * fac;
      }
      float* to = &s_o[wave][n][32 * i + 8 * hg];
      *reinterpret_cast<float4*>(to) = float4{o[0], o[1], o[2], o[3]};
      *reinterpret_cast<float4*>(to + 4) = float4{o[4], o[5], o[6], o[7]};
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

// Joins the splits of (query, head) rows.  S groups of HD / 4 lanes a row share its splits: one
// where rows are many or splits few.
template <int HD, int S>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8AttnArgs g, int group, Attn8Plan plan) {
  constexpr int LPR = HD / 4, RPB = 256 / LPR / S;  // lanes of a row's group, rows of a block
  const int b = blockIdx.z, kvh = blockIdx.y;
  const int part = (threadIdx.x / LPR) % S, slot = threadIdx.x / LPR / S;
  const int rr = int(blockIdx.x) * RPB + slot, d = (threadIdx.x % LPR) * 4;
  const AttnSeq sq = attn_seq(g, b);
  int count = 0;
  if (rr < sq.q_len * group) {
    const int row0 = rr / plan.rows * plan.rows, rows = sq.q_len * group - row0;
    count = attn8_tiles(g, sq, row0, rows < plan.rows ? rows : plan.rows, group, plan, 0).count;
  }
  const int64_t row = (int64_t(sq.q0) + rr / group) * g.n_q + kvh * group + rr % group, R0 = g.T * g.n_q;
  const float* po = static_cast<const float*>(g.ws);
  const float* pm = po + plan.nsplit * R0 * HD;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  if (count > 1) {
    const float qs = pm[plan.nsplit * R0 * 2 + row];
    float mm = -INFINITY;
    if constexpr (S > 1) {  // a split a lane (each lane all of them: 256 splits of 8 rows 35 us, so 23)
      for (int s = threadIdx.x % LPR; s < count; s += LPR) mm = fmaxf(mm, pm[(s * R0 + row) * 2]);
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    } else {
#pragma unroll 4
      for (int s = 0; s < count; ++s) mm = fmaxf(mm, pm[(s * R0 + row) * 2]);
    }
#pragma unroll 8
    for (int s = part; s < count; s += S) {
      const int64_t at = s * R0 + row;
      const float x = (pm[at * 2] - mm) * qs, f = exp2_hw(x);
      const float4 v = *reinterpret_cast<const float4*>(po + at * HD + d);
      // prompts' maxima hold the values' scales, which alone may lie 2^136 apart: such outputs vanish, their weights do not
      float sum = pm[at * 2 + 1], w = f;
      if (x < -120.f) w = exp2_hw(0.5f * x), sum *= w;
      l = fmaf(sum, w, l);
      o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    }
  }
  if constexpr (S > 1) {
    __shared__ float4 s_o[256];
    __shared__ float s_l[256];
    s_o[threadIdx.x] = o;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int i = 1; i < S; ++i) {
        const float4 v = s_o[threadIdx.x + i * LPR];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        l += s_l[threadIdx.x + i * LPR];
      }
    }
  }
  if (count > 1 && part == 0) attn_store4(g, row * HD + d, o, l);
}

template <int HD, bool PG32, int NW>
int launch_nw(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv;
  const int64_t rts = (int64_t(a.max_q) * group + 15) / 16;
  const dim3 grid(uint32_t(a.c.n_kv), uint32_t(p.nsplit * rts), uint32_t(a.B));
  if (rts == 1) kv8_decode_kernel<HD, PG32, NW, true><<<grid, NW * 64, 0, s>>>(a, group, p);
  else kv8_decode_kernel<HD, PG32, NW, false><<<grid, NW * 64, 0, s>>>(a, group, p);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}
template <int HD>
int launch_hd(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  if (a.c.page_shift >= 5) return p.waves == 8 ? launch_nw<HD, true, 8>(a, p, s) : launch_nw<HD, true, 4>(a, p, s);
  return p.waves == 8 ? launch_nw<HD, false, 8>(a, p, s) : launch_nw<HD, false, 4>(a, p, s);
}

template <int HD>
int join_hd(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  constexpr int RPB = 1024 / HD;  // groups of HD / 4 lanes in a block
  const int group = a.n_q / a.c.n_kv;
  const uint32_t rows = uint32_t(a.max_q * group);
  if (p.nsplit > 8)
    kv8_join_kernel<HD, RPB><<<dim3(rows, uint32_t(a.c.n_kv), uint32_t(a.B)), 256, 0, s>>>(a, group, p);
  else
    kv8_join_kernel<HD, 1><<<dim3((rows + RPB - 1) / RPB, uint32_t(a.c.n_kv), uint32_t(a.B)), 256, 0, s>>>(a, group, p);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

// Which calls run here, others as prompts: those of few rows for each KV head, whose prompt blocks would be mostly empty,
// and those of few row tiles in all, which as prompts would be few blocks.  One rule for all sequences of a call: single tokens
// beside a prompt run in blocks of 128 or 256 rows, unsplit (63 of them on 100 to 8000 keys and a prompt of 512 on 2048, one
// call and two: 40 / 8 heads x 128 723 and 176 us, 24 / 4 x 256 1281 and 202, 14 / 2 x 64 187 and 48).
// Here and as prompts, us, contexts of 4000, 4 KV heads a sequence:
//   64 sequences x 128 dims   96 rows 145, 155   128 rows 184, 158
//   16 sequences x 256 dims   30 rows 44, 54     48 rows 64, 59
//    4 sequences x 256 dims  128 rows 43, 47    192 rows 61, 48
//    4 sequences x 128 dims  256 rows 39, 47
//   64 sequences x 64 dims    48 rows 61, 80    64 rows 74, 78    96 rows 98, 84   128 rows 119, 84
//   32 sequences x 64 dims    64 rows 44, 48    80 rows 53, 50
//   16 sequences x 64 dims    64 rows 27, 31    96 rows 36, 34   128 rows 43, 36
//    4 sequences x 64 dims   128 rows 19, 24   256 rows 27, 26
bool few_rows(int64_t rows, int64_t heads, int64_t hd) {
  return rows <= (hd == 256 ? 16 : hd == 128 ? 96 : 64) ||
         (rows <= 256 && (rows + 15) / 16 * heads <= (hd == 256 ? 128 : 256));
}

}  // namespace

Attn8Plan attn8_plan(int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv, int64_t window,
                     int64_t sinks) {
  const int64_t rows = max_q * (n_q / n_kv), cus = device_cus();
  // keys that the rows of a block can see at most
  int64_t seen = max_kv;
  if (window > 0 && window + max_q + sinks + 64 < max_kv) seen = window + max_q + sinks + 64;
  Attn8Plan p;
  p.rows = few_rows(rows, B * n_kv, hd) ? 16 : attn8_rows(hd);
  const int64_t blocks = B * n_kv * ((rows + p.rows - 1) / p.rows);
  int64_t ns;
  if (p.rows != 16) {
    p.shift = 6, p.keys = 512, p.waves = 4;
    ns = cus / blocks;
    const int64_t longs = (seen + p.keys - 1) / p.keys;
    ns = ns > longs ? longs : ns;
    p.nsplit = int(ns > 256 ? 256 : ns < 1 ? 1 : ns);
    return p;
  }
  // Contexts are often much shorter than the table: few sequences are split however short (16 contexts of 1000 keys in
  // tables of 16384, 8 heads x 128: 22.4 -> 15.4 us), many fill the GPU anyhow.
  p.shift = 5, p.keys = 1024;
  while (p.keys > 128 && blocks * 1024 / p.keys < 2 * cus) p.keys /= 2;
  ns = 8 * cus / blocks < 4 ? 8 * cus / blocks : 4;
  if (ns < cus / blocks) ns = cus / blocks;
  // (a second launch joins them: one token of 40 / 8 heads x 128 in splits and without: 320 keys 10.8, 8.8 us; 512 10.7, 9.9;
  // 768 11.4, 11.2; 1024 11.1, 12.7; 16 of them: 512 10.3, 10.4; 768 14.0, 11.8; 1024 15.0, 14.4; 1500 17.7, 19.0)
  if (seen <= 768 || seen <= 2 * p.keys) ns = 1;
  const int64_t most = (seen + p.keys - 1) / p.keys;
  ns = ns > most ? most : ns;
  p.nsplit = int(ns > 256 ? 256 : ns < 1 ? 1 : ns);
  // 8 waves where they halve a chain of several steps and nothing else could (one token, 4 and 8 waves, us; 40 / 8 heads x
  // 128: 200 keys 8.0, 8.5; 400 10.1, 10.0; 517 11.0, 10.1; 760 12.1, 11.3; split: 1200 11.1, 11.6; 4000 12.5, 13.0.
  // 14 / 2 heads x 64: 517 keys 8.6, 7.8; 24 / 4 x 256: 400 15.1, 15.7; 517 16.9, 16.3; 760 18.7, 18.9; 4000 14.6, 16.2)
  p.waves = p.nsplit == 1 && seen > 448 && blocks <= cus / 2 ? 8 : 4;
  return p;
}

int launch_kv8_decode(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  if (a.c.hd == 64) return launch_hd<64>(a, p, s);
  if (a.c.hd == 128) return launch_hd<128>(a, p, s);
  return launch_hd<256>(a, p, s);
}

int launch_kv8_join(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  if (a.c.hd == 64) return join_hd<64>(a, p, s);
  if (a.c.hd == 128) return join_hd<128>(a, p, s);
  return join_hd<256>(a, p, s);
}

uint64_t kv8_attn_workspace(int64_t T, int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd,
                            int64_t max_kv, int64_t window, int64_t sinks) {
  const uint64_t ns = uint64_t(attn8_plan(B, max_q, n_q, n_kv, hd, max_kv, window, sinks).nsplit);
  // of a row: each split's output, maximum and sum; the factor of its scores
  return ns > 1 && T > 0 ? uint64_t(T) * uint64_t(n_q) * (ns * uint64_t(hd + 2) + 1) * 4 : 256;
}

int launch_kv8_attn(const Kv8AttnArgs& a, hipStream_t s) {
  const Attn8Plan p = attn8_plan(a.B, a.max_q, a.n_q, a.c.n_kv, a.c.hd, int64_t(a.max_pages) << a.c.page_shift,
                                 a.window, a.sinks);
  const int st = p.rows == 16 ? launch_kv8_decode(a, p, s) : launch_kv8_prefill(a, p, s);
  return st || p.nsplit == 1 ? st : launch_kv8_join(a, p, s);
}

}  // namespace qmm
