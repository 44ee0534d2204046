// Attention of prompts over the paged 8-bit cache (qmm_kv8_attn's prompt form).
//
// Mathematics.  Codes enter both products exactly, as fp16 numbers in LDS, queries too (bf16 values
// times a power of two).  With a block's scales s_k and s_v a key's weight times its value scale is
//   2^(s_k (q . c) + log2 s_v - m),
// one multiply-add and one exponential, m being the running maximum of that exponent: so the weights
// that are rounded to fp16 (2^-11) are those of the output's own terms, and off by 2^-36 of the largest
// one where they are below 2^-25 of it.  The sum of the weights alone is that of each block's, in fp32,
// over its s_v.  Scales may be anything (append stores 0 and 2^-127 to 2^9): those below 2^-80 of the largest one that
// the block's rows have met are taken as that, so that weights stay within fp32, and sums and outputs are held in a unit
// that leaves them within fp32 for scales up to 2^88.  And so that it holds for scores of any size: from 2^22 on (as a
// bound, taken from the scales of keys) fp32 maxima lie too far from exact products, and a row takes its scores rounded
// and all exponents from an offset of its own.
//
// Bound: one wave a SIMD (three at 64 dims) that issues its vector work (7 slots a score, the exponential being 4, and 1.3 a
// code) and its matrix instructions in turn, and waits for LDS and two barriers a tile alone: neither unit is full
// (prompts of 128 dims: vector unit 33 % busy, matrix cores 27 %).
//
// Split.  A block of 4 waves takes (query, head) rows of one KV head (the heads of a group share the
// tile) and walks the keys 64 at a time, in two steps of 32.  A wave keeps 64 rows at 128 dims, their queries as
// operands and their outputs in registers: each LDS operand serves two products, as reading it takes as long as
// one.  At 256 dims registers end at 32 rows; at 64 dims 32 rows leave room for three blocks a unit (168 registers), which
// fill each other's waits (four prompts of 2000 over 6000 keys, 14 / 2 heads: 315 us with 64 rows, 263).  Keys and dims are the
// rows of the products,
// so that a lane's scores are its share of the next operand.  A step is ordered by hand: a wave issues
// in order, so vector work is placed between matrix instructions, beside which it runs.
// Measured: 815, 673 and 870 TFLOP/s at 128, 64 and 256 dims where blocks fill the GPU evenly (at 128 dims once 952 without
// the codes' conversion, 872 without barriers, of 806).  Four ragged chunks of prompts behind 1500 to 8000 keys (40 / 8
// heads x 128): 270 us, 676 TFLOP/s: 376 blocks on 256 units, so that a second round is half empty; cutting all blocks by
// keys cost more than it brought (286 to 337 us), and so did blocks of 128 rows (355 us).
#include <hip/hip_runtime.h>

#include "kv8_attn.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kKeys = 64;
constexpr int NW = 4;             // waves of a block
constexpr float kFloor = -3e38f;  // maximum of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 4.f;     // a row's reference maximum may lag by 2^4,
constexpr float kShift = 11.f;    // weights are 2^11 of it: below 2^15, within fp16's range
constexpr float kWild = 0x1p22f;  // exponents from which a rounded maximum lies too far from their exact products for that

// Scores: keys (LDS operands) x queries.  The compiler would keep every product's result in accumulation
// registers, and queries in turn spilled: scores are wanted by the vector unit, outputs (and queries, which
// the matrix cores read there as well) are not.  So this product is written out, with its result in
// vector registers; what reads it is kept away by score_settle or by the products in between.
__device__ __forceinline__ void score_first(f32x16_t& d, f16x8_t k, f16x8_t q) {
  asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(d) : "v"(k), "a"(q));
}
__device__ __forceinline__ void score_more(f32x16_t& d, f16x8_t k, f16x8_t q) {
  asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(d) : "v"(k), "a"(q));
}
// Wait states between a score product and the vector unit's read (12 are needed).
__device__ __forceinline__ void score_settle(f32x16_t& d) { asm volatile("s_nop 15" : "+v"(d)); }

// The largest of a wave's values, within the vector unit (row_shr:1, 2, 4, 8, row_bcast:15, 31).
template <int CTRL>
__device__ __forceinline__ float max_with(float x) {
  const int w = int(__float_as_uint(x));
  return fmaxf(x, __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(w, w, CTRL, 0xf, 0xf, false))));
}
__device__ __forceinline__ float max_wave(float x) {
  x = max_with<0x118>(max_with<0x114>(max_with<0x112>(max_with<0x111>(x))));
  return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(max_with<0x143>(max_with<0x142>(x)))), 63)));
}

// A lane's number and the one 32 lanes on (of the wave's halves, in that order): the larger, and the sum.
__device__ __forceinline__ float2 halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return float2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ float max_halves(float x) {
  const float2 v = halves(x);
  return fmaxf(v.x, v.y);
}
__device__ __forceinline__ float sum_halves(float x) {
  const float2 v = halves(x);
  return v.x + v.y;
}

template <int N>
using Int = std::integral_constant<int, N>;

// LDS rows, in fp16: 16 bytes more than a key's dims or a tile's keys, so that rows at one
// chunk meet no bank twice.
template <int HD>
constexpr int kRowK = HD + 8;
constexpr int kRowV = kKeys + 8;

template <int HD>
__global__ __launch_bounds__(NW * 64, HD == 64 ? 2 : 1) void kv8_prefill_kernel(Kv8AttnArgs g, int group, Attn8Plan plan, int tiles) {
  constexpr int CT = HD == 128 ? 2 : 1;  // column tiles of 32 rows
  constexpr int ROWS = NW * 32 * CT, OT = HD / 32, NS = HD / 16, NV = 2 * OT, PER = HD / 64;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = attn8_split(plan);
  int b = blockIdx.z;
  const int kvh = blockIdx.x, rt = tiles - 1 - int(blockIdx.y) / plan.nsplit;  // longest rows first

  const AttnSeq sq = attn_longest_first(g, b, lane);
  const int row0 = rt * ROWS, rows = sq.q_len * group - row0;
  if (rows <= 0) return;
  const Attn8Tiles pl = attn8_tiles(g, sq, row0, rows < ROWS ? rows : ROWS, group, plan, split);
  if (split >= pl.count) return;

  __shared__ __attribute__((aligned(16))) _Float16 s_k[2][kKeys * kRowK<HD>], s_v[2][HD * kRowV];

  // Where exponents may be wild, scores are rounded and a row's maximum and exponents are held from an offset of its own.
  __shared__ float s_off[CT][NW * 64];
  static_for<CT>([&](auto cx) { s_off[decltype(cx)::value][wave * 64 + lane] = 0.f; });

  // the lane's rows, and the keys that they see
  int c_lo[CT], c_hi[CT], u_lo = 0, u_hi = sq.kv_len;  // u: that all rows of the wave see
  const int sinks = int(g.sinks < sq.kv_len ? g.sinks : sq.kv_len);
  f16x8_t qf[CT][NS];
  float qs[CT];
  static_for<CT>([&](auto cx) {
    constexpr int c = decltype(cx)::value;
    const int r = wave * 32 * CT + 32 * c + n, j = (row0 + r) / group;
    const bool ok = r < rows;
    c_lo[c] = 0, c_hi[c] = sq.kv_len;
    if (g.causal) {  // columns without a row see what the last row does
      const int64_t p = int64_t(sq.first) + (ok ? j : (row0 + rows - 1) / group);
      c_hi[c] = p < 0 ? 0 : int(p) + 1;
      c_lo[c] = g.window > 0 && p - g.window + 1 > 0 ? int(p - g.window + 1) : 0;
    }
    u_lo = max(u_lo, c_lo[c]);
    u_hi = min(u_hi, c_hi[c]);
    // q as operands: operand e takes dims 16e + 8 hh .. + 7; fp16 scaled by a power of two so that the
    // row's largest is in [2^7, 2^8)
    const int64_t qrow = (int64_t(sq.q0) + j) * g.n_q + kvh * group + (row0 + r) % group;
    u32x4_t raw[NS];
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < NS; ++e) {
      raw[e] = u32x4_t{0, 0, 0, 0};
      if (ok) raw[e] = *reinterpret_cast<const u32x4_t*>(g.q + qrow * HD + 16 * e + 8 * hh);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(raw[e][i])), fabsf(bf16_hi(raw[e][i]))));
    }
    mx = max_halves(mx);
    const int ex = mx > 0.f ? int((__float_as_uint(mx) >> 23) & 255) - 127 : 0;
    const int sh = 7 - ex;
    qs[c] = fminf(g.scale * kLog2e * ldexpf(1.f, -sh), 1e35f);
#pragma unroll
    for (int e = 0; e < NS; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[c][e][2 * i] = static_cast<_Float16>(ldexpf(bf16_lo(raw[e][i]), sh));
        qf[c][e][2 * i + 1] = static_cast<_Float16>(ldexpf(bf16_hi(raw[e][i]), sh));
      }
#pragma unroll
    for (int e = 0; e < NS; ++e) asm volatile("" : "+a"(qf[c][e]));
  });
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    u_lo = max(u_lo, __shfl_xor(u_lo, o));
    u_hi = min(u_hi, __shfl_xor(u_hi, o));
  }
  u_lo = __builtin_amdgcn_readfirstlane(u_lo);
  u_hi = __builtin_amdgcn_readfirstlane(u_hi);

  // Pages, 16 tiles (a window) at a time: lane i has the 16 keys i % 4 of tile window + i / 4.
  const int psh = g.c.page_shift, pmask = (1 << psh) - 1;
  const int32_t* __restrict__ table = g.table + int64_t(b) * g.max_pages;
  const int last_key = sq.kv_len > 0 ? sq.kv_len - 1 : 0;
  auto key_of = [&](int v) { return pl.at(v + (lane >> 2)) * kKeys + 16 * (lane & 3); };  // below 2^31 some tiles ahead
  auto page_of = [&](int v) {
    const int k = key_of(v);
    return table[(k < last_key ? k : last_key) >> psh];
  };
  const uint32_t n_pages = uint32_t(g.c.n_pages);

  // the window of the tiles whose codes are loaded: the cache's row of a lane's 16 keys (of page 0 where there is
  // no page)
  int lw = pl.begin, l_next = 0;
  int64_t l_row = 0;
  auto rows_of = [&](int v, int page) {
    return ((int64_t(uint32_t(page) < n_pages ? page : 0) * g.c.n_kv + kvh) << psh) + (key_of(v) & pmask);
  };
  auto place = [&](int v, int t16) {  // that of 16 keys of tile v
    const int i = 4 * (v - lw) + t16;
    const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(l_row), i);
    const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(l_row >> 32), i);
    return int64_t(uint64_t(hi) << 32 | lo);
  };
  // the window of the tiles that are computed: the scales of lane i's 16 keys, the logarithm and the
  // reciprocal of the values' one; whether any of the keys is there
  int sw = pl.begin;
  float s_ks = 0.f, s_lv = 0.f, s_iv = 0.f, n_ks = 0.f, n_vs = 0.f;
  uint64_t there = 0;
  auto fetch_scales = [&](int v, int page) {  // of the window from v on
    const int k = key_of(v);
    // only blocks that some row sees: others' scales may be anything
    const bool ok = uint32_t(page) < n_pages && k < pl.hi && (k + 16 > pl.lo || k < sinks);
    n_ks = 0.f, n_vs = 0.f;
    if (ok) {
      const int64_t at = (((int64_t(page) * g.c.n_kv + kvh) << psh) + (k & pmask)) >> 4;
      n_ks = g.c.k_scale[at];
      n_vs = g.c.v_scale[at];
    }
    return __ballot(ok);
  };
  uint64_t n_there = 0;
  // Of a sum: up to 2^15 2^128 for each key (scales count as 2^-128 at least) stays below 2^127, and 2^11 / 2^88 above 2^-126.
  const float unit = __uint_as_float(uint32_t(127 - 18 - 32 + __builtin_clz(sq.kv_len | 1)) << 23);
  // the key scale from which exponents may be wild (as bits, which are ordered as the numbers are)
  uint32_t wild_from = 0;
  uint32_t wild = 0;       // 4: they may be, from here on
  float v_top = 0x1p-48f;  // the largest value scale so far
  auto take_scales = [&]() {
    wild |= __any(__float_as_uint(n_ks) > wild_from) ? 4 : 0;
    v_top = max_wave(fmaxf(n_vs, v_top));
    const float vs = fmaxf(n_vs, v_top * 0x1p-80f);
    s_ks = n_ks;
    s_lv = vs < 0x1p-100f ? __builtin_amdgcn_logf(vs * 0x1p64f) - 64.f : __builtin_amdgcn_logf(vs);  // of normal numbers
    s_iv = unit / vs;
    there = n_there;
  };

  // a lane's share of a tile's codes: 16 dims of a key, two dims of 8 keys
  constexpr int KL = HD / 16, UK = 64 / KL;  // lanes of a key, keys of a wave's load
  const int k_key = lane / KL, k_dim = 16 * (lane % KL);
  const uint32_t k_off = uint32_t(16 * lane);
  u32x4_t ck[2][PER], cv[2][PER];  // of the next two tiles
  auto load_k = [&](int set, int i, int v) {
    const int key = UK * (wave + NW * i);  // of the tile
    const int8_t* from = g.c.k_codes + (place(v, key >> 4) + (key & 15)) * HD;
    ck[set][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(from + k_off));
  };
  auto load_v = [&](int set, int i, int v) {
    const int unit = wave + NW * i;  // of 1 KB: 128 / HD octets of keys
    const int8_t* from = g.c.v_codes + place(v, unit * 64 / HD) * HD + unit * 1024 % (16 * HD);
    cv[set][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(from + k_off));
  };
  // Codes into LDS, four at a time: word a of the lane's share (of all loads).
  constexpr int WORDS = 4 * PER;
  uint32_t held[4];
  auto unpack_k = [&](int set, auto ac, int buf) {
    constexpr int i = decltype(ac)::value / 4, w = decltype(ac)::value % 4;
    code_pairs(ck[set][i][w], held[2 * (w & 1)], held[2 * (w & 1) + 1]);
    if constexpr (w & 1)
      *reinterpret_cast<u32x4_t*>(&s_k[buf][(UK * (wave + NW * i) + k_key) * kRowK<HD> + k_dim + 8 * (w >> 1)]) =
          u32x4_t{held[0], held[1], held[2], held[3]};
  };
  auto unpack_v = [&](int set, auto ac, int buf) {
    constexpr int i = decltype(ac)::value / 4, w = decltype(ac)::value % 4;
    code_pairs(cv[set][i][w], held[2 * (w & 1)], held[2 * (w & 1) + 1]);
    if constexpr (w & 1) {
      const int at = (wave + NW * i) * 64 + lane;  // of the tile's 16-byte units, HD / 2 an octet
      const int octet = at / (HD / 2), dim = 2 * (at % (HD / 2)) + (w >> 1);
      *reinterpret_cast<u32x4_t*>(&s_v[buf][dim * kRowV + 8 * octet]) = u32x4_t{held[0], held[1], held[2], held[3]};
    }
  };

  f32x16_t acc[CT][OT], sa[CT], sb[CT];  // scores of this step and the next, in turn
  float m[CT], l[CT];
  float kq[CT][2], ad[CT][2];  // of a step's two blocks of 16 keys: a score's factor and what is added
  static_for<CT>([&](auto cx) {
    constexpr int c = decltype(cx)::value;
    m[c] = kFloor, l[c] = 0.f;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[c][i][e] = 0.f;
  });
  // rows 8a + 4h + e of a product's 32 are keys 16 (a / 2) + 8h + 4 (a % 2) + e, so that a lane's
  // eight scores of 16 keys are neighbours
  const int krow = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
  const int k_src = krow * kRowK<HD> + 8 * hh, v_src = n * kRowV + 8 * hh;

  // What a step of 32 keys, half of tile v, needs besides its scores.
  struct Facts {
    float ks[2], lv[2], iv[2];  // of its two blocks of 16 keys
    int key;                    // the first one
    uint32_t blocks;            // those that are there; bit 2: wild
    bool masked;                // some row does not see all of them, or wild
  };
  auto facts = [&](int v, int half) {
    Facts f;
    const int i = 4 * (v - sw) + 2 * half;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f.ks[k] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s_ks), i + k));
      f.lv[k] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s_lv), i + k));
      f.iv[k] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s_iv), i + k));
    }
    f.blocks = (uint32_t(there >> i) & 3) | wild;
    f.key = pl.at(v) * kKeys + 32 * half;
    f.masked = f.key + 32 > u_hi || (f.key < u_lo && f.key + 32 > sinks) || f.blocks != 3;
    return f;
  };
  // Scores before their exponentials: factors and what is added; hidden keys leave; the reference
  // maximum moves where the scores ran away from it.  gm: the largest scores of the two blocks if none is hidden.
  auto settle = [&](f32x16_t (&x)[CT], const float (&gm)[CT][2], const Facts& f) __attribute__((always_inline)) {
    float mx[CT];
    bool run = false;
    static_for<CT>([&](auto cx) {
      constexpr int c = decltype(cx)::value;
      kq[c][0] = f.ks[0] * qs[c], kq[c][1] = f.ks[1] * qs[c];
      ad[c][0] = f.lv[0], ad[c][1] = f.lv[1];
      mx[c] = fmaxf(fmaf(gm[c][0], kq[c][0], f.lv[0]), fmaf(gm[c][1], kq[c][1], f.lv[1]));
    });
    if (f.masked) {
      static_for<CT>([&](auto cx) {
        constexpr int c = decltype(cx)::value;
        mx[c] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = f.key + 16 * (e >> 3) + 8 * hh + (e & 7);
          const bool see = ((f.blocks >> (e >> 3)) & 1) && (k >= c_lo[c] || k < sinks) && k < c_hi[c];
          x[c][e] = see ? fmaf(x[c][e], kq[c][e >> 3], ad[c][e >> 3]) : -INFINITY;
          mx[c] = fmaxf(mx[c], x[c][e]);
        }
        kq[c][0] = kq[c][1] = 1.f;
        ad[c][0] = ad[c][1] = 0.f;
        if (f.blocks & 4) {
          float& off = s_off[c][wave * 64 + lane];  // the largest rounded score where not 0
          const float top = fmaxf(off != 0.f ? off : m[c], max_halves(mx[c]));
          m[c] += off - top;
          off = top;
          mx[c] -= top;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[c][e] -= top;
        }
      });
    }
    static_for<CT>([&](auto cx) {
      constexpr int c = decltype(cx)::value;
      run |= mx[c] > m[c] + kSlack;
    });
    if (__any(run)) {
      static_for<CT>([&](auto cx) {
        constexpr int c = decltype(cx)::value;
        const float top = fmaxf(m[c], max_halves(mx[c]));
        const float half = exp2_hw(0.5f * (m[c] - top)), fac = half * half;
        m[c] = top;
        l[c] = l[c] * half * half;  // scales alone may move a maximum by 2^136, where outputs vanish and sums do not
#pragma unroll
        for (int i = 0; i < OT; ++i) acc[c][i] *= fac;
      });
    }
    static_for<CT>([&](auto cx) {
      constexpr int c = decltype(cx)::value;
      ad[c][0] -= m[c] - kShift, ad[c][1] -= m[c] - kShift;
    });
  };

  // The first key operands of a step are read before its weights' factors are settled.
  constexpr int LEAD = 4;
  f16x8_t kf[NS];
  auto lead = [&](int kbuf, int ka) {
    const _Float16* kb = &s_k[kbuf][k_src + 32 * ka * kRowK<HD>];
    static_for<LEAD>([&](auto ec) {
      constexpr int e = decltype(ec)::value;
      kf[e] = *reinterpret_cast<const f16x8_t*>(kb + 16 * e);
    });
  };
  f16x8_t pv[CT][2];
  float ps[CT][2];
  // Weights 2p, 2p + 1 of a lane's 16 of rows c: their exponentials, and, one turn later so that nothing waits for
  // them, the rest.
  float e0, e1;
  auto raise = [&](const f32x16_t (&sc)[CT], auto cc, auto pc) __attribute__((always_inline)) {
    constexpr int c = decltype(cc)::value, w = 2 * decltype(pc)::value;
    e0 = exp2_hw(fmaf(sc[c][w], kq[c][w >> 3], ad[c][w >> 3]));
    e1 = exp2_hw(fmaf(sc[c][w + 1], kq[c][w >> 3], ad[c][w >> 3]));
  };
  auto gather = [&](auto cc, auto pc) __attribute__((always_inline)) {
    constexpr int c = decltype(cc)::value, w = 2 * decltype(pc)::value;
    const f16x2_t h = half_pair(e0, e1);
    pv[c][w >> 3][w & 7] = h[0], pv[c][w >> 3][(w & 7) + 1] = h[1];
    ps[c][w >> 3] = (w & 7) == 0 ? e0 + e1 : ps[c][w >> 3] + (e0 + e1);
    asm volatile("" : "+v"(ps[c][w >> 3]));  // here, not behind the products
  };
  // One step of 32 keys (half of tile v, in buffer buf): the next step's scores (from kbuf, its half ka), then the
  // values.  Each matrix instruction is a turn, with its share of the vector work behind it: pairs of weights, which
  // have to be there by the products that take them (so all by the last PV / 2 turns), the next tile's
  // unpacking, and at the end the next scores' maxima.
  auto step = [&](auto half, auto set, const f32x16_t (&sc)[CT], f32x16_t (&next)[CT], int kbuf, int ka, int buf,
                  float (&gm)[CT][2], int v, const Facts& now, Facts& then) __attribute__((always_inline)) {
    constexpr int h = decltype(half)::value, st = decltype(set)::value;
    constexpr int TURNS = CT * (NS + NV), PAIRS = 8 * CT, DUE = TURNS - NV / 2;
    const int dst = buf ^ 1;
    const _Float16* kb = &s_k[kbuf][k_src + 32 * ka * kRowK<HD>];
    const _Float16* vb = &s_v[buf][v_src + 32 * h];
    f16x8_t vf[NV];
    auto read_k = [&](auto ec) {
      constexpr int e = decltype(ec)::value;
      if constexpr (e < NS) kf[e] = *reinterpret_cast<const f16x8_t*>(kb + 16 * e);
    };
    auto read_v = [&](auto qc) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q >= 0 && q < NV) vf[q] = *reinterpret_cast<const f16x8_t*>(vb + 32 * (q % OT) * kRowV + 16 * (q / OT));
    };
    static_for<TURNS>([&](auto tc) {
      constexpr int t = decltype(tc)::value;
      if constexpr (t < CT * NS) {
        constexpr int e = t / CT, c = t % CT;
        if constexpr (c == 0) {
          read_k(Int<e + LEAD>{});
          read_v(Int<e + LEAD - NS>{});
        }
        if constexpr (e == 0) score_first(next[c], kf[e], qf[c][e]);
        else score_more(next[c], kf[e], qf[c][e]);
        // two tiles ahead, into the set that the step before emptied
        if constexpr (e < PER && c == CT - 1 && h == 0) load_v(1 - st, e, v + 2);
        if constexpr (e < PER && c == CT - 1 && h == 1) load_k(st, e, v + 3);
      } else {
        constexpr int c = (t - CT * NS) / NV, q = (t - CT * NS) % NV;
        if constexpr (c == 0) read_v(Int<q + LEAD>{});
        acc[c][q % OT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[q], pv[c][q / OT], acc[c][q % OT], 0, 0, 0);
      }
      static_for<PAIRS + 1>([&](auto kc) {  // pair k's turn is k DUE / PAIRS
        constexpr int k = decltype(kc)::value;
        if constexpr (k < PAIRS ? k * DUE / PAIRS == t : t == DUE - 1) {
          if constexpr (k > 0) gather(Int<(k - 1) / 8>{}, Int<(k - 1) % 8>{});
          if constexpr (k < PAIRS) raise(sc, Int<k / 8>{}, Int<k % 8>{});
        }
      });
      static_for<WORDS>([&](auto ac) {
        constexpr int a = decltype(ac)::value;
        if constexpr (a * (TURNS - NV) / WORDS == t) {
          if constexpr (h == 0) unpack_k(st, ac, dst);
          else unpack_v(st, ac, dst);
        }
      });
      if constexpr (t == CT * NS) then = facts(h ? v + 1 : v, 1 - h);
      constexpr int M = NV / 2, m0 = TURNS - M;  // the next scores have long been through
      if constexpr (t >= m0) {
        static_for<CT * 8>([&](auto xc) {
          constexpr int x = decltype(xc)::value, k = x / 8, e = 2 * (x % 8);
          if constexpr (x * M / (CT * 8) == t - m0) {
            const float top = fmaxf(next[k][e], next[k][e + 1]);
            gm[k][e >> 3] = (e & 7) == 0 ? top : fmaxf(gm[k][e >> 3], top);
            asm volatile("" : "+v"(gm[k][e >> 3]));
          }
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    static_for<CT>([&](auto cx) {
      constexpr int c = decltype(cx)::value;
      l[c] = fmaf(ps[c][0], now.iv[0], fmaf(ps[c][1], now.iv[1], l[c]));
    });
  };

  if (pl.begin < pl.end) {
    const int page = page_of(pl.begin);
    l_row = rows_of(pl.begin, page);
    l_next = page_of(pl.begin + 16);
    n_there = fetch_scales(pl.begin, page);
    static_for<PER>([&](auto i) {
      load_k(0, i, pl.begin);
      load_v(0, i, pl.begin);
    });
    static_for<PER>([&](auto i) {
      load_k(1, i, pl.begin + 1);
      load_v(1, i, pl.begin + 1);
    });
    float q_top = qs[0];  // codes and queries multiply to 2^15 for each dim at most
    static_for<CT>([&](auto cx) { q_top = fmaxf(q_top, qs[decltype(cx)::value]); });
    wild_from = uint32_t(__builtin_amdgcn_readfirstlane(int(__float_as_uint(kWild / (HD * 0x1p15f) / max_wave(q_top)))));
    take_scales();
    static_for<WORDS>([&](auto a) { unpack_k(0, a, 0); });
    static_for<WORDS>([&](auto a) { unpack_v(0, a, 0); });
    static_for<PER>([&](auto i) { load_k(0, i, pl.begin + 2); });
    __syncthreads();
    float gm[CT][2];
    static_for<CT>([&](auto cx) {
      constexpr int c = decltype(cx)::value;
      static_for<NS>([&](auto ec) {
        constexpr int e = decltype(ec)::value;
        const f16x8_t k = *reinterpret_cast<const f16x8_t*>(&s_k[0][k_src + 16 * e]);
        if constexpr (e == 0) score_first(sa[c], k, qf[c][e]);
        else score_more(sa[c], k, qf[c][e]);
      });
      score_settle(sa[c]);
#pragma unroll
      for (int e = 0; e < 16; ++e) gm[c][e >> 3] = (e & 7) == 0 ? sa[c][e] : fmaxf(gm[c][e >> 3], sa[c][e]);
    });
    lead(0, 1);
    Facts fa = facts(pl.begin, 0), fb;
    settle(sa, gm, fa);
    // a tile: `set` holds the next tile's codes, the other one the keys of the one after (its values are loaded in the
    // first step)
    auto tile = [&](auto set, int v) __attribute__((always_inline)) {
      constexpr int buf = 1 - decltype(set)::value;
      step(Int<0>{}, set, sa, sb, buf, 1, buf, gm, v, fa, fb);
      __syncthreads();
      lead(buf ^ 1, 0);
      settle(sb, gm, fb);
      if (v + 3 - lw >= 16) {  // the window of the loads moves on
        lw += 16;
        l_row = rows_of(lw, l_next);
        l_next = page_of(lw + 16);
      }
      // the next window's scales, some tiles before it begins (the loads' window moves on 4 tiles later)
      if (v - sw == 9) n_there = fetch_scales(sw + 16, l_next);
      if (v - sw == 15) {
        sw += 16;
        take_scales();
      }
      step(Int<1>{}, set, sb, sa, buf ^ 1, 0, buf, gm, v, fb, fa);
      __syncthreads();
      lead(buf ^ 1, 1);
      settle(sa, gm, fa);
    };
    for (int v = pl.begin;;) {
      tile(Int<1>{}, v);
      if (++v >= pl.end) break;
      tile(Int<0>{}, v);
      if (++v >= pl.end) break;
    }
  }

  const int64_t R0 = g.T * g.n_q;
  float* po = static_cast<float*>(g.ws);
  static_for<CT>([&](auto cx) {
    constexpr int c = decltype(cx)::value;
    const float off = s_off[c][wave * 64 + lane], fold = off != 0.f ? exp2_hw(m[c]) : 1.f;
    const float sum = sum_halves(l[c]) * fold, scale = unit * fold;
    const int r = wave * 32 * CT + 32 * c + n;
    if (r >= rows) return;
    const int64_t qrow = (int64_t(sq.q0) + (row0 + r) / group) * g.n_q + kvh * group + (row0 + r) % group;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float4 o = {acc[c][i][4 * a] * scale, acc[c][i][4 * a + 1] * scale, acc[c][i][4 * a + 2] * scale,
                          acc[c][i][4 * a + 3] * scale};
        const int d = 32 * i + 8 * a + 4 * hh;
        if (pl.count == 1) attn_store4(g, qrow * HD + d, o, sum);
        else *reinterpret_cast<float4*>(po + (split * R0 + qrow) * HD + d) = o;
      }
    if (pl.count > 1 && hh == 0) {
      float* pm = po + plan.nsplit * R0 * HD;
      pm[(split * R0 + qrow) * 2] = off != 0.f ? off : m[c];
      pm[(split * R0 + qrow) * 2 + 1] = sum;
      if (split == 0) pm[plan.nsplit * R0 * 2 + qrow] = 1.f;  // maxima are in powers of two
    }
  });
}

template <int HD>
int launch(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv, tiles = int((int64_t(a.max_q) * group + p.rows - 1) / p.rows);
  kv8_prefill_kernel<HD>
      <<<dim3(uint32_t(a.c.n_kv), uint32_t(p.nsplit * tiles), uint32_t(a.B)), NW * 64, 0, s>>>(a, group, p, tiles);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

int launch_kv8_prefill(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s) {
  if (a.c.hd == 256) return launch<256>(a, p, s);
  return a.c.hd == 128 ? launch<128>(a, p, s) : launch<64>(a, p, s);
}

}  // namespace qmm
