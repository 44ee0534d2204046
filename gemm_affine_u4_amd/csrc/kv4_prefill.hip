// Attention of prompts over the paged 4-bit cache (qmm_kv4_attn's prompt form).
//
// Mathematics: that of kv4_decode.hip, but a key tile serves many queries here, so its codes are
// dequantized once per block: fp16(s c + b), one rounding (2^-11 of the key or value), into LDS.
// Queries times scale log2(e) are rounded to fp16 likewise (below 2^-14 by 2^-25); scores, maxima and
// sums are fp32, probabilities fp16 (below 2^-14 by 2^-25, the largest being 1 or more).  Together the roundings
// add a quarter of the output's own rounding to bf16 (prompts of 2048 and of 100 to 1500 against 64 bits).
//
// Bound: no unit by itself.  Matrix cores, vector unit and LDS (each 32x32x16 product takes 1 KB of the
// shared tile, its rate at the matrix rate) are busy for 28, 37 and 32 % of a prompt of 2048 x 128 dims and
// 28, 34 and 36 % of five prompts x 256 dims, one after the other for the most part: a SIMD has two waves or
// one.  At 128 dims its two places are filled for 68 % of the time, until the longest block ends.
//
// Split.  A block of 4 waves takes 128 (query, head) rows of one KV head (the heads of a
// group share the tile) and walks the keys 64 at a time, in two steps of 32; a wave keeps 32
// rows: their queries as operands and their output in registers.  Keys and dims are the rows
// of the products, as in kv4_decode.hip, so a lane's scores are its share of the next operand.
// A step is ordered by hand (step() below): a wave issues in order, so vector work placed
// behind a run of matrix instructions waits for all of them, while one placed between two
// runs beside them.
//
// Measured: a prompt of 2048, 40/8 heads x 128, causal: 63 us, 0.68 PFLOP/s (before the hand order
// 77, with tiles dequantized by each wave for itself 129); five prompts on up to 9000 keys,
// 24/4 heads x 256: 398 us, 0.70 PFLOP/s (sequences in the order given: 456).  8 waves, 16-column
// tiles and 32-key tiles were slower.
#include <hip/hip_runtime.h>

#include "kv4_attn.h"
#include "kv4_device.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kKeys = 64;
constexpr int NW = 4;  // waves of a block
constexpr float kFloor = -1e30f;  // maximum of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // a row's reference maximum may lag by 2^8: p stays below fp16's range

template <int N>
using Int = std::integral_constant<int, N>;

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

// LDS rows, in fp16: 16 bytes more than a key's dims or a tile's keys, so that 16 rows at one
// chunk meet no bank twice and every chunk is a constant offset from the lane's first.
template <int HD>
constexpr int kRowK = HD + 8;
constexpr int kRowV = kKeys + 8;

// A lane's share of a tile's key codes, and of its value codes: PER units of WPL words.
template <int HD>
struct Units {
  static constexpr int kWords = HD / (8 * NW);
  static constexpr int WPL = kWords < 4 ? kWords : 4;
  static constexpr int PER = kWords / WPL;
  static constexpr int UK = 512 * WPL / HD;  // keys of a unit: 8 or 16, in one page
  static_assert(WPL * PER == kWords && WPL >= 1 && UK <= 16);
};

template <int WPL>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[WPL]) {
  if constexpr (WPL == 4) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
    w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
  } else if constexpr (WPL == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *p;
  }
}

template <int HD>
__global__ __launch_bounds__(NW * 64, HD == 256 ? 1 : 2) void kv4_prefill_kernel(Kv4AttnArgs g, int group,
                                                                                 AttnPlan plan, int tiles) {
  using U = Units<HD>;
  constexpr int NG = HD / 64, WPL = U::WPL, PER = U::PER, UK = U::UK, ROWS = kAttnRows, OT = HD / 32;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x;
  int b = blockIdx.z;
  const int kvh = blockIdx.y % g.c.n_kv, rt = tiles - 1 - int(blockIdx.y) / g.c.n_kv;  // longest rows first

  const AttnSeq sq = attn_longest_first(g, b, lane);
  const int row0 = rt * ROWS, rows = sq.q_len * group - row0;
  if (rows <= 0) return;
  const AttnSplit pl = attn_split(g, sq, row0, rows < ROWS ? rows : ROWS, group, plan, split);
  if (split >= pl.count) return;

  __shared__ __attribute__((aligned(16))) _Float16 s_k[2][kKeys * kRowK<HD>], s_v[2][HD * kRowV];

  // the lane's row
  const int r = wave * 32 + n;
  const bool row_ok = r < rows;
  const int cj = (row0 + r) / group, ch = kvh * group + (row0 + r) % group;
  const int64_t qrow = (int64_t(sq.q0) + cj) * g.n_q + ch;
  int c_lo = 0, c_hi = sq.kv_len;  // keys that it sees
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

  // q times scale log2(e): operand e takes chunks 2e + hh, in the order of the codes of a
  // word (0 4 1 5 2 6 3 7)
  f16x8_t qf[HD / 16];
#pragma unroll
  for (int e = 0; e < HD / 16; ++e) {
    u32x4_t raw = {0, 0, 0, 0};
    if (row_ok) raw = *reinterpret_cast<const u32x4_t*>(g.q + qrow * HD + 16 * e + 8 * hh);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = fminf(fmaxf(bf16_lo(raw[i]) * (g.scale * kLog2e), -65504.f), 65504.f);
      x[2 * i + 1] = fminf(fmaxf(bf16_hi(raw[i]) * (g.scale * kLog2e), -65504.f), 65504.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qf[e][2 * i] = static_cast<_Float16>(x[i]);
      qf[e][2 * i + 1] = static_cast<_Float16>(x[i + 4]);
    }
  }

  // Pages, a window of 1024 keys at a time: lane i holds the page of the 16 keys from
  // window + 16 i on (0 if there is none, with its bit of `there` clear).
  const int psh = g.c.page_shift, pmask = (1 << psh) - 1;
  const int32_t* __restrict__ table = g.table + int64_t(b) * g.max_pages;
  const int last_key = sq.kv_len > 0 ? sq.kv_len - 1 : 0;
  const int t_begin = pl.begin * kKeys, t_end = pl.end * kKeys;
  int window = t_begin, pages = 0, pages_next = 0;
  uint64_t there = 0;
  auto pages_from = [&](int t) {
    const int k = t + 16 * lane;
    return table[(k < last_key ? k : last_key) >> psh];
  };
  auto enter = [&](int ids) {
    const bool ok = uint32_t(ids) < uint32_t(g.c.n_pages);
    there = __ballot(ok);
    pages = ok ? ids : 0;
  };
  // Where a unit's keys are: the row of its first key in the cache, and how many of its keys
  // there are.
  struct Place {
    int64_t row;
    int keys;
  };
  auto place = [&](int t) {
    const int i = (t - window) >> 4;
    Place p;
    p.row = ((int64_t(__builtin_amdgcn_readlane(pages, i)) * g.c.n_kv + kvh) << psh) + (t & pmask);
    p.keys = (there >> i) & 1 ? sq.kv_len - t : 0;
    return p;
  };

  // a lane's share of a unit: words of one key; words (key pairs) of one quad of dims of 8 keys
  constexpr int KL = HD / 8 / WPL, SUBS = 4 / WPL;
  const int k_key = lane / KL, k_place = (lane % KL) * WPL;
  const int v_sub = (lane >> 4) % SUBS, v_rest = (lane >> 4) / SUBS;
  const int v_quad = 16 * (v_rest % NG) + (lane & 15), v_key = 8 * (v_rest / NG) + 2 * WPL * v_sub;
  // place in the stored row -> first dim (qmm_mix.h); a share of 4 words has two groups
  const int k_word = HD == 64 ? k_place : 16 * (k_place >> 4) + 8 * ((k_place >> 1) & 1) + 2 * ((k_place >> 2) & 3) + (k_place & 1);
  const int k_meta = HD == 64 ? 0 : 2 * (k_place >> 4) + ((k_place >> 1) & 1);
  const int k_dst = k_key * kRowK<HD> + 8 * k_word, v_dst = 4 * v_quad * kRowV + v_key;
  const int v_meta = v_key + (lane & (2 * WPL - 1));  // the key whose scale the lane fetches
  struct Codes {
    uint32_t w[WPL], m0, m1;
    int keys;
  };
  Codes ck[2][PER], cv[2][PER];  // of the next two tiles
  Place at[PER];
  auto load_k = [&](Codes (&xk)[PER], int i, int t0) {
    at[i] = place(t0 + UK * (wave + NW * i));
    load_words<WPL>(g.c.k_codes + at[i].row * (HD / 8) + (k_key * (HD / 8) + k_place), xk[i].w);
    const uint32_t* mp = g.c.k_meta + at[i].row * NG + (k_key * NG + k_meta);
    xk[i].m0 = mp[0];
    xk[i].m1 = WPL == 4 && HD > 64 ? mp[1] : 0u;
    xk[i].keys = at[i].keys;
  };
  auto load_v = [&](Codes (&xv)[PER], int i) {  // of the tile whose keys were loaded last
    load_words<WPL>(reinterpret_cast<const uint32_t*>(g.c.v_codes) + (at[i].row >> 3) * HD +
                        ((v_key >> 3) * HD + v_quad * 4 + WPL * v_sub), xv[i].w);
    xv[i].m0 = g.c.v_meta[at[i].row * NG + (v_meta * NG + (v_quad >> 4))];
    xv[i].keys = at[i].keys;
  };

  // Dequantization, a pair of codes at a time: K pair i of word j, stored with the word's
  // last; V dim j of key pair i, stored with the dim's last.  Absent keys become zeros (their
  // scales may be anything).
  constexpr int PAIRS = 4 * WPL * PER;
  const uint32_t magic = in_vgpr(0x64006400u);
  struct Half {
    f16x2_t s[4], b[4];
    uint32_t o[4];
  };
  Half hf;
  auto pair_k = [&](const Codes (&xk)[PER], auto ac, int buf) {
    constexpr int u = decltype(ac)::value / (4 * WPL), j = decltype(ac)::value / 4 % WPL, i = decltype(ac)::value % 4;
    if constexpr (i == 0) {
      const uint32_t m = HD == 64 || j < 2 ? xk[u].m0 : xk[u].m1;
      const f16x2_t sb = h2(k_key < xk[u].keys ? m : 0u);
      hf.s[0] = f16x2_t{sb[0], sb[0]}, hf.b[0] = f16x2_t{sb[1], sb[1]};
    }
    hf.o[i] = u32(__builtin_elementwise_fma(code_pair<i>(xk[u].w[j], magic), hf.s[0], hf.b[0]));
    if constexpr (i == 3) {
      constexpr int w = HD == 64 ? j : 8 * (j >> 1) + (j & 1);  // words from the share's first
      *reinterpret_cast<u32x4_t*>(&s_k[buf][UK * (wave + NW * u) * kRowK<HD> + k_dst + 8 * w]) =
          u32x4_t{hf.o[0], hf.o[1], hf.o[2], hf.o[3]};
    }
  };
  auto pair_v = [&](Codes (&xv)[PER], auto ac, int buf) {
    constexpr int u = decltype(ac)::value / (4 * WPL), j = decltype(ac)::value / WPL % 4, i = decltype(ac)::value % WPL;
    if constexpr (j == 0) {
      if constexpr (i == 0) xv[u].m0 = v_meta < xv[u].keys ? xv[u].m0 : 0u;
      const uint32_t a = __float_as_uint(row_bcast<2 * i>(__uint_as_float(xv[u].m0)));
      const uint32_t c = __float_as_uint(row_bcast<2 * i + 1>(__uint_as_float(xv[u].m0)));
      hf.s[i] = h2(__builtin_amdgcn_perm(c, a, 0x05040100u));
      hf.b[i] = h2(__builtin_amdgcn_perm(c, a, 0x07060302u));
    }
    hf.o[i] = u32(__builtin_elementwise_fma(code_pair<j>(xv[u].w[i], magic), hf.s[i], hf.b[i]));
    if constexpr (i == WPL - 1) {
      _Float16* d = &s_v[buf][UK * (wave + NW * u) + v_dst + j * kRowV];
      if constexpr (WPL == 4) *reinterpret_cast<u32x4_t*>(d) = u32x4_t{hf.o[0], hf.o[1], hf.o[2], hf.o[3]};
      else if constexpr (WPL == 2) *reinterpret_cast<uint2*>(d) = uint2{hf.o[0], hf.o[1]};
      else *reinterpret_cast<uint32_t*>(d) = hf.o[0];
    }
  };
  constexpr Int<0> kKeysHalf{};
  constexpr Int<1> kValuesHalf{};
  auto unpack = [&](auto half, auto set, auto ac, int buf) {
    if constexpr (decltype(ac)::value < PAIRS) {
      if constexpr (decltype(half)::value == 0) pair_k(ck[decltype(set)::value], ac, buf);
      else pair_v(cv[decltype(set)::value], ac, buf);
    }
  };

  // A row's reference maximum m follows its scores with a slack of 2^8; until the row has
  // seen a key, any score moves it.  `start` is -m: the products begin from it.
  f32x16_t acc[OT], start;
  float m = 0.f, l = 0.f, slack = -1e30f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    start[e] = 0.f;
#pragma unroll
    for (int i = 0; i < OT; ++i) acc[i][e] = 0.f;
  }
  // rows 8a + 4h + e of a product's 32 are keys 16 (a / 2) + 8h + 4 (a % 2) + e, so that a lane's
  // eight scores of 16 keys are neighbours
  const int krow = 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
  const int k_src = krow * kRowK<HD> + 8 * hh, v_src = n * kRowV + 8 * hh;

  // Hidden keys leave (blocks: which 16-key blocks there are); the reference maximum moves
  // where the scores ran away from it.  `mx`: the largest score if none is hidden.
  auto settle = [&](f32x16_t& sc, float mx, int tb, uint32_t blocks) {
    if (tb < u_lo || tb + 32 > u_hi || blocks != 3) {
      const int lo = c_lo - tb, hi = c_hi - tb;
      mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int k = 16 * (e >> 3) + 8 * hh + (e & 7);
        const bool see = ((blocks >> (e >> 3)) & 1) && k >= lo && k < hi;
        sc[e] = see ? sc[e] : -INFINITY;
        mx = fmaxf(mx, sc[e]);
      }
    }
    if (__any(mx > slack)) {
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const bool any = mx > -INFINITY, set = slack > 0.f;
      const float d = !any ? 0.f : set ? fmaxf(mx, 0.f) : mx;
      const float fac = set ? exp2_hw(-d) : 0.f;
      slack = any || set ? kSlack : slack;
      m += d;
      l *= fac;
#pragma unroll
      for (int i = 0; i < OT; ++i) acc[i] *= fac;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sc[e] -= d;
        start[e] = -m;
      }
    }
  };
  // One step of 32 keys.  First the next step's scores (keys kbuf, half ka) beside this step's
  // weights and a tile's loads, then this step's values (vbuf, half va) beside the next tile's
  // dequantization into buffer `dst` and the next scores' maximum.
  constexpr int NS = HD / 16, NV = 2 * OT, LEAD = 6, P = (PAIRS + NV - 1) / NV;
  auto step = [&](auto half, auto set, const f32x16_t& sc, f32x16_t& next, int kbuf, int ka, int vbuf, int va,
                  int t_load) {
    const int dst = vbuf ^ 1;
    const _Float16* kb = &s_k[kbuf][k_src + 32 * ka * kRowK<HD>];
    const _Float16* vb = &s_v[vbuf][v_src + 32 * va];
    f16x8_t kf[NS], vf[NV];
    f16x2_t p[8];
    auto read_k = [&](auto ec) {
      constexpr int e = decltype(ec)::value;
      if constexpr (e < NS) kf[e] = *reinterpret_cast<const f16x8_t*>(kb + 16 * e);
    };
    auto read_v = [&](auto qc) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q < NV) vf[q] = *reinterpret_cast<const f16x8_t*>(vb + 32 * (q % OT) * kRowV + 16 * (q / OT));
    };
    static_for<LEAD>([&](auto ec) {
      constexpr int e = decltype(ec)::value;
      if constexpr (e < NS) read_k(ec);
      else read_v(Int<e - NS>{});
    });
    next = start;
    static_for<NS>([&](auto ec) {
      constexpr int e = decltype(ec)::value;
      if constexpr (e + LEAD < NS) read_k(Int<e + LEAD>{});
      else read_v(Int<e + LEAD - NS>{});
      next = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[e], qf[e], next, 0, 0, 0);
      static_for<8>([&](auto wc) {  // this step's weights: elements 16 e / NS on
        constexpr int w = 2 * decltype(wc)::value;
        if constexpr (w * NS >= 16 * e && w * NS < 16 * (e + 1)) {
          p[w / 2] = f16x2_t{static_cast<_Float16>(exp2_hw(sc[w])), static_cast<_Float16>(exp2_hw(sc[w + 1]))};
          l = __builtin_amdgcn_fdot2(p[w / 2], f16x2_t{(_Float16)1.f, (_Float16)1.f}, l, false);
          asm volatile("" : "+v"(l));  // here, not behind the products
        }
      });
      // three tiles ahead: keys into the set that the step before emptied, values likewise
      if constexpr (e < PER && decltype(half)::value == 0) load_v(cv[1 - decltype(set)::value], e);
      if constexpr (e < PER && decltype(half)::value == 1) load_k(ck[decltype(set)::value], e, t_load);
      __builtin_amdgcn_sched_barrier(0);
    });
    f16x8_t pv[2];
#pragma unroll
    for (int e = 0; e < 16; ++e) pv[e >> 3][e & 7] = p[e >> 1][e & 1];
    float mx = -INFINITY;
    static_for<NV>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      read_v(Int<q + LEAD>{});
      acc[q % OT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[q], pv[q / OT], acc[q % OT], 0, 0, 0);
      static_for<P>([&](auto ic) { unpack(half, set, Int<q * P + decltype(ic)::value>{}, dst); });
      static_for<8>([&](auto wc) {  // behind the first products, when the scores are through
        constexpr int w = 2 * decltype(wc)::value;
        if constexpr (w * (NV / 4) >= 16 * (q - 3 * NV / 4) && w * (NV / 4) < 16 * (q + 1 - 3 * NV / 4)) {
          mx = fmaxf(fmaxf(mx, next[w]), next[w + 1]);
          if constexpr (w == 14) asm volatile("" : "+v"(mx));
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    return mx;
  };

  if (t_begin < t_end) {
    enter(pages_from(t_begin));
    pages_next = pages_from(t_begin + 1024);
    // 16-key blocks there are, of this tile and the next two
    auto blocks = [&](int t) { return uint32_t(there >> ((t - window) >> 4)) & 15; };
    uint32_t blocks0 = blocks(t_begin), blocks1 = blocks(t_begin + kKeys), blocks2 = blocks(t_begin + 2 * kKeys);
    static_for<PER>([&](auto i) {
      load_k(ck[0], i, t_begin);
      load_v(cv[0], i);
    });
    static_for<PER>([&](auto i) {
      load_k(ck[1], i, t_begin + kKeys);
      load_v(cv[1], i);
    });
    static_for<PAIRS>([&](auto a) { unpack(kKeysHalf, Int<0>{}, a, 0); });
    static_for<PAIRS>([&](auto a) { unpack(kValuesHalf, Int<0>{}, a, 0); });
    static_for<PER>([&](auto i) { load_k(ck[0], i, t_begin + 2 * kKeys); });
    __syncthreads();
    f32x16_t sc = start, next;
#pragma unroll
    for (int e = 0; e < NS; ++e)
      sc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8_t*>(&s_k[0][k_src + 16 * e]), qf[e],
                                                  sc, 0, 0, 0);
    float mx = sc[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[e]);
    settle(sc, mx, t_begin, blocks0 & 3);
    // a tile: `set` holds the next tile's codes, the other the one's after (its values are loaded
    // in the first step)
    auto tile = [&](auto set, int t0) {
      constexpr int buf = 1 - decltype(set)::value;
      mx = step(kKeysHalf, set, sc, next, buf, 1, buf, 0, 0);
      settle(next, mx, t0 + 32, blocks0 >> 2);
      __syncthreads();
      if (t0 + 3 * kKeys - window >= 1024) {  // the page window moves on
        window = t0 + 3 * kKeys;
        enter(pages_next);
        pages_next = pages_from(window + 1024);
      }
      mx = step(kValuesHalf, set, next, sc, buf ^ 1, 0, buf, 1, t0 + 3 * kKeys);
      blocks0 = blocks1, blocks1 = blocks2, blocks2 = blocks(t0 + 3 * kKeys);
      settle(sc, mx, t0 + kKeys, blocks0 & 3);
      __syncthreads();
    };
    for (int t0 = t_begin;;) {
      tile(Int<1>{}, t0);
      if ((t0 += kKeys) >= t_end) break;
      tile(Int<0>{}, t0);
      if ((t0 += kKeys) >= t_end) break;
    }
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
    pm[(split * R0 + qrow) * 2] = slack > 0.f ? m : kFloor;
    pm[(split * R0 + qrow) * 2 + 1] = l;
  }
}

template <int HD>
int launch(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int group = a.n_q / a.c.n_kv, tiles = int((int64_t(a.max_q) * group + p.rows - 1) / p.rows);
  kv4_prefill_kernel<HD>
      <<<dim3(uint32_t(p.nsplit), uint32_t(a.c.n_kv * tiles), uint32_t(a.B)), NW * 64, 0, s>>>(a, group, p, tiles);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

int launch_kv4_prefill(const Kv4AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  if (a.c.hd == 256) return launch<256>(a, p, s);
  return a.c.hd == 128 ? launch<128>(a, p, s) : launch<64>(a, p, s);
}

}  // namespace qmm
