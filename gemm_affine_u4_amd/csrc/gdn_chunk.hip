// The gated delta rule in chunks of 64 tokens on the matrix cores (qmm_gdn's prompt form).
//
// Mathematics.  With c_i the running sum of g inside a chunk, unit keys k, S the state at
// the chunk's start, L_ij = beta_i (k_i.k_j) e^{c_i - c_j} for j < i and T = (I + L)^-1:
//   D = T diag(beta) (V - diag(e^c) K S)          what the tokens really write
//   Y = scale (diag(e^c) Q S + tril((q_i.k_j) e^{c_i - c_j}) D)
//   S <- e^{c_64} S + K^T diag(e^{c_64 - c}) D
// every exponent <= 0.  T and the masked scores do not depend on the state, so a first launch
// (prep, parallel over chunks) computes them; a second walks each sequence's chunks in order,
// a block per value head and 16 NT of its Dv columns, with S in registers.
//
// Precision.  Keys, queries and values are bf16 and enter exactly (their norms are factors
// of rows).  An fp32 factor x enters as h + m + l, three bf16 values that hold its 24 bits; a
// product of two such factors takes the six partial products down to 2^-24.  What only a
// bf16 output reads (scores, D as their factor, S as Q's) enters as h + m: each part left out is at
// most 2^-16 of its product, 1/256 of that output's own rounding; an fp32 output takes l too (PO
// planes; the state always does).  T comes from
// forward substitution and fp32 matrix products; sums are fp32, the running sum of g fp64.
//
// Bound: the walk's stages, three barriers a chunk, one after the other.  A chunk takes 1.6 us with 16
// columns and 3.3 with 32, so a stage's time follows its work; matrix cores, vector unit and LDS
// are busy for 20, 33 and 28 % (21, 33 and 30 % with 32 columns) and a wave waits for half of its
// time, at barriers and for its own operands, with nothing beside it (loads that all hit L2 take
// off 5%).  All slices of a head sit on one XCD, so that its L2 serves them.  A wave's operands
// go straight to its registers, for the next chunk as soon as this one's were used.
//
// Measured: 4096 tokens, 32 heads x 128 x 128: prep 30 us, walk 104 to 111 us; 6813 tokens of six
// sequences, 48 heads: prep 77 us, walk 258 to 276 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdn.h"
#include "kv4_attn.h"
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
constexpr int C = 64;  // tokens of a chunk

// Workspace of one (chunk, value head): operands in fragment order (1 KB: 64 lanes x 16 bytes),
// then the tokens' factors.  Fragments of T diag(beta) and of the scores: row tile w (16
// tokens), 32 columns s <= w / 2, plane p; tiles 0, 1 have one s, tiles 2, 3 two.
constexpr int kTri = 6;                        // (w, s) pairs
__host__ __device__ constexpr int tri_at(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }
constexpr int64_t kFragM = 0, kFragA = kTri * 3 * 1024, kFactors = 2 * kTri * 3 * 1024;
constexpr int64_t kHeadBytes = kFactors + C * 16;
// Workspace of one (chunk, key head): K^T (dim tiles x 2 token halves), K and Q (quarters of
// the dims x row tiles), each as a wave of the walk loads it: read by rows, the 16 lanes of a
// load's quarter would touch 16 cache lines.
__host__ __device__ constexpr int64_t part_bytes(int64_t dk) { return dk * C * 2; }
__host__ __device__ constexpr int64_t key_bytes(int64_t dk) { return 3 * part_bytes(dk); }

__device__ __forceinline__ bf16x8_t frag8(const u32x4_t& v) { return __builtin_bit_cast(bf16x8_t, v); }
__device__ __forceinline__ f32x4_t mma(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag8(a), frag8(b), c, 0, 0, 0);
}

// (x, y) as three words of bf16 pairs that add up to them.
__device__ __forceinline__ void split2(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack_bf16x2(x, y);
  x -= bf16_lo(h), y -= bf16_hi(h);
  m = pack_bf16x2(x, y);
  x -= bf16_lo(m), y -= bf16_hi(m);
  l = pack_bf16x2(x, y);
}

__device__ __forceinline__ int64_t chunk_slot(const GdnSeq& s, int b, int c) { return (s.t0 >> 6) + c + b; }

// ---- prep: one (chunk, value head) ---------------------------------------------------------

// Wave w makes row tile w (16 tokens) of L, T and the scores, as transposed products: lane
// (n, hg) then holds columns 4 hg .. +3 of every 16 of row n, which is the fragment order that the
// walk loads, with the tokens of a 32-wide step taken as 16 (j / 4) + 4 hg + j % 4.
template <int DK, int PO>
__global__ __launch_bounds__(256, 4) void gdn_prep_kernel(GdnArgs g, int64_t n_slots_ws) {
  constexpr int KSTEP = DK / 32;
  constexpr int LS = 20;  // LDS row of a 16 x 16 fp32 tile
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x, hv = blockIdx.y, b = blockIdx.z, rep = g.Hv / g.Hk, hk = hv / rep;
  const GdnSeq sq = gdn_seq(g, b);
  if (c * C >= sq.len) return;
  const int left = sq.len - c * C;  // tokens from the chunk's start on
  const int64_t tok0 = int64_t(sq.t0) + c * C;

  __shared__ u32x4_t s_k[4][KSTEP][64];
  __shared__ __attribute__((aligned(16))) float s_l[10][16 * LS], s_t[4][16 * LS];
  __shared__ __attribute__((aligned(16))) float s_rk[C], s_rq[C], s_beta[C], s_hi[C], s_lo[C];
  auto tile = [](int i, int j) { return i * (i + 1) / 2 + j; };

  // keys and queries of the wave's rows; tokens behind the sequence repeat its last one (their beta is 0)
  const int row = 16 * w + n;
  u32x4_t ak[KSTEP], aq[KSTEP];
  {
    const int64_t at = ((tok0 + (row < left ? row : left - 1)) * g.Hk + hk) * DK;
#pragma unroll
    for (int s = 0; s < KSTEP; ++s) {
      if constexpr (DK == 128) {
        ak[s] = *reinterpret_cast<const u32x4_t*>(g.k + at + 32 * s + 8 * hg);
        aq[s] = *reinterpret_cast<const u32x4_t*>(g.q + at + 32 * s + 8 * hg);
      } else {
        const uint16_t *kp = g.k + at + 32 * s + 4 * hg, *qp = g.q + at + 32 * s + 4 * hg;
        const uint2 k0 = *reinterpret_cast<const uint2*>(kp), k1 = *reinterpret_cast<const uint2*>(kp + 16);
        const uint2 q0 = *reinterpret_cast<const uint2*>(qp), q1 = *reinterpret_cast<const uint2*>(qp + 16);
        ak[s] = u32x4_t{k0.x, k0.y, k1.x, k1.y};
        aq[s] = u32x4_t{q0.x, q0.y, q1.x, q1.y};
      }
    }
  }
  if (w == 0) {
    const bool in = lane < left;
    const int64_t at = (tok0 + (in ? lane : left - 1)) * g.Hv + hv;
    s_beta[lane] = in ? g.beta[at] : 0.f;
    // e^-200 is 0 in fp32 as all below it are: held there, the chunk's sums stay exact and finite
    double x = in ? double(fmaxf(g.g[at], -200.f)) : 0.0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    x *= 1.4426950408889634;  // in powers of two
    const float hi = float(x);
    s_hi[lane] = hi;
    s_lo[lane] = float(x - double(hi));
  }
  float rk = 1.f, rq = 1.f;
#pragma unroll
  for (int s = 0; s < KSTEP; ++s) s_k[w][s][lane] = ak[s];
  if (g.l2norm) {
    rk = rq = 0.f;
#pragma unroll
    for (int s = 0; s < KSTEP; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rk = fmaf(bf16_lo(ak[s][i]), bf16_lo(ak[s][i]), fmaf(bf16_hi(ak[s][i]), bf16_hi(ak[s][i]), rk));
        rq = fmaf(bf16_lo(aq[s][i]), bf16_lo(aq[s][i]), fmaf(bf16_hi(aq[s][i]), bf16_hi(aq[s][i]), rq));
      }
    }
    rk += __shfl_xor(rk, 16), rq += __shfl_xor(rq, 16);
    rk += __shfl_xor(rk, 32), rq += __shfl_xor(rq, 32);
    rk = 1.f / sqrtf(rk + kGdnEps), rq = 1.f / sqrtf(rq + kGdnEps);
  }
  rq *= g.scale;
  if (hg == 0) s_rk[row] = rk, s_rq[row] = rq;
  __syncthreads();

  const int64_t slot = chunk_slot(sq, b, c);
  unsigned char* ws = static_cast<unsigned char*>(g.ws);
  unsigned char* mine = ws + (slot * g.Hv + hv) * kHeadBytes;
  if (hv % rep == 0) {  // fragments of K^T, K and Q, once per key head
    unsigned char* kt = ws + n_slots_ws * g.Hv * kHeadBytes + (slot * g.Hk + hk) * key_bytes(DK);
    unsigned char *kf = kt + part_bytes(DK), *qf = kf + part_bytes(DK);
#pragma unroll
    for (int s = 0; s < KSTEP; ++s) {
      if constexpr (DK == 128) {
        const int at = s * 4096 + w * 1024 + lane * 16;
        *reinterpret_cast<u32x4_t*>(kf + at) = ak[s];
        *reinterpret_cast<u32x4_t*>(qf + at) = aq[s];
      } else {
        const int at = s * 4096 + w * 512 + lane * 8;
        *reinterpret_cast<uint2*>(kf + at) = uint2{ak[s][0], ak[s][1]};
        *reinterpret_cast<uint2*>(kf + at + 2048) = uint2{ak[s][2], ak[s][3]};
        *reinterpret_cast<uint2*>(qf + at) = uint2{aq[s][0], aq[s][1]};
        *reinterpret_cast<uint2*>(qf + at + 2048) = uint2{aq[s][2], aq[s][3]};
      }
    }
#pragma unroll
    for (int f = 0; f < DK / 16 * 2 / 4; ++f) {
      const int fr = f * 4 + w, dt = fr >> 1, s = fr & 1;  // dim tile, token half
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(
                                &s_k[2 * s + (i >> 1)][dt >> 1][(n >> 2) * 16 + 4 * hg + 2 * (i & 1)]) +
                            4 * (dt & 1) + (n & 3);
        v[i] = uint32_t(p[0]) | (uint32_t(p[8]) << 16);
      }
      *reinterpret_cast<u32x4_t*>(kt + fr * 1024 + lane * 16) = v;
    }
  }
  // row tile w of K K^T and Q K^T, transposed
  const float beta = s_beta[row], hi = s_hi[row], lo = s_lo[row];
  f32x4_t sc[4] = {};  // the scores
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j > w) continue;
    f32x4_t kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
    for (int s = 0; s < KSTEP; ++s) {
      const u32x4_t bk = s_k[j][s][lane];
      kk = mma(bk, ak[s], kk);
      qk = mma(bk, aq[s], qk);
    }
    const int col = 16 * j + 4 * hg;
    const f32x4_t rkc = *reinterpret_cast<const f32x4_t*>(&s_rk[col]), hic = *reinterpret_cast<const f32x4_t*>(&s_hi[col]),
                  loc = *reinterpret_cast<const f32x4_t*>(&s_lo[col]);
    f32x4_t l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float fall = row >= col + i ? exp2_hw((hi - hic[i]) + (lo - loc[i])) : 0.f;
      l[i] = row > col + i ? beta * rk * rkc[i] * fall * kk[i] : 0.f;
      sc[j][i] = row >= col + i ? rq * rkc[i] * fall * qk[i] : 0.f;
    }
    *reinterpret_cast<f32x4_t*>(&s_l[tile(w, j)][n * LS + 4 * hg]) = l;
  }
  auto put = [&](int64_t part, int planes, int s, const f32x4_t& x0, const f32x4_t& x1) {
    u32x4_t f[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t& x = i < 2 ? x0 : x1;
      uint32_t h, m, l;
      split2(x[2 * (i & 1)], x[2 * (i & 1) + 1], h, m, l);
      f[0][i] = h, f[1][i] = m, f[2][i] = l;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      if (p < planes) *reinterpret_cast<u32x4_t*>(mine + part + (tri_at(w, s) * 3 + p) * 1024 + uint32_t(lane * 16)) = f[p];
    }
  };
  put(kFragA, PO, 0, sc[0], sc[1]);
  if (w >= 2) put(kFragA, PO, 1, sc[2], sc[3]);
  // T_ww by forward substitution, column n in each lane of it ...
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  {
    float x[16];
    const float* lb = s_l[tile(w, w)];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a = i == n ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) a = fmaf(-lb[i * LS + j], x[j], a);
      x[i] = a;
      if ((i >> 2) == hg) s_t[w][i * LS + n] = a;
    }
  }
  __syncthreads();
  // ... and left of it, T (I + L) = I: T_wj = -(sum_{k > j} T_wk L_kj) T_jj, all in this wave
  f32x4_t tt[4] = {};
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    if (j > w) continue;
    if (j == w) {
      tt[j] = *reinterpret_cast<const f32x4_t*>(&s_t[w][n * LS + 4 * hg]);
      continue;
    }
    f32x4_t x = {0.f, 0.f, 0.f, 0.f}, t = x;
#pragma unroll
    for (int k = j + 1; k < 4; ++k) {
      if (k > w) continue;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x = __builtin_amdgcn_mfma_f32_16x16x4f32(s_l[tile(k, j)][(4 * hg + s) * LS + n], tt[k][s], x, 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
      t = __builtin_amdgcn_mfma_f32_16x16x4f32(-s_t[j][(4 * hg + s) * LS + n], x[s], t, 0, 0, 0);
    tt[j] = t;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) tt[j] *= *reinterpret_cast<const f32x4_t*>(&s_beta[16 * j + 4 * hg]);
  put(kFragM, 3, 0, tt[0], tt[1]);
  if (w >= 2) put(kFragM, 3, 1, tt[2], tt[3]);
  if (tid < C) {  // factors of the rows: of K S, of Q S, of K in the state's update; the state's decay
    const float top = s_hi[C - 1], tol = s_lo[C - 1];
    const float e = exp2_hw(s_hi[tid] + s_lo[tid]);
    const bool in = tid < left;
    float* f = reinterpret_cast<float*>(mine + kFactors);
    f[tid] = in ? e * s_rk[tid] : 0.f;
    f[C + tid] = in ? e * s_rq[tid] : 0.f;
    f[2 * C + tid] = in ? exp2_hw((top - s_hi[tid]) + (tol - s_lo[tid])) * s_rk[tid] : 0.f;
    f[3 * C + tid] = exp2_hw(top + tol);
  }
}

// ---- walk: one value head's 16 NT columns through a sequence -------------------------------

// Eight waves.  Four carry the state: wave w holds dims w DK/4 .. of it in registers, in an
// order that makes them the operand of K S and Q S as they stand, so only sums of partial
// products, X, D and U = D e^{c_64 - c} cross waves (LDS, three barriers a chunk).  The other four
// make the outputs of the chunk whose D they were given while the first four go on.
template <int DK, int NT, int PO>
__global__ __launch_bounds__(512, 2) void gdn_walk_kernel(GdnArgs g, int64_t n_slots_ws, int slices, int heads) {
  constexpr int XS = C + 8;    // LDS row of a column's tokens in bf16 ...
  constexpr int DS = C + 4;    // ... and in fp32
  constexpr int DT = DK / 64;  // dim tiles of a wave
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  // block L runs on XCD L % 8: the slices of a (sequence, head) share one
  const int xi = int(blockIdx.x) >> 3, unit = (int(blockIdx.x) & 7) + 8 * (xi / slices), slice = xi % slices;
  if (unit >= heads) return;
  const int b = unit / g.Hv, hv = unit % g.Hv, hk = hv / (g.Hv / g.Hk);
  const GdnSeq sq = gdn_seq(g, b);
  const bool kept = uint32_t(sq.slot) < uint32_t(g.n_slots);
  if (sq.len == 0 && (!kept || g.state_in == g.state_out)) return;

  __shared__ f32x4_t s_ks[4][NT][4][64], s_qs[4][NT][4][64];  // partial sums: of wave, for row tile
  __shared__ __attribute__((aligned(16))) uint16_t s_x[3][16 * NT * XS], s_u[3][16 * NT * XS];
  __shared__ __attribute__((aligned(16))) float s_d[16 * NT * DS];

  const int v0 = slice * 16 * NT;
  const int chunks = (sq.len + C - 1) / C;
  const unsigned char* ws = static_cast<const unsigned char*>(g.ws);
  const unsigned char* head0 = ws + (chunk_slot(sq, b, 0) * g.Hv + hv) * kHeadBytes;
  const int64_t head_step = g.Hv * kHeadBytes;
  auto head_at = [&](int c) { return head0 + c * head_step; };
  // A column's tokens of V and y: 32 bits from the chunk's first one (64 rows of Hv Dv).
  const uint32_t row_bytes = uint32_t(g.Hv) * uint32_t(g.Dv) * 2u;
  auto load_tri = [&](int c, int64_t part, int planes, u32x4_t (&f)[2][3]) {
    const unsigned char* at = head_at(c) + part;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        if (p < planes)
          f[s][p] = *reinterpret_cast<const u32x4_t*>(at + (tri_at(w, s <= (w >> 1) ? s : 0) * 3 + p) * 1024 + uint32_t(lane * 16));
      }
    }
  };
  // the partial products that `planes` planes can hold
  auto mma_planes = [&](int planes, const u32x4_t (&f)[3], const u32x4_t (&x)[3], f32x4_t (&a)[3]) {
    a[0] = mma(f[0], x[0], a[0]);
    a[1] = mma(f[0], x[1], a[1]);
    if (planes == 3) a[2] = mma(f[0], x[2], a[2]);
    a[1] = mma(f[1], x[0], a[1]);
    if (planes == 3) a[2] = mma(f[1], x[1], a[2]);
    if (planes == 3) a[2] = mma(f[2], x[0], a[2]);
  };

  if (wave >= 4) {  // outputs
    u32x4_t fa[2][3];
    f32x4_t fy;
    auto load = [&](int c) {
      load_tri(c, kFragA, PO, fa);
      fy = *reinterpret_cast<const f32x4_t*>(head_at(c) + kFactors + (C + 16 * w) * 4 + uint32_t(hg * 16));
    };
    if (chunks) load(0);
    for (int c = 0; c < chunks; ++c) {
      __syncthreads();
      __syncthreads();
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4_t a[3] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s > (w >> 1)) continue;
          const float* at = &s_d[(16 * nt + n) * DS + 32 * s + 8 * hg];
          const f32x4_t d0 = *reinterpret_cast<const f32x4_t*>(at), d1 = *reinterpret_cast<const f32x4_t*>(at + 4);
          u32x4_t x[3];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h, m, l;
            if (i < 2) split2(d0[2 * i], d0[2 * i + 1], h, m, l);
            else split2(d1[2 * i - 4], d1[2 * i - 3], h, m, l);
            x[0][i] = h, x[1][i] = m, x[2][i] = l;
          }
          mma_planes(PO, fa[s], x, a);
        }
        const f32x4_t q = (s_qs[0][nt][w][lane] + s_qs[1][nt][w][lane]) + (s_qs[2][nt][w][lane] + s_qs[3][nt][w][lane]);
        const f32x4_t y = a[0] + (a[1] + a[2]);
        f32x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(fy[i], q[i], y[i]);
        asm volatile("" : "+v"(v));  // whole before the branches, which else wait for each other's stores
        const int left = sq.len - c * C - 16 * w;  // tokens from the row tile's first on
        const int64_t y0 = ((int64_t(sq.t0) + c * C + 16 * w) * g.Hv + hv) * g.Dv + v0 + 16 * nt;
        const uint32_t at = uint32_t(4 * hg) * row_bytes + uint32_t(2 * n);
        if (g.f32_out) {
          unsigned char* to = static_cast<unsigned char*>(g.y) + y0 * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * hg + i < left) *reinterpret_cast<float*>(to + uint64_t(at + uint32_t(i) * row_bytes) * 2) = v[i];
        } else {
          unsigned char* to = static_cast<unsigned char*>(g.y) + y0 * 2;
          uint16_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = f32_to_bf16_bits(v[i]);
          if (left >= 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint16_t*>(to + (at + uint32_t(i) * row_bytes)) = r[i];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (4 * hg + i < left) *reinterpret_cast<uint16_t*>(to + (at + uint32_t(i) * row_bytes)) = r[i];
          }
        }
      }
      if (c + 1 < chunks) load(c + 1);
    }
    return;
  }

  // state: row 4 hg + i of tile dt is dim w DK/4 + 4 DT hg + 4 dt + i, column v0 + 16 nt + n
  const int64_t sbase = ((int64_t(kept ? sq.slot : 0) * g.Hv + hv) * g.Dv + v0 + n) * DK + w * (DK / 4) + 4 * DT * hg;
  f32x4_t st[DT][NT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      st[dt][nt] = kept ? *reinterpret_cast<const f32x4_t*>(g.state_in + sbase + int64_t(16 * nt) * DK + 4 * dt)
                        : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  // rows 16 w + 4 hg .. +3 of a column stand where a fragment's lane finds its eight in one piece
  const int pos = 32 * (w >> 1) + 8 * hg + 4 * (w & 1);
  auto put4 = [&](uint16_t (*pl)[16 * NT * XS], int nt, f32x4_t x) {  // of column 16 nt + n
    uint32_t h0, m0, l0, h1, m1, l1;
    split2(x[0], x[1], h0, m0, l0);
    split2(x[2], x[3], h1, m1, l1);
    const int at = (16 * nt + n) * XS + pos;
    *reinterpret_cast<uint2*>(&pl[0][at]) = uint2{h0, h1};
    *reinterpret_cast<uint2*>(&pl[1][at]) = uint2{m0, m1};
    *reinterpret_cast<uint2*>(&pl[2][at]) = uint2{l0, l1};
  };
  auto get = [&](const uint16_t (*pl)[16 * NT * XS], int nt, int s, u32x4_t (&x)[3]) {
#pragma unroll
    for (int p = 0; p < 3; ++p)
      x[p] = *reinterpret_cast<const u32x4_t*>(&pl[p][(16 * nt + n) * XS + 32 * s + 8 * hg]);
  };

  const unsigned char* key0 = ws + n_slots_ws * g.Hv * kHeadBytes + (chunk_slot(sq, b, 0) * g.Hk + hk) * key_bytes(DK);
  const int64_t key_step = g.Hk * key_bytes(DK);
  auto key_at = [&](int c) { return key0 + c * key_step; };
  u32x4_t fk[4], fq[4], fm[2][3], ft[DT][2];
  f32x4_t fx, fz;
  float decay;
  uint16_t fv[NT][4];
  auto load_rows = [&](int part, int c, u32x4_t (&f)[4]) {  // this wave's dims of all 64 tokens: K (1), Q (2)
    const unsigned char* at = key_at(c) + part * part_bytes(DK) + w * (512 * 4 * DT);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (DT == 2) {
        f[t] = *reinterpret_cast<const u32x4_t*>(at + t * 1024 + uint32_t(lane * 16));
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(at + t * 512 + uint32_t(lane * 8));
        f[t] = u32x4_t{v.x, v.y, 0u, 0u};
      }
    }
  };
  uint32_t voff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) voff[i] = uint32_t(16 * w + 4 * hg + i) * row_bytes;
  auto load_v = [&](int c) {
    const int left = sq.len - c * C;
    const uint32_t last = uint32_t(left < C ? left - 1 : C - 1) * row_bytes;
    const unsigned char* from = reinterpret_cast<const unsigned char*>(g.v) +
                                2 * (((int64_t(sq.t0) + c * C) * g.Hv + hv) * g.Dv + v0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the sequence's last token stands for those behind it
      const uint32_t at = voff[i] < last ? voff[i] : last;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        fv[nt][i] = *reinterpret_cast<const uint16_t*>(from + 32 * nt + (at + uint32_t(2 * n)));
    }
  };
  auto load_fac = [&](int c, int which) {
    return *reinterpret_cast<const f32x4_t*>(head_at(c) + kFactors + (which * C + 16 * w) * 4 + uint32_t(hg * 16));
  };
  auto load_decay = [&](int c) { return *reinterpret_cast<const float*>(head_at(c) + kFactors + 3 * C * 4 + uint32_t(lane * 4)); };
  auto load_kt = [&](int c) {
    const unsigned char* kt = key_at(c) + w * (2048 * DT);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ft[dt][s] = *reinterpret_cast<const u32x4_t*>(kt + (dt * 2 + s) * 1024 + uint32_t(lane * 16));
    }
  };
  if (chunks) {
    load_rows(1, 0, fk);
    fx = load_fac(0, 0);
    load_v(0);
    load_rows(2, 0, fq);
    load_tri(0, kFragM, 3, fm);
    fz = load_fac(0, 2);
    decay = load_decay(0);
    load_kt(0);
  }
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {  // arrived before the loop, which then counts its own loads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) asm volatile("" : "+v"(st[dt][nt]));
  }
  auto chunk = [&](int c, auto more) {  // more: load the next one's operands as this one's were used
    const int cn = c + 1;
    u32x4_t sp[NT][3];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h = 0, m = 0, l = 0;
        if (i / 2 < DT) split2(st[i / 2 < DT ? i / 2 : 0][nt][2 * (i & 1)], st[i / 2 < DT ? i / 2 : 0][nt][2 * (i & 1) + 1], h, m, l);
        sp[nt][0][i] = h, sp[nt][1][i] = m, sp[nt][2][i] = l;
      }
    }
    // K S: this wave's dims, smallest parts first
    f32x4_t ks[NT][4], qs[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int p = 2; p >= 0; --p) {
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[nt][t] = mma(fk[t], sp[nt][p], p == 2 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : ks[nt][t]);
      }
    }
    if constexpr (more.value) load_rows(1, cn, fk);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int t = 0; t < 4; ++t) s_ks[w][nt][t][lane] = ks[nt][t];
    }
    __syncthreads();
    f32x4_t x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = s_ks[i][nt][w][lane];
    }
    auto qs_mul = [&](int t0) {  // Q S of two row tiles, while LDS answers
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int p = PO - 1; p >= 0; --p) {
#pragma unroll
          for (int t = t0; t < t0 + 2; ++t)
            qs[nt][t] = mma(fq[t], sp[nt][p], p == PO - 1 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : qs[nt][t]);
        }
      }
    };
    qs_mul(0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const f32x4_t sum = (x[nt][0] + x[nt][1]) + (x[nt][2] + x[nt][3]);
      f32x4_t r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = fmaf(-fx[i], sum[i], bf16_bits_to_f32(fv[nt][i]));
      put4(s_x, nt, r);
    }
    if constexpr (more.value) fx = load_fac(cn, 0);
    if constexpr (more.value) load_v(cn);
    __syncthreads();
    qs_mul(2);
    if constexpr (more.value) load_rows(2, cn, fq);
    // D, as it is (for the outputs) and faded to the chunk's end (for the state)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4_t a[3] = {};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s > (w >> 1)) continue;
        u32x4_t xp[3];
        get(s_x, nt, s, xp);
        mma_planes(3, fm[s], xp, a);
      }
      const f32x4_t d = a[0] + (a[1] + a[2]);
      *reinterpret_cast<f32x4_t*>(&s_d[(16 * nt + n) * DS + pos]) = d;
      put4(s_u, nt, d * fz);
#pragma unroll
      for (int t = 0; t < 4; ++t) s_qs[w][nt][t][lane] = qs[nt][t];
    }
    if constexpr (more.value) load_tri(cn, kFragM, 3, fm);
    if constexpr (more.value) fz = load_fac(cn, 2);
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4_t a[DT][2];
      u32x4_t up[2][3];
      get(s_u, nt, 0, up[0]);
      get(s_u, nt, 1, up[1]);
#pragma unroll
      for (int p = 2; p >= 0; --p) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
#pragma unroll
          for (int s = 0; s < 2; ++s) a[dt][s] = mma(ft[dt][s], up[s][p], p == 2 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : a[dt][s]);
        }
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) st[dt][nt] = st[dt][nt] * decay + (a[dt][0] + a[dt][1]);
    }
    if constexpr (more.value) load_kt(cn);
    if constexpr (more.value) decay = load_decay(cn);
  };
  for (int c = 0; c + 1 < chunks; ++c) chunk(c, std::true_type{});
  if (chunks) chunk(chunks - 1, std::false_type{});
  if (kept) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<f32x4_t*>(g.state_out + sbase + int64_t(16 * nt) * DK + 4 * dt) = st[dt][nt];
    }
  }
}

int64_t ws_slots(int64_t T, int64_t B) { return T / C + B + 1; }

template <int DK, int NT, int PO>
void walk(const GdnArgs& a, int64_t n, hipStream_t s) {
  const int slices = a.Dv / (16 * NT), heads = a.B * a.Hv;
  const uint32_t grid = uint32_t((heads + 7) / 8 * 8) * uint32_t(slices);
  gdn_walk_kernel<DK, NT, PO><<<dim3(grid), 512, 0, s>>>(a, n, slices, heads);
}

template <int DK, int PO>
int launch(const GdnArgs& a, hipStream_t s) {
  const int64_t n = ws_slots(a.T, a.B);
  const uint32_t chunks = uint32_t((int64_t(a.max_len < a.T ? a.max_len : a.T) + C - 1) / C);
  gdn_prep_kernel<DK, PO><<<dim3(chunks ? chunks : 1, uint32_t(a.Hv), uint32_t(a.B)), 256, 0, s>>>(a, n);
  if (hipGetLastError() != hipSuccess) return 6;
  // 32 columns a block share its operands' loads where 16 would more than fill the GPU (six
  // ragged sequences of 48 heads: walk 269 us, with 16 columns 356 us)
  if (int64_t(a.B) * a.Hv * (a.Dv / 16) > int64_t(device_cus())) walk<DK, 2, PO>(a, n, s);
  else walk<DK, 1, PO>(a, n, s);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

uint64_t gdn_chunk_workspace(int64_t T, int64_t B, int64_t Hk, int64_t Hv, int64_t Dk) {
  return uint64_t(ws_slots(T, B)) * uint64_t(Hv * kHeadBytes + Hk * key_bytes(Dk));
}

int launch_gdn_chunk(const GdnArgs& a, hipStream_t s) {
  if (a.f32_out) return a.Dk == 64 ? launch<64, 3>(a, s) : launch<128, 3>(a, s);
  return a.Dk == 64 ? launch<64, 2>(a, s) : launch<128, 2>(a, s);
}

}  // namespace qmm
