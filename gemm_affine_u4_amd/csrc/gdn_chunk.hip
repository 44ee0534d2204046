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
// product of two such factors takes the six partial products down to 2^-24.  T comes from
// forward substitution and fp32 matrix products; sums are fp32, the running sum of g fp64.
//
// Bound: latency of the chunk's dependent products for few sequences (three barriers a
// chunk), the loads of T, scores and keys from L2 for many.  All slices of a head sit on
// one XCD, so that its L2 serves them.  The operands that only one wave needs go straight to
// its registers, for the next chunk as soon as this one's were used.
#include <hip/hip_runtime.h>

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

template <int DK>
__global__ __launch_bounds__(256) void gdn_prep_kernel(GdnArgs g, int64_t n_slots_ws) {
  constexpr int KS = DK + 8;   // LDS row of keys, in bf16: 16-byte reads of 16 rows meet no bank twice
  constexpr int FS = C + 4;    // LDS row of a 64 x 64 fp32 matrix
  constexpr int DT = DK / 64;  // dim tiles of a wave of the walk
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x, hv = blockIdx.y, b = blockIdx.z, rep = g.Hv / g.Hk, hk = hv / rep;
  const GdnSeq sq = gdn_seq(g, b);
  if (c * C >= sq.len) return;
  const int left = sq.len - c * C;  // tokens from the chunk's start on
  const int64_t tok0 = int64_t(sq.t0) + c * C;

  constexpr int kKQ = 2 * C * KS * 2, kLA = 2 * C * FS * 4;
  __shared__ __attribute__((aligned(16))) unsigned char s_pool[(kKQ > kLA ? kKQ : kLA)];
  uint16_t* s_k = reinterpret_cast<uint16_t*>(s_pool);
  uint16_t* s_q = s_k + C * KS;
  float* s_l = reinterpret_cast<float*>(s_pool);  // over the keys, once they are used
  float* s_a = s_l + C * FS;
  __shared__ __attribute__((aligned(16))) float s_t[C * FS];
  __shared__ float s_rk[C], s_rq[C], s_beta[C], s_hi[C], s_lo[C];

  // keys and queries; tokens behind the sequence repeat its last one (their beta is 0)
  constexpr int LPR = DK / 8;
#pragma unroll
  for (int it = 0; it < C * LPR / 256; ++it) {
    const int e = it * 256 + tid, r = e / LPR, d = (e % LPR) * 8;
    const int64_t tok = tok0 + (r < left ? r : left - 1);
    const int64_t at = (tok * g.Hk + hk) * DK + d;
    const u32x4_t kv = *reinterpret_cast<const u32x4_t*>(g.k + at), qv = *reinterpret_cast<const u32x4_t*>(g.q + at);
    *reinterpret_cast<u32x4_t*>(s_k + r * KS + d) = kv;
    *reinterpret_cast<u32x4_t*>(s_q + r * KS + d) = qv;
    float kk = 0.f, qq = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kk = fmaf(bf16_lo(kv[i]), bf16_lo(kv[i]), fmaf(bf16_hi(kv[i]), bf16_hi(kv[i]), kk));
      qq = fmaf(bf16_lo(qv[i]), bf16_lo(qv[i]), fmaf(bf16_hi(qv[i]), bf16_hi(qv[i]), qq));
    }
    if (g.l2norm) {
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) kk += __shfl_xor(kk, o), qq += __shfl_xor(qq, o);
      kk = 1.f / sqrtf(kk + kGdnEps), qq = 1.f / sqrtf(qq + kGdnEps);
    } else {
      kk = qq = 1.f;
    }
    if (d == 0) s_rk[r] = kk, s_rq[r] = qq * g.scale;
  }
  if (w == 0) {
    const bool in = lane < left;
    const int64_t at = (tok0 + (in ? lane : left - 1)) * g.Hv + hv;
    s_beta[lane] = in ? g.beta[at] : 0.f;
    double x = in ? double(g.g[at]) : 0.0;
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
  __syncthreads();

  const int64_t slot = chunk_slot(sq, b, c);
  unsigned char* ws = static_cast<unsigned char*>(g.ws);
  unsigned char* mine = ws + (slot * g.Hv + hv) * kHeadBytes;
  if (hv % rep == 0) {  // K^T fragments, once per key head
    unsigned char* kt = ws + n_slots_ws * g.Hv * kHeadBytes + (slot * g.Hk + hk) * key_bytes(DK);
#pragma unroll
    for (int f = 0; f < DK / 16 * 2 / 4; ++f) {
      const int fr = f * 4 + w, s = fr & 1;
      const int dim = (fr >> 1) / DT * (DK / 4) + 4 * DT * (n >> 2) + 4 * ((fr >> 1) % DT) + (n & 3);
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* p = s_k + (32 * s + 8 * hg + 2 * i) * KS + dim;
        v[i] = uint32_t(p[0]) | (uint32_t(p[KS]) << 16);
      }
      *reinterpret_cast<u32x4_t*>(kt + fr * 1024 + lane * 16) = v;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int from = (16 * t + n) * KS + w * (DK / 4) + 4 * DT * hg;
      unsigned char* to = kt + part_bytes(DK) + ((w * 4 + t) * 64 + lane) * (8 * DT);
      if constexpr (DT == 2) {
        *reinterpret_cast<u32x4_t*>(to) = *reinterpret_cast<const u32x4_t*>(s_k + from);
        *reinterpret_cast<u32x4_t*>(to + part_bytes(DK)) = *reinterpret_cast<const u32x4_t*>(s_q + from);
      } else {
        *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(s_k + from);
        *reinterpret_cast<uint2*>(to + part_bytes(DK)) = *reinterpret_cast<const uint2*>(s_q + from);
      }
    }
  }
  // row tile w of K K^T and Q K^T
  f32x4_t kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = qk[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (j > w) continue;
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      const u32x4_t bk = *reinterpret_cast<const u32x4_t*>(s_k + (16 * j + n) * KS + 32 * s + 8 * hg);
      const u32x4_t ak = *reinterpret_cast<const u32x4_t*>(s_k + (16 * w + n) * KS + 32 * s + 8 * hg);
      const u32x4_t aq = *reinterpret_cast<const u32x4_t*>(s_q + (16 * w + n) * KS + 32 * s + 8 * hg);
      kk[j] = mma(ak, bk, kk[j]);
      qk[j] = mma(aq, bk, qk[j]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 16 * j + n;
    const float rkj = s_rk[col], hj = s_hi[col], lj = s_lo[col];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * w + 4 * hg + i;
      const float fall = row >= col ? exp2_hw((s_hi[row] - hj) + (s_lo[row] - lj)) : 0.f;
      s_l[row * FS + col] = row > col ? s_beta[row] * s_rk[row] * rkj * fall * kk[j][i] : 0.f;
      s_a[row * FS + col] = row >= col ? s_rq[row] * rkj * fall * qk[j][i] : 0.f;
      s_t[row * FS + col] = 0.f;
    }
  }
  __syncthreads();
  // T: the four diagonal blocks by forward substitution (lane: block hg, column n) ...
  if (w == 0) {
    float x[16];
    const float* lb = s_l + (16 * hg) * FS + 16 * hg;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a = i == n ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) a = fmaf(-lb[i * FS + j], x[j], a);
      x[i] = a;
      s_t[(16 * hg + i) * FS + 16 * hg + n] = a;
    }
  }
  __syncthreads();
  // ... and below them T_ij = -T_ii sum_k L_ik T_kj, one block diagonal after the other
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    const int i = w + d, j = w;
    if (i < 4) {
      f32x4_t p = {0.f, 0.f, 0.f, 0.f};
      for (int k = j; k < i; ++k) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          p = __builtin_amdgcn_mfma_f32_16x16x4f32(s_l[(16 * i + n) * FS + 16 * k + 4 * s + hg],
                                                   s_t[(16 * k + 4 * s + hg) * FS + 16 * j + n], p, 0, 0, 0);
      }
      f32x4_t t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s)  // the product's rows 4 hg + s are in this lane already
        t = __builtin_amdgcn_mfma_f32_16x16x4f32(-s_t[(16 * i + n) * FS + 16 * i + 4 * hg + s], p[s], t, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) s_t[(16 * i + 4 * hg + r) * FS + 16 * j + n] = t[r];
    }
    __syncthreads();
  }
  // fragments of T diag(beta) and of the scores
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > (w >> 1)) continue;
    const int col = 32 * s + 8 * hg, at = (16 * w + n) * FS + col;
    u32x4_t pm[3], pa[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h, m, l;
      split2(s_t[at + 2 * i] * s_beta[col + 2 * i], s_t[at + 2 * i + 1] * s_beta[col + 2 * i + 1], h, m, l);
      pm[0][i] = h, pm[1][i] = m, pm[2][i] = l;
      split2(s_a[at + 2 * i], s_a[at + 2 * i + 1], h, m, l);
      pa[0][i] = h, pa[1][i] = m, pa[2][i] = l;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const int64_t o = (tri_at(w, s) * 3 + p) * 1024 + lane * 16;
      *reinterpret_cast<u32x4_t*>(mine + kFragM + o) = pm[p];
      *reinterpret_cast<u32x4_t*>(mine + kFragA + o) = pa[p];
    }
  }
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
template <int DK, int NT>
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
  auto load_tri = [&](int c, int64_t part, u32x4_t (&f)[2][3]) {
    const unsigned char* at = head_at(c) + part;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int p = 0; p < 3; ++p)
        f[s][p] = *reinterpret_cast<const u32x4_t*>(at + (tri_at(w, s <= (w >> 1) ? s : 0) * 3 + p) * 1024 + uint32_t(lane * 16));
    }
  };
  // six partial products
  auto mma6 = [&](const u32x4_t (&f)[3], const u32x4_t (&x)[3], f32x4_t (&a)[3]) {
    a[0] = mma(f[0], x[0], a[0]);
    a[1] = mma(f[0], x[1], a[1]);
    a[2] = mma(f[0], x[2], a[2]);
    a[1] = mma(f[1], x[0], a[1]);
    a[2] = mma(f[1], x[1], a[2]);
    a[2] = mma(f[2], x[0], a[2]);
  };

  if (wave >= 4) {  // outputs
    u32x4_t fa[2][3];
    f32x4_t fy;
    auto load = [&](int c) {
      load_tri(c, kFragA, fa);
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
          mma6(fa[s], x, a);
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
      load(c + 1 < chunks ? c + 1 : c);
    }
    return;
  }

  __builtin_amdgcn_s_setprio(2);  // the chain that the sequence waits for
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
  auto put4 = [&](uint16_t (*pl)[16 * NT * XS], int nt, f32x4_t x) {  // rows 16 w + 4 hg .. +3 of column 16 nt + n
    uint32_t h0, m0, l0, h1, m1, l1;
    split2(x[0], x[1], h0, m0, l0);
    split2(x[2], x[3], h1, m1, l1);
    const int at = (16 * nt + n) * XS + 16 * w + 4 * hg;
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
    load_tri(0, kFragM, fm);
    fz = load_fac(0, 2);
    decay = load_decay(0);
    load_kt(0);
  }
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {  // arrived before the loop, which then counts its own loads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) asm volatile("" : "+v"(st[dt][nt]));
  }
  for (int c = 0; c < chunks; ++c) {
    const int cn = c + 1 < chunks ? c + 1 : c;
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
    load_rows(1, cn, fk);
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
        for (int p = 2; p >= 0; --p) {
#pragma unroll
          for (int t = t0; t < t0 + 2; ++t)
            qs[nt][t] = mma(fq[t], sp[nt][p], p == 2 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : qs[nt][t]);
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
    fx = load_fac(cn, 0);
    load_v(cn);
    __syncthreads();
    qs_mul(2);
    load_rows(2, cn, fq);
    // D, as it is (for the outputs) and faded to the chunk's end (for the state)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4_t a[3] = {};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s > (w >> 1)) continue;
        u32x4_t xp[3];
        get(s_x, nt, s, xp);
        mma6(fm[s], xp, a);
      }
      const f32x4_t d = a[0] + (a[1] + a[2]);
      *reinterpret_cast<f32x4_t*>(&s_d[(16 * nt + n) * DS + 16 * w + 4 * hg]) = d;
      put4(s_u, nt, d * fz);
#pragma unroll
      for (int t = 0; t < 4; ++t) s_qs[w][nt][t][lane] = qs[nt][t];
    }
    load_tri(cn, kFragM, fm);
    fz = load_fac(cn, 2);
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
    load_kt(cn);
    decay = load_decay(cn);
  }
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

template <int DK, int NT>
void walk(const GdnArgs& a, int64_t n, hipStream_t s) {
  const int slices = a.Dv / (16 * NT), heads = a.B * a.Hv;
  const uint32_t grid = uint32_t((heads + 7) / 8 * 8) * uint32_t(slices);
  gdn_walk_kernel<DK, NT><<<dim3(grid), 512, 0, s>>>(a, n, slices, heads);
}

template <int DK>
int launch(const GdnArgs& a, hipStream_t s) {
  const int64_t n = ws_slots(a.T, a.B);
  const uint32_t chunks = uint32_t((int64_t(a.max_len < a.T ? a.max_len : a.T) + C - 1) / C);
  gdn_prep_kernel<DK><<<dim3(chunks ? chunks : 1, uint32_t(a.Hv), uint32_t(a.B)), 256, 0, s>>>(a, n);
  if (hipGetLastError() != hipSuccess) return 6;
  // 32 columns a block share its operands' loads where 16 would more than fill the GPU
  if (int64_t(a.B) * a.Hv * (a.Dv / 16) > int64_t(device_cus())) walk<DK, 2>(a, n, s);
  else walk<DK, 1>(a, n, s);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

uint64_t gdn_chunk_workspace(int64_t T, int64_t B, int64_t Hk, int64_t Hv, int64_t Dk) {
  return uint64_t(ws_slots(T, B)) * uint64_t(Hv * kHeadBytes + Hk * key_bytes(Dk));
}

int launch_gdn_chunk(const GdnArgs& a, hipStream_t s) { return a.Dk == 64 ? launch<64>(a, s) : launch<128>(a, s); }

}  // namespace qmm
