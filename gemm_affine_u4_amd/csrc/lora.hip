// Low-rank adapters of many requests beside a shared projection (qmm_lora; include/qmm_serve.h).
//
// Mathematics: h = A x, then y = base + s B h, with the adapter of each token.  Both products are
// small (a rank of 8 to 128), so they are bound by the bytes of x, base, y and the adapters
// in use; each adapter's weights are read once for a tile of tokens that use it.
// Split.  Tokens go in tiles of 16 (up to 256 tokens in all) or, of more, of 64 to shrink and 32 to expand, as they
// stand: a block finds the adapters of its tile and takes those that are its share, each as a product of
// the adapter's weights with the whole tile, of which it keeps the columns of that adapter's tokens.
// So nothing is sorted, requests that stand side by side share their weights' reads, and a
// batch of many adapters is spread over blocks.
//   shrink: weights' rows x tokens over a range of K; the block's waves take 64 inputs in turn and
//     join in LDS; each range's sums go to the workspace.
//   join (more than 256 tokens): adds the ranges' sums in order, times s, and writes them as three bf16
//     pieces (24 bits).  Of fewer tokens each expanding block does so itself: a launch costs more there.
//   expand: the pieces follow each other along the matrix product's k: for ranks up to 16 they fit
//     in one or two instructions.  A lane ends with 4 neighbouring outputs of a token, four lanes with 16.
// Measured.  Rank 16, K 5120, parts of 5120, 1024 and 1024 rows: one token 8.5 us, 64 tokens of 48 adapters 16 us,
// two launches, each of them one chain of loads.  Rank 64, K 13824, 5120 rows, 4464 tokens of prompts beside a fp32
// projection: 120 us, of which shrinking 57 us, joining 5 us, expanding 58 us (183 MB, 3.1 TB/s).  Both launches have two blocks
// a unit there: shrinking by its 64 KB of LDS (560 blocks for 512 places), expanding by its 174 registers.
#include <hip/hip_runtime.h>

#include "qmm_device.h"
#include "qmm_internal.h"
#include "serve_internal.h"

namespace qmm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;

__device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// Waits until the last matrix instruction has written its result.  The compiler does so itself in
// straight code, but not where a loop's last product is stored to LDS behind the loop, inside
// another loop (seen in its output, and as a register stored too early).
__device__ __forceinline__ void mma_settle(f32x4_t& c) { asm volatile("s_nop 7\n\ts_nop 7" : "+v"(c)); }
__device__ __forceinline__ void mma_settle(f32x4_t (&c)[4]) {
  asm volatile("s_nop 7\n\ts_nop 7" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
}

// The adapters of a tile of up to 64 tokens, lane t having token t, and which of them a block (a share of the tile)
// takes.  Of few tokens share i takes token i's adapter if no token in front has the same one; of
// many, where tiles of one adapter are the rule, each shares-th of the distinct ones.
constexpr int kNone = -1, kNoToken = -2;
template <int TT>
struct Tile {
  int id;  // of the lane's token
  int list = 0, count = 0;  // lane i: the i-th distinct one (many tokens), or this block's only one
  __device__ __forceinline__ Tile(const LoraArgs& g, int64_t t0, int lane, int share) {
    id = kNoToken;
    if (lane < 16 * TT && t0 + lane < g.T) {
      id = g.ids[t0 + lane];
      if (uint32_t(id) >= uint32_t(g.n_adapters)) id = kNone;
    }
    if constexpr (TT == 1) {
      list = __builtin_amdgcn_readlane(id, share);
      const uint64_t same = __ballot(id == list);
      count = list != kNoToken && __ffsll(static_cast<unsigned long long>(same)) - 1 == share;
    } else {
      uint64_t left = __ballot(id != kNoToken);
      while (left) {
        const int next = __builtin_amdgcn_readlane(id, __ffsll(static_cast<unsigned long long>(left)) - 1);
        left &= ~__ballot(id == next);
        if (lane == count) list = next;
        ++count;
      }
    }
  }
  // turns of this block: from(share) on in steps(shares) up to count
  __device__ __forceinline__ static int from(int share) { return TT == 1 ? 0 : share; }
  __device__ __forceinline__ int at(int turn) const { return __builtin_amdgcn_readlane(list, turn); }
};

// TT column tiles of 16 tokens, RT row tiles of 16 ranks, KS steps of 32 inputs at a time.
template <int TT, int RT, int KS>
__global__ __launch_bounds__(kWaves * 64, 2) void lora_shrink_kernel(LoraArgs g, int row_groups, int splits,
                                                                     int shares) {
  const int lane = threadIdx.x & 63, n = lane & 15, hg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // ranges of K side by side: with 8 of them each die, to which blocks go in turn, keeps its own range of the
  // adapters' weights in its cache
  const uint32_t block = blockIdx.x / uint32_t(splits);
  const int split = int(blockIdx.x % uint32_t(splits)), share = blockIdx.y;
  const int64_t t0 = int64_t(block / uint32_t(row_groups)) * (16 * TT);
  const int R = g.n_parts * g.rank, r0 = int(block % uint32_t(row_groups)) * (16 * RT);
  using T = Tile<TT>;
  const T tile(g, t0, lane, share);
  if (T::from(share) >= tile.count) return;

  const int units = g.K / 64, u0 = units * split / splits, u1 = units * (split + 1) / splits;
  // the wave's steps: two of each fourth unit of 64
  const int steps = u0 + wave < u1 ? (u1 - u0 - wave + kWaves - 1) / kWaves * 2 : 0;
  auto input = [&](int q) { return (u0 + wave + (q >> 1) * kWaves) * 64 + (q & 1) * 32; };
  const uint16_t* xp[TT];
  int ids[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int64_t t = t0 + 16 * i + n;
    xp[i] = g.x + (t < g.T ? t : g.T - 1) * g.K + 8 * hg;
    ids[i] = __shfl(tile.id, 16 * i + n);
  }
  __shared__ f32x4_t s_acc[kWaves][TT * RT][64];
  for (int turn = T::from(share); turn < tile.count; turn += shares) {
    const int id = tile.at(turn);
    if (id < 0) continue;
    const uint16_t* ap[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = r0 + 16 * i + n;
      ap[i] = g.a + (int64_t(id) * R + (r < R ? r : R - 1)) * g.K + 8 * hg;
    }
    f32x4_t acc[TT][RT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // KS steps at a time: whole lines of 128 bytes; columns of other adapters are not read
    u32x4_t xv[KS][TT], av[KS][RT];
    auto fetch = [&](int q) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int at = input(q + k < steps ? q + k : steps - 1);  // behind the last step that one again, not used
#pragma unroll
        for (int i = 0; i < RT; ++i) av[k][i] = *reinterpret_cast<const u32x4_t*>(ap[i] + at);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          xv[k][i] = u32x4_t{0, 0, 0, 0};
          if (ids[i] == id) xv[k][i] = *reinterpret_cast<const u32x4_t*>(xp[i] + at);
        }
      }
    };
    auto use = [&](int q) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if (q + k >= steps) continue;
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[i][j] = mma(av[k][j], xv[k][i], acc[i][j]);
      }
    };
    for (int q = 0; q < steps; q += KS) {
      fetch(q);
      use(q);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        mma_settle(acc[i][j]);
        s_acc[wave][i * RT + j][lane] = acc[i][j];
      }
    __syncthreads();
    for (int e = wave; e < TT * RT; e += kWaves) {
      f32x4_t v = s_acc[0][e][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += s_acc[w][e][lane];
      const int tt = 16 * (e / RT) + n, r = r0 + 16 * (e % RT) + 4 * hg;
      if (__shfl(tile.id, tt) == id && r < R)
        *reinterpret_cast<f32x4_t*>(g.ws + (int64_t(split) * g.T + t0 + tt) * R + r) = v;
    }
    __syncthreads();
  }
}

// Rows of the part `p` from n0 on: 64 of them a wave.
template <int RANK>
struct Expand {
  static constexpr int kChunks = RANK / 8;                        // of 8 along k
  static constexpr int kSteps = (3 * kChunks + 3) / 4;            // matrix instructions of the three pieces
  static constexpr int kLoads = RANK > 32 ? RANK / 32 : 1;        // distinct weight operands
};

template <bool BASE32>
__device__ __forceinline__ float base_at(const void* p, int64_t at) {
  if constexpr (BASE32) return static_cast<const float*>(p)[at];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
}

// Four neighbours of h (the ranges' sums in order, times the adapter's factor) in three bf16 pieces.
template <int N>
__device__ __forceinline__ void add_ranges(const float* p, int64_t stride, int splits, int& i, f32x4_t& v) {
  for (; i + N <= splits; i += N) {
    f32x4_t x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = *reinterpret_cast<const f32x4_t*>(p + (i + k) * stride);
#pragma unroll
    for (int k = 0; k < N; ++k) v += x[k];
  }
}
__device__ __forceinline__ void pieces4(const float* p, int64_t stride, int splits, float f, uint2 (&h)[3]) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  int i = 0;
  add_ranges<8>(p, stride, splits, i, v);
  add_ranges<4>(p, stride, splits, i, v);
  add_ranges<1>(p, stride, splits, i, v);
  v *= f;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    h[k] = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    v -= f32x4_t{bf16_lo(h[k].x), bf16_hi(h[k].x), bf16_lo(h[k].y), bf16_hi(h[k].y)};
  }
}

// Many tokens: the pieces once, for all blocks of the expanding launch.  to: bf16 [3][T][R].
__global__ __launch_bounds__(256) void lora_join_kernel(LoraArgs g, uint16_t* to, int splits) {
  const int R = g.n_parts * g.rank;
  const int64_t n = g.T * R, at = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  const int id = g.ids[at / R];
  if (uint32_t(id) >= uint32_t(g.n_adapters)) return;
  uint2 h[3];
  pieces4(g.ws + at, n, splits, g.scales ? g.scales[id] : 1.f, h);
#pragma unroll
  for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(to + k * n + at) = h[k];
}

// VEC: every part's rows are a multiple of 16 and its arrays 16-byte aligned.
// pieces: bf16 [3][T][R] where they were made by the launch before, else made here, in LDS.
template <int TT, int RANK, bool BASE32, bool OUT32, bool VEC>
__global__ __launch_bounds__(kWaves * 64, TT == 1 && RANK <= 32 ? 4 : 2) void lora_expand_kernel(
    LoraArgs g, const uint16_t* pieces, int row_chunks, int splits, int shares) {
  using E = Expand<RANK>;
  constexpr int TOK = 16 * TT, ROW = RANK + 8;  // bf16 of a token's piece in LDS, 16 bytes of pad
  constexpr bool MADE = TT > 1;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = int64_t(blockIdx.x / row_chunks) * TOK;
  const int share = blockIdx.y;
  // the block's part and rows
  int chunk = blockIdx.x % row_chunks, part = 0, first = 0;
  for (;; ++part) {
    const int c = (g.rows[part] + 255) / 256;
    if (chunk < c) break;
    chunk -= c;
    first += g.rows[part];
  }
  const int N = g.rows[part], n0 = chunk * 256 + wave * 64;
  const void* base = g.base[part];
  void* y = g.y[part];
  const int total = g.rows[0] + g.rows[1] + g.rows[2], R = g.n_parts * RANK;

  using T = Tile<TT>;
  const T tile(g, t0, lane, share);
  if (T::from(share) >= tile.count) return;
  const int id0 = tile.at(T::from(share));

  // Rows 4h + i of product j are outputs n0 + 16j + 4h + i: four lanes have 16 neighbours of a token.  Weights,
  // and what is added to, are under way before anything is waited for.
  const bool mine = n0 < N;
  constexpr int J = 4;  // products of 16 rows
  auto weights_of = [&](int id, u32x4_t (&w)[J][E::kLoads]) {
    const uint16_t* b = g.b + (int64_t(id) * total + first) * RANK;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = n0 + 16 * j + n < N ? n0 + 16 * j + n : N - 1;
#pragma unroll
      for (int l = 0; l < E::kLoads; ++l)
        w[j][l] = *reinterpret_cast<const u32x4_t*>(b + int64_t(row) * RANK + 8 * ((4 * l + hg) % E::kChunks));
    }
  };
  u32x4_t w[J][E::kLoads];
  if (mine && id0 >= 0) weights_of(id0, w);
  using BaseRaw = std::conditional_t<BASE32, u32x4_t, uint2>;
  BaseRaw from[TT][J];
  if constexpr (VEC) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const int64_t t = t0 + 16 * i + n;
        const int id = __shfl(tile.id, 16 * i + n);  // of many tokens all are taken on by one block, but for rare tiles
        if (TT == 1 ? id != id0 : id == kNoToken) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int64_t at = t * N + (n0 + 16 * j < N ? n0 + 16 * j : N - 16) + 4 * hg;
          from[i][j] = *reinterpret_cast<const BaseRaw*>(static_cast<const char*>(base) + at * (BASE32 ? 4 : 2));
        }
      }
    }
  }

  // h of the tile's tokens that are this block's, in three pieces
  __shared__ __attribute__((aligned(16))) uint16_t s_h[3][MADE ? 1 : TOK][ROW];
  if constexpr (!MADE) {
    for (int e0 = 0; e0 < TOK * RANK / 4; e0 += kWaves * 64) {
      const int e = e0 + tid, t = e / (RANK / 4), r = e % (RANK / 4) * 4;
      const int id = __shfl(tile.id, t & 63);
      if (t >= TOK || id != id0 || id < 0) continue;
      uint2 h[3];
      pieces4(g.ws + (t0 + t) * R + part * RANK + r, g.T * R, splits, g.scales ? g.scales[id] : 1.f, h);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(&s_h[k][t][r]) = h[k];
    }
    __syncthreads();
  }
  if (!mine) return;

  auto columns = [&](int id, const f32x4_t (&acc)[TT][J]) {
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t t = t0 + 16 * i + n;
      if (__shfl(tile.id, 16 * i + n) != id) continue;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int o = n0 + 16 * j + 4 * hg;
        const int64_t at = t * N + o;
        if constexpr (VEC) {
          if (n0 + 16 * j >= N) continue;
          f32x4_t v;
          if constexpr (BASE32) {
            v = __builtin_bit_cast(f32x4_t, from[i][j]);
          } else {
            v = f32x4_t{bf16_lo(from[i][j].x), bf16_hi(from[i][j].x), bf16_lo(from[i][j].y), bf16_hi(from[i][j].y)};
          }
          v += acc[i][j];
          if constexpr (OUT32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(y) + at) = v;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
                uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (o + e < N) store_out(y, at + e, base_at<BASE32>(base, at + e) + acc[i][j][e], OUT32);
        }
      }
    }
  };
  f32x4_t acc[TT][J];
  for (int turn = T::from(share); turn < tile.count; turn += shares) {
    const int id = tile.at(turn);
    if (turn != T::from(share) && id >= 0) weights_of(id, w);
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (id < 0) {  // tokens without an adapter
      if (base != y || BASE32 != OUT32) columns(id, acc);
      continue;
    }
#pragma unroll
    for (int m = 0; m < E::kSteps; ++m) {
      const int c = 4 * m + hg, piece = c / E::kChunks, k8 = c % E::kChunks;
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        u32x4_t h = {0, 0, 0, 0};
        if (piece < 3) {
          if constexpr (MADE) {
            const int64_t t = t0 + 16 * i + n < g.T ? t0 + 16 * i + n : g.T - 1;
            h = *reinterpret_cast<const u32x4_t*>(pieces + (piece * g.T + t) * R + part * RANK + 8 * k8);
          } else {
            h = *reinterpret_cast<const u32x4_t*>(&s_h[piece][16 * i + n][8 * k8]);
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = mma(w[j][m % E::kLoads], h, acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) mma_settle(acc[i]);
    columns(id, acc);
  }
}

// How a call is cut: a function of the sizes that its workspace is asked for with.
struct Plan {
  int tt, rt, row_groups, splits, shares;  // column and row tiles of a shrinking block; shares of a tile's adapters
  int64_t tiles;
};
// Tokens from which on tiles are larger, and h is joined by a launch of its own.  300 tokens of prompts of 100 so 18 and
// 22 us (rank 16 and 64), as few 31 and 37; 300 of as many requests 72 and 65, as few 54 and 69.
constexpr int kMany = 256;
Plan plan_of(int64_t T, int64_t K, int64_t rank, int64_t n_parts) {
  Plan p;
  const int64_t rows = (rank * n_parts + 15) / 16, cus = device_cus();
  const bool many = T > kMany;
  p.tt = many ? 4 : 1;
  p.rt = rows % 4 == 0 ? 4 : rows % 3 == 0 ? 3 : rows % 2 == 0 ? 2 : 1;
  p.tiles = (T + 16 * p.tt - 1) / (16 * p.tt);
  p.row_groups = int(rows / p.rt);
  // of tiles' adapters: blocks without one cost a start (4464 tokens of 5 prompts: 4 shares 126 us, one 121), but a tile's
  // adapters in turn take long where tiles are few (1000 tokens, each its own: 146 and 192 us; 4000: 510 and 471)
  p.shares = !many ? int(T < 16 ? T < 1 ? 1 : T : 16) : T > 2048 ? 1 : 4;
  const int64_t blocks = p.tiles * p.row_groups * (many ? 1 : p.shares), most = (K / 64 + kWaves - 1) / kWaves;
  // Two blocks for each unit, whose LDS holds no more where tokens and ranks are many.  There 8 or 16 ranges, a multiple
  // of the dies, keep each die to its own ranges of the adapters' weights (8 ranges 126 us, 7 of them 130 us).
  int64_t s = blocks ? 2 * cus / blocks : 1;
  if (many && s >= 6) s = s >= 12 ? 16 : 8;
  s = s > most ? most : s;
  p.splits = int(s < 1 ? 1 : s > 16 ? 16 : s);
  return p;
}

template <int TT, int RT, int KS>
void shrink_as(const LoraArgs& a, const Plan& p, hipStream_t s) {
  const dim3 grid(uint32_t(p.tiles * p.row_groups * p.splits), uint32_t(p.shares));
  lora_shrink_kernel<TT, RT, KS><<<grid, kWaves * 64, 0, s>>>(a, p.row_groups, p.splits, p.shares);
}

template <int TT, int KS>
void shrink(const LoraArgs& a, const Plan& p, hipStream_t s) {
  switch (p.rt) {
    case 1: return shrink_as<TT, 1, KS>(a, p, s);
    case 2: return shrink_as<TT, 2, KS>(a, p, s);
    case 3: return shrink_as<TT, 3, KS>(a, p, s);
    default: return shrink_as<TT, 4, KS>(a, p, s);
  }
}

// Behind the ranges' sums in the workspace.
uint16_t* pieces_of(const LoraArgs& a, const Plan& p) {
  return reinterpret_cast<uint16_t*>(a.ws + int64_t(p.splits) * a.T * a.rank * a.n_parts);
}

template <int TT, int RANK, bool B32, bool O32>
void expand_v(const LoraArgs& a, const Plan& p, hipStream_t s) {
  int chunks = 0;
  bool vec = true;
  for (int i = 0; i < 3; ++i) {
    chunks += (a.rows[i] + 255) / 256;
    vec = vec && a.rows[i] % 16 == 0 &&
          (reinterpret_cast<uintptr_t>(a.base[i]) | reinterpret_cast<uintptr_t>(a.y[i])) % 16 == 0;
  }
  const int64_t tiles = (a.T + 16 * TT - 1) / (16 * TT);
  const dim3 grid(uint32_t(tiles * chunks), uint32_t(p.shares));
  const uint16_t* h = pieces_of(a, p);
  if (vec) lora_expand_kernel<TT, RANK, B32, O32, true><<<grid, kWaves * 64, 0, s>>>(a, h, chunks, p.splits, p.shares);
  else lora_expand_kernel<TT, RANK, B32, O32, false><<<grid, kWaves * 64, 0, s>>>(a, h, chunks, p.splits, p.shares);
}
template <int TT, int RANK>
void expand_r(const LoraArgs& a, const Plan& p, hipStream_t s) {
  if (a.base_f32) a.out_f32 ? expand_v<TT, RANK, true, true>(a, p, s) : expand_v<TT, RANK, true, false>(a, p, s);
  else a.out_f32 ? expand_v<TT, RANK, false, true>(a, p, s) : expand_v<TT, RANK, false, false>(a, p, s);
}
template <int TT>
void expand(const LoraArgs& a, const Plan& p, hipStream_t s) {
  switch (a.rank) {
    case 8: return expand_r<TT, 8>(a, p, s);
    case 16: return expand_r<TT, 16>(a, p, s);
    case 32: return expand_r<TT, 32>(a, p, s);
    case 64: return expand_r<TT, 64>(a, p, s);
    default: return expand_r<TT, 128>(a, p, s);
  }
}

}  // namespace

bool lora_launches(int64_t T, const int32_t (&rows)[3]) {
  const int64_t chunks = (int64_t(rows[0]) + 255) / 256 + (int64_t(rows[1]) + 255) / 256 + (int64_t(rows[2]) + 255) / 256;
  return ((T + 31) / 32 + 16) * chunks < int64_t(1) << 24;
}

uint64_t lora_workspace(int64_t T, int64_t K, int64_t rank, int64_t n_parts) {
  const Plan p = plan_of(T, K, rank, n_parts);
  const uint64_t n = uint64_t(T) * uint64_t(rank * n_parts) * (uint64_t(p.splits) * 4 + (p.tt > 1 ? 6 : 0));
  return n ? n : 256;
}

int launch_lora(const LoraArgs& a, hipStream_t s) {
  const Plan p = plan_of(a.T, a.K, a.rank, a.n_parts);
  if (a.T <= kMany) {
    shrink<1, 4>(a, p, s);
    expand<1>(a, p, s);
  } else {
    shrink<4, 2>(a, p, s);
    const int64_t n = (a.T * a.rank * a.n_parts / 4 + 255) / 256;
    lora_join_kernel<<<dim3(uint32_t(n)), 256, 0, s>>>(a, pieces_of(a, p), p.splits);
    expand<2>(a, p, s);
  }
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace qmm
