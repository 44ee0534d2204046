// What the attention kernels over the paged 8-bit cache share: the keys that a block's rows can
// see, their split over blocks, and the codes as operands.
#pragma once
#include "kv4_attn.h"
#include "qmm_device.h"
#include "serve_internal.h"

namespace qmm {

// How a call is cut: a function of its sizes alone (host), the same for its workspace.
struct Attn8Plan {
  int rows;    // (query, head) rows of a block: 16 (kv8_decode.hip) or attn8_rows (kv8_prefill.hip)
  int waves;   // of a block
  int shift;   // log2 of the keys of a tile
  int nsplit;  // at most this many splits of a block's keys ...
  int keys;    // ... of at least this many keys
};
constexpr int attn8_rows(int64_t hd) { return hd == 128 ? 256 : 128; }
Attn8Plan attn8_plan(int64_t B, int64_t max_q, int64_t n_q, int64_t n_kv, int64_t hd, int64_t max_kv, int64_t window,
                     int64_t sinks);

// The block's split.  Blocks go to the dies in turn: heads are neighbours, as they have equal work; splits, of which
// short sequences leave the last ones empty, follow, from elsewhere on in every sequence; then row tiles, which read the
// same keys, mostly on the same die (64 contexts of 1000 keys, 8 heads x
// 128, in tables of 16384 keys: 78 us with the splits as neighbours, 41 us).
__device__ __forceinline__ int attn8_split(const Attn8Plan& p) { return int((blockIdx.y + blockIdx.z) % uint32_t(p.nsplit)); }

// The tiles of keys that some rows of a sequence can see, numbered without a gap: the first `sink`
// ones, then those from `first` on.  A split has those from begin to end.
struct Attn8Tiles {
  int sink, first, count;  // count: splits of the block's keys
  int begin, end;
  int lo, hi;  // every key from lo to hi - 1, and of the first `sinks` before lo, is seen by some row
  __device__ __forceinline__ int at(int v) const { return v < sink ? v : v - sink + first; }
};
__device__ __forceinline__ Attn8Tiles attn8_tiles(const Kv8AttnArgs& g, const AttnSeq& s, int row0, int rows, int group,
                                                  const Attn8Plan& p, int split) {
  int64_t lo = 0, hi = s.kv_len;
  if (g.causal) {
    hi = int64_t(s.first) + (row0 + rows - 1) / group + 1;
    const int64_t w = int64_t(s.first) + row0 / group - g.window + 1;
    if (g.window > 0 && w > 0) lo = w;
  }
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  const int tile = 1 << p.shift;
  const int64_t sinks = g.sinks < lo ? g.sinks : lo;
  Attn8Tiles r;
  r.sink = int((sinks + tile - 1) >> p.shift);
  r.first = int(lo >> p.shift);
  if (r.sink >= r.first) r.sink = r.first = 0;  // they meet
  const int tiles = r.sink + int((hi + tile - 1) >> p.shift) - r.first, least = p.keys >> p.shift;
  int c = (tiles + least - 1) / least;
  c = c > p.nsplit ? p.nsplit : c < 1 ? 1 : c;
  const int per = (tiles + c - 1) / c;
  r.count = per > 0 ? (tiles + per - 1) / per : 1;
  r.lo = int(lo), r.hi = int(hi);
  r.begin = split * per;
  r.end = r.begin + per < tiles ? r.begin + per : tiles;
  return r;
}

// Four codes as fp16 numbers, exact: the byte c + 128 under the exponent of 1024, less 1152.
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const f16x2_t off = {(_Float16)-1152.f, (_Float16)-1152.f};
  lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + off);
  hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + off);
}
// Eight of them as an operand.
__device__ __forceinline__ f16x8_t code_operand(uint32_t a, uint32_t b) {
  u32x4_t r;
  uint32_t x, y;
  code_pairs(a, x, y);
  r[0] = x, r[1] = y;
  code_pairs(b, x, y);
  r[2] = x, r[3] = y;
  return __builtin_bit_cast(f16x8_t, r);
}
__device__ __forceinline__ f16x2_t half_pair(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_convertvector(f32x2_t{a, b}, f16x2_t);
}

int launch_kv8_decode(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s);
int launch_kv8_prefill(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s);
int launch_kv8_join(const Kv8AttnArgs& a, const Attn8Plan& p, hipStream_t s);

}  // namespace qmm
