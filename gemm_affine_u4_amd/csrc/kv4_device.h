// Device helpers of the paged 4-bit cache (layout: include/qmm_mix.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

// Place of logical word w (dims 8w .. 8w+7) in a stored key row.  A lane (token, h) of the
// score product loads the 16 bytes at places 16p + 4h .. +3: words 0, 1 of its four belong
// to group 2p and words 2, 3 to group 2p + 1, so each matrix instruction stays inside a group.
template <int HD>
__host__ __device__ constexpr int k_word_place(int w) {
  return HD == 64 ? w : 16 * (w / 16) + 4 * ((w % 8) / 2) + 2 * ((w % 16) / 8) + w % 2;
}
// The logical word of load p, lane group h, word j (j < 4; head_dim 64: 2 words at 2h).
template <int HD>
__host__ __device__ constexpr int k_word_of(int p, int h, int j) {
  return HD == 64 ? 2 * h + j : 16 * p + 8 * (j >> 1) + 2 * h + (j & 1);
}

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float x) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(x)), CTRL, 0xf, 0xf, true)));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kRowMirror = 0x140;

// Over the 8 lanes that share lane / 8 (all of them active).
__device__ __forceinline__ float max8_lanes(float x) {
  x = fmaxf(x, dpp_mov<kQuadXor1>(x));
  x = fmaxf(x, dpp_mov<kQuadXor2>(x));
  return fmaxf(x, dpp_mov<kHalfMirror>(x));
}
__device__ __forceinline__ float min8_lanes(float x) {
  x = fminf(x, dpp_mov<kQuadXor1>(x));
  x = fminf(x, dpp_mov<kQuadXor2>(x));
  return fminf(x, dpp_mov<kHalfMirror>(x));
}

}  // namespace qmm
