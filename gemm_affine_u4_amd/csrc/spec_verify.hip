// Drafted tokens against the target's probabilities (qmm_spec_verify; include/qmm_serve.h).
//
// Mathematics: draft j is kept while u q_j(d) < p_j(d); at the first one that is not, the new token
// is drawn from max(p_j - q_j, 0), by the inverse of its cumulative sum: so kept and new tokens are
// distributed as the target's whatever the drafts' distribution is.  Products of two fp32
// values are exact in 64 bits; sums are 64-bit, so that a number within 2^-50 or so of a border between
// two tokens is all that their order could move.
// Bound: HBM, one row of p and one of q a sequence, and for few sequences two launches of
// three dependent round trips to memory.
// Split: a block takes kChunk entries of a sequence's row, finds by itself how many of its drafts are
// kept (a few gathered numbers) and writes the chunk's sums; a second launch, a block a
// sequence, adds the chunks' sums in order, and goes through the chunk that the number falls in.
#include <hip/hip_runtime.h>

#include "qmm_device.h"
#include "serve_internal.h"

namespace qmm {
namespace {

constexpr int kChunk = 4096, kThreads = 256, kPer = kChunk / kThreads;

template <bool F32>
__device__ __forceinline__ double prob(const void* p, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(p)[at];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[at]);
}

struct Row {
  int64_t start, row;  // the sequence's first draft; the row of p that the new token is drawn from
  int n, kept;
};
// Every thread of a block gets the same; s_first: one int of LDS.
template <bool F32>
__device__ __forceinline__ Row verify_row(const VerifyArgs& g, int b, int* s_first) {
  int64_t a = g.start[b], e = g.start[b + 1];
  a = a < 0 ? 0 : a > g.D ? g.D : a;
  e = e < a ? a : e > g.D ? g.D : e;
  Row r;
  r.start = a;
  r.n = int(e - a < g.max_draft ? e - a : g.max_draft);
  if (threadIdx.x == 0) *s_first = r.n;
  __syncthreads();
  for (int j = threadIdx.x; j < r.n; j += kThreads) {
    const int64_t d = g.draft[a + j];
    bool kept = false;
    if (d >= 0 && d < g.V) {
      const double u = g.u[a + b + j], q = g.q ? prob<F32>(g.q, (a + j) * g.V + d) : 1.0;
      kept = u * q < prob<F32>(g.p, (a + b + j) * g.V + d);
    }
    if (!kept) {
      atomicMin(s_first, j);
      break;  // later drafts of this thread lie behind it
    }
  }
  __syncthreads();
  r.kept = *s_first;
  r.row = a + b + r.kept;
  return r;
}

// Weight of entry v, before the fallback and of the fallback.
struct Weight {
  double rest, p;
};
template <bool F32>
__device__ __forceinline__ Weight weight(double p, double q) {
  const double d = p - q;
  return {d > 0 ? d : 0.0, p > 0 ? p : 0.0};
}

template <bool F32>
__device__ __forceinline__ Weight weight_at(const VerifyArgs& g, const Row& r, int64_t v) {
  const double p = prob<F32>(g.p, r.row * g.V + v);
  double q = 0.0;
  if (r.kept < r.n) {
    if (g.q) q = prob<F32>(g.q, (r.start + r.kept) * g.V + v);
    else q = v == g.draft[r.start + r.kept] ? 1.0 : 0.0;
  }
  return weight<F32>(p, q);
}

// Sum over a wave, then over the block's waves in order (s: 4 doubles of LDS).
__device__ __forceinline__ double block_sum(double x, double* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  return s[0] + s[1] + s[2] + s[3];
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs g, int chunks) {
  __shared__ int s_first;
  __shared__ double s_sum[4];
  const int b = blockIdx.y, chunk = blockIdx.x;
  const Row r = verify_row<F32>(g, b, &s_first);
  double rest = 0.0, all = 0.0;
#pragma unroll 4
  for (int i = 0; i < kPer; ++i) {
    const int64_t v = int64_t(chunk) * kChunk + i * kThreads + threadIdx.x;
    if (v < g.V) {
      const Weight w = weight_at<F32>(g, r, v);
      rest += w.rest;
      all += w.p;
    }
  }
  rest = block_sum(rest, s_sum);
  all = block_sum(all, s_sum);
  if (threadIdx.x == 0) {
    double* to = g.ws + (int64_t(b) * chunks + chunk) * 2;
    to[0] = rest;
    to[1] = all;
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs g, int chunks) {
  __shared__ int s_first, s_chunk, s_last, s_token, s_least;
  __shared__ double s_sum[4], s_pre[kThreads], s_before;
  const int b = blockIdx.x, tid = threadIdx.x;
  const Row r = verify_row<F32>(g, b, &s_first);
  const double* sums = g.ws + int64_t(b) * chunks * 2;
  double rest = 0.0, all = 0.0;
  for (int i = tid; i < chunks; i += kThreads) {
    rest += sums[2 * i];
    all += sums[2 * i + 1];
  }
  rest = block_sum(rest, s_sum);
  const bool use_p = !(rest > 0.0);  // nothing is left of p - q: the target itself
  (void)all;
  if (tid == 0) {
    // chunks in order: the first one in which the cumulative sum passes the number's share
    double total = 0.0;
    for (int i = 0; i < chunks; ++i) total += sums[2 * i + use_p];
    const double x = double(g.u[r.start + b + r.n]) * total;
    double before = 0.0, c = 0.0;
    int hit = -1, last = -1;
    for (int i = 0; i < chunks && hit < 0; ++i) {
      const double w = sums[2 * i + use_p];
      if (w > 0.0) {
        last = i, before = c;
        if (c + w > x) hit = i;
      }
      c += w;
    }
    s_chunk = hit >= 0 ? hit : last;
    s_before = x - before;  // what the chunk's own sum has to pass
    s_least = kChunk;
    s_last = -1;
  }
  __syncthreads();
  const int chunk = s_chunk;
  if (chunk >= 0) {
    double w[kPer], sum = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t v = int64_t(chunk) * kChunk + tid * kPer + i;
      w[i] = 0.0;
      if (v < g.V) {
        const Weight x = weight_at<F32>(g, r, v);
        w[i] = use_p ? x.p : x.rest;
      }
      sum += w[i];
    }
    s_pre[tid] = sum;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
      const double y = tid >= o ? s_pre[tid - o] : 0.0;
      __syncthreads();
      s_pre[tid] += y;
      __syncthreads();
    }
    double c = tid ? s_pre[tid - 1] : 0.0;
    int least = kChunk, last = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c += w[i];
      if (w[i] > 0.0) {
        last = tid * kPer + i;
        if (c > s_before && least == kChunk) least = last;
      }
    }
    if (least < kChunk) atomicMin(&s_least, least);
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    if (tid == 0) s_token = chunk * kChunk + (s_least < kChunk ? s_least : s_last);
  } else if (tid == 0) {
    s_token = -1;
  }
  __syncthreads();
  int32_t* to = g.tokens + int64_t(b) * (g.max_draft + 1);
  for (int j = tid; j <= g.max_draft; j += kThreads)
    to[j] = j < r.kept ? g.draft[r.start + j] : j == r.kept ? s_token : -1;
  if (tid == 0) g.accepted[b] = r.kept;
}

int chunks_of(int64_t V) { return int((V + kChunk - 1) / kChunk); }

template <bool F32>
int launch(const VerifyArgs& a, hipStream_t s) {
  const int chunks = chunks_of(a.V);
  verify_sums_kernel<F32><<<dim3(uint32_t(chunks), uint32_t(a.B)), kThreads, 0, s>>>(a, chunks);
  verify_pick_kernel<F32><<<dim3(uint32_t(a.B)), kThreads, 0, s>>>(a, chunks);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

uint64_t verify_workspace(int64_t B, int64_t V) { return uint64_t(B) * uint64_t(chunks_of(V)) * 16; }

int launch_verify(const VerifyArgs& a, hipStream_t s) { return a.f32 ? launch<true>(a, s) : launch<false>(a, s); }

}  // namespace qmm
