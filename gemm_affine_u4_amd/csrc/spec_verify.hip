// Drafted tokens against the target's probabilities (qmm_spec_verify; include/qmm_serve.h).
//
// Mathematics: draft j is kept while u q_j(d) < p_j(d); at the first one that is not, the new token
// is drawn from max(p_j - q_j, 0), by the inverse of its cumulative sum: so kept and new tokens are
// distributed as the target's whatever the drafts' distribution is.  Products of two fp32
// values are exact in 64 bits; sums are 64-bit, so that a number within 2^-50 or so of a border between
// two tokens is all that their order could move.
// Bound: HBM, one row of p and one of q a sequence (64 sequences x 152001 fp32 entries with draft probabilities: 19 us, of it
// the sums 14 at 5.6 TB/s and the pick 6), and for few sequences the round trips to memory that depend on each other:
// the sequence's drafts, their probabilities, the row, and the launches (5 drafts of one sequence, 32000 entries: 9.1 us).
// Split: a block takes kChunk entries of a sequence's row, finds by itself how many of its drafts are
// kept (a few gathered numbers) and writes the chunk's sums; a second launch, a block a sequence,
// finds by a scan of the chunks' sums in which of them the number falls, and in that one by a
// scan of its weights at which entry.
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
// Four neighbours as loaded; a row may begin at any entry.
template <bool F32>
struct Four {
  uint32_t w[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    __builtin_memcpy(w, static_cast<const char*>(p) + at * (F32 ? 4 : 2), sizeof w);
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    else return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

struct Row {
  int start, n, kept;  // the sequence's first draft, how many there are, how many are kept
};
// Every thread of a block gets the same; s_first: one int of LDS.
template <bool F32, int THREADS>
__device__ __forceinline__ Row verify_row(const VerifyArgs& g, int b, int* s_first) {
  int64_t a = g.start[b], e = g.start[b + 1];
  a = a < 0 ? 0 : a > g.D ? g.D : a;
  e = e < a ? a : e > g.D ? g.D : e;
  Row r;
  r.start = int(a);
  r.n = int(e - a < g.max_draft ? e - a : g.max_draft);
  if (threadIdx.x == 0) *s_first = r.n;
  __syncthreads();
  for (int j = threadIdx.x; j < r.n; j += THREADS) {
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
  return r;
}

// Weight of an entry, before the fallback and of the fallback.
struct Weight {
  double rest, p;
};
__device__ __forceinline__ Weight weight(double p, double q) { return {fmax(p - q, 0.0), fmax(p, 0.0)}; }  // NaN: 0

// The row that the weights come from, and what is taken off.
template <bool F32>
struct Weights {
  const VerifyArgs& g;
  int64_t p_row, q_row;  // first entries; q_row < 0: nothing is taken off but the draft `gone`
  int64_t gone;
  __device__ __forceinline__ Weights(const VerifyArgs& args, const Row& r, int b)
      : g(args), p_row((int64_t(r.start) + b + r.kept) * args.V), q_row(-1), gone(-1) {
    if (r.kept < r.n) {
      if (g.q) q_row = (int64_t(r.start) + r.kept) * g.V;
      else gone = g.draft[r.start + r.kept];
    }
  }
  // N groups of entries v + i step .. + 3, zeros behind the last: use(i, weights).  All loads are under way before the
  // first is waited for: a group that leaves the row is read from the row's last four and moved.
  template <int N, class Use>
  __device__ __forceinline__ void groups(int64_t v, int step, int count, Use&& use) const {
    if (q_row >= 0) groups_of<N, true>(v, step, count, use);
    else groups_of<N, false>(v, step, count, use);
  }
  template <int N, bool HAS_Q, class Use>
  __device__ __forceinline__ void groups_of(int64_t v, int step, int count, Use&& use) const {
    Four<F32> p[N], q[N];
    if (g.V >= 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= count) continue;
        const int64_t at = v + i * step < g.V - 4 ? v + i * step : g.V - 4;
        p[i].load(g.p, p_row + at);
        if constexpr (HAS_Q) q[i].load(g.q, q_row + at);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= count) continue;
      const int64_t first = v + i * step;
      float x[4], y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = p[i].at(k), y[k] = HAS_Q ? q[i].at(k) : 0.f;
      if (__any(first + 4 > g.V)) {
        const int64_t off = g.V >= 4 ? first - (g.V - 4) : 4;  // places that the group was moved by
        float a[4], c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = off > 0 ? 0.f : x[k], c[k] = off > 0 ? 0.f : y[k];
#pragma unroll
          for (int m = k + 1; m < 4; ++m)
            if (off == m - k) a[k] = x[m], c[k] = y[m];
          if (g.V < 4 && first + k < g.V) {
            a[k] = float(prob<F32>(g.p, p_row + first + k));
            if constexpr (HAS_Q) c[k] = float(prob<F32>(g.q, q_row + first + k));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = a[k], y[k] = c[k];
      }
      Weight w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = weight(x[k], first + k == gone ? 1.0 : double(y[k]));
      use(i, w);
    }
  }
};

// Sum over a wave, then over the block's waves in order (s: 4 doubles of LDS).
__device__ __forceinline__ double block_sum(double x, double* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  return s[0] + s[1] + s[2] + s[3];
}

// Behind the sums in the workspace: what the first launch found out about each sequence.
__device__ __forceinline__ int4* rows_of(const VerifyArgs& g, int chunks) {
  return reinterpret_cast<int4*>(g.ws + int64_t(g.B) * chunks * 2);
}

// A sequence's answer, by all threads of a block.
template <int THREADS>
__device__ __forceinline__ void answer(const VerifyArgs& g, int b, const Row& r, int token) {
  int32_t* to = g.tokens + int64_t(b) * (g.max_draft + 1);
  for (int j = threadIdx.x; j <= g.max_draft; j += THREADS)
    to[j] = j < r.kept ? g.draft[r.start + j] : j == r.kept ? token : -1;
  if (threadIdx.x == 0) g.accepted[b] = r.kept;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs g, int chunks) {
  __shared__ int s_first;
  __shared__ double s_sum[4];
  const int b = blockIdx.y, chunk = blockIdx.x;
  const Row r = verify_row<F32, kThreads>(g, b, &s_first);
  const Weights<F32> weights(g, r, b);
  double rest = 0.0, all = 0.0;
  weights.template groups<kPer / 4>(int64_t(chunk) * kChunk + 4 * int(threadIdx.x), 4 * kThreads, kPer / 4,
                                    [&](int, const Weight (&w)[4]) {
#pragma unroll
                                      for (int k = 0; k < 4; ++k) rest += w[k].rest, all += w[k].p;
                                    });
  rest = block_sum(rest, s_sum);
  all = block_sum(all, s_sum);
  if (threadIdx.x == 0) {
    double* to = g.ws + (int64_t(b) * chunks + chunk) * 2;
    to[0] = rest;
    to[1] = all;
    if (chunk == 0) rows_of(g, chunks)[b] = int4{r.start, r.n, r.kept, 0};
  }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
// The sum over the lanes in front of each.
__device__ __forceinline__ double wave_before(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  x = __shfl_up(x, 1);
  return lane ? x : 0.0;
}
// Where the running sum first passes x, of N weights that all lanes hold; else the last one above 0, or -1.
template <int N>
__device__ __forceinline__ int first_past(const double (&w)[N], double x, double& before) {
  int hit = -1, last = -1;
  double c = 0.0, hit_before = 0.0, last_before = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double next = c + w[i];
    if (w[i] > 0.0) {
      last = i, last_before = c;
      if (hit < 0 && next > x) hit = i, hit_before = c;
    }
    c = next;
  }
  before = hit >= 0 ? hit_before : last_before;
  return hit >= 0 ? hit : last;
}

// The entry at which the running sum of a range's weights first passes a number (else the last one above 0, -1 if
// there is none), by all threads of a block.  The range is WAVES parts of `steps` (up to STEPS) times 256
// neighbouring entries, a part a wave: the one in whose part the number falls finds the step, then the entry.
// share(total, x): the number, or false where the range's sum is of no use.
template <int WAVES>
struct FindShared {
  double sums[WAVES];
  int at;
};
template <bool F32, int WAVES, int STEPS, class Share>
__device__ __forceinline__ bool find(const Weights<F32>& weights, int64_t first, int steps, bool use_p,
                                     FindShared<WAVES>* s, Share&& share, int& found) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t v0 = first + int64_t(wave) * steps * 256;
  auto weight_of = [&](const Weight& w) { return use_p ? w.p : w.rest; };
  double sums[STEPS], own = 0.0;  // the lane's
  weights.template groups<STEPS>(v0 + 4 * lane, 256, steps, [&](int i, const Weight (&w)[4]) {
    sums[i] = weight_of(w[0]) + weight_of(w[1]) + weight_of(w[2]) + weight_of(w[3]);
    own += sums[i];
  });
  own = wave_sum(own);
  __syncthreads();
  if (lane == 0) s->sums[wave] = own;
  if (threadIdx.x == 0) s->at = -1;
  __syncthreads();
  double part[WAVES], total = 0.0, x, before;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) part[i] = s->sums[i], total += part[i];
  if (!share(total, x)) return false;
  if (first_past(part, x, before) == wave) {
    x -= before;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) sums[i] = wave_sum(i < steps ? sums[i] : 0.0);
    const int step = first_past(sums, x, before);
    x -= before;
    double w[4];  // the step's entries again, from the caches
    weights.template groups<1>(v0 + 256 * step + 4 * lane, 0, 1, [&](int, const Weight (&four)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = weight_of(four[k]);
    });
    double c = wave_before(w[0] + w[1] + w[2] + w[3], lane);
    int hit = -1, last = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c += w[k];
      if (w[k] > 0.0) {
        last = k;
        if (hit < 0 && c > x) hit = k;
      }
    }
    const uint64_t hits = __ballot(hit >= 0), lasts = __ballot(last >= 0);
    const int from = hits ? __ffsll(static_cast<unsigned long long>(hits)) - 1
                          : 63 - __clzll(static_cast<long long>(lasts));
    const int k = __shfl(hits ? hit : last, from);
    if (lane == 0) s->at = int(v0 - first) + 256 * step + 4 * from + k;
  }
  __syncthreads();
  found = s->at;
  return true;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs g, int chunks) {
  __shared__ FindShared<4> s_find;
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  const int4 found = rows_of(g, chunks)[b];
  const Row r = {found.x, found.y, found.z};
  const double* sums = g.ws + int64_t(b) * chunks * 2;
  // every wave: the chunks' sum, then 64 chunks at a time in order
  double rest = 0.0, all = 0.0;
  for (int i = lane; i < chunks; i += 64) rest += sums[2 * i], all += sums[2 * i + 1];
  rest = wave_sum(rest);
  const bool use_p = !(rest > 0.0);  // nothing is left of p - q: the target itself
  if (use_p) rest = wave_sum(all);
  const double x = double(g.u[int64_t(r.start) + b + r.n]) * rest;
  int chunk = -1, last = -1;
  double front = 0.0, before = 0.0, last_before = 0.0;
  for (int i0 = 0; i0 < chunks && chunk < 0; i0 += 64) {
    const double w = i0 + lane < chunks ? sums[2 * (i0 + lane) + use_p] : 0.0;
    const double c = front + wave_before(w, lane);
    const uint64_t some = __ballot(w > 0.0), hits = __ballot(w > 0.0 && c + w > x);
    if (hits) {
      const int k = __ffsll(static_cast<unsigned long long>(hits)) - 1;
      chunk = i0 + k, before = __shfl(c, k);
    } else if (some) {
      const int k = 63 - __clzll(static_cast<long long>(some));
      last = i0 + k, last_before = __shfl(c, k);
    }
    front = __shfl(c + w, 63);
  }
  if (chunk < 0) chunk = last, before = last_before;
  int token = -1;
  if (chunk >= 0) {
    const Weights<F32> weights(g, r, b);
    find<F32, 4, kChunk / 1024>(weights, int64_t(chunk) * kChunk, kChunk / 1024, use_p, &s_find,
                                [&](double, double& y) { return y = x - before, true; }, token);
    token += chunk * kChunk;
  }
  answer<kThreads>(g, b, r, token);
}

// Rows of up to kRow entries: a block of 16 waves a sequence does all of it (4000 entries, 64 sequences: 7.9 us, in two
// launches 10.0; 16000 of 8: 9.1 and 9.4; of 32000 entries two launches are faster: one sequence 8.8 us against 10.1, 64 of
// them 12.6 against 15.0).
constexpr int kWaves = 16, kSteps = 4, kRow = kWaves * kSteps * 256;

template <bool F32>
__global__ __launch_bounds__(kWaves * 64) void verify_row_kernel(VerifyArgs g) {
  __shared__ int s_first;
  __shared__ FindShared<kWaves> s_find;
  const int b = blockIdx.x;
  const Row r = verify_row<F32, kWaves * 64>(g, b, &s_first);
  const Weights<F32> weights(g, r, b);
  const double u = g.u[int64_t(r.start) + b + r.n];
  const int steps = int((g.V + kWaves * 256 - 1) / (kWaves * 256));
  int token = -1;
  // once more with the target itself where nothing is left of p - q
  for (int use_p = 0; use_p < 2; ++use_p)
    if (find<F32, kWaves, kSteps>(weights, 0, steps, use_p, &s_find,
                                  [&](double total, double& x) { return x = u * total, total > 0.0 || use_p; }, token))
      break;
  answer<kWaves * 64>(g, b, r, token);
}

int chunks_of(int64_t V) { return int((V + kChunk - 1) / kChunk); }

template <bool F32>
int launch(const VerifyArgs& a, hipStream_t s) {
  const int chunks = chunks_of(a.V);
  if (a.V <= kRow) {
    verify_row_kernel<F32><<<dim3(uint32_t(a.B)), kWaves * 64, 0, s>>>(a);
    return hipGetLastError() == hipSuccess ? 0 : 6;
  }
  verify_sums_kernel<F32><<<dim3(uint32_t(chunks), uint32_t(a.B)), kThreads, 0, s>>>(a, chunks);
  verify_pick_kernel<F32><<<dim3(uint32_t(a.B)), kThreads, 0, s>>>(a, chunks);
  return hipGetLastError() == hipSuccess ? 0 : 6;
}

}  // namespace

uint64_t verify_workspace(int64_t B, int64_t V) { return uint64_t(B) * uint64_t(chunks_of(V) + 1) * 16; }

int launch_verify(const VerifyArgs& a, hipStream_t s) { return a.f32 ? launch<true>(a, s) : launch<false>(a, s); }

}  // namespace qmm
