// logprobs.cu -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
//
// With x a row, m its maximum and S = sum e^(x - m):
//   log p_i = (x_i - m) - log S,   H = log S - sum e^(x - m) (x - m) / S,
// both from one pass that keeps m, S and the weighted sum (in powers of two),
// and every thread's largest entry.  H is a sum of two terms >= 0, so nothing
// cancels.
//
// The k largest.  Entries are ordered by (value, then lower index), as 64-bit
// keys, so no two are equal.  The k-th largest of the threads' own largest
// entries is no more than the row's k-th largest entry, and only the k threads
// whose largest reach it can hold entries that do: their entries alone (a few
// hundred) are read again, from the L2, and those that reach it are ranked by
// counting.  Nothing depends on the order in which threads get there.
#include <cuda_fp16.h>

#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTop = kLogprobsMaxTop;
constexpr int kCandidates = 1024;
constexpr int kMaxCluster = 8;
constexpr float kL = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A sum of 2^(x L - m) and one of 2^(x L - m) (x L - m), m the largest x L.
struct Sums {
  float m, s, e;
};
// Its terms in units of 2^m2 >= 2^m.  (What has seen nothing above -inf has m =
// -inf and zeros, or NaN, which is kept.)
__device__ __forceinline__ void lower(Sums& a, float m2) {
  if (a.m == -INFINITY || a.m == m2) return;
  const float d = fmaxf(a.m - m2, -300.f), f = ex2(d);
  a.e = f * fmaf(d, a.s, a.e);
  a.s *= f;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  lower(a, m);
  lower(b, m);
  return {m, a.s + b.s, a.e + b.e};
}
__device__ __forceinline__ Sums shuffled(const Sums& a, int off) {
  return {__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
          __shfl_xor_sync(0xffffffffu, a.e, off)};
}

template <typename T>
constexpr int kPer = 16 / sizeof(T);  // entries of 16 bytes

__device__ __forceinline__ void floats_of(const uint4& w, const float*, float (&x)[4]) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void floats_of(const uint4& w, const __nv_bfloat16*, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(v[i]);
    x[2 * i + 1] = bf16hi(v[i]);
  }
}
__device__ __forceinline__ void floats_of(const uint4& w, const __half*, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// A row as 16-byte pieces of memory: piece j holds entries j * kPer - skew ..;
// the first and the last may be partly outside and are read one by one.
template <typename T>
struct Row {
  const T* p;
  int V, skew, begin, end, pieces;  // whole pieces: [begin, end)

  __device__ __forceinline__ Row(const T* row, int n) : p(row), V(n) {
    skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    begin = skew ? 1 : 0;
    end = (V + skew) / kPer<T>;
    pieces = (V + skew + kPer<T> - 1) / kPer<T>;
  }
  __device__ __forceinline__ bool whole(int j) const { return j >= begin && j < end; }
  __device__ __forceinline__ uint4 raw(int j) const {
    return *reinterpret_cast<const uint4*>(p + (static_cast<int64_t>(j) * kPer<T> - skew));
  }
  // Entries of any piece; bit i of the result: entry i is inside the row.
  __device__ __forceinline__ unsigned entries(int j, float (&x)[kPer<T>]) const {
    if (whole(j)) {
      floats_of(raw(j), p, x);
      return (1u << kPer<T>) - 1;
    }
    unsigned in = 0;
#pragma unroll
    for (int i = 0; i < kPer<T>; ++i) {
      const int at = j * kPer<T> - skew + i;
      x[i] = -INFINITY;
      if (at >= 0 && at < V) {
        x[i] = to_f(p[at]);
        in |= 1u << i;
      }
    }
    return in;
  }
};

__device__ __forceinline__ uint64_t key_of(float x, int at) {
  return static_cast<uint64_t>(float_key(x)) << 32 | static_cast<uint32_t>(~at);
}

// What a thread has seen: its sums, and the piece with its largest entry.
struct Seen {
  Sums a{-INFINITY, 0.f, 0.f};
  float best = -INFINITY;
  int piece = -1;
};

template <int kN, int kPieces>
__device__ __forceinline__ void take(Seen& t, const float (&x)[kPieces][kN], int j0, int step) {
  float top = -INFINITY;
#pragma unroll
  for (int b = 0; b < kPieces; ++b) {
    float m = x[b][0];
#pragma unroll
    for (int i = 1; i < kN; ++i) m = fmaxf(m, x[b][i]);
    if (m > t.best) {
      t.best = m;
      t.piece = j0 + b * step;
    }
    top = fmaxf(top, m);
  }
  top *= kL;
  if (top > t.a.m) {
    lower(t.a, top);
    t.a.m = top;
  }
  const float off = t.a.m == -INFINITY ? 0.f : -t.a.m;
  float s[2] = {0.f, 0.f}, e[2] = {0.f, 0.f};
#pragma unroll
  for (int b = 0; b < kPieces; ++b)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float y = fmaf(x[b][i], kL, off), w = ex2(y);
      s[i & 1] += w;
      e[i & 1] = fmaf(w, fmaxf(y, -200.f), e[i & 1]);  // (0 times -inf would be NaN)
    }
  t.a.s += s[0] + s[1];
  t.a.e += e[0] + e[1];
}

// One step of a sorting network over the warp: the larger of each two at the
// lower lane where `down`.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int off, bool down, int lane) {
  const uint64_t o = __shfl_xor_sync(0xffffffffu, v, off);
  return ((lane & off) == 0) == down ? (v > o ? v : o) : (v > o ? o : v);
}
__device__ __forceinline__ uint64_t sort_down(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off; off >>= 1) v = exchange(v, off, size == 32 || (lane & size) == 0, lane);
  return v;
}
__device__ __forceinline__ uint64_t merge_down(uint64_t v, int lane) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v = exchange(v, off, true, lane);
  return v;
}

struct Shared {
  Sums warp_sum[kWarps];
  uint64_t lists[kWarps][32];
  uint64_t candidates[kCandidates];
  uint64_t result[kTop];
  uint64_t best;
  int flagged[kTop];
  int n_flagged, n_candidates;
  Sums sum;
};

// The k largest of sh.candidates into sh.result (sorted; 0 where there are
// fewer).  Called by the whole CTA, result cleared.
__device__ __forceinline__ void rank(Shared& sh, int n, int k) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = sh.candidates[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += sh.candidates[j] > key;
    if (r < k && key) sh.result[r] = key;
  }
}

template <typename T>
__device__ __forceinline__ void largest(Shared& sh, const Row<T>& row, const Seen& t, int k, int first, int total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t own = 0;
  const int mine = first + threadIdx.x;
  if (mine < row.pieces) {
    float x[kPer<T>];
    const int j = t.piece >= 0 ? t.piece : mine;  // (nothing above -inf: the first of them)
    const unsigned in = row.entries(j, x);
#pragma unroll
    for (int i = kPer<T> - 1; i >= 0; --i)
      if ((in >> i & 1) && x[i] == t.best) own = key_of(x[i], j * kPer<T> - row.skew + i);
  }
  uint64_t v = sort_down(own, lane);
  sh.lists[warp][lane] = v;
  __syncthreads();
  for (int half = 1; half < kWarps; half <<= 1) {
    if ((warp & (2 * half - 1)) == 0) {
      const uint64_t o = sh.lists[warp + half][31 - lane];
      v = merge_down(v > o ? v : o, lane);
      sh.lists[warp][lane] = v;
    }
    __syncthreads();
  }
  const uint64_t least = sh.lists[0][k - 1];
  if (own && own >= least) sh.flagged[atomicAdd(&sh.n_flagged, 1)] = mine;
  __syncthreads();
  const int n_flagged = sh.n_flagged;
  auto each = [&](auto&& f) {  // the entries of the flagged threads, a warp a thread's
    for (int i = warp; i < n_flagged; i += kWarps)
      for (int j = sh.flagged[i] + lane * total; j < row.pieces; j += 32 * total) {
        float x[kPer<T>];
        const unsigned in = row.entries(j, x);
#pragma unroll
        for (int b = 0; b < kPer<T>; ++b)
          if ((in >> b & 1) && x[b] == x[b]) f(key_of(x[b], j * kPer<T> - row.skew + b));
      }
  };
  each([&](uint64_t key) {
    if (key >= least) {
      const int at = atomicAdd(&sh.n_candidates, 1);
      if (at < kCandidates) sh.candidates[at] = key;
    }
  });
  __syncthreads();
  if (sh.n_candidates <= kCandidates) {
    rank(sh, sh.n_candidates, k);
  } else {
    // Many entries above the threshold in few threads' shares: one by one.
    uint64_t below = ~0ull;
    for (int i = 0; i < k; ++i) {
      uint64_t m = 0;
      each([&](uint64_t key) { m = key < below && key > m ? key : m; });
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, m, off);
        m = o > m ? o : m;
      }
      if (lane == 0) sh.lists[0][warp] = m;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) m = sh.lists[0][w] > m ? sh.lists[0][w] : m;
      if (threadIdx.x == 0) sh.result[i] = m;
      below = m;
      __syncthreads();
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsArgs a, int cluster) {
  __shared__ Shared sh;
  previous_done();
  next_may_begin();
  const int r = static_cast<int>(blockIdx.x / cluster);
  const int at = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = a.tokens ? a.tokens[r] : 0;
  if (token < 0) return;  // every CTA of the cluster alike
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.stride, a.V);
  if (tid < kTop) sh.result[tid] = 0;
  if (tid == 0) sh.n_flagged = sh.n_candidates = 0;

  const int total = cluster * kThreads, first = at * kThreads;
  Seen t;
  int j = first + tid;
  constexpr int kBatch = 4;
  if (j < row.pieces && !row.whole(j)) {
    float x[1][kPer<T>];
    row.entries(j, x[0]);
    take(t, x, j, 0);
    j += total;
  }
  for (; j + (kBatch - 1) * total < row.end; j += kBatch * total) {
    uint4 w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) w[b] = row.raw(j + b * total);
    float x[kBatch][kPer<T>];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) floats_of(w[b], row.p, x[b]);
    take(t, x, j, total);
  }
  for (; j < row.pieces; j += total) {
    float x[1][kPer<T>];
    row.entries(j, x[0]);
    take(t, x, j, 0);
  }

  Sums sum = t.a;
#pragma unroll
  for (int off = 16; off; off >>= 1) sum = join(sum, shuffled(sum, off));
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  sum = sh.warp_sum[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) sum = join(sum, sh.warp_sum[w]);
  if (a.k > 0) largest(sh, row, t, a.k, first, total);

  if (cluster > 1) {
    if (tid == 0) sh.sum = sum;
    cluster_sync();
    if (at == 0) {
      for (int c = 1; c < cluster; ++c)
        sum = join(sum, Sums{load_remote(&sh.sum.m, c), load_remote(&sh.sum.s, c), load_remote(&sh.sum.e, c)});
      if (a.k > 0) {
        for (int i = tid; i < cluster * kTop; i += kThreads) {
          const uint64_t* from = &sh.result[i % kTop];
          const uint32_t lo = __float_as_uint(load_remote(reinterpret_cast<const float*>(from), i / kTop));
          const uint32_t hi = __float_as_uint(load_remote(reinterpret_cast<const float*>(from) + 1, i / kTop));
          sh.candidates[i] = static_cast<uint64_t>(hi) << 32 | lo;
        }
        __syncthreads();
        if (tid < kTop) sh.result[tid] = 0;
        __syncthreads();
        rank(sh, cluster * kTop, a.k);
        __syncthreads();
      }
    }
    cluster_sync();  // no CTA leaves while its shared memory is read
    if (at != 0) return;
  }
  const float off = sum.m == -INFINITY ? 0.f : -sum.m, log_s = log2f(sum.s);
  auto logprob = [&](float x) { return (fmaf(x, kL, off) - log_s) * kLn2; };
  if (tid == 0) {
    if (a.logprobs && a.tokens) a.logprobs[r] = token < a.V ? logprob(to_f(row.p[token])) : -INFINITY;
    if (a.entropy) a.entropy[r] = (log_s - sum.e / sum.s) * kLn2;
  }
  if (tid < a.k) {
    const uint64_t key = sh.result[tid];
    const int64_t to = static_cast<int64_t>(r) * a.k + tid;
    a.top_ids[to] = key ? static_cast<int32_t>(~static_cast<uint32_t>(key)) : -1;
    a.top_logprobs[to] = key ? logprob(key_float(static_cast<uint32_t>(key >> 32))) : -INFINITY;
  }
}

template <typename T>
cudaError_t launch_t(const LogprobsArgs& a, cudaStream_t s) {
  const int pieces = a.V / kPer<T> + 2;
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(a.rows) * cluster * 2 <= 4 * 152 &&
         cluster * kThreads * 2 <= pieces)
    cluster *= 2;
  return launch_early(logprobs_kernel<T>, static_cast<unsigned>(a.rows) * cluster, kThreads, 0, s, cluster, a,
                      cluster);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.type == kBf16) return launch_t<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}

cudaError_t preload_logprobs_kernels() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, logprobs_kernel<__nv_bfloat16>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, logprobs_kernel<__half>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, logprobs_kernel<float>);
  return e;
}

}  // namespace oasis
