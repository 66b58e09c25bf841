// logprobs.cu -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
//
// With x a row, m its maximum and S = sum e^(x - m):
//   log p_i = (x_i - m) - log S,   H = log S - sum e^(x - m) (x - m) / S,
// both from one pass that keeps m, S and the weighted sum (in powers of two),
// and every thread's largest entry.  H is a sum of two terms >= 0 (m lags behind
// the maximum by a factor of 2^4 at most, so but for 4), so nothing much cancels.
// m is kept as it is, and x - m formed before anything else: a product
// with log2 e would be off by more than whole powers of two from |x| of 10^8 on
// and overflow near the type's largest, where masks are.
//
// Roundings of S, in 2^-24 of it: 4 of a weight, 9 in a group of entries, 2 of the
// running sum, 24 where m is moved while what was summed still counts, three
// lowerings of 5 and 11 additions where threads, warps and CTAs are joined: 65, and
// 2.2 times the mean of |y| (under 13) for the y's.
//
// The k largest.  Entries are ordered by (value, then lower index), as 64-bit
// keys, so no two are equal.  The k-th largest of the threads' own largest
// entries is no more than the row's k-th largest entry.  Every thread keeps the
// largest of each of 16 slots of its entries too: the slots that reach that
// threshold (some k of them) are read again, and their entries that reach it are
// ranked by counting.  Nothing depends on the order in which threads get there.
//
// Bound by memory in fp32 without alternatives, else by latency: no pipe is busy
// over 41 % of the time, 49 % of the issue slots are used, 44 % of the memory's
// rate (bf16, k = 20), and all CTAs of the one wave read, then rank, at the same
// time.  A thread's next four pieces are on their way while four are looked at.
// GB300, 512 rows of 151936, calls in a row: bf16 k = 0 36 us, 1 40, 20 47 (3.3
// TB/s); fp32 k = 0 51 (6.1 TB/s), 20 61; bf16, k = 20, all but a thousandth -inf 57
// (the weighted sum is formed twice).  x - m in place of one multiply-add costs 2
// of the 47.  On the way (of then 44): without the next pieces on their way and
// packed arithmetic 47; the entries of the k threads read again, 20 us more at k =
// 20 (16 bytes of each sector of memory that has left the L2).
#include <cuda_fp16.h>

#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

// Warps a CTA: eight where the clusters of eight CTAs of all rows run at once (a
// row's latency counts), else four, whose CTAs fill the SMs more evenly.  GB300,
// calls in a row, us with four and eight: 4 rows of 32000, fp32, k = 5, 10.7, 9.2; 1
// of 151936, bf16, k = 1, 10.5, 8.6; 256 of 128256, k = 20, 27.7, 30.5; 512 of 151936
// 46.5, 50.3.  Just past the rule's border, of 57 rows, eight would still be better:
// 64 of 128256, k = 20, 26.6, 17.7 (clusters of eight and of four CTAs).
constexpr int kFewRows = 8, kManyRows = 4;
template <int kWarps>
constexpr int kPerSM = 28 / kWarps;  // CTAs
constexpr int kBatch = 4, kSlots = 16;
constexpr int kTop = kLogprobsMaxTop;
constexpr int kCandidates = 1024;
constexpr int kMaxCluster = 8;
constexpr float kL = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A sum of 2^y and one of 2^y y, y = (x - m) L, m the largest x but for a few
// powers of two.
struct Sums {
  float m, s, e;
};
// Its terms in units of e^m2 >= e^m.  (What has seen nothing above -inf has m =
// -inf and zeros, or NaN, which is kept.)
__device__ __forceinline__ void lower(Sums& a, float m2) {
  if (a.m == -INFINITY || a.m == m2) return;
  const float d = fmaxf((a.m - m2) * kL, -300.f), f = ex2(d);
  a.e = f * fmaf(d, a.s, a.e);
  a.s *= f;
}
// The sums of the warp's lanes, or of each kLanes of them, as one.  (The maximum
// first: so each is lowered, and rounded, once.)
template <int kLanes = 32>
__device__ __forceinline__ Sums joined(Sums a) {
  float m = a.m;
#pragma unroll
  for (int off = kLanes / 2; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  lower(a, m);
#pragma unroll
  for (int off = kLanes / 2; off; off >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, off);
    a.e += __shfl_xor_sync(0xffffffffu, a.e, off);
  }
  return {m, a.s, a.e};
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

// What a thread has seen: its sums, and the piece with its largest entry.  A
// thread of a long row adds up to 512 times, equal entries with roundings of one
// sign: so each sum's rounding is carried along into the next addition (over:
// what the sums are too large by).
struct Seen {
  Sums a{-INFINITY, 0.f, 0.f};
  float over_s = 0.f, over_e = 0.f;
  float best = -INFINITY;
  int piece = -1;
};
__device__ __forceinline__ void settle(Seen& t) {
  t.a.s -= t.over_s;
  t.a.e -= t.over_e;
  t.over_s = t.over_e = 0.f;
}
__device__ __forceinline__ void add(Seen& t, float s, float e) {
  const float ds = s - t.over_s, de = e - t.over_e;
  const float to_s = t.a.s + ds, to_e = t.a.e + de;
  t.over_s = (to_s - t.a.s) - ds;
  t.over_e = (to_e - t.a.e) - de;
  t.a.s = to_s;
  t.a.e = to_e;
}
// An entry x is to be added.  (The maximum is left where it is until weights would
// pass 2^4: each time it is moved rounds the sums.)
__device__ __forceinline__ void reach(Seen& t, float x) {
  if ((x - t.a.m) * kL > 4.f) {
    settle(t);
    lower(t.a, x);
    t.a.m = x;
  }
}

// Two entries a word, their largest, and as floats (an fp32 row: one a word).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, const __nv_bfloat16*) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, const __half*) {
  const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ float largest_of(const uint4& w) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmax3(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z)), __uint_as_float(w.w));
  } else {
    const T* p = nullptr;
    const uint32_t m = max2(max2(w.x, w.y, p), max2(w.z, w.w, p), p);
    const T* v = reinterpret_cast<const T*>(&m);
    return fmaxf(to_f(v[0]), to_f(v[1]));
  }
}

template <typename T, int kPieces>
__device__ __forceinline__ float take(Seen& t, const uint4 (&w)[kPieces], int j0, int step) {
  float top = -INFINITY;
#pragma unroll
  for (int b = 0; b < kPieces; ++b) {
    const float m = largest_of<T>(w[b]);
    if (m > t.best) {
      t.best = m;
      t.piece = j0 + b * step;
    }
    top = fmaxf(top, m);
  }
  reach(t, top);
  const float off = -finite_or_0(t.a.m);
  const uint64_t by = f2pack(kL, kL), off2 = f2pack(off, off);
  uint64_t s[2] = {0, 0}, e[2] = {0, 0};
  const T* p = nullptr;
#pragma unroll
  for (int b = 0; b < kPieces; ++b) {
    float x[kPer<T>];
    floats_of(w[b], p, x);
#pragma unroll
    for (int i = 0; i < kPer<T>; i += 2) {
      const uint64_t y2 = fmul2(fadd2(f2pack(x[i], x[i + 1]), off2), by);
      float y0, y1;
      f2unpack(y2, y0, y1);
      const uint64_t w2 = f2pack(ex2(y0), ex2(y1));
      s[i >> 1 & 1] = fadd2(s[i >> 1 & 1], w2);
      e[i >> 1 & 1] = ffma2(w2, y2, e[i >> 1 & 1]);
    }
  }
  float weighted = f2sum(fadd2(e[0], e[1]));
  if (weighted != weighted) {  // a y of -inf, 0 times it: again, with what has no weight held (or NaN, which stays)
    weighted = 0.f;
#pragma unroll
    for (int b = 0; b < kPieces; ++b) {
      float x[kPer<T>];
      floats_of(w[b], p, x);
#pragma unroll
      for (int i = 0; i < kPer<T>; ++i) {
        const float y = (x[i] + off) * kL;
        weighted = fmaf(ex2(y), fmaxf(y, -200.f), weighted);
      }
    }
  }
  add(t, f2sum(fadd2(s[0], s[1])), weighted);
  return top;
}
// The same of one piece that may be partly outside the row.
template <typename T>
__device__ __forceinline__ float take_edge(Seen& t, const Row<T>& row, int j) {
  float x[kPer<T>], most = -INFINITY;
  row.entries(j, x);
  for (int i = 0; i < kPer<T>; ++i) {
    if (x[i] > t.best) {
      t.best = x[i];
      t.piece = j;
    }
    reach(t, x[i]);
    const float y = (x[i] - finite_or_0(t.a.m)) * kL, w = ex2(y);
    add(t, w, w * fmaxf(y, -200.f));
    most = fmaxf(most, x[i]);
  }
  return most;
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

template <int kWarps>
struct Shared {
  static constexpr int kThreads = kWarps * 32;
  Sums warp_sum[kWarps];
  uint64_t lists[kWarps][32];
  uint64_t candidates[kCandidates];
  uint64_t result[kTop];
  float most[kSlots][kThreads];
  uint16_t reached[kSlots * kThreads];
  int n_reached, n_candidates;
  Sums sum;
};

// The k largest of sh.candidates into sh.result (sorted; 0 where there are
// fewer).  Called by the whole CTA, result cleared.
template <int kWarps>
__device__ __forceinline__ void rank(Shared<kWarps>& sh, int n, int k) {
  for (int i = threadIdx.x; i < n; i += kWarps * 32) {
    const uint64_t key = sh.candidates[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += sh.candidates[j] > key;
    if (r < k && key) sh.result[r] = key;
  }
}

template <typename T, int kWarps>
__device__ __forceinline__ void largest(Shared<kWarps>& sh, const Row<T>& row, const Seen& t, int k, int first, int total, int slot) {
  constexpr int kThreads = kWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t own = 0;
  const int mine = first + threadIdx.x;
  for (int j = t.piece >= 0 ? t.piece : mine; j < row.pieces && !own; j += total) {  // (nothing above -inf: the first of them)
    float x[kPer<T>];
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
  if (k == 1) {
    if (threadIdx.x == 0) sh.result[0] = least;
    __syncthreads();
    return;
  }
  // The slots that reach the threshold, and of their pieces the entries that do.
  const uint32_t least_x = static_cast<uint32_t>(least >> 32);
#pragma unroll 4
  for (int i = 0; i < kSlots; ++i)
    if (float_key(sh.most[i][threadIdx.x]) >= least_x)
      sh.reached[atomicAdd(&sh.n_reached, 1)] = static_cast<uint16_t>(i * kThreads + threadIdx.x);
  __syncthreads();
  const int pieces = sh.n_reached * slot;
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int e = threadIdx.x; e < pieces; e += kThreads) {
      const int n = e / slot, at = sh.reached[n];
      const int j = first + at % kThreads + (at / kThreads * slot + e - n * slot) * total;
      if (j >= row.pieces || (row.whole(j) && float_key(largest_of<T>(row.raw(j))) < least_x)) continue;
#pragma unroll 1
      for (int i = max(j * kPer<T> - row.skew, 0); i < min((j + 1) * kPer<T> - row.skew, row.V); ++i) {
        const float x = to_f(row.p[i]);
        const uint64_t key = key_of(x, i);
        if (x == x && key >= least) f(key);
      }
    }
  };
  each([&](uint64_t key) {
    const int at = atomicAdd(&sh.n_candidates, 1);
    if (at < kCandidates) sh.candidates[at] = key;
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

template <typename T, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kPerSM<kWarps>) logprobs_kernel(const LogprobsArgs a, int cluster) {
  constexpr int kThreads = kWarps * 32;
  __shared__ Shared<kWarps> sh;
  previous_done();
  next_may_begin();
  const int r = static_cast<int>(blockIdx.x / cluster);
  const int at = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = a.tokens ? a.tokens[r] : 0;
  if (token < 0) return;  // every CTA of the cluster alike
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.stride, a.V);
  if (tid < kTop) sh.result[tid] = 0;
  if (tid == 0) sh.n_reached = sh.n_candidates = 0;

  const int total = cluster * kThreads, first = at * kThreads;
  Seen t;
  // A thread's pieces in fours, in at most kSlots slots of so many each.
  const int fours = (row.pieces + kBatch * total - 1) / (kBatch * total);
  const int slot = (fours + kSlots - 1) / kSlots * kBatch;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) sh.most[i][tid] = -INFINITY;
  auto whole = [&](int j) { return j >= row.begin && j + (kBatch - 1) * total < row.end; };
  uint4 w[kBatch], next[kBatch];
  auto load = [&](uint4 (&to)[kBatch], int j) {
    if (whole(j))
#pragma unroll
      for (int b = 0; b < kBatch; ++b) to[b] = row.raw(j + b * total);
  };
  int j = first + tid;
  load(w, j);
#pragma unroll 1
  for (int n = 0, i = 0; n < fours; ++n) {
    load(next, j + kBatch * total);
    float top = -INFINITY;
    if (whole(j)) {
      top = take<T>(t, w, j, total);
    } else {
#pragma unroll 1
      for (int at = j; at < min(j + kBatch * total, row.pieces); at += total) {
        if (row.whole(at)) {
          const uint4 one[1] = {row.raw(at)};
          top = fmaxf(top, take<T>(t, one, at, 0));
        } else {
          top = fmaxf(top, take_edge(t, row, at));
        }
      }
    }
    sh.most[i][tid] = fmaxf(sh.most[i][tid], top);
    if ((n + 1) * kBatch >= (i + 1) * slot) ++i;
    j += kBatch * total;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) w[b] = next[b];
  }

  settle(t);
  Sums sum = joined(t.a);
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  sum = joined<kWarps>(sh.warp_sum[lane % kWarps]);
  if (a.k > 0) largest(sh, row, t, a.k, first, total, slot);

  if (cluster > 1) {
    if (tid == 0) sh.sum = sum;
    cluster_sync();
    if (at == 0) {
      Sums of{-INFINITY, 0.f, 0.f};  // a CTA of the cluster
      if (const int c = lane % kMaxCluster; c < cluster)
        of = {load_remote(&sh.sum.m, c), load_remote(&sh.sum.s, c), load_remote(&sh.sum.e, c)};
      sum = joined<kMaxCluster>(of);
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
  const float log_s = log2f(sum.s);
  auto logprob = [&](float x) { return fmaf(-log_s, kLn2, x - finite_or_0(sum.m)); };
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

template <typename T, int kWarps>
cudaError_t launch_w(const LogprobsArgs& a, cudaStream_t s) {
  const int pieces = a.V / kPer<T> + 2;
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(a.rows) * cluster * 2 <= kPerSM<kWarps> * 152 &&
         cluster * kWarps * 32 * 2 <= pieces)
    cluster *= 2;
  return launch_early(logprobs_kernel<T, kWarps>, static_cast<unsigned>(a.rows) * cluster, kWarps * 32, 0, s, cluster,
                      a, cluster);
}
template <typename T>
cudaError_t launch_t(const LogprobsArgs& a, cudaStream_t s) {
  const bool few = static_cast<int64_t>(a.rows) * kMaxCluster <= kPerSM<kFewRows> * 152;
  return few ? launch_w<T, kFewRows>(a, s) : launch_w<T, kManyRows>(a, s);
}
template <typename T>
cudaError_t preload_t() {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, logprobs_kernel<T, kFewRows>);
  return e == cudaSuccess ? cudaFuncGetAttributes(&at, logprobs_kernel<T, kManyRows>) : e;
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.type == kBf16) return launch_t<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}

cudaError_t preload_logprobs_kernels() {
  cudaError_t e = preload_t<__nv_bfloat16>();
  if (e == cudaSuccess) e = preload_t<__half>();
  if (e == cudaSuccess) e = preload_t<float>();
  return e;
}

}  // namespace oasis
