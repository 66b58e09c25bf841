// verify.cu -- which drafted tokens the target's probabilities accept, and
// the token that follows (speculative decoding).
//
// Draft i of a request is accepted while u_i * q_i(x_i) < p_i(x_i).  With k
// the first refused draft, the next token is drawn from max(p_k - q_k, 0) by
// the given u: the first j whose running sum exceeds u * total (from p_n when
// all are accepted, and from p_k where the difference leaves nothing).
//
// Tokens are whole numbers, so a sum that is off by one unit in the last
// place of 32 bits can name another token (a vocabulary's neighbouring
// borders are about 1e-5 apart).  The sums are therefore held to about 48
// bits: pairs of floats (an error-free sum and its remainder, as Dekker and
// Knuth give them), two entries an instruction within a segment of the row.
// 64-bit arithmetic would bound the kernel: the card's rate for it is two
// lanes a clock and SM.
//
// One cluster of CTAs per request reads the one or two rows that are needed
// once, segment by segment; the segments' sums go to every CTA through
// distributed shared memory, each finds the segment that the threshold falls
// in, and the CTA that read it reads those entries again, all its threads
// together.  No scratch in global memory, one launch.
#include "q8.cuh"
#include "q8.h"

#include <cuda_fp16.h>

namespace oasis {
namespace {

constexpr int kVerifyWarps = 16;
constexpr int kThreads = kVerifyWarps * 32;
constexpr int kMaxSegs = 1024;        // of 1024 entries: vocabularies up to 2^20
constexpr int kShortSeg = 256, kLongSeg = 1024;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// ---- four consecutive entries, of any alignment, or with 0 past the row's end
template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T x[4];
};
// As floats.  (Of bf16 by shifts: conversions run at a quarter of the rate.)
__device__ __forceinline__ void floats_of(const Four<float>& f, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f.x[i];
}
__device__ __forceinline__ void floats_of(const Four<__nv_bfloat16>& f, float (&x)[4]) {
  uint32_t w[2];
  memcpy(w, f.x, 8);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ void floats_of(const Four<__half>& f, float (&x)[4]) {
  __half2 w[2];
  memcpy(w, f.x, 8);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 v = __half22float2(w[i]);
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ Four<T> row4(const T* p) {
  if constexpr (kVec) {
    return *reinterpret_cast<const Four<T>*>(p);
  } else {
    Four<T> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.x[i] = p[i];
    return r;
  }
}
template <typename T>
__device__ __forceinline__ Four<T> row4(const T* p, int at, int V) {
  Four<T> r;
  const T none = T(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) r.x[i] = at + i < V ? p[at + i] : none;
  return r;
}

// ---- sums of pairs: hi + lo, hi the rounded sum (no contraction: __f*_rn)
struct alignas(8) Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair join(Pair s, Pair x) {
  const float t = __fadd_rn(s.hi, x.hi);
  const float z = __fsub_rn(t, s.hi);
  const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, z)), __fsub_rn(x.hi, z));
  return {t, __fadd_rn(s.lo, __fadd_rn(e, x.lo))};
}
// The same with lo under half a unit of hi again, for the long chains.
__device__ __forceinline__ Pair join_tight(Pair s, Pair x) {
  const Pair t = join(s, x);
  const float hi = __fadd_rn(t.hi, t.lo);
  return {hi, __fsub_rn(t.lo, __fsub_rn(hi, t.hi))};
}
// a < b.
__device__ __forceinline__ bool less(Pair a, Pair b) {
  const Pair d = join(b, Pair{-a.hi, -a.lo});
  return __fadd_rn(d.hi, d.lo) > 0.f;
}
// max(p - q, 0) exactly, negative numbers and NaN counting as 0: with the
// larger of the two first, the remainder of the difference takes three steps.
__device__ __forceinline__ Pair rest(float p, float q) {
  q = fmaxf(q, 0.f);
  p = fmaxf(p, q);
  const float d = __fsub_rn(p, q);
  return {d, -__fadd_rn(q, __fsub_rn(d, p))};
}
// The same for two entries at a time, added to two running sums (a - b as
// -1 * b + a, one rounding).
struct Pair2 {
  uint64_t hi, lo;
};
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b, uint64_t minus) { return ffma2(b, minus, a); }
__device__ __forceinline__ void add_rest2(Pair2& s, float p0, float p1, float q0, float q1, uint64_t minus) {
  q0 = fmaxf(q0, 0.f);
  q1 = fmaxf(q1, 0.f);
  const uint64_t q = f2pack(q0, q1), p = f2pack(fmaxf(p0, q0), fmaxf(p1, q1));
  const uint64_t d = sub2(p, q, minus);
  const uint64_t less = fadd2(q, sub2(d, p, minus));  // minus the remainder
  const uint64_t t = fadd2(s.hi, d), z = sub2(t, s.hi, minus);
  const uint64_t e = fadd2(sub2(s.hi, sub2(t, z, minus), minus), sub2(d, z, minus));
  s.hi = t;
  s.lo = fadd2(s.lo, sub2(e, less, minus));
}
__device__ __forceinline__ Pair half_of(const Pair2& s, int i) {
  float h0, h1, l0, l1;
  f2unpack(s.hi, h0, h1);
  f2unpack(s.lo, l0, l1);
  return i ? Pair{h1, l1} : Pair{h0, l0};
}
__device__ __forceinline__ Pair shuffled(Pair a, int off) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)};
}
// Sums over the lanes up to this one.
__device__ __forceinline__ Pair scan(Pair a, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair o = {__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
    if (lane >= off) a = join_tight(o, a);
  }
  return a;
}

// What a request's threshold falls on.
template <typename T>
struct Rows {
  const T* p;
  const T* q;      // null: nothing to subtract
  int certain;     // the token that a certain draft takes out, or -1
  int V;
};

// A warp's sums over a segment's entries, each lane its own.
template <typename T, bool kVec, int kSeg, bool kQ>
__device__ __forceinline__ Pair segment(const Rows<T>& rows, int seg, int lane) {
  const uint64_t minus = f2pack(-1.f, -1.f);
  Pair2 s0{}, s1{};
  auto add = [&](int at, const Four<T>& from, const Four<T>& less) {
    float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
    floats_of(from, x);
    if constexpr (kQ) {
      floats_of(less, y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = rows.certain == at + i ? 0.f : x[i];
    }
    add_rest2(s0, x[0], x[1], y[0], y[1], minus);
    add_rest2(s1, x[2], x[3], y[2], y[3], minus);
  };
  const int begin = seg * kSeg + lane * 4;
  constexpr int kLoads = kSeg / 128;
  if ((seg + 1) * kSeg <= rows.V) {
    // Nothing between the loads, so that a batch is in flight together.  (With
    // a test for the row's end at each load the code waits between them: 128
    // rows of 151936 took 28.3 us in fp32 and 40 in bf16 instead of 24 and 21.)
    constexpr int kBatch = kLoads < 4 ? kLoads : 4;
#pragma unroll
    for (int i0 = 0; i0 < kLoads; i0 += kBatch) {
      Four<T> x[kBatch], y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        x[i] = row4<T, kVec>(rows.p + begin + (i0 + i) * 128);
        if constexpr (kQ) y[i] = row4<T, kVec>(rows.q + begin + (i0 + i) * 128);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) add(begin + (i0 + i) * 128, x[i], y[i]);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < kLoads; ++i) {
      const int at = begin + i * 128;
      Four<T> x, y;
      x = row4<T>(rows.p, at, rows.V);
      if constexpr (kQ) y = row4<T>(rows.q, at, rows.V);
      add(at, x, y);
    }
  }
  return join(join(half_of(s0, 0), half_of(s0, 1)), join(half_of(s1, 0), half_of(s1, 1)));
}

// The segment that u of the total falls in, and what of it the segment has to
// exceed; -1 where there is nothing, -2 where there is no sum.  By one warp: the
// sums before each lane's share of the segments, then the segments of one
// share.  (64-bit operations took as long as this in pairs, 1 us alone and 3
// beside another CTA that reads; run ahead on a made-up table, to have the code
// at hand, it cost 3 us.)
struct Found {
  int seg;
  Pair rest;
};
__device__ __noinline__ Found find(const Pair* sums, int segs, float u, int lane) {
  const int share = (segs + 31) / 32;
  Pair own{};
  for (int i = 0; i < share; ++i)
    if (lane * share + i < segs) own = join_tight(own, sums[lane * share + i]);
  const Pair incl = scan(own, lane);
  const Pair total = {__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
  Found f = {total.hi == 0.f ? -1 : -2, {}};
  if (!(total.hi > 0.f && total.hi + total.lo < INFINITY)) return f;
  const float high = __fmul_rn(u, total.hi);
  const Pair threshold = {high, __fmaf_rn(u, total.lo, __fmaf_rn(u, total.hi, -high))};
  // The lane whose share holds it; past the end (u = 1, or a rounding), the
  // last lane with anything.
  const unsigned over = __ballot_sync(0xffffffffu, own.hi > 0.f && less(threshold, incl));
  const unsigned some = __ballot_sync(0xffffffffu, own.hi > 0.f);
  const int at = over ? __ffs(over) - 1 : 31 - __clz(some);
  Pair before = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
  if (lane == 0) before = Pair{};
  before = {__shfl_sync(0xffffffffu, before.hi, at), __shfl_sync(0xffffffffu, before.lo, at)};
  for (int i = 0; i < share && at * share + i < segs; ++i) {
    const Pair v = sums[at * share + i];
    if (v.hi > 0.f) {
      f.seg = at * share + i;
      f.rest = join(threshold, Pair{-before.hi, -before.lo});
      if (less(f.rest, v)) break;
    }
    before = join_tight(before, v);
  }
  return f;
}

template <typename T, bool kVec, int kSeg>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a, int cluster) {
  __shared__ Pair sums[2][kMaxSegs];
  __shared__ int first_s, bad_s, seg_s, last_s;
  __shared__ Pair target_s;            // the threshold, from its segment's start
  __shared__ Pair warp_sum[kVerifyWarps];
  previous_done();
  next_may_begin();
  const int r = blockIdx.x / cluster;
  const int rank = static_cast<int>(cluster_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.n_drafts ? min(max(a.n_drafts[r], 0), a.n) : a.n;
  const int V = a.V;
  const T* target = static_cast<const T*>(a.target) + static_cast<int64_t>(r) * (a.n + 1) * a.target_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + static_cast<int64_t>(r) * a.n * a.draft_stride
                           : nullptr;
  const int32_t* tokens = a.tokens + static_cast<int64_t>(r) * a.n;
  int32_t* out = a.out_tokens + static_cast<int64_t>(r) * (a.n + 1);
  const float u = a.u_sample[r];

  // The first refused draft.  Products of two floats are exact in 64 bits.
  if (tid == 0) {
    first_s = n;
    bad_s = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int x = tokens[i];
    const float ua = a.u_accept[static_cast<int64_t>(r) * a.n + i];
    if (x < 0 || x >= V) {
      bad_s = 1;
    } else {
      const float p = fmaxf(to_f(target[i * a.target_stride + x]), 0.f);
      const float q = draft ? fmaxf(to_f(draft[i * a.draft_stride + x]), 0.f) : 1.f;
      if (!(static_cast<double>(ua) * static_cast<double>(q) < static_cast<double>(p))) atomicMin(&first_s, i);
    }
  }
  cluster_sync();  // also: every CTA runs before the first remote store
  const int k = first_s;
  const bool bad = bad_s != 0;
  if (rank == 0) {
    for (int i = tid; i <= a.n; i += kThreads)
      if (i != k || bad) out[i] = (i < k && !bad) ? tokens[i] : -1;
    if (tid == 0) a.n_accept[r] = bad ? -1 : k;
  }
  if (bad) return;  // every CTA of the cluster alike

  Rows<T> rows;
  rows.p = target + k * a.target_stride;
  rows.q = k < n && draft ? draft + k * a.draft_stride : nullptr;
  rows.certain = k < n && !draft ? tokens[k] : -1;
  rows.V = V;
  const int segs = (V + kSeg - 1) / kSeg;
  const int stride = cluster * kVerifyWarps;
  for (int pass = 0; pass < 2; ++pass) {
    Pair* mine = sums[pass];
    for (int at = rank * kVerifyWarps + warp; at < segs; at += stride) {
      Pair t = rows.q ? segment<T, kVec, kSeg, true>(rows, at, lane) : segment<T, kVec, kSeg, false>(rows, at, lane);
#pragma unroll
      for (int off = 16; off; off >>= 1) t = join(t, shuffled(t, off));
      t = {__shfl_sync(0xffffffffu, t.hi, 0), __shfl_sync(0xffffffffu, t.lo, 0)};
      if (lane < cluster) store_remote(&mine[at], lane, f2pack(t.hi, t.lo));
    }
    cluster_sync();

    if (warp == 0) {
      const Found f = find(mine, segs, u, lane);
      if (lane == 0) {
        seg_s = f.seg;
        target_s = f.rest;
        first_s = 0x7fffffff;
        last_s = -1;
      }
    }
    __syncthreads();
    const int seg = seg_s;
    if (seg < 0) {
      // Nothing is left of the difference: draw from p itself.
      if (seg == -1 && pass == 0 && (rows.q || rows.certain >= 0)) {
        rows.q = nullptr;
        rows.certain = -1;
        __syncthreads();  // seg_s is written again
        continue;
      }
      if (rank == 0 && tid == 0) out[k] = -1;  // no entry above zero, or an infinite one
      return;
    }
    if (seg % stride / kVerifyWarps != rank) return;

    // The segment again, two entries a thread: the first whose running sum
    // exceeds the threshold; past the end, the last above zero.
    constexpr int kWarps = kSeg / 64;
    static_assert(kWarps <= kVerifyWarps, "two entries a thread");
    Pair w[2] = {}, before{};
    const int e = seg * kSeg + tid * 2;
    if (warp < kWarps) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (e + i < V && e + i != rows.certain)
          w[i] = rest(to_f(rows.p[e + i]), rows.q ? to_f(rows.q[e + i]) : 0.f);
      const Pair incl = scan(join(w[0], w[1]), lane);
      before = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      if (lane == 0) before = {0.f, 0.f};
      if (lane == 31) warp_sum[warp] = incl;
    }
    __syncthreads();
    if (warp < kWarps) {
      const Pair sum = scan(lane < kWarps ? warp_sum[lane] : Pair{0.f, 0.f}, lane);
      const int left = warp > 0 ? warp - 1 : 0;
      Pair at = {__shfl_sync(0xffffffffu, sum.hi, left), __shfl_sync(0xffffffffu, sum.lo, left)};
      if (warp == 0) at = {0.f, 0.f};
      at = join(join(at, before), Pair{-target_s.hi, -target_s.lo});
      int found = 0x7fffffff, last = -1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        at = join(at, w[i]);
        if (w[i].hi > 0.f) {
          last = e + i;
          if (__fadd_rn(at.hi, at.lo) > 0.f && found == 0x7fffffff) found = e + i;
        }
      }
      found = __reduce_min_sync(0xffffffffu, found);
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        if (found != 0x7fffffff) atomicMin(&first_s, found);
        if (last >= 0) atomicMax(&last_s, last);
      }
    }
    __syncthreads();
    if (tid == 0) out[k] = first_s != 0x7fffffff ? first_s : last_s;
    return;
  }
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.target) % (4 * sizeof(T)) == 0 &&
                   a.target_stride % 4 == 0 &&
                   (!a.draft || (reinterpret_cast<uintptr_t>(a.draft) % (4 * sizeof(T)) == 0 &&
                                 a.draft_stride % 4 == 0));
  // CTAs a request: as many as find a segment for each warp, up to two CTAs
  // an SM over all requests.  Short segments where even so the long ones
  // leave warps without work (few requests: the time is one segment's).
  const int longs = (a.V + kLongSeg - 1) / kLongSeg;
  const bool brief = static_cast<int64_t>(a.R) * longs < 152 * kVerifyWarps && a.V <= kMaxSegs * kShortSeg;
  const int segs = brief ? (a.V + kShortSeg - 1) / kShortSeg : longs;
  int cluster = 1;
  while (cluster < 8 && cluster * kVerifyWarps < segs && 2 * cluster * a.R <= 2 * 152) cluster *= 2;
  const auto kernel = brief ? (vec ? verify_kernel<T, true, kShortSeg> : verify_kernel<T, false, kShortSeg>)
                            : (vec ? verify_kernel<T, true, kLongSeg> : verify_kernel<T, false, kLongSeg>);
  return launch_early(kernel, static_cast<unsigned>(a.R) * cluster, kThreads, 0, s, cluster, a, cluster);
}

template <typename T>
cudaError_t preload() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, verify_kernel<T, true, kShortSeg>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, verify_kernel<T, false, kShortSeg>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, verify_kernel<T, true, kLongSeg>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, verify_kernel<T, false, kLongSeg>);
  return e;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  if (a.type == kBf16) return launch_t<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}

cudaError_t preload_verify_kernels() {
  cudaError_t e = preload<float>();
  if (e == cudaSuccess) e = preload<__half>();
  if (e == cudaSuccess) e = preload<__nv_bfloat16>();
  return e;
}

}  // namespace oasis
