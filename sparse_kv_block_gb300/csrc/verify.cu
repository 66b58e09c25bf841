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
// Knuth give them) inside a segment of 1024 entries, 64 bits between the
// segments.  64-bit arithmetic throughout would bound the kernel: the card's
// rate for it is two lanes a clock and SM.
//
// One cluster of CTAs per request reads the one or two rows that are needed
// once, segment by segment; the segments' sums go to every CTA through
// distributed shared memory, each finds the segment that the threshold falls
// in, and the CTA that read it reads those 1024 entries again.  No scratch in
// global memory, no atomics on results, one launch.
#include "common.cuh"
#include "q8.h"

#include <cuda_fp16.h>

namespace oasis {
namespace {

constexpr int kSeg = 1024;            // entries of a segment (32 lanes x 8 x 4)
#ifndef VW
#define VW 16
#define VS 2
#endif
constexpr int kVerifyWarps = VW;
constexpr int kMaxSegs = 1024;        // vocabularies up to 2^20

// ---- four consecutive entries as floats, whatever the alignment
template <typename T, bool kVec>
__device__ __forceinline__ float4 row4(const T* p, int at, int V);
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

template <typename T, bool kVec>
__device__ __forceinline__ float4 row4(const T* p, int at, int V) {
  if (kVec && at + 4 <= V) {
    if constexpr (sizeof(T) == 4) {
      return __ldg(reinterpret_cast<const float4*>(p + at));
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + at));
      T t[4];
      memcpy(t, &w, 8);
      return make_float4(to_f(t[0]), to_f(t[1]), to_f(t[2]), to_f(t[3]));
    }
  }
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at < V) r.x = to_f(p[at]);
  if (at + 1 < V) r.y = to_f(p[at + 1]);
  if (at + 2 < V) r.z = to_f(p[at + 2]);
  if (at + 3 < V) r.w = to_f(p[at + 3]);
  return r;
}

// ---- sums of pairs: hi + lo, hi the rounded sum (no contraction: __f*_rn)
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ void add(Pair& s, float x, float x_lo) {
  const float t = __fadd_rn(s.hi, x);
  const float z = __fsub_rn(t, s.hi);
  const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, z)), __fsub_rn(x, z));
  s.hi = t;
  s.lo = __fadd_rn(s.lo, __fadd_rn(e, x_lo));
}
// max(p - q, 0) as a pair, exactly; NaN counts as 0.
__device__ __forceinline__ void add_rest(Pair& s, float p, float q) {
  const float d = __fsub_rn(p, q);
  const float b = __fsub_rn(d, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
  if (d > 0.f) add(s, d, e);
}
__device__ __forceinline__ Pair join(Pair a, Pair b) {
  add(a, b.hi, b.lo);
  return a;
}
__device__ __forceinline__ double value(Pair a) {
  return static_cast<double>(a.hi) + static_cast<double>(a.lo);
}
__device__ __forceinline__ double rest(float p, float q) {
  const double d = static_cast<double>(p) - static_cast<double>(q);
  return d > 0.0 ? d : 0.0;
}

// What a request's threshold falls on.
template <typename T, bool kVec>
struct Rows {
  const T* p;
  const T* q;      // null: nothing to subtract
  int certain;     // the token that a certain draft takes out, or -1
  int V;
  __device__ __forceinline__ void load(int at, float4& x, float4& y) const {
    x = row4<T, kVec>(p, at, V);
    y = q ? row4<T, kVec>(q, at, V) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (certain >= at && certain < at + 4) {
      x.x = certain == at ? 0.f : x.x;
      x.y = certain == at + 1 ? 0.f : x.y;
      x.z = certain == at + 2 ? 0.f : x.z;
      x.w = certain == at + 3 ? 0.f : x.w;
    }
  }
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kVerifyWarps * 32)
    verify_kernel(const VerifyArgs a, int cluster) {
  __shared__ double sums[2][kMaxSegs];
  __shared__ int first_s, bad_s;
  const int r = blockIdx.x / cluster;
  const uint32_t rank = cluster_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.n_drafts ? min(max(a.n_drafts[r], 0), a.n) : a.n;
  const int V = a.V;
  const T* target = static_cast<const T*>(a.target) + static_cast<int64_t>(r) * (a.n + 1) * a.target_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + static_cast<int64_t>(r) * a.n * a.draft_stride
                           : nullptr;
  const int32_t* tokens = a.tokens + static_cast<int64_t>(r) * a.n;
  int32_t* out = a.out_tokens + static_cast<int64_t>(r) * (a.n + 1);

  // The first refused draft.  Products of two floats are exact in 64 bits.
  if (tid == 0) {
    first_s = n;
    bad_s = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int x = tokens[i];
    if (x < 0 || x >= V) {
      bad_s = 1;
    } else {
      const float p = to_f(target[i * a.target_stride + x]);
      const float q = draft ? to_f(draft[i * a.draft_stride + x]) : 1.f;
      const double u = a.u_accept[static_cast<int64_t>(r) * a.n + i];
      if (!(u * static_cast<double>(q) < static_cast<double>(p))) atomicMin(&first_s, i);
    }
  }
  cluster_sync();  // also: every CTA runs before the first remote store
  const int k = first_s;
  const bool bad = bad_s != 0;
  if (rank == 0) {
    for (int i = tid; i <= a.n; i += blockDim.x)
      if (i != k || bad) out[i] = (i < k && !bad) ? tokens[i] : -1;
    if (tid == 0) a.n_accept[r] = bad ? -1 : k;
  }
  if (bad) return;  // every CTA of the cluster alike

  Rows<T, kVec> rows;
  rows.p = target + k * a.target_stride;
  rows.q = k < n && draft ? draft + k * a.draft_stride : nullptr;
  rows.certain = k < n && !draft ? tokens[k] : -1;
  rows.V = V;
  const int segs = (V + kSeg - 1) / kSeg;
  const int stride = cluster * kVerifyWarps;
  for (int pass = 0; pass < 2; ++pass) {
    double* mine = sums[pass];
    for (int seg = rank * kVerifyWarps + warp; seg < segs; seg += stride) {
      Pair s[4] = {};
      float4 x[8], y[8];  // all of the segment's loads in flight
#pragma unroll
      for (int i = 0; i < 8; ++i) rows.load(seg * kSeg + i * 128 + lane * 4, x[i], y[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        add_rest(s[0], x[i].x, y[i].x);
        add_rest(s[1], x[i].y, y[i].y);
        add_rest(s[2], x[i].z, y[i].z);
        add_rest(s[3], x[i].w, y[i].w);
      }
      Pair t = join(join(s[0], s[1]), join(s[2], s[3]));
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        Pair o;
        o.hi = __shfl_xor_sync(0xffffffffu, t.hi, off);
        o.lo = __shfl_xor_sync(0xffffffffu, t.lo, off);
        t = join(t, o);
      }
      const double v = __shfl_sync(0xffffffffu, value(t), 0);
      if (lane < cluster) store_remote(&mine[seg], lane, v);
    }
    cluster_sync();

    // Every warp: the sums before each lane's share of the segments, the
    // total, and the segment that the threshold falls in.
    const int share = (segs + 31) / 32;
    double own = 0.0;
    for (int i = 0; i < share; ++i)
      if (lane * share + i < segs) own += mine[lane * share + i];
    double incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const double total = __shfl_sync(0xffffffffu, incl, 31);
    if (!(total > 0.0)) {
      // Nothing is left of the difference: draw from p itself.
      if (pass == 0 && (rows.q || rows.certain >= 0)) {
        rows.q = nullptr;
        rows.certain = -1;
        continue;
      }
      if (rank == 0 && tid == 0) out[k] = -1;  // no entry above zero
      return;
    }
    const double threshold = static_cast<double>(a.u_sample[r]) * total;
    // The lane whose share holds it; past the end (u = 1, or a rounding), the
    // last lane with anything.
    unsigned over = __ballot_sync(0xffffffffu, incl > threshold && own > 0.0);
    const unsigned some = __ballot_sync(0xffffffffu, own > 0.0);
    const int at = over ? __ffs(over) - 1 : 31 - __clz(some);
    double before = __shfl_sync(0xffffffffu, incl - own, at);
    int seg = -1, last = -1;
    double last_before = before;
    for (int i = 0; i < share && at * share + i < segs; ++i) {
      const double v = mine[at * share + i];
      if (v > 0.0) {
        last = at * share + i;
        last_before = before;
        if (before + v > threshold) {
          seg = last;
          break;
        }
      }
      before += v;
    }
    if (seg < 0) seg = last;
    before = last_before;
    if ((seg % stride) / kVerifyWarps != static_cast<int>(rank) || seg % kVerifyWarps != warp) return;

    // The segment's own warp: 32 consecutive entries a lane, then one entry a
    // lane of the 32 that hold the threshold.
    Pair s[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float4 x, y;
      rows.load(seg * kSeg + lane * 32 + i * 4, x, y);
      add_rest(s[0], x.x, y.x);
      add_rest(s[1], x.y, y.y);
      add_rest(s[2], x.z, y.z);
      add_rest(s[3], x.w, y.w);
    }
    own = value(join(join(s[0], s[1]), join(s[2], s[3])));
    incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    over = __ballot_sync(0xffffffffu, before + incl > threshold && own > 0.0);
    const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
    const int part = over ? __ffs(over) - 1 : 31 - __clz(any);
    before += __shfl_sync(0xffffffffu, incl - own, part);
    const int e = seg * kSeg + part * 32 + lane;
    float p = 0.f, q = 0.f;
    if (e < V && e != rows.certain) {
      p = to_f(rows.p[e]);
      q = rows.q ? to_f(rows.q[e]) : 0.f;
    }
    const double d = rest(p, q);
    incl = d;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    over = __ballot_sync(0xffffffffu, before + incl > threshold && d > 0.0);
    const unsigned pos = __ballot_sync(0xffffffffu, d > 0.0);
    const int j = over ? __ffs(over) - 1 : 31 - __clz(pos);
    if (lane == 0) out[k] = seg * kSeg + part * 32 + j;
    return;
  }
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.target) % (4 * sizeof(T)) == 0 &&
                   a.target_stride % 4 == 0 &&
                   (!a.draft || (reinterpret_cast<uintptr_t>(a.draft) % (4 * sizeof(T)) == 0 &&
                                 a.draft_stride % 4 == 0));
  const int segs = (a.V + kSeg - 1) / kSeg;
  int cluster = 1;
  while (cluster < 8 && cluster * kVerifyWarps < segs && 2 * cluster * a.R <= VS * 152) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.R) * cluster);
  cfg.blockDim = dim3(kVerifyWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return vec ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, a, cluster)
             : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, a, cluster);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  if (a.type == kBf16) return launch_t<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}

cudaError_t preload_verify_kernels() {
  cudaFuncAttributes at;
  const void* fns[] = {reinterpret_cast<const void*>(verify_kernel<float, true>),
                       reinterpret_cast<const void*>(verify_kernel<float, false>),
                       reinterpret_cast<const void*>(verify_kernel<__half, true>),
                       reinterpret_cast<const void*>(verify_kernel<__half, false>),
                       reinterpret_cast<const void*>(verify_kernel<__nv_bfloat16, true>),
                       reinterpret_cast<const void*>(verify_kernel<__nv_bfloat16, false>)};
  for (const void* f : fns) {
    const cudaError_t e = cudaFuncGetAttributes(&at, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace oasis
