// tree.cu -- attention of a request's tree of drafted tokens over its 8-bit
// pages.  A warp per node and query head.
#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

constexpr int kTreeWarps = 8;

__device__ __forceinline__ float4 load_row4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}
__device__ __forceinline__ float4 load_row4(const __half* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 codes4(uint32_t w) {
  const uint32_t lo = q8_unpack2(w & 0xffffu), hi = q8_unpack2(w >> 16);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

template <typename T>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_kernel(const TreeArgs a) {
  previous_done();
  next_may_begin();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTreeWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.R) * a.N * a.Hq) return;
  const int hq = static_cast<int>(row % a.Hq), h = hq / a.G;
  const int i = static_cast<int>(row / a.Hq % a.N), r = static_cast<int>(row / a.Hq / a.N);
  const int nodes = a.size ? min(max(a.size[r], 0), a.N) : a.N;
  if (i >= nodes) return;
  int len = max(a.len[r], 0);
  if (len > a.max_blocks * kBlock || (len > 0 && len < nodes)) {
    if (lane == 0) raise_error(a.err, kErrBadBlock);
    len = len < nodes ? 0 : a.max_blocks * kBlock;
  }
  const int base = len - nodes;
  const uint64_t word = a.words[static_cast<int64_t>(r) * a.N + i];
  float4 q = load_row4(static_cast<const T*>(a.q) + row * kHeadDim + lane * 4);
  scale4(q, a.scale_log2);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int b = 0; b * kBlock < len; ++b) {
    const int page = a.table[static_cast<int64_t>(r) * a.max_blocks + b];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) raise_error(a.err, kErrBadBlock);
      continue;
    }
    const uint8_t* unit = a.pages + (static_cast<int64_t>(page) * a.Hkv + h) * kQ8UnitBytes;
    for (int j = 0; j < kBlock; ++j) {
      const int pos = b * kBlock + j;
      if (pos >= len || (pos >= base && !(word >> (pos - base) & 1))) continue;
      float4 k = codes4(*reinterpret_cast<const uint32_t*>(unit + q8_key_at(j, lane * 4)));
      float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      x *= pow2f(unit[kQ8ExpOffset + j] - 127);
      uint32_t w = 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) w |= static_cast<uint32_t>(unit[q8_value_at(j, lane * 4 + d)]) << (8 * d);
      float4 v = codes4(w);
      scale4(v, pow2f(unit[kQ8ExpOffset + kBlock + j] - 127));
      const float top = fmaxf(m, x), old = scale_of(m, top), p = ex2(x - finite_or_0(top));
      scale4(o, old);
      add4(o, p, v);
      l = l * old + p;
      m = top;
    }
  }
  const float4 v = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / l, o.y / l, o.z / l, o.w / l);
  if (a.out_fp32) store4_finite(static_cast<float*>(a.out) + row * kHeadDim + lane * 4, v);
  else store4_finite(static_cast<T*>(a.out) + row * kHeadDim + lane * 4, v);
}

template <typename T>
cudaError_t launch_t(const TreeArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.R) * a.N * a.Hq;
  return launch_early(tree_kernel<T>, static_cast<unsigned>((rows + kTreeWarps - 1) / kTreeWarps), kTreeWarps * 32, 0,
                      s, 0, a);
}

}  // namespace

cudaError_t launch_q8_tree(const TreeArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  return a.type == kBf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

cudaError_t preload_tree_kernels() {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, tree_kernel<__nv_bfloat16>);
  return e == cudaSuccess ? cudaFuncGetAttributes(&at, tree_kernel<__half>) : e;
}

}  // namespace oasis
