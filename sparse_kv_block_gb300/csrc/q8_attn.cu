// q8_attn.cu -- attention over the 8-bit paged cache, with or without a
// prefix that all requests share.
#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

constexpr int kWarps = 4;

// One CTA per query vector (query s of request r, head hq): each warp takes
// every fourth token with a running maximum and sum; the four are joined in
// shared memory.  A lane holds four dims.
template <typename T>
__global__ void simple_kernel(const Q8AttnArgs a) {
  const int vec = blockIdx.x;  // ((s * R) + r) * Hq + hq
  const int hq = vec % a.Hq, r = (vec / a.Hq) % a.R, s = vec / a.Hq / a.R;
  const int h = hq / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len = max(a.len[r], 0);
  if (len > a.max_blocks * kBlock) {
    if (threadIdx.x == 0) raise_error(a.err, kErrBadBlock);
    len = a.max_blocks * kBlock;
  }
  const int limit = max(a.causal ? len - (a.S - 1 - s) : len, 0);
  float q[4];
  const T* qp = static_cast<const T*>(a.q) + static_cast<int64_t>(vec) * kHeadDim + lane * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = static_cast<float>(qp[i]) * a.scale_log2;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  auto token = [&](const float* k, const float* v) {
    float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float mn = fmaxf(m, x);
    const float al = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(x - mn);
    m = mn;
    l = l * al + p;
    for (int i = 0; i < 4; ++i) o[i] = o[i] * al + p * v[i];
  };
  for (int t = warp; t < a.prefix_len; t += kWarps) {
    const __nv_bfloat16* u = static_cast<const __nv_bfloat16*>(a.prefix) +
        (static_cast<int64_t>(h) * a.prefix_blocks + t / kBlock) * kUnitElems + (t % kBlock) * kHeadDim + lane * 4;
    float k[4], v[4];
    for (int i = 0; i < 4; ++i) {
      k[i] = __bfloat162float(u[i]);
      v[i] = __bfloat162float(u[kBlock * kHeadDim + i]);
    }
    token(k, v);
  }
  for (int t = warp; t < limit; t += kWarps) {
    const int page = a.table[static_cast<int64_t>(r) * a.max_blocks + t / kBlock];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) raise_error(a.err, kErrBadBlock);
      continue;
    }
    const uint8_t* u = a.pages + (static_cast<int64_t>(page) * a.Hkv + h) * kQ8UnitBytes;
    const int j = t % kBlock;
    const float ks = pow2f(u[kQ8ExpOffset + j] - 127), vs = pow2f(u[kQ8ExpOffset + kBlock + j] - 127);
    float k[4], v[4];
    for (int i = 0; i < 4; ++i) {
      k[i] = ks * __half2float(__ushort_as_half(q8_unpack2(u[q8_key_at(j, lane * 4 + i)])));
      v[i] = vs * __half2float(__ushort_as_half(q8_unpack2(u[q8_value_at(j, lane * 4 + i)])));
    }
    token(k, v);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kHeadDim];
  for (int i = 0; i < 4; ++i) so[warp][lane * 4 + i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  const int d = threadIdx.x;
  float mx = -INFINITY, acc = 0.f, den = 0.f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mx);
    acc += f * so[w][d];
    den += f * sl[w];
  }
  const float v = den == 0.f ? 0.f : acc / den;
  const int64_t at = static_cast<int64_t>(vec) * kHeadDim + d;
  if (a.out_fp32) static_cast<float*>(a.out)[at] = v;
  else static_cast<T*>(a.out)[at] = static_cast<T>(v);
}

}  // namespace

cudaError_t launch_q8_attn(const Q8AttnArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.S) * a.R * a.Hq;
  if (grid == 0) return cudaSuccess;
  if (a.type == kBf16) simple_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(a);
  else simple_kernel<__half><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t preload_q8_attn_kernels() {
  cudaFuncAttributes at;
  const void* fns[] = {reinterpret_cast<const void*>(simple_kernel<__nv_bfloat16>),
                       reinterpret_cast<const void*>(simple_kernel<__half>)};
  for (const void* f : fns) {
    const cudaError_t e = cudaFuncGetAttributes(&at, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace oasis
