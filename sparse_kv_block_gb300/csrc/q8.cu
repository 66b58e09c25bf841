// q8.cu -- writing keys and values into the 8-bit paged cache, and reading
// them back.
#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

// Four consecutive elements as floats.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// |x| of a finite x, else 0 (an infinity or NaN does not set the scale).
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// A warp's row of 128 values, four a lane: its exponent and the lane's codes.
__device__ __forceinline__ uint32_t quantise_row(float4 x, int& e) {
  const uint32_t m = max(max(finite_abs_bits(x.x), finite_abs_bits(x.y)),
                         max(finite_abs_bits(x.z), finite_abs_bits(x.w)));
  e = q8_exponent(__reduce_max_sync(0xffffffffu, m));
  const float s = pow2f(-e);
  return q8_pack4(x.x * s, x.y * s, x.z * s, x.w * s);
}

// One warp per (token, KV head).
template <typename T>
__global__ void write_kernel(const Q8WriteArgs a) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(a.T) * a.Hkv) return;
  const int t = static_cast<int>(row / a.Hkv), h = static_cast<int>(row - static_cast<int64_t>(t) * a.Hkv);
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) raise_error(a.err, kErrBadUnit);
    return;
  }
  const int j = static_cast<int>(slot & (kBlock - 1));
  uint8_t* unit = a.pages + ((slot >> 4) * a.Hkv + h) * static_cast<int64_t>(kQ8UnitBytes);
  int ke, ve;
  const uint32_t kc = quantise_row(
      load4(static_cast<const T*>(a.k) + t * a.k_stride + h * kHeadDim + lane * 4), ke);
  const uint32_t vc = quantise_row(
      load4(static_cast<const T*>(a.v) + t * a.v_stride + h * kHeadDim + lane * 4), ve);
  *reinterpret_cast<uint32_t*>(unit + q8_key_at(j, lane * 4)) = kc;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    unit[q8_value_at(j, lane * 4 + i)] = static_cast<uint8_t>(vc >> (8 * i));
  if (lane == 0) {
    unit[kQ8ExpOffset + j] = static_cast<uint8_t>(ke + 127);
    unit[kQ8ExpOffset + kBlock + j] = static_cast<uint8_t>(ve + 127);
  }
}

__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half* p, float x) { *p = __float2half_rn(x); }

__device__ __forceinline__ float q8_value(uint8_t code, uint8_t exp) {
  const uint32_t h2 = q8_unpack2(code);
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h2))) * pow2f(exp - 127);
}

// One CTA per (request, block): every KV head's unit.
template <typename T>
__global__ void read_kernel(const Q8ReadArgs a) {
  const int r = blockIdx.y, b = blockIdx.x;
  const int len = a.len[r];
  const int n = len - b * kBlock;
  if (n <= 0) return;
  if (b == 0 && threadIdx.x == 0 && (len - 1) / kBlock >= min(a.max_blocks, a.out_blocks))
    raise_error(a.err, kErrBadBlock);
  if (b >= a.out_blocks) return;
  const int page = a.table[static_cast<int64_t>(r) * a.max_blocks + b];
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0) raise_error(a.err, kErrBadBlock);
    return;
  }
  const int valid = min(n, kBlock);
  for (int h = 0; h < a.Hkv; ++h) {
    const uint8_t* unit = a.pages + (static_cast<int64_t>(page) * a.Hkv + h) * kQ8UnitBytes;
    T* out = static_cast<T*>(a.out) +
             ((static_cast<int64_t>(r) * a.Hkv + h) * a.out_blocks + b) * kUnitElems;
    for (int x = threadIdx.x; x < valid * kHeadDim; x += blockDim.x) {
      const int j = x / kHeadDim, i = x % kHeadDim;
      store1(out + x, q8_value(unit[q8_key_at(j, i)], unit[kQ8ExpOffset + j]));
      store1(out + kBlock * kHeadDim + x,
             q8_value(unit[q8_value_at(j, i)], unit[kQ8ExpOffset + kBlock + j]));
    }
  }
}

}  // namespace

cudaError_t launch_q8_write(const Q8WriteArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv;
  if (rows == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (a.type == kBf16) write_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  else if (a.type == kFp16) write_kernel<__half><<<grid, 256, 0, s>>>(a);
  else write_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  const dim3 grid(a.max_blocks, a.R);
  if (a.type == kBf16) read_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  else if (a.type == kFp16) read_kernel<__half><<<grid, 256, 0, s>>>(a);
  else read_kernel<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t preload_q8_cache_kernels() {
  cudaFuncAttributes at;
  const void* fns[] = {reinterpret_cast<const void*>(write_kernel<__nv_bfloat16>),
                       reinterpret_cast<const void*>(write_kernel<__half>),
                       reinterpret_cast<const void*>(write_kernel<float>),
                       reinterpret_cast<const void*>(read_kernel<__nv_bfloat16>),
                       reinterpret_cast<const void*>(read_kernel<__half>),
                       reinterpret_cast<const void*>(read_kernel<float>)};
  for (const void* f : fns) {
    const cudaError_t e = cudaFuncGetAttributes(&at, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace oasis
