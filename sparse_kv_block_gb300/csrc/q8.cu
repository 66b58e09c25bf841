// q8.cu -- writing keys and values into the 8-bit paged cache, and reading
// them back.
#include "q8.cuh"
#include "q8.h"
#include "q8_rows.cuh"

namespace oasis {
namespace {

constexpr int kWriteWarps = 4;

// Rounding into the pages.  Bound by memory: 256 values are read and 258
// bytes written a token and head.  What holds it back is latency (the slots,
// then the rows): 16 rows a warp are asked for at once, and seven CTAs of
// four warps an SM were the best of what registers allow (32768 tokens x 8
// heads, bf16: 39.6 us, six 42, eight 41, nine 48, ten 50; CTAs of eight warps
// 43 to 53).  Then integer work (70 % of its pipe): maxima of two 16-bit
// values at a time 35.8 us, a row's exponent made by one lane 35.0 us = 5.8
// TB/s.
template <typename T, int kSpan>
__global__ void __launch_bounds__(kWriteWarps * 32, sizeof(T) == 4 ? 5 : 7) write_kernel(const Q8WriteArgs a) {
  previous_done();
  next_may_begin();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t spans = (static_cast<int64_t>(a.T) + kSpan - 1) / kSpan;
  if (item >= spans * a.Hkv * 2) return;
  const bool values = item & 1;
  const int h = static_cast<int>((item >> 1) % a.Hkv);
  const int64_t t0 = (item >> 1) / a.Hkv * kSpan;
  write_item<T, kSpan>(a, t0, h, values, lane);
}

// Two codes times a power of two, as two values of the output's type.
__device__ __forceinline__ float2 values2(uint32_t codes, float s) {
  const uint32_t h = q8_unpack2(codes);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return make_float2(f.x * s, f.y * s);
}

// Four codes of a row and its scale -> four values at p.
template <typename T>
__device__ __forceinline__ void put4(T* p, uint32_t codes, float s) {
  const float2 a = values2(codes & 0xffffu, s), b = values2(codes >> 16, s);
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(finite(a.x), finite(a.y), finite(b.x), finite(b.y));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2_finite(p, a.x, a.y), pack2_finite(p, b.x, b.y));
  }
}

// Reading back: a warp per unit, whose 4128 bytes are asked for at once; a
// token's row of 128 values is then four values a lane (values are transposed
// in registers).  Bound by memory, mostly by what it writes.
template <typename T>
__global__ void __launch_bounds__(256) read_kernel(const Q8ReadArgs a, int blocks) {
  previous_done();
  next_may_begin();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.R) * blocks * a.Hkv) return;
  const int h = static_cast<int>(item % a.Hkv);
  const int b = static_cast<int>(item / a.Hkv % blocks);
  const int r = static_cast<int>(item / a.Hkv / blocks);
  const int len = max(a.len[r], 0);
  const int page = a.table[static_cast<int64_t>(r) * a.max_blocks + b];
  const int valid = min(len - b * kBlock, kBlock);
  if (b == 0 && h == 0 && lane == 0 && len > 0 && (len - 1) / kBlock >= blocks) raise_error(a.err, kErrBadBlock);
  if (valid <= 0) return;
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) raise_error(a.err, kErrBadBlock);
    return;
  }
  const uint8_t* unit = a.pages + (static_cast<int64_t>(page) * a.Hkv + h) * kQ8UnitBytes;
  T* out = static_cast<T*>(a.out) + ((static_cast<int64_t>(r) * a.Hkv + h) * a.out_blocks + b) * kUnitElems +
           lane * 4;
  uint32_t k[kBlock], v[kBlock];
#pragma unroll
  for (int j = 0; j < kBlock; ++j) k[j] = *reinterpret_cast<const uint32_t*>(unit + q8_key_at(j, lane * 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(unit + q8_value_at(0, lane * 4 + i));
    v[i] = w.x;
    v[4 + i] = w.y;
    v[8 + i] = w.z;
    v[12 + i] = w.w;
  }
  const float scale = pow2f(unit[kQ8ExpOffset + lane] - 127);  // lane: key, then value exponents
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    transpose4(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * q + i] = w[i];
  }
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    const float ks = __shfl_sync(0xffffffffu, scale, j), vs = __shfl_sync(0xffffffffu, scale, kBlock + j);
    if (j < valid) {
      put4(out + j * kHeadDim, k[j], ks);
      put4(out + (kBlock + j) * kHeadDim, v[j], vs);
    }
  }
}

}  // namespace

namespace {

constexpr int kLongSpan = 16;

template <typename T>
cudaError_t launch_write(const Q8WriteArgs& a, cudaStream_t s) {
  // A span of 16 tokens a warp, or of one where that leaves SMs without work (a
  // decode step's tokens, each in a page of its own).  GB300, 8 heads, bf16,
  // us with one and sixteen: 128 scattered tokens 2.9, 5.6, a run of them 3.4,
  // 2.4; 256 3.8, 6.1 and 4.4, 2.3; 600 6.5, 6.6 and 7.1, 2.9.
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv * 2;
  const bool one = rows < 152 * 32;
  const int64_t items = one ? rows : (static_cast<int64_t>(a.T) + kLongSpan - 1) / kLongSpan * a.Hkv * 2;
  const unsigned grid = static_cast<unsigned>((items + kWriteWarps - 1) / kWriteWarps);
  return launch_early(one ? write_kernel<T, 1> : write_kernel<T, kLongSpan>, grid, kWriteWarps * 32, 0, s, 0, a);
}

template <typename T>
cudaError_t launch_read(const Q8ReadArgs& a, cudaStream_t s) {
  const int blocks = a.max_blocks < a.out_blocks ? a.max_blocks : a.out_blocks;
  const int64_t items = static_cast<int64_t>(a.R) * blocks * a.Hkv;
  if (items == 0) return cudaSuccess;
  return launch_early(read_kernel<T>, static_cast<unsigned>((items + 7) / 8), 256, 0, s, 0, a, blocks);
}

template <typename T>
cudaError_t preload() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, write_kernel<T, 1>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, write_kernel<T, kLongSpan>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, read_kernel<T>);
  return e;
}

}  // namespace

cudaError_t launch_q8_write(const Q8WriteArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.type == kBf16) return launch_write<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_write<__half>(a, s);
  return launch_write<float>(a, s);
}

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  if (a.type == kBf16) return launch_read<__nv_bfloat16>(a, s);
  if (a.type == kFp16) return launch_read<__half>(a, s);
  return launch_read<float>(a, s);
}

cudaError_t preload_q8_cache_kernels() {
  cudaError_t e = preload<__nv_bfloat16>();
  if (e == cudaSuccess) e = preload<__half>();
  if (e == cudaSuccess) e = preload<float>();
  return e;
}

}  // namespace oasis
