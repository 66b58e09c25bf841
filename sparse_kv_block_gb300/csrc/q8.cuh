// q8.cuh -- the 8-bit page format shared by the quantised-cache kernels.
//
// A unit is one KV head's block of 16 tokens, 4128 bytes:
//   [0, 2048)     key codes    [16 tokens][128 dims], the two 64-byte halves
//                 of an odd token's row exchanged
//   [2048, 4096)  value codes  [128 dims][16 tokens]
//   [4096, 4112)  key exponents, one byte a token
//   [4112, 4128)  value exponents
// A code c (e4m3) with exponent byte b stands for c * 2^(b - 127).
//
// Why this layout.  Attention reads a unit as mma.sync m16n8k16 fragments.
// Keys: a lane needs 16-byte pieces of a token's row, and two neighbouring
// tokens' pieces at once; the exchange puts those in different banks.
// Values: the contraction runs over tokens, so a lane needs consecutive
// tokens of one dim: they are stored that way, once, when written.  A unit's
// 4128 bytes are a multiple of 16 (one bulk copy) and 32 mod 128, so the
// same place of four units lies in four different bank groups.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace oasis {

constexpr int kQ8HalfBytes = kBlock * kHeadDim;                  // 2048
constexpr int kQ8ExpOffset = 2 * kQ8HalfBytes;                   // 4096
constexpr int kQ8UnitBytes = kQ8ExpOffset + 2 * kBlock;          // 4128
constexpr int kQ8MinExp = -100, kQ8MaxExp = 120;

// Byte of dim i of token j inside a unit.
__host__ __device__ __forceinline__ int q8_key_at(int j, int i) {
  return j * kHeadDim + (i ^ ((j & 1) << 6));
}
__host__ __device__ __forceinline__ int q8_value_at(int j, int i) {
  return kQ8HalfBytes + i * kBlock + j;
}

// The least e with amax <= 448 * 2^e, held in [lowest, kQ8MaxExp];
// `bits` are those of amax >= 0 (fp32).  448 = 1.75 * 2^8.
__device__ __forceinline__ int q8_exponent(uint32_t bits, int lowest = kQ8MinExp) {
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, lowest), kQ8MaxExp);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two floats -> two e4m3 codes (lo in the low byte), to nearest even; beyond
// 448 (an infinity) the largest code, NaN stays NaN.
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  return q8_pack2(a, b) | (q8_pack2(c, d) << 16);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two floats that codes stand for, or averages of them -> two of an output's
// type, to nearest even, NaN as NaN.  A row's largest value may have the code of
// the power of two past its type's range, 65536 or 2^128: that is given as the
// type's largest value.  (Nothing else reaches 2^128; in fp16 what is larger
// still, of a wider type, is an infinity as ever.)
__device__ __forceinline__ uint32_t pack2_finite(const __nv_bfloat16*, float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2_finite(const __half*, float lo, float hi) {
  auto held = [](float x) {  // 65536, and 2^-11 of it for the rounding of sums
    return fabsf(x) <= 65568.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
  };
  return pack_f16x2(held(lo), held(hi));
}
__device__ __forceinline__ float finite(float x) {
  return fabsf(x) == INFINITY ? copysignf(__uint_as_float(0x7f7fffffu), x) : x;
}

// Two e4m3 codes -> two halves (exact).
__device__ __forceinline__ uint32_t q8_unpack2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// 2^x, to two units in the last place (results under 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- launches that overlap (see launch_early)
// Wait until the launch ahead in the stream has ended and its writes are seen.
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The launch behind may begin (when all CTAs have said so).
__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;"); }

// ---- parts of a softmax, each (outputs, sum) in units of 2^m
// 2^(m - mx); where no part has seen a score (mx = -inf) the parts are zeros,
// or NaN, and are added as they are.
__device__ __forceinline__ float scale_of(float m, float mx) {
  return mx == -INFINITY ? 1.f : ex2(m - mx);
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }
// The sums (m, l) and (m2, l2), each in units of 2^m, as one.
__device__ __forceinline__ void join_sum(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  l = l * scale_of(m, mx) + l2 * scale_of(m2, mx);
  m = mx;
}
__device__ __forceinline__ void scale4(float4& a, float f) {
  a.x *= f;
  a.y *= f;
  a.z *= f;
  a.w *= f;
}
__device__ __forceinline__ void add4(float4& a, float f, const float4& x) {
  a.x = fmaf(f, x.x, a.x);
  a.y = fmaf(f, x.y, a.y);
  a.z = fmaf(f, x.z, a.z);
  a.w = fmaf(f, x.w, a.w);
}
// A warp joins a row's shares, `stride` rows apart: each lane a share's maximum
// and sum, then four dims of every share.  (Loads past L1: the launches that
// write them may have run beside this one's beginning.)
__device__ __forceinline__ float4 join_shares(const float4* part, const float2* stat, int64_t stride, int shares,
                                              int lane, float& sum) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY;
  sum = 0.f;
  for (int i0 = 0; i0 < shares; i0 += 32) {
    const int some = min(shares - i0, 32);
    constexpr int kBatch = 8;
    const float2 st = lane < some ? __ldcg(stat + (i0 + lane) * stride) : make_float2(-INFINITY, 0.f);
    const float4* from = part + i0 * stride * 32 + lane;
    float4 x[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) x[b] = __ldcg(from + min(b, some - 1) * stride * 32);
    float top = st.x;
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    top = fmaxf(top, m);
    const float old = scale_of(m, top), w = scale_of(st.x, top);
    float l = w * st.y;
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    sum = fmaf(sum, old, l);
    scale4(acc, old);
    m = top;
    for (int i = 0; i < some; i += kBatch) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float f = __shfl_sync(0xffffffffu, w, (i + b) & 31);
        if (i + b < some) add4(acc, f, x[b]);
      }
      if (i + kBatch < some)
#pragma unroll
        for (int b = 0; b < kBatch; ++b) x[b] = __ldcg(from + min(i + kBatch + b, some - 1) * stride * 32);
    }
  }
  return acc;
}
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
// An output over codes.
__device__ __forceinline__ void store4_finite(float* p, const float4& v) {
  store4(p, make_float4(finite(v.x), finite(v.y), finite(v.z), finite(v.w)));
}
template <typename T>
__device__ __forceinline__ void store4_finite(T* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2_finite(p, v.x, v.y), pack2_finite(p, v.z, v.w));
}

}  // namespace oasis
