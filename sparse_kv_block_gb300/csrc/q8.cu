// q8.cu -- writing keys and values into the 8-bit paged cache, and reading
// them back.
#include <type_traits>

#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

// Four consecutive elements, as they lie and as floats.  (The loads are
// volatile so that a row of them is issued before the first is used.)
template <typename T>
struct Raw {
  uint2 w;
};
template <>
struct Raw<float> {
  uint4 w;
};
template <typename T>
__device__ __forceinline__ Raw<T> load4(const T* p) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4)
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w.x), "=r"(r.w.y), "=r"(r.w.z), "=r"(r.w.w)
                 : "l"(p));
  else
    asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(r.w.x), "=r"(r.w.y) : "l"(p));
  return r;
}
__device__ __forceinline__ float4 floats(const Raw<float>& r) {
  return make_float4(__uint_as_float(r.w.x), __uint_as_float(r.w.y), __uint_as_float(r.w.z),
                     __uint_as_float(r.w.w));
}
__device__ __forceinline__ float4 floats(const Raw<__nv_bfloat16>& r) {
  return make_float4(bf16lo(r.w.x), bf16hi(r.w.x), bf16lo(r.w.y), bf16hi(r.w.y));
}
__device__ __forceinline__ float4 floats(const Raw<__half>& r) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r.w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// The warp's largest |x| of a row, as its type's bits without the sign
// (16-bit types two at a time).
template <typename T>
__device__ __forceinline__ uint32_t row_max(const Raw<T>& r) {
  uint32_t m;
  if constexpr (sizeof(T) == 4) {
    m = max(max(r.w.x & 0x7fffffffu, r.w.y & 0x7fffffffu), max(r.w.z & 0x7fffffffu, r.w.w & 0x7fffffffu));
  } else {
    const uint32_t two = __vmaxu2(r.w.x & 0x7fff7fffu, r.w.y & 0x7fff7fffu);
    m = max(two >> 16, two & 0xffffu);
  }
  return __reduce_max_sync(0xffffffffu, m);
}
// Such a maximum's fp32 bits; an infinity or NaN gives 0x7f800000 or more.
template <typename T>
__device__ __forceinline__ uint32_t float_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  if constexpr (std::is_same_v<T, __half>)
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
  return m << 16;
}
// The fp32 bits of the largest |x| of finite x: infinities and NaN do not set
// a row's scale.
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t finite_row_max(float4 x) {
  return __reduce_max_sync(0xffffffffu, max(max(finite_abs_bits(x.x), finite_abs_bits(x.y)),
                                            max(finite_abs_bits(x.z), finite_abs_bits(x.w))));
}
__device__ __forceinline__ uint32_t codes_of(float4 x, float s) {
  return q8_pack4(x.x * s, x.y * s, x.z * s, x.w * s);
}

// Four words of four bytes, transposed: byte i of word j to byte j of word i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
  const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, c, 0x5410);
  w[1] = __byte_perm(a, c, 0x7632);
  w[2] = __byte_perm(b, d, 0x5410);
  w[3] = __byte_perm(b, d, 0x7632);
}

// 32 bytes of a unit, 16-byte aligned: a whole sector in one store where they
// are one, which the instruction requires (a unit's 4128 bytes are a multiple
// of 32, so that is so for all of a pool's units or for none), else two.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

constexpr int kWriteWarps = 4;

// Rounding into the pages.  Bound by memory: 256 values are read and 258
// bytes written a token and head.  What holds it back is latency (the slots,
// then the rows): 16 rows a warp are asked for at once, and seven CTAs of
// four warps an SM were the best of what registers allow (32768 tokens x 8
// heads, bf16: 39.6 us, six 42, eight 41, nine 48, ten 50; CTAs of eight warps
// 43 to 53).  Then integer work (70 % of its pipe): maxima of two 16-bit
// values at a time 35.8 us, a row's exponent made by one lane 35.0 us = 5.8
// TB/s.
//
// Values are stored with a block's tokens consecutive, so single tokens mean
// single bytes 16 apart; whole blocks (16 consecutive slots from a block's
// first, wherever in the call they begin) are worth finding.  A warp takes 16
// consecutive tokens, one head and keys or values; it treats the whole blocks
// that begin among them, reading on past its tokens where they do, transposed
// in registers and stored in whole sectors; then, all together, those of its
// tokens that no whole block has.  With kSpan = 1 a warp takes one token.

// The codes of 16 rows, `have` a bit for each that is there; lane i makes row
// i's exponent, which it returns, and scale (the whole warp doing each row's
// would double the integer work, which is what fills the SM).
template <typename T, int kRows>
__device__ __forceinline__ int quantise_rows(const T* const (&x)[kRows], unsigned have, int lane,
                                             uint32_t (&codes)[kRows]) {
  Raw<T> v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    v[i] = have >> i & 1 ? load4(x[i]) : Raw<T>{};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t m = row_max(v[i]);
    if (lane == i) top = m;
  }
  top = float_bits<T>(top);
  if (__any_sync(0xffffffffu, top >= 0x7f800000u)) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t m = finite_row_max(floats(v[i]));
      if (lane == i) top = m;
    }
  }
  const int e = q8_exponent(top);
  const float scale = pow2f(-e);
#pragma unroll
  for (int i = 0; i < kRows; ++i) codes[i] = codes_of(floats(v[i]), __shfl_sync(0xffffffffu, scale, i));
  return e;
}

// Bit i of the result: bits i .. i + 14 of x are set.
__device__ __forceinline__ uint64_t fifteen(uint64_t x) {
  x &= x >> 1;
  x &= x >> 2;
  x &= x >> 4;
  return x & x >> 7;
}

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
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const T* src = static_cast<const T*>(values ? a.v : a.k) + h * kHeadDim + lane * 4 + t0 * stride;
  const int exps = kQ8ExpOffset + (values ? kBlock : 0);
  auto slot_of = [&](int64_t t) { return t >= 0 && t < a.T ? a.slots[t] : -1; };
  auto unit_of = [&](int64_t slot) {
    return a.pages + ((slot >> 4) * a.Hkv + h) * static_cast<int64_t>(kQ8UnitBytes);
  };
  uint32_t codes[kSpan];
  const T* x[kSpan];
  // Lane i: the slot of token t0 + i of the span.
  int64_t slot;
  uint64_t whole = 0, mine = 1;  // whole blocks' first tokens; tokens of none (bit i: token t0 + i)
  uint64_t follows = 0;          // tokens in the slot behind the token before
  if constexpr (kSpan == 1) {
    slot = slot_of(t0);
  } else {
    // Tokens t0 - 16 .. t0 + 31, bits 0 .. 47: which stand in the slot behind
    // the token before, and which in a block's first.
    const int64_t s0 = slot_of(t0 - 16 + lane), s1 = lane < 16 ? slot_of(t0 + 16 + lane) : -1;
    int64_t p0 = __shfl_up_sync(0xffffffffu, s0, 1), p1 = __shfl_up_sync(0xffffffffu, s1, 1);
    const int64_t last = __shfl_sync(0xffffffffu, s0, 31);
    if (lane == 0) {
      p0 = -1;  // of no consequence: no block that reaches the span began before
      p1 = last;
    }
    auto bits = [](bool b0, bool b1) {
      return static_cast<uint64_t>(__ballot_sync(0xffffffffu, b0)) |
             static_cast<uint64_t>(__ballot_sync(0xffffffffu, b1)) << 32;
    };
    const uint64_t next = bits(p0 >= 0 && s0 == p0 + 1, p1 >= 0 && s1 == p1 + 1);
    const uint64_t begins = bits(s0 >= 0 && (s0 & (kBlock - 1)) == 0, s1 >= 0 && (s1 & (kBlock - 1)) == 0);
    const uint64_t there = bits(s0 >= 0, s1 >= 0);
    const uint64_t first = begins & fifteen(next >> 1);
    uint64_t member = first | first << 1;
    member |= member << 2;
    member |= member << 4;
    member |= member << 8;
    whole = first >> 16 & 0xffffu;
    mine = (there & ~member) >> 16 & 0xffffu;
    follows = next >> 16;
    slot = __shfl_sync(0xffffffffu, s0, (lane + 16) & 31);  // of the span's tokens, lanes 0 .. 15
  }

  if constexpr (kSpan > 1) {
    for (; whole; whole &= whole - 1) {
      const int at = __ffsll(static_cast<long long>(whole)) - 1;
      const int64_t begin = __shfl_sync(0xffffffffu, slot, at);
      if (begin >= a.num_slots) {
        if (lane == 0) raise_error(a.err, kErrBadUnit);
        continue;
      }
#pragma unroll
      for (int i = 0; i < kSpan; ++i) x[i] = src + (at + i) * stride;
      const int e = quantise_rows(x, 0xffffu, lane, codes);
      uint8_t* unit = unit_of(begin);
      if (values) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4] = {codes[4 * q], codes[4 * q + 1], codes[4 * q + 2], codes[4 * q + 3]};
          transpose4(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) codes[4 * q + i] = w[i];
        }
        // codes[4 q + i]: tokens 4 q .. + 3 of dim 4 lane + i
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const uint32_t two[8] = {codes[i], codes[4 + i], codes[8 + i], codes[12 + i],
                                   codes[i + 1], codes[5 + i], codes[9 + i], codes[13 + i]};
          store32(unit + q8_value_at(0, lane * 4 + i), two);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSpan; ++i)
          *reinterpret_cast<uint32_t*>(unit + q8_key_at(i, lane * 4)) = codes[i];
      }
      if (lane < kBlock) unit[exps + lane] = static_cast<uint8_t>(e + 127);
    }
  }

  // The other tokens.  Values: four of them in four slots that make a word go
  // as words, the rest as bytes 16 apart (each a sector of its own, which is
  // what such writes cost: 16384 scattered tokens 145 us, runs of 13 as bytes
  // 111).
  const bool in = lane < kSpan && (mine >> lane & 1) && slot >= 0;
  if (in && slot >= a.num_slots) raise_error(a.err, kErrBadUnit);
  const unsigned have = __ballot_sync(0xffffffffu, in && slot < a.num_slots);
  if (have == 0) return;
#pragma unroll
  for (int i = 0; i < kSpan; ++i) x[i] = src + i * stride;
  const int e = quantise_rows(x, have, lane, codes);
  const unsigned on = have & static_cast<unsigned>(follows);
  const unsigned quads = __ballot_sync(0xffffffffu, (slot & 3) == 0) & have & on >> 1 & on >> 2 & on >> 3;
  unsigned bytes = have & ~(quads | quads << 1 | quads << 2 | quads << 3);
#pragma unroll
  for (int i = 0; i < kSpan; ++i) {
    if (!(have >> i & 1)) continue;
    const int64_t to = __shfl_sync(0xffffffffu, slot, i);
    const int j = static_cast<int>(to & (kBlock - 1));
    uint8_t* unit = unit_of(to);
    if (!values) {
      *reinterpret_cast<uint32_t*>(unit + q8_key_at(j, lane * 4)) = codes[i];
    } else if (bytes >> i & 1) {
#pragma unroll
      for (int d = 0; d < 4; ++d) unit[q8_value_at(j, lane * 4 + d)] = static_cast<uint8_t>(codes[i] >> (8 * d));
    } else if constexpr (kSpan > 3) {
      if (i + 3 < kSpan && (quads >> i & 1)) {
        uint32_t w[4] = {codes[i], codes[(i + 1) % kSpan], codes[(i + 2) % kSpan], codes[(i + 3) % kSpan]};
        transpose4(w);
#pragma unroll
        for (int d = 0; d < 4; ++d) *reinterpret_cast<uint32_t*>(unit + q8_value_at(j, lane * 4 + d)) = w[d];
      }
    }
  }
  if (have >> lane & 1) unit_of(slot)[exps + (slot & (kBlock - 1))] = static_cast<uint8_t>(e + 127);
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
