// append.cu -- a step's queries, keys and values: queries and keys turned by
// their positions, keys and values rounded into the 8-bit pages; and moving
// an accepted path's tokens inside the pages.
#include "q8.cuh"
#include "q8.h"
#include "q8_rows.cuh"

namespace oasis {
namespace {

constexpr int kAppendWarps = 4;

// Four values as T at p (16-bit types to nearest even).
__device__ __forceinline__ void put(float* p, const float (&x)[4]) { store4(p, make_float4(x[0], x[1], x[2], x[3])); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[4]) {
  store4(p, make_float4(x[0], x[1], x[2], x[3]));
}
__device__ __forceinline__ void put(__half* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]));
}

// Rows of two tokens and some heads, queries or keys: half a warp a token.  A
// lane holds eight dims, four whole pairs, in two pieces of four: (i, i + half)
// pairs i = 4 c .. + 3 and their partners, neighbouring pairs dims 8 c .. + 7;
// dims past the turned ones go to the lanes that have no pairs.
//
// The angle.  A position times a frequency, in turns, is taken modulo one as
// 64-bit integers: a frequency is a multiple of 2^-64 turns, so the product is
// exact whatever the position.  (In fp32 a position of 10^6 would be off by 2^-4
// radians.)  cos and sin of a pair are made once for all of the token's heads
// that the warp has.
//
// Bound by memory for long runs (16384 tokens of a prompt, 32 / 8 heads, bf16: 66
// us, 5.6 TB/s; 65536 of 8 / 2, the same bytes but four times the angles, 79) and
// by a chain of latencies for a step's (position, angle, row, maximum: 16 tokens 4
// us, 128 in scattered slots 5, on the device).  Between, 4999 tokens of 28 / 4
// heads with three axes take 22.5 us, 1.7 times their bytes' time.
template <typename T>
__device__ __forceinline__ void turn_item(const AppendArgs& a, int64_t pair, int chunk, int lane) {
  const Q8WriteArgs& kv = a.kv;
  const int c = lane & 15;
  const int64_t t = 2 * pair + (lane >> 4);
  const bool there = t < kv.T;
  const int quarter = a.half / 4;
  const bool turns = c < quarter;
  const int o0 = a.interleaved ? 8 * c : turns ? 4 * c : 2 * a.half + 8 * (c - quarter);
  const int o1 = a.interleaved || !turns ? o0 + 4 : a.half + 4 * c;
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (there && turns) {
      const uint64_t phase =
          static_cast<uint64_t>(a.positions[a.axis[4 * c + i] * static_cast<int64_t>(kv.T) + t]) * a.turn[4 * c + i];
      // The nearest quarter turn, and what is left of the angle, an eighth of a
      // turn at most, in half turns: so fp32 holds it to 2^-28 of a turn.
      const uint32_t quarter_turn = (static_cast<uint32_t>(phase >> 32) + 0x20000000u) >> 30;
      const int32_t rest = static_cast<int32_t>(
          static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter_turn) << 62)) >> 30);
      float s, c;
      sincospif(static_cast<float>(rest) * 0x1p-33f, &s, &c);
      cs[i] = quarter_turn & 1 ? -s : c;
      sn[i] = quarter_turn & 1 ? c : s;
      if (quarter_turn & 2) {
        cs[i] = -cs[i];
        sn[i] = -sn[i];
      }
      cs[i] *= a.scale;
      sn[i] *= a.scale;
    }
  }
  const int64_t slot = there ? kv.slots[t] : -1;
  const bool fits = slot >= 0 && slot < kv.num_slots;
  const int heads = a.Hq + kv.Hkv;
  const int h0 = chunk * a.chunk, h1 = min(h0 + a.chunk, heads);
  if (h1 > a.Hq && slot >= kv.num_slots && c == 0) raise_error(kv.err, kErrBadUnit);
  const T* q = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* k = static_cast<const T*>(kv.k) + t * kv.k_stride;
  T* out = static_cast<T*>(a.out) + t * a.out_stride;
  const int j = static_cast<int>(slot & (kBlock - 1));
  constexpr int kBatch = 4;
  for (int h = h0; h < h1; h += kBatch) {
    Raw<T> lo[kBatch], hi[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      lo[b] = hi[b] = Raw<T>{};
      if (there && h + b < h1) {
        const T* row = h + b < a.Hq ? q + (h + b) * kHeadDim : k + (h + b - a.Hq) * kHeadDim;
        lo[b] = load4(row + o0);
        hi[b] = load4(row + o1);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (h + b >= h1) break;
      const float4 u = floats(lo[b]), v = floats(hi[b]);
      float x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
      if (turns) {
        auto turn = [&](float& p, float& r, int i) {
          const float p1 = p * cs[i] - r * sn[i];
          r = p * sn[i] + r * cs[i];
          p = p1;
        };
        if (a.interleaved) {
          turn(x[0], x[1], 0);
          turn(x[2], x[3], 1);
          turn(y[0], y[1], 2);
          turn(y[2], y[3], 3);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) turn(x[i], y[i], i);
        }
      }
      if (h + b < a.Hq) {
        if (there) {
          put(out + (h + b) * kHeadDim + o0, x);
          put(out + (h + b) * kHeadDim + o1, y);
        }
        continue;
      }
      // A key: its turned values are rounded once, to codes.
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(finite_abs_bits(x[i]), finite_abs_bits(y[i])));
#pragma unroll
      for (int off = 8; off; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      const int e = q8_exponent(top);
      const float s = pow2f(-e);
      if (fits) {
        uint8_t* unit = kv.pages + ((slot >> 4) * kv.Hkv + (h + b - a.Hq)) * static_cast<int64_t>(kQ8UnitBytes);
        *reinterpret_cast<uint32_t*>(unit + q8_key_at(j, o0)) = q8_pack4(x[0] * s, x[1] * s, x[2] * s, x[3] * s);
        *reinterpret_cast<uint32_t*>(unit + q8_key_at(j, o1)) = q8_pack4(y[0] * s, y[1] * s, y[2] * s, y[3] * s);
        if (c == 0) unit[kQ8ExpOffset + j] = static_cast<uint8_t>(e + 127);
      }
    }
  }
}

// The first CTAs turn queries and keys, the others write values.
template <typename T, int kSpan>
__global__ void __launch_bounds__(kAppendWarps * 32, sizeof(T) == 4 ? 5 : 7)
    append_kernel(const AppendArgs a, const __grid_constant__ unsigned turn_blocks) {
  previous_done();
  next_may_begin();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x < turn_blocks) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t pair = item / a.chunks;
    if (2 * pair < a.kv.T) turn_item<T>(a, pair, static_cast<int>(item - pair * a.chunks), lane);
  } else {
    const int64_t item = static_cast<int64_t>(blockIdx.x - turn_blocks) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t span = item / a.kv.Hkv;
    if (span * kSpan < a.kv.T)
      write_item<T, kSpan>(a.kv, span * kSpan, static_cast<int>(item - span * a.kv.Hkv), true, lane);
  }
}

template <typename T>
cudaError_t launch_t(AppendArgs a, cudaStream_t s) {
  // Heads a warp: so many that 16 warps an SM have work, but four at least, whose
  // rows are asked for together.  More share a token's angles, fewer give more
  // warps.  GB300, 32 / 8 heads, bf16, us with all heads, this, and four: 16
  // tokens 21.6, 9.4, 9.4; 1024 27.8, 20.6, 33.9; 8192 42, 42, 60; 32768 130, 130,
  // 204 (with a launch of some 5).  32 warps an SM: 1024 34.0, 8192 48.
  const int heads = a.Hq + a.kv.Hkv;
  const int64_t pairs = (static_cast<int64_t>(a.kv.T) + 1) / 2;
  int64_t chunk = pairs * heads / (152 * 16);
  chunk = chunk < 4 ? 4 : chunk > heads ? heads : chunk;
  a.chunk = static_cast<int>(chunk);
  a.chunks = (heads + a.chunk - 1) / a.chunk;
  const unsigned turn_blocks = static_cast<unsigned>((pairs * a.chunks + kAppendWarps - 1) / kAppendWarps);
  // As oasis_q8_write chooses: a token a warp while that fills the SMs (values alone
  // are written so here, yet the border is that call's, for keys and values).  GB300,
  // 32 / 8 heads, on the device, us with one token and sixteen: 128 tokens in whole
  // blocks 5.0, 4.6, in scattered slots 5.0, 9.2; 303 7.8, 5.8 and 7.8, 10.0; past the
  // border 607 10.0, 8.7 and 9.9, 26.6; 2432 24.4, 16.7 and 24.0, 44.7.
  const bool one = static_cast<int64_t>(a.kv.T) * a.kv.Hkv * 2 < 152 * 32;
  const int64_t spans = one ? a.kv.T : (static_cast<int64_t>(a.kv.T) + 15) / 16;
  const unsigned grid = turn_blocks + static_cast<unsigned>((spans * a.kv.Hkv + kAppendWarps - 1) / kAppendWarps);
  return launch_early(one ? append_kernel<T, 1> : append_kernel<T, 16>, grid, kAppendWarps * 32, 0, s, 0, a,
                      turn_blocks);
}

template <typename T>
cudaError_t preload() {
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, append_kernel<T, 1>);
  return e == cudaSuccess ? cudaFuncGetAttributes(&at, append_kernel<T, 16>) : e;
}

// ------------------------------------------------------------------ keeping
constexpr int kKeepThreads = 128;

// One request and KV head a CTA.  All tokens that move are read into shared
// memory before the first is written, so the places may overlap in any way.
// Bound by latency: two chains of dependent loads, then bytes 16 apart.
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a) {
  __shared__ uint32_t key[kTreeMaxNodes][32];     // four codes a lane
  __shared__ uint32_t value[kTreeMaxNodes][32];
  __shared__ uint8_t exps[kTreeMaxNodes][2];
  __shared__ uint8_t* from_s[kTreeMaxNodes];      // units; null: the token stays
  __shared__ uint8_t* to_s[kTreeMaxNodes];
  __shared__ int places[kTreeMaxNodes];           // tokens in their blocks: from, then 16 * to
  previous_done();
  next_may_begin();
  const int h = static_cast<int>(blockIdx.x % a.Hkv), r = static_cast<int>(blockIdx.x / a.Hkv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = a.len[r];
  const int nodes = a.size ? min(max(a.size[r], 0), a.N) : a.N;
  const int keep = min(max(a.keep[r], 0), min(a.M, nodes));
  const int64_t base = static_cast<int64_t>(len) - nodes;
  if (len <= 0 || keep == 0) return;
  if (base < 0 || len > a.max_blocks * kBlock) {
    if (tid == 0) raise_error(a.err, kErrBadBlock);
    return;
  }
  if (tid < keep) {
    const int node = a.nodes[static_cast<int64_t>(r) * a.M + tid];
    uint8_t *from = nullptr, *to = nullptr;
    const int64_t dst = base + tid;
    int64_t src = dst;
    if (node < 0 || node >= nodes) {
      raise_error(a.err, kErrBadUnit);
    } else if (node != tid) {
      src = base + node;
      const int32_t* row = a.table + static_cast<int64_t>(r) * a.max_blocks;
      const int p = row[src / kBlock], w = row[dst / kBlock];
      if (p < 0 || p >= a.num_pages || w < 0 || w >= a.num_pages) {
        raise_error(a.err, kErrBadBlock);
      } else {
        from = a.pages + (static_cast<int64_t>(p) * a.Hkv + h) * kQ8UnitBytes;
        to = a.pages + (static_cast<int64_t>(w) * a.Hkv + h) * kQ8UnitBytes;
      }
    }
    from_s[tid] = from;
    to_s[tid] = to;
    places[tid] = static_cast<int>(src % kBlock) + kBlock * static_cast<int>(dst % kBlock);
  }
  __syncthreads();
  for (int i = warp; i < keep; i += kKeepThreads / 32) {
    const uint8_t* unit = from_s[i];
    if (!unit) continue;
    const int j = places[i] % kBlock;
    key[i][lane] = *reinterpret_cast<const uint32_t*>(unit + q8_key_at(j, lane * 4));
    uint32_t v = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) v |= static_cast<uint32_t>(unit[q8_value_at(j, lane * 4 + d)]) << (8 * d);
    value[i][lane] = v;
    if (lane < 2) exps[i][lane] = unit[kQ8ExpOffset + lane * kBlock + j];
  }
  __syncthreads();
  for (int i = warp; i < keep; i += kKeepThreads / 32) {
    uint8_t* unit = to_s[i];
    if (!unit) continue;
    const int j = places[i] / kBlock;
    *reinterpret_cast<uint32_t*>(unit + q8_key_at(j, lane * 4)) = key[i][lane];
    const uint32_t v = value[i][lane];
#pragma unroll
    for (int d = 0; d < 4; ++d) unit[q8_value_at(j, lane * 4 + d)] = static_cast<uint8_t>(v >> (8 * d));
    if (lane < 2) unit[kQ8ExpOffset + lane * kBlock + j] = exps[i][lane];
  }
}

}  // namespace

cudaError_t launch_q8_append(const AppendArgs& a, cudaStream_t s) {
  if (a.kv.T == 0) return cudaSuccess;
  if (a.kv.type == kBf16) return launch_t<__nv_bfloat16>(a, s);
  if (a.kv.type == kFp16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}

cudaError_t launch_q8_keep(const KeepArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  return launch_early(keep_kernel, static_cast<unsigned>(a.R) * a.Hkv, kKeepThreads, 0, s, 0, a);
}

cudaError_t preload_append_kernels() {
  cudaError_t e = preload<__nv_bfloat16>();
  if (e == cudaSuccess) e = preload<__half>();
  if (e == cudaSuccess) e = preload<float>();
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, keep_kernel);
  return e;
}

}  // namespace oasis
