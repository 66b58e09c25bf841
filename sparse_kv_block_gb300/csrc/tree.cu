// tree.cu -- attention of a request's tree of drafted tokens over its 8-bit
// pages.
//
// The nodes' queries that read one KV head (row node * G + gi) are the rows of
// a matrix, at most 256 of them a CTA, so its pages are read once: 4 * 128
// operations a row and token against 258 bytes a token, bound by HBM up to
// some 140 rows, by the tensor cores (tcgen05) beyond.
//
// Both operands are used as they lie in the pages, as far as they can be:
// * Keys go in as e4m3 (kind::f8f6f4).  A query row is a sum of e4m3 rows times
//   one power of two: two of them hold bf16's eight bits, three fp16's eleven
//   (exact for entries down to 2^-10 and 2^-7 of the row's largest; below, off
//   by at most 2^-19 of it).  A tile of 128 tokens is eight units, whose even
//   and odd tokens are two operands of 64 tokens: the odd ones have their
//   halves exchanged, which costs nothing but another order of the steps.
// * Values have a unit's 16 tokens consecutive, which is an operand's layout
//   without a swizzle for 16 rows of 8-bit weights.  Weights of 8 bits would be
//   too coarse, so four warps turn the values into fp16, in units of the
//   largest value exponent so far, and the weights are fp16 (tensor memory).
//
// One CTA an SM.  The tiles of all (request, KV head, 256 rows) are one
// sequence, which the CTAs share out evenly, whatever the lengths: a CTA's range
// is made of segments, each a run of tiles of one pair.  A pair wholly inside
// one CTA's range is written straight out, others as shares (average, maximum,
// sum) that a second launch joins.
//
// Roles: warps 0..7 softmax, one thread a row, two streams of four warps; 8..11
// values to fp16; 12 loads (TMA with the 128-byte swizzle for keys, bulk copies
// for values and exponents); 13 issues the products.  The two streams have
// scores and outputs of their own in tensor memory (2 x (128 + 128) columns), so
// that the products of one run while the other's weights are formed: with more
// than 128 rows they are two row tiles over the same tokens, else they take
// turns at the same rows' tiles and are joined at the end.
#include <cuda_fp16.h>

#include <type_traits>

#include "q8.cuh"
#include "q8.h"
#include "tcgen05.cuh"

namespace oasis {
namespace {

constexpr int kTile = 128;                              // rows, tokens
constexpr int kUnits = kTile / kBlock;                  // of a tile
constexpr int kRest = kQ8UnitBytes - kQ8HalfBytes;      // values and exponents of a unit
constexpr int kKeyStage = kUnits * kQ8HalfBytes;        // 16 KiB
constexpr int kValueStage = kUnits * kRest;
constexpr int kHalfStage = kTile * kHeadDim * 2;        // values in fp16: 32 KiB
constexpr int kTerm = kTile * kHeadDim;                 // one e4m3 row tile of queries: 16 KiB
constexpr int kTreeThreads = 14 * 32;
constexpr int kSoftmaxThreads = 256, kConvertThreads = 128;
constexpr float kLazy = 8.f;                            // growth of a maximum let pass (log2)
constexpr float kWeight = 7.f;                          // a weight is 2^(x - m + 7), at most 2^15
constexpr int kValueUp = 6;                             // a value is code * 2^(e - U + 6), at most 448 * 64

template <int kTerms, int kTiles>
struct TreeLayout {
  static constexpr int kK = 3, kV = kTiles == 1 ? 3 : 2, kC = 2;  // stages
  static constexpr int kQ = 0;
  static constexpr int kKeys = kQ + kTiles * kTerms * kTerm;
  static constexpr int kHalves = kKeys + kK * kKeyStage;
  static constexpr int kValues = kHalves + kC * kHalfStage;
  static constexpr int kScale = kValues + kV * kValueStage;     // [kC][128] of a token's key, in score columns
  static constexpr int kInfo = kScale + kC * kTile * 4;         // [kC] int4: first token, whole, U, -
  static constexpr int kNan = kInfo + kC * 16;                  // [kC + 1][128] words, then [kC + 1] int4 flags
  static constexpr int kNanFlag = kNan + (kC + 1) * kHeadDim * 8;
  static constexpr int kFactor = kNanFlag + (kC + 1) * 16;      // [kTiles][128] of a row's scores
  static constexpr int kStat = kFactor + kTiles * kTile * 4;    // [2][128] float4: m, sum, U of a stream's rows
  static constexpr int kHalfScale = kStat + 2 * kTile * 16;     // [2][128] half: of a token's value
  static constexpr int kValid = kHalfScale + 2 * kTile * 2;     // [kV][8] tokens of a unit
  static constexpr int kConvert = kValid + kV * kUnits * 4;     // [4] int2 of the converting warps
  static constexpr int kScan = kConvert + 32;                   // [16] int64, then [4] results
  static constexpr int kBars = kScan + 20 * 8;
  static constexpr int kBytes = kBars + 256 + 1024;             // + alignment
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kHalves % 128 == 0 && kValues % 128 == 0 && kScale % 16 == 0 && kBars % 8 == 0, "alignment");
};

constexpr uint32_t kScoreInstr = kMmaF32 | mma_shape(128, 64);
constexpr uint32_t kOutInstr = kMmaF32 | mma_shape(128, 128);

__device__ __forceinline__ void load_keys(void* dst, const CUtensorMap* map, int head, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
template <int kId, int kThreads>
__device__ __forceinline__ void named_barrier() {
  asm volatile("barrier.cta.sync %0, %1;" ::"n"(kId), "n"(kThreads) : "memory");
}
// The same; true where all say so.  (Threads whose waits ran out meet the
// others here, so that none is left waiting.)
template <int kId, int kThreads>
__device__ __forceinline__ bool all_of(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "n"(kId), "n"(kThreads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return r != 0;
}
// 2^e as fp16 bits, -24 <= e <= 15 (0 below).
__device__ __forceinline__ uint16_t pow2h(int e) {
  return static_cast<uint16_t>(e >= -14 ? (e + 15) << 10 : e >= -24 ? 1 << (e + 24) : 0);
}
// A power of two from its exponent, held to the normal range.
__device__ __forceinline__ float pow2_held(int e) { return pow2f(max(e, -126)); }

// A request's tokens, nodes, blocks of rows a KV head, and tiles of 128 tokens
// (none where there is nothing to do).
struct Request {
  int len, nodes, blocks, tiles;
};
template <int kRows>
__device__ __forceinline__ Request request(const TreeArgs& a, int r) {
  Request q;
  q.nodes = a.size ? min(max(__ldg(a.size + r), 0), a.N) : a.N;
  q.len = min(max(__ldg(a.len + r), 0), a.max_blocks * kBlock);
  q.blocks = (q.nodes * a.G + kRows - 1) / kRows;
  q.tiles = q.nodes > 0 && q.len >= q.nodes ? (q.len + kTile - 1) / kTile : 0;
  return q;
}

// The segments of a CTA's range, in order: runs of tiles [i0, i0 + n) of block
// `block` of rows of KV head h of request r.
template <int kRows>
struct Walk {
  int r, pair, i0;     // pair: h * blocks + block
  int64_t left;        // tiles
  Request q;
  int h, block, first, n;
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    if (left == 0) return false;
    if (pair == a.Hkv * q.blocks) {
      pair = 0;
      do q = request<kRows>(a, ++r);
      while (q.tiles == 0);
    }
    h = pair / q.blocks;
    block = pair - h * q.blocks;
    first = i0;
    n = static_cast<int>(min(static_cast<int64_t>(q.tiles - i0), left));
    left -= n;
    ++pair;
    i0 = 0;
    return true;
  }
  __device__ __forceinline__ int rows(const TreeArgs& a) const {
    return min(q.nodes * a.G - block * kRows, kRows);
  }
  __device__ __forceinline__ bool whole() const { return first == 0 && n == q.tiles; }
};

template <typename T, int kTiles>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap map) {
  constexpr int kTerms = std::is_same_v<T, __half> ? 3 : 2;
  using Lay = TreeLayout<kTerms, kTiles>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* key_full = reinterpret_cast<uint64_t*>(smem + Lay::kBars);  // [kK] keys have landed
  uint64_t* key_empty = key_full + Lay::kK;                             // [kK] their products are done
  uint64_t* value_full = key_empty + Lay::kK;                           // [kV]
  uint64_t* value_empty = value_full + Lay::kV;                         // [kV] (four warps)
  uint64_t* half_full = value_empty + Lay::kV;                          // [kC] values are fp16 (four warps)
  uint64_t* half_empty = half_full + Lay::kC;                           // [kC]
  uint64_t* s_full = half_empty + Lay::kC;                              // [2] scores of a stream
  uint64_t* p_full = s_full + 2;                                        // [2] its weights (four warps)
  uint64_t* o_done = p_full + 2;                                        // [2] its outputs
  uint64_t* q_ready = o_done + 2;                                       // a segment's queries (eight warps)
  uint64_t* drain = q_ready + 1;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + Lay::kScan);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kTreeThreads / 32;
  previous_done();
  // (Not before: a kernel ahead that takes tensor memory after it has let its
  // dependents begin would wait for this one's.)
  if (warp == 13) tmem_alloc(tmem_s, 512);
  next_may_begin();
  if (tid == 12 * 32) {
    prefetch_tensormap(&map);
    for (int i = 0; i < 2 * Lay::kK; ++i) mbar_init(key_full + i, 1);
    for (int i = 0; i < Lay::kV; ++i) {
      mbar_init(value_full + i, 1);
      mbar_init(value_empty + i, 4);
    }
    for (int i = 0; i < Lay::kC; ++i) {
      mbar_init(half_full + i, 4);
      mbar_init(half_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(drain, 1);
    fence_barrier_init();
  }

  // Requests without a tile: their nodes give zeros, and bad lengths are
  // reported, each by one CTA.
  constexpr int kRows = kTiles * kTile;
  if (tid == 0) a.info[blockIdx.x] = make_int4(-1, 0, 0, 0);
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const Request q = request<kRows>(a, r);
    const int len = a.len[r];
    if (tid == 0 && (len > a.max_blocks * kBlock || (len > 0 && len < q.nodes))) raise_error(a.err, kErrBadBlock);
    if (q.tiles == 0 && q.nodes > 0) {
      const int64_t bytes = static_cast<int64_t>(a.Hq) * kHeadDim * (a.out_fp32 ? 4 : 2);
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(r) * a.N * bytes);
      for (int64_t i = tid; i < q.nodes * bytes / 16; i += kTreeThreads) out[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // This CTA's range of the sequence.
  auto tiles_of = [&](int r) {
    const Request q = request<kRows>(a, r);
    return static_cast<int64_t>(q.tiles) * q.blocks * a.Hkv;
  };
  int64_t total = 0;
  for (int r = tid; r < a.R; r += kTreeThreads) total += tiles_of(r);
#pragma unroll
  for (int off = 16; off; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (lane == 0) scan[warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kWarps; ++w) total += scan[w];
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  const int c = blockIdx.x;
  const int64_t u0 = c < ctas ? total * c / ctas : 0, u1 = c < ctas ? total * (c + 1) / ctas : 0;
  int64_t* found = scan + 16;
  int64_t before = 0;  // tiles of the requests before the ones looked at
  for (int r0 = 0; u0 < u1; r0 += kTreeThreads) {
    const int r = r0 + tid;
    const int64_t t = r < a.R ? tiles_of(r) : 0;
    int64_t incl = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) incl += all;
      all += scan[w];
    }
    incl += before;
    if (incl - t <= u0 && u0 < incl) {
      const int tiles = request<kRows>(a, r).tiles;
      found[0] = r;
      found[1] = (u0 - (incl - t)) / tiles;
      found[2] = (u0 - (incl - t)) % tiles;
    }
    before += all;
    if (before > u0) break;  // every thread alike
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_s, 0);
  Walk<kRows> walk;
  walk.left = u1 - u0;
  if (walk.left > 0) {
    walk.r = static_cast<int>(found[0]);
    walk.pair = static_cast<int>(found[1]);
    walk.i0 = static_cast<int>(found[2]);
    walk.q = request<kRows>(a, walk.r);
  }
  auto reached = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_limit)) != 0;
  };

  bool ok = true;
  if (warp == 12) {
    // ---- loads: a lane a unit
    int gk = 0, gv = 0;  // tiles whose keys, whose values are on their way
    while (ok && walk.next(a)) {
      const int32_t* row = a.table + static_cast<int64_t>(walk.r) * a.max_blocks;
      auto page_of = [&](int i) {
        const int b = (walk.first + i) * kUnits + lane;
        return lane < kUnits && i < walk.n && b * kBlock < walk.q.len ? __ldg(row + b) : -1;
      };
      int page = page_of(0);
      for (int i = 0; i < walk.n && ok; ++i) {
        const int left = walk.q.len - ((walk.first + i) * kUnits + lane) * kBlock;
        const bool inside = lane < kUnits && left > 0;
        const bool there = inside && page >= 0 && page < a.num_pages;
        if (inside && !there) raise_error(a.err, kErrBadBlock);
        const int at = page;
        page = page_of(i + 1);
        const int units = __popc(__ballot_sync(0xffffffffu, there));
        const int ks = gk % Lay::kK, vs = gv % Lay::kV;
        ok = gk < Lay::kK || reached(key_empty + ks, (gk / Lay::kK - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(key_full + ks, units * kQ8HalfBytes);
        __syncwarp();
        if (there)
          load_keys(smem + Lay::kKeys + ks * kKeyStage + lane * kQ8HalfBytes, &map, walk.h, at, key_full + ks);
        ++gk;
        ok = gv < Lay::kV || reached(value_empty + vs, (gv / Lay::kV - 1) & 1);
        if (!ok) break;
        if (lane < kUnits)
          reinterpret_cast<int*>(smem + Lay::kValid)[vs * kUnits + lane] = there ? min(left, kBlock) : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(value_full + vs, units * kRest);
        __syncwarp();
        if (there)
          bulk_g2s(smem + Lay::kValues + vs * kValueStage + lane * kRest,
                   a.pages + (static_cast<int64_t>(at) * a.Hkv + walk.h) * kQ8UnitBytes + kQ8HalfBytes, kRest,
                   value_full + vs);
        ++gv;
      }
    }
    // No copy may outlive the CTA, whatever the other warps met.
    for (int j = max(gk - Lay::kK, 0); j < gk; ++j) (void)mbar_wait(key_full + j % Lay::kK, (j / Lay::kK) & 1);
    for (int j = max(gv - Lay::kV, 0); j < gv; ++j) (void)mbar_wait(value_full + j % Lay::kV, (j / Lay::kV) & 1);
  } else if (warp == 13) {
    // ---- products
    const uint32_t lead = elected();
    const uint64_t q_desc = smem_desc(smem_u32(smem + Lay::kQ), 16);
    const uint64_t k_desc = smem_desc(smem_u32(smem + Lay::kKeys), 16, 2048);
    const uint64_t v_desc = smem_desc_plain(smem_u32(smem + Lay::kHalves), 2048, 128);
    int g0 = 0, weights = 0;  // tiles before the segment; bit t: the parity of stream t's weights
    for (int segments = 0; ok && walk.next(a); ++segments, g0 += walk.n) {
      const bool two = kTiles == 2 && walk.rows(a) > kTile;
      const int jobs = two ? 2 * walk.n : walk.n;  // a stream's tile each, the streams in turn
      ok = reached(q_ready, segments & 1);
      auto scores = [&](int k) {
        const int t = k & 1, g = g0 + (two ? k >> 1 : k), st = g % Lay::kK;
        if ((!two || t == 0) && !reached(key_full + st, (g / Lay::kK) & 1)) return false;
        fence_after();
        const uint64_t q = q_desc + (two ? t * kTerms * (kTerm >> 4) : 0), kd = k_desc + st * (kKeyStage >> 4);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
#pragma unroll
          for (int term = 0; term < kTerms; ++term)
#pragma unroll
            for (int s = 0; s < 4; ++s)  // 32 dims a step
              mma_ss_8bit<kScoreInstr>(tmem + t * 128 + odd * 64, q + term * (kTerm >> 4) + s * 2,
                                       kd + odd * (1024 >> 4) + (odd ? s ^ 2 : s) * 2, term > 0 || s > 0, lead);
        mma_commit(s_full + t, lead);
        if (!two || t == 1) mma_commit(key_empty + st, lead);
        return true;
      };
      ok = ok && scores(0) && (jobs < 2 || scores(1));
      for (int k = 0; k < jobs && ok; ++k) {
        const int t = k & 1, i = k >> 1, g = g0 + (two ? k >> 1 : k), st = g % Lay::kC;
        ok = ((two && t == 1) || reached(half_full + st, (g / Lay::kC) & 1)) &&
             reached(p_full + t, weights >> t & 1);
        weights ^= 1 << t;
        if (!ok) break;
        fence_after();
        const uint64_t v = v_desc + st * (kHalfStage >> 4);
#pragma unroll
        for (int s = 0; s < 8; ++s)  // a unit's 16 tokens a step
          mma_ts<kOutInstr>(tmem + 256 + t * 128, tmem + t * 128 + s * 8, v + s * (4096 >> 4), i > 0 || s > 0, lead);
        if (!two || t == 1) mma_commit(half_empty + st, lead);
        if (k + 2 < jobs) ok = scores(k + 2);
        else mma_commit(o_done + t, lead);
      }
    }
    // No product may outlive its operands and accumulators, either.
    mma_commit(drain, lead);
    (void)mbar_wait(drain, 0);
  } else if (warp >= 8) {
    // ---- values to fp16: a thread a dim
    const int d = tid - kSoftmaxThreads, unit = d >> 4, j = d & 15;
    const int* valid_s = reinterpret_cast<const int*>(smem + Lay::kValid);
    int2* seen = reinterpret_cast<int2*>(smem + Lay::kConvert);
    uint16_t* half_scale = reinterpret_cast<uint16_t*>(smem + Lay::kHalfScale);
    int g = 0;
    while (ok && walk.next(a)) {
      const int base = walk.q.len - walk.q.nodes;
      int U = 0;         // the largest exponent byte so far
      uint64_t nan = 0;  // nodes whose value of dim d is NaN
      for (int i = 0; i < walk.n; ++i, ++g) {
        const int vs = g % Lay::kV, st = g % Lay::kC, t0 = (walk.first + i) * kTile;
        ok = reached(value_full + vs, (g / Lay::kV) & 1) &&
             (g < Lay::kC || reached(half_empty + st, (g / Lay::kC - 1) & 1));
        const uint8_t* raw = smem + Lay::kValues + vs * kValueStage;
        // First a thread a token.
        const bool valid = ok && j < valid_s[vs * kUnits + unit];
        const int ke = valid ? raw[unit * kRest + kQ8HalfBytes + j] : 0;
        const int ve = valid ? raw[unit * kRest + kQ8HalfBytes + kBlock + j] : 0;
        const int top = __reduce_max_sync(0xffffffffu, ve);
        const int low = __reduce_min_sync(0xffffffffu, valid ? ve : 255);
        const bool every = __all_sync(0xffffffffu, valid);
        if (lane == 0) seen[warp - 8] = make_int2(every ? top : top - 1024, low);
        ok = all_of<2, kConvertThreads>(ok);
        if (!ok) break;
        bool all_valid = true;
        int least = 255;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int2 s = seen[w];
          all_valid = all_valid && s.x >= 0;
          U = max(U, s.x >= 0 ? s.x : s.x + 1024);
          least = min(least, s.y);
        }
        // 2^(e - U + 6), as two factors where fp16 does not hold it.
        const int up = ve - U + kValueUp;
        half_scale[d] = valid ? pow2h(max(up, -14)) : 0;
        half_scale[kTile + d] = pow2h(min(up + 14, 0));
        reinterpret_cast<float*>(smem + Lay::kScale)[st * kTile + (j & 1) * 64 + unit * 8 + (j >> 1)] =
            valid ? __uint_as_float(static_cast<uint32_t>(ke) << 23) : -1.f;
        if (d == 0)
          reinterpret_cast<int4*>(smem + Lay::kInfo)[st] = make_int4(t0, all_valid && t0 + kTile <= base, U, 0);
        named_barrier<2, kConvertThreads>();
        // Then a thread a dim.
        const bool small = least - U + kValueUp < -14, tail = t0 + kTile > base;
        uint8_t* to = smem + Lay::kHalves + st * kHalfStage + d * 16;
#pragma unroll 2
        for (int u = 0; u < kUnits; ++u) {
          uint4 w4 = *reinterpret_cast<const uint4*>(raw + u * kRest + d * 16);
          uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          if (!all_valid || tail) {
            // A NaN code times a zero weight is NaN: codes past the end are
            // cleared, and NaN codes of nodes, whose NaN is given to the rows
            // that see them at the end.
            const int have = valid_s[vs * kUnits + u], node0 = t0 + u * kBlock - base;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int n = have - 4 * b;
              w[b] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
              if (node0 + 4 * b + 3 >= 0) {
                uint32_t bad = __vcmpeq4(w[b] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                if (node0 + 4 * b < 0) bad &= ~0u << (8 * -(node0 + 4 * b));
                w[b] &= ~bad;
                for (; bad; bad &= bad - 1) nan |= 1ull << (node0 + 4 * b + ((__ffs(bad) - 1) >> 3));
              }
            }
          }
          const uint4 f0 = *reinterpret_cast<const uint4*>(half_scale + u * kBlock);
          const uint4 f1 = *reinterpret_cast<const uint4*>(half_scale + u * kBlock + 8);
          const uint32_t f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
          uint32_t o[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t v = q8_unpack2(w[b >> 1] >> (16 * (b & 1)));
            const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&f[b]));
            o[b] = *reinterpret_cast<const uint32_t*>(&x);
          }
          if (small) {
            const uint32_t* f2 = reinterpret_cast<const uint32_t*>(half_scale + kTile + u * kBlock);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&o[b]), *reinterpret_cast<const __half2*>(f2 + b));
              o[b] = *reinterpret_cast<const uint32_t*>(&x);
            }
          }
          *reinterpret_cast<uint4*>(to + u * 4096) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(to + u * 4096 + 2048) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        if (i == walk.n - 1) {
          const int ring = g % (Lay::kC + 1);
          reinterpret_cast<uint64_t*>(smem + Lay::kNan)[ring * kHeadDim + d] = nan;
          const int any = __any_sync(0xffffffffu, nan != 0);
          if (lane == 0) reinterpret_cast<int*>(smem + Lay::kNanFlag)[ring * 4 + warp - 8] = any;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(half_full + st);
          mbar_arrive(value_empty + vs);
        }
      }
    }
  } else {
    // ---- softmax: row `rr` of stream t
    const int t = warp >> 2, rr = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256;
    float* factor = reinterpret_cast<float*>(smem + Lay::kFactor);
    float4* stat = reinterpret_cast<float4*>(smem + Lay::kStat);
    int g0 = 0;
    uint32_t score_phase = 0, done_phase = 0;
    while (ok && walk.next(a)) {
      const int rows = walk.rows(a), row0 = walk.block * kRows;
      const bool two = kTiles == 2 && rows > kTile;
      // The segment's queries: half a warp a row, eight rows at a time.  (The
      // last ones' products are done: every stream has waited for its own.)
      for (int r0 = warp * 2 + (lane >> 4); r0 < (two ? 2 : 1) * kTile; r0 += 128) {
        uint4 v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int row = r0 + 16 * b, at = row0 + row;
          v[b] = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows)
            v[b] = __ldg(reinterpret_cast<const uint4*>(
                             static_cast<const T*>(a.q) +
                             ((static_cast<int64_t>(walk.r) * a.N + at / a.G) * a.Hq + walk.h * a.G + at % a.G) *
                                 kHeadDim) +
                         (lane & 15));
        }
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int row = r0 + 16 * b;
          float x[8];
          if constexpr (kTerms == 2) {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[2 * i] = bf16lo(w[i]);
              x[2 * i + 1] = bf16hi(w[i]);
            }
          } else {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
              x[2 * i] = f.x;
              x[2 * i + 1] = f.y;
            }
          }
          uint32_t amax = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
          for (int off = 8; off; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
          const bool finite_row = amax < 0x7f800000u;
          const int e = q8_exponent(finite_row ? amax : 0);
          const float down = pow2f(-e);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= down;
          uint8_t* tile = smem + Lay::kQ + (row >> 7) * kTerms * kTerm + (row & 127) * 128 +
                          ((((lane & 15) >> 1) ^ (row & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
          for (int term = 0; term < kTerms; ++term) {
            const uint32_t lo = q8_pack4(x[0], x[1], x[2], x[3]), hi = q8_pack4(x[4], x[5], x[6], x[7]);
            *reinterpret_cast<uint2*>(tile + term * kTerm) = make_uint2(lo, hi);
            const uint32_t c[4] = {q8_unpack2(lo & 0xffffu), q8_unpack2(lo >> 16), q8_unpack2(hi & 0xffffu),
                                   q8_unpack2(hi >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // what is left, exactly
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
              x[2 * i] -= f.x;
              x[2 * i + 1] -= f.y;
            }
          }
          // (Held above 0: -inf times a factor has to stay.)
          if ((lane & 15) == 0)
            factor[row] = finite_row ? fmaxf(a.scale_log2 * pow2f(e), 0x1p-126f) : __int_as_float(0x7fffffff);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      named_barrier<1, kSoftmaxThreads>();
      if (lane == 0) mbar_arrive(q_ready);
      const int row = (two ? t * kTile : 0) + rr;  // of the block
      const bool busy = __any_sync(0xffffffffu, row < rows);
      const float f = factor[row];
      const int base = walk.q.len - walk.q.nodes;
      uint64_t word = 0;
      if (row < rows) {
        word = __ldg(a.words + static_cast<int64_t>(walk.r) * a.N + (row0 + row) / a.G);
        if (walk.q.nodes < 64) word &= (1ull << walk.q.nodes) - 1;
      }

      float m = -INFINITY, l = 0.f;
      int U = 0, jobs = 0;
      for (int i = two ? 0 : t; i < walk.n; i += two ? 1 : 2, ++jobs) {
        const int g = g0 + i, st = g % Lay::kC;
        ok = reached(s_full + t, score_phase) && reached(half_full + st, (g / Lay::kC) & 1);
        score_phase ^= 1;
        if (!ok) break;
        fence_after();
        if (busy) {
          const int4 info = reinterpret_cast<const int4*>(smem + Lay::kInfo)[st];
          const float4* scale = reinterpret_cast<const float4*>(smem + Lay::kScale + st * kTile * 4);
          const bool whole = info.y != 0;
          // Which of the tile's tokens the row sees, in score columns (even
          // tokens, then odd ones).
          uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t bits = 0;
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                const float4 k4 = scale[c * 8 + b];
                const float k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  const int col = (c & 1) * 32 + b * 4 + n;
                  const int node = info.x + (col >> 3) * kBlock + (col & 7) * 2 + (c >> 1) - base;
                  const bool in = k[n] >= 0.f && (node < 0 || (word >> (node & 63) & 1));
                  bits |= static_cast<uint32_t>(in) << (b * 4 + n);
                }
              }
              see[c] = bits;
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float s[32];
            tmem_ld32(s_at + c * 32, s);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const float4 k4 = scale[c * 8 + b];
              s[4 * b] *= k4.x;
              s[4 * b + 1] *= k4.y;
              s[4 * b + 2] *= k4.z;
              s[4 * b + 3] *= k4.w;
            }
            if (!whole) {
#pragma unroll
              for (int n = 0; n < 32; ++n)
                if (!(see[c] >> n & 1)) s[n] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < 32; n += 2) top = fmax3(top, s[n], s[n + 1]);
          }
          top *= f;
          float to = m, alpha = 1.f;
          if (top > m + kLazy || m == -INFINITY) {
            to = fmaxf(top, m);
            alpha = m == -INFINITY ? 0.f : ex2(m - to);
            m = to;
          }
          l *= alpha;
          alpha *= pow2_held(U - info.z);
          U = info.z;
          if (jobs > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // (The scores' arrival says that the stream's last output product is done.)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[32];
              tmem_ld32(o_at + t * 128 + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int n = 0; n < 32; ++n) o[n] *= alpha;
              tmem_st32(o_at + t * 128 + c * 32, reinterpret_cast<const uint32_t*>(o));
            }
          }
          const float off = kWeight - finite_or_0(m);
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float s[2][32];
            tmem_ld32(s_at + c * 32, s[0]);
            tmem_ld32(s_at + 64 + c * 32, s[1]);
            tmem_wait_ld();
            uint32_t w[32];
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                const float4 k4 = scale[odd * 16 + c * 8 + b];
                const float k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  float& x = s[odd][4 * b + n];
                  x = ex2(fmaf(x * k[n], f, off));
                  if (!whole && !(see[odd * 2 + c] >> (4 * b + n) & 1)) x = 0.f;
                  sum[odd] += x;
                }
              }
            }
#pragma unroll
            for (int n = 0; n < 32; ++n) w[n] = pack_f16x2(s[0][n], s[1][n]);
            tmem_st32(s_at + c * 32, w);
          }
          l += sum[0] + sum[1];
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + t);
      }
      if (ok && jobs > 0) {
        ok = reached(o_done + t, done_phase);
        done_phase ^= 1;
      }
      stat[t * kTile + rr] = make_float4(m, l, __int_as_float(U), 0.f);
      fence_before();
      ok = all_of<1, kSoftmaxThreads>(ok);
      if (!ok) break;
      fence_after();

      // The rows' outputs, in units of 2^8, averages: of this stream's row, or
      // of half the dims of both streams' shares of it.
      const float4 s0 = stat[(two ? t : 0) * kTile + rr];
      const float4 s1 = two || walk.n < 2 ? make_float4(-INFINITY, 0.f, 0.f, 0.f) : stat[kTile + rr];
      const float mx = fmaxf(s0.x, s1.x);
      float c0 = scale_of(s0.x, mx), c1 = scale_of(s1.x, mx);
      const float sum = s0.y * c0 + s1.y * c1;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      c0 *= inv;
      c1 *= inv;
      const float p0 = pow2_held(__float_as_int(s0.z) - 127 - kValueUp - 8);
      const float p1 = pow2_held(__float_as_int(s1.z) - 127 - kValueUp - 8);
      const int last = g0 + walk.n - 1, ring = last % (Lay::kC + 1);
      const int4 flags = reinterpret_cast<const int4*>(smem + Lay::kNanFlag)[ring];
      const bool some_nan = (flags.x | flags.y | flags.z | flags.w) != 0;
      const uint64_t* nan = reinterpret_cast<const uint64_t*>(smem + Lay::kNan) + ring * kHeadDim;
      const int64_t share = static_cast<int64_t>(2 * c + (walk.first > 0 ? 0 : 1)) * a.part_rows + row;
      const int at = row0 + row;
      const int64_t to_row =
          ((static_cast<int64_t>(walk.r) * a.N + at / a.G) * a.Hq + walk.h * a.G + at % a.G) * kHeadDim;
      if (busy) {
#pragma unroll 1
        for (int d0 = two ? 0 : t * 64; d0 < (two ? 128 : t * 64 + 64); d0 += 32) {
          float o[32], o1[32];
          tmem_ld32(o_at + (two ? t * 128 : 0) + d0, o);
          if (!two && walk.n > 1) tmem_ld32(o_at + 128 + d0, o1);
          tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            o[n] = o[n] * c0 * p0;
            if (!two && walk.n > 1) o[n] += o1[n] * c1 * p1;
          }
          if (some_nan) {
#pragma unroll
            for (int n = 0; n < 32; ++n)
              if (nan[d0 + n] & word) o[n] = __int_as_float(0x7fffffff);
          }
          if (row < rows) {
            if (!walk.whole()) {
#pragma unroll
              for (int n = 0; n < 4; ++n) store8(a.part + share * kHeadDim + d0 + 8 * n, o + 8 * n);
            } else if (a.out_fp32) {
#pragma unroll
              for (int n = 0; n < 8; ++n)
                store4_finite(static_cast<float*>(a.out) + to_row + d0 + 4 * n,
                              make_float4(o[4 * n] * 256.f, o[4 * n + 1] * 256.f, o[4 * n + 2] * 256.f,
                                          o[4 * n + 3] * 256.f));
            } else {
              T* out = static_cast<T*>(a.out) + to_row + d0;
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                uint32_t w[4];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  w[b] = pack2_finite(out, o[8 * n + 2 * b] * 256.f, o[8 * n + 2 * b + 1] * 256.f);
                *reinterpret_cast<uint4*>(out + 8 * n) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        fence_before();
        if (!walk.whole() && row < rows && (two || t == 0)) a.stat[share] = make_float2(mx, sum);
      }
      // The CTA where a pair begins that others go on with names the shares.
      if (tid == 0 && walk.first == 0 && !walk.whole()) {
        const int64_t end = u1 - walk.left - walk.n + walk.q.tiles;  // of the pair, in the sequence
        const int64_t owner = (end * ctas + total - 1) / total - 1;
        a.info[c] = make_int4(walk.r, walk.h, walk.block, static_cast<int>(owner) - c + 1);
      }
      g0 += walk.n;
    }
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout);
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 13) tmem_free(tmem, 512);
}

// The shares of the pair that begins in a CTA and goes on in others: a warp a
// row, eight rows a CTA of this launch.
constexpr int kJoinRows = 8;
template <typename T, int kRows>
__global__ void __launch_bounds__(kJoinRows * 32) tree_join(const TreeArgs a) {
  previous_done();
  next_may_begin();
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int4 info = __ldcg(a.info + c);
  if (info.x < 0) return;
  const Request q = request<kRows>(a, info.x);
  if (row >= min(q.nodes * a.G - info.z * kRows, kRows)) return;
  auto share = [&](int i) {
    return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.part_rows + row;
  };
  float mx = -INFINITY, sum = 0.f;
  for (int i = lane; i < info.w; i += 32) {
    const float2 st = __ldcg(a.stat + share(i));
    join_sum(mx, sum, st.x, st.y);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1)
    join_sum(mx, sum, __shfl_xor_sync(0xffffffffu, mx, off), __shfl_xor_sync(0xffffffffu, sum, off));
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < info.w; ++i) {
    const float2 st = __ldcg(a.stat + share(i));
    const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part + share(i) * kHeadDim) + lane);
    add4(acc, scale_of(st.x, mx) * st.y * inv, x);
  }
  scale4(acc, 256.f);
  const int at = info.z * kRows + row;
  const int64_t to =
      ((static_cast<int64_t>(info.x) * a.N + at / a.G) * a.Hq + info.y * a.G + at % a.G) * kHeadDim + lane * 4;
  if (a.out_fp32) store4_finite(static_cast<float*>(a.out) + to, acc);
  else store4_finite(static_cast<T*>(a.out) + to, acc);
}

template <typename T, int kTiles>
cudaError_t launch_t(const TreeArgs& a, const CUtensorMap& map, cudaStream_t s) {
  using Lay = TreeLayout<std::is_same_v<T, __half> ? 3 : 2, kTiles>;
  const cudaError_t e = launch_early(tree_kernel<T, kTiles>, a.ctas, kTreeThreads, Lay::kBytes, s, 0, a, map);
  if (e != cudaSuccess) return e;
  return launch_early(tree_join<T, kTiles * kTile>, dim3(a.ctas, (a.part_rows + kJoinRows - 1) / kJoinRows),
                      kJoinRows * 32, 0, s, 0, a);
}

template <typename T, int kTiles>
cudaError_t configure() {
  using Lay = TreeLayout<std::is_same_v<T, __half> ? 3 : 2, kTiles>;
  cudaError_t e = cudaFuncSetAttribute(tree_kernel<T, kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, tree_join<T, kTiles * kTile>);
  return e;
}

}  // namespace

TreeShape tree_shape(int R, int N, int G, int Hkv, int max_blocks, int type) {
  TreeShape p{};
  const int rows = N * G;
  // 256 rows a CTA where there are so many: its pages are read once for all.
  // (fp16's third term of the queries leaves no room for a second row tile.)
  p.tiles = type == kBf16 && rows > kTile ? 2 : 1;
  const int block = p.tiles * kTile;
  const int64_t most = static_cast<int64_t>(R) * Hkv * ((rows + block - 1) / block) *
                       ((static_cast<int64_t>(max_blocks) + kUnits - 1) / kUnits);
  p.ctas = static_cast<int>(most < 152 ? most : 152);
  p.rows = rows < block ? rows : block;
  auto up = [](int64_t n) { return static_cast<size_t>((n + 255) / 256 * 256); };
  const int64_t shares = 2ll * p.ctas * p.rows;
  p.part_bytes = up(shares * kHeadDim * 4);
  p.stat_bytes = up(shares * 8);
  p.bytes = p.part_bytes + p.stat_bytes + up(p.ctas * 16);
  return p;
}

cudaError_t launch_q8_tree(const TreeArgs& a, int tiles, const CUtensorMap& map, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  if (a.type == kFp16) return launch_t<__half, 1>(a, map, s);
  return tiles == 2 ? launch_t<__nv_bfloat16, 2>(a, map, s) : launch_t<__nv_bfloat16, 1>(a, map, s);
}

cudaError_t preload_tree_kernels() {
  cudaError_t e = configure<__half, 1>();
  if (e == cudaSuccess) e = configure<__nv_bfloat16, 1>();
  if (e == cudaSuccess) e = configure<__nv_bfloat16, 2>();
  return e;
}

}  // namespace oasis
