// tree.cu -- attention of a request's tree of drafted tokens over its 8-bit
// pages.
//
// The nodes' queries that read one KV head (row node * G + gi) are the rows of
// a matrix, at most 256 of them a CTA, so its pages are read once: 4 * 128
// operations a row and token against 258 bytes a token, bound by HBM up to
// some 140 rows, by the tensor cores (tcgen05) beyond.
//
// Both operands are used as they lie in the pages, as far as they can be:
// * Keys go in as e4m3 with their exponent bytes (kind::mxf8f6f4, scales in
//   tensor memory), so scores come out whole.  A query row is a sum of e4m3 rows
//   times one power of two: two of them hold bf16's eight bits, three fp16's
//   eleven (exact for entries down to 2^-9 and 2^-6 of the row's largest; below,
//   off by half of e4m3's least step, 2^-10, where the largest is over 224: 2^-17.8
//   of it).  A tile of 128 tokens is eight units, whose even
//   and odd tokens are two operands of 64 tokens: the odd ones have their
//   halves exchanged, which costs nothing but another order of the steps.
// * Values have a unit's 16 tokens consecutive, which is an operand's layout
//   without a swizzle for 16 rows of 8-bit weights.  Weights of 8 bits would be
//   too coarse, so four warps turn the values into fp16, in units of the
//   largest value exponent so far, and the weights are fp16 (tensor memory).
//   In the tree's own tiles a row's unit is held to what the row sees, so that
//   no other node's exponent costs it bits.
//
// One CTA an SM.  The tiles of all (request, KV head, 256 rows) are one
// sequence, which the CTAs share out evenly, whatever the lengths: a CTA's range
// is made of segments, each a run of tiles of one pair.  A pair wholly inside
// one CTA's range is written straight out, others as shares (average, maximum,
// sum) that a second launch joins.
//
// Roles: warps 0..7 softmax, one thread a row, two streams of four warps; 8..11
// values to fp16; 12 loads (TMA with the 128-byte swizzle for keys, bulk copies
// for values and exponents); 13 issues outputs' products, 14 scores'; 15 plans.
// The streams take turns, so that the products of one run while the other's
// weights are formed: with more than 128 rows they are two row tiles over the
// same tokens, else the even and the odd tokens of the same rows, joined at the
// end.  A job is 128 rows x 64 tokens; its scores are in one of three buffers of
// tensor memory, where its weights take their place.
//
// GB300, us: 16 requests x 64 nodes x 32 / 8 heads over 16384 tokens 241 (tensor
// cores 146 at the measured bf16 rate), in fp16 320 (its pages are read twice), 24
// ragged ones up to 9001 tokens, fp16, 73, one of 16 nodes over 4096 22.  With many
// rows what holds it back is a job's way through the buffers (scores 400 cycles,
// 384 of them for the operands that its steps of 64 columns read from shared
// memory; the softmax of its 64 columns 700 to 1000, outputs 270, 100 to 300 from
// each hand to the next): 960 cycles a job where the products alone take 640.  With
// few rows it is the loads (16 x 4 nodes 160, as the large case with nothing but its
// loads: 3.4 TB/s), in ragged batches also what a segment begins and ends with,
// some 9000 cycles that nothing covers and the share-out does not count.  Measured
// on the way, the first case (of then 243): 128 columns a
// job and two buffers 288; two buffers for scores and three for weights, released
// as soon as they are read, 278; sixteen softmax warps 317; more registers for
// the softmax warps (setmaxnreg) spilled.  The elected lane must not change in
// the issuing loops: a lane that turned 0 when a wait had run out cost 460 cycles
// a job, 282 in all; outputs' products unrolled over a tile's jobs 252 (their code
// is fetched in turn with seven other roles').
#include <cuda_fp16.h>

#include <type_traits>

#include "q8.cuh"
#include "q8.h"
#include "tcgen05.cuh"
#include "tree_place.h"

namespace oasis {
namespace {

constexpr int kTile = 128;                              // rows, tokens
constexpr int kUnits = kTile / kBlock;                  // of a tile
constexpr int kRest = kQ8UnitBytes - kQ8HalfBytes;      // values and exponents of a unit
constexpr int kKeyStage = kUnits * kQ8HalfBytes;        // 16 KiB
constexpr int kValueStage = kUnits * kRest;
constexpr int kHalfStage = kTile * kHeadDim * 2;        // values in fp16: 32 KiB
constexpr int kTerm = kTile * kHeadDim;                 // one e4m3 row tile of queries: 16 KiB
constexpr int kSoftmaxWarps = 8, kConvertWarp = 8, kLoadWarp = 12, kOutWarp = 13, kScoreWarp = 14, kPlanWarp = 15;
constexpr int kTreeThreads = 16 * 32;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32, kConvertThreads = 128;
constexpr float kWeight = 7.f;                          // a weight is 2^(x - m + 7): 2^7 where the maximum is its own
constexpr float kMostSum = 32768.f;                     // of a row's weights over a tile, each under it
constexpr int kValueUp = 6;                             // a value is code * 2^(e - U + 6), at most 448 * 64
constexpr int kReach = 14 + kValueUp;                   // U - e up to which that is a code times one fp16 number, exactly

template <int kTerms, int kTiles>
struct TreeLayout {
  static constexpr int kK = 3, kV = kTiles == 1 ? 3 : 2, kC = 2;  // stages
  static constexpr int kQ = 0;
  static constexpr int kKeys = kQ + kTiles * kTerms * kTerm;
  static constexpr int kHalves = kKeys + kK * kKeyStage;
  static constexpr int kValues = kHalves + kC * kHalfStage;
  static constexpr int kKeyScale = kValues + kV * kValueStage;  // [kC][2][32][4] words: of even, of odd tokens' keys
  static constexpr int kQueryScale = kKeyScale + kC * 1024;     // [kTiles][32][4]
  static constexpr int kInfo = kQueryScale + kTiles * 512;         // [kC] int4: first token, whole, U, wide; valid tokens
  static constexpr int kNan = kInfo + kC * 32;                  // [kC + 1][128] words, then [kC + 1] int4 flags
  static constexpr int kNanFlag = kNan + (kC + 1) * kHeadDim * 8;
  static constexpr int kFactor = kNanFlag + (kC + 1) * 16;      // [kTiles][128] of a row's scores
  static constexpr int kStat = kFactor + kTiles * kTile * 4;    // [2][128] float4: m, sum, U of a stream's rows
  static constexpr int kPlan = kStat + 2 * kTile * 16;          // [4] segments
  static constexpr int kHalfScale = kPlan + 4 * 64;             // [2][128] half: of a token's value
  static constexpr int kValid = kHalfScale + 2 * kTile * 2;     // [kV][8] tokens of a unit
  static constexpr int kConvert = kValid + kV * kUnits * 4;     // [4] int2 of the converting warps
  static constexpr int kExps = kConvert + 32;                   // [kC][128] bytes: values' exponents of even, of odd tokens
  static constexpr int kBars = kExps + kC * kTile;
  static constexpr int kBytes = kBars + 384 + 1024;             // + alignment
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kHalves % 128 == 0 && kValues % 128 == 0 && kKeyScale % 128 == 0 && kBars % 8 == 0, "alignment");
};

constexpr uint32_t kScoreInstr = kMmaScaleE8 | mma_shape(128, 64);
// Columns of tensor memory: three buffers of 64 for scores, two streams' outputs,
// scales of two query tiles and of two tiles' even and odd tokens.
constexpr int kOutAt = 192, kQueryScaleAt = 448, kKeyScaleAt = 456;
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
template <int kThreads>
__device__ __forceinline__ bool all_of(int id, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "n"(kThreads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return r != 0;
}
// Bits 0, 2, 4, .. of x, together.
__device__ __forceinline__ uint32_t even_bits(uint32_t x) {
  x &= 0x55555555u;
  x = (x | x >> 1) & 0x33333333u;
  x = (x | x >> 2) & 0x0f0f0f0fu;
  x = (x | x >> 4) & 0x00ff00ffu;
  return (x | x >> 8) & 0xffffu;
}
// 2^e as fp16 bits, -24 <= e <= 15 (0 below).
__device__ __forceinline__ uint16_t pow2h(int e) {
  return static_cast<uint16_t>(e >= -14 ? (e + 15) << 10 : e >= -24 ? 1 << (e + 24) : 0);
}
// mbar_wait in few instructions, for its many places: limits under 2^20 cycles are
// for tests, and polled without sleeping.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint32_t limit) {
  const bool brief = limit < kShortWaitCycles;
  if (!brief && mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
  while (!(brief ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)))
    if (static_cast<uint32_t>(clock()) - t0 > limit) return false;
  return true;
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

// A segment as the other warps have it.
struct alignas(16) Plan {
  int n, rows, row0, base;             // tiles (0: the last one has been), rows, the block's first, tokens before the tree
  int nodes, len, whole, share;        // share: row 0 of the CTA's share of the pair
  int64_t query;                       // where row 0 of node 0 begins in q and out
  int r, h, first, pad;                // request, KV head, first tile
};
constexpr int kPlans = 4;

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
  uint64_t* scale_full = half_empty + Lay::kC;                          // [kC] keys' scales (four warps)
  uint64_t* s_full = scale_full + Lay::kC;                              // [3] scores in a buffer
  uint64_t* p_full = s_full + 3;                                        // [3] weights (four warps)
  uint64_t* o_done = p_full + 3;                                        // [3] outputs with them
  uint64_t* q_ready = o_done + 3;                                       // a segment's queries (eight warps)
  uint64_t* plan_full = q_ready + 1;                                    // [4]
  uint64_t* plan_empty = plan_full + kPlans;                            // [4] (all but the planning warp)
  uint64_t* drain = plan_empty + kPlans;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kWarps = kTreeThreads / 32;
  previous_done();
  // (Not before: a kernel ahead that takes tensor memory after it has let its
  // dependents begin would wait for this one's.)
  if (warp == kScoreWarp) tmem_alloc(tmem_s, 512);
  next_may_begin();
  if (tid == kLoadWarp * 32) {
    prefetch_tensormap(&map);
    for (int i = 0; i < 2 * Lay::kK; ++i) mbar_init(key_full + i, 1);
    for (int i = 0; i < Lay::kV; ++i) {
      mbar_init(value_full + i, 1);
      mbar_init(value_empty + i, 4);
    }
    for (int i = 0; i < Lay::kC; ++i) {
      mbar_init(half_full + i, 4);
      mbar_init(half_empty + i, 1);
      mbar_init(scale_full + i, 4);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < kPlans; ++i) {
      mbar_init(plan_full + i, 1);
      mbar_init(plan_empty + i, kWarps - 1);
    }
    mbar_init(q_ready, kSoftmaxWarps);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    fence_barrier_init();
  }

  constexpr int kRows = kTiles * kTile;
  // This CTA's range of the sequence: for the planning warp, a lane a request,
  // and where there are more than 32, in rounds.
  const int c = blockIdx.x;
  Walk<kRows> walk = {};
  int64_t per = 0, u1 = 0;
  int ctas = 1, rem = 0;
  auto begin = [&](int at) { return per * at + rem * at / ctas; };  // total * at / ctas
  if (warp == kPlanWarp) {
    if (lane == 0) a.info[c] = make_int4(-1, 0, 0, 0);
    auto tiles_of = [&](const Request& q) { return static_cast<int64_t>(q.tiles) * q.blocks * a.Hkv; };
    auto sum_up = [&](int64_t t) {  // over the lanes up to this one
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += o;
      }
      return t;
    };
    Request own = {};
    if (lane < a.R) own = request<kRows>(a, lane);
    int64_t t = tiles_of(own), incl = sum_up(t), more = 0;
    int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    if (a.R > 32) {
#pragma unroll 4
      for (int r = lane + 32; r < a.R; r += 32) more += tiles_of(request<kRows>(a, r));
      total += __shfl_sync(0xffffffffu, sum_up(more), 31);
    }
    ctas = static_cast<int>(max(min(static_cast<int64_t>(gridDim.x), total), static_cast<int64_t>(1)));
    per = total >> 32 ? total / ctas : static_cast<uint32_t>(total) / ctas;
    rem = static_cast<int>(total - per * ctas);
    const int64_t u0 = c < ctas ? begin(c) : 0;
    u1 = c < ctas ? begin(c + 1) : 0;
    walk.left = u1 - u0;
    for (int r0 = 0; u0 < u1;) {
      const uint32_t found = __ballot_sync(0xffffffffu, incl - t <= u0 && u0 < incl);
      if (found) {
        const int from = __ffs(found) - 1;
        walk.q = {__shfl_sync(0xffffffffu, own.len, from), __shfl_sync(0xffffffffu, own.nodes, from),
                  __shfl_sync(0xffffffffu, own.blocks, from), __shfl_sync(0xffffffffu, own.tiles, from)};
        const TreePlace at = tree_place(__shfl_sync(0xffffffffu, u0 - (incl - t), from), walk.q.tiles);
        walk.r = r0 + from;
        walk.pair = at.pair;
        walk.i0 = at.tile;
        break;
      }
      const int64_t before = __shfl_sync(0xffffffffu, incl, 31);
      r0 += 32;
      own = Request{};
      if (r0 + lane < a.R) own = request<kRows>(a, r0 + lane);
      t = tiles_of(own);
      incl = before + sum_up(t);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  // (All of the tensor memory is this CTA's: it begins at 0.)
  const uint32_t limit = static_cast<uint32_t>(min(a.wait_limit, static_cast<long long>(kWaitLimitCycles)));
  auto reached = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_for(bar, parity, limit)) != 0;
  };

  // Segment k's plan, once it is there.
  const Plan* plans = reinterpret_cast<const Plan*>(smem + Lay::kPlan);
  auto plan_there = [&](int k) { return reached(plan_full + k % kPlans, k / kPlans & 1); };
  auto plan_read = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(plan_empty + k % kPlans);
  };

  bool ok = true;
  if (warp == kPlanWarp) {
    // ---- the segments of this CTA's range
    for (int k = 0; ok; ++k) {
      const bool more = walk.next(a);
      ok = k < kPlans || reached(plan_empty + k % kPlans, (k / kPlans - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        Plan& p = reinterpret_cast<Plan*>(smem + Lay::kPlan)[k % kPlans];
        p.n = more ? walk.n : 0;
        if (more) {
          p.rows = walk.rows(a);
          p.row0 = walk.block * kRows;
          p.base = walk.q.len - walk.q.nodes;
          p.nodes = walk.q.nodes;
          p.len = walk.q.len;
          p.whole = walk.whole();
          p.share = (2 * c + (walk.first > 0 ? 0 : 1)) * a.part_rows;
          p.query = (static_cast<int64_t>(walk.r) * a.N * a.Hq + walk.h * a.G) * kHeadDim;
          p.r = walk.r;
          p.h = walk.h;
          p.first = walk.first;
        }
        mbar_arrive(plan_full + k % kPlans);
        // The CTA where a pair begins that others go on with names the shares.
        if (more && walk.first == 0 && !walk.whole()) {
          const int64_t end = u1 - walk.left - walk.n + walk.q.tiles;  // of the pair, in the sequence
          int owner = c + 1;                                            // of its last tile
          while (begin(owner + 1) < end) ++owner;
          a.info[c] = make_int4(walk.r, walk.h, walk.block, owner - c + 1);
        }
      }
      __syncwarp();
      if (!more) break;
    }
    // Requests without a tile: their nodes give zeros, and bad lengths are
    // reported, each by one CTA.
    for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
      const Request q = request<kRows>(a, r);
      const int len = a.len[r];
      if (lane == 0 && (len > a.max_blocks * kBlock || (len > 0 && len < q.nodes))) raise_error(a.err, kErrBadBlock);
      if (q.tiles == 0 && q.nodes > 0) {
        const int64_t bytes = static_cast<int64_t>(a.Hq) * kHeadDim * (a.out_fp32 ? 4 : 2);
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(r) * a.N * bytes);
        for (int64_t i = lane; i < q.nodes * bytes / 16; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else if (warp == kLoadWarp) {
    // ---- loads: a lane a unit
    int gk = 0, gv = 0;  // tiles whose keys, whose values are on their way
    for (int k = 0; ok; ++k) {
      ok = plan_there(k);
      if (!ok) break;
      const Plan p = plans[k % kPlans];
      plan_read(k);
      if (p.n == 0) break;
      const int32_t* row = a.table + static_cast<int64_t>(p.r) * a.max_blocks;
      auto page_of = [&](int i) {
        const int b = (p.first + i) * kUnits + lane;
        return lane < kUnits && i < p.n && b * kBlock < p.len ? __ldg(row + b) : -1;
      };
      int page = page_of(0);
#pragma unroll 1
      for (int i = 0; i < p.n; ++i) {
        const int left = p.len - ((p.first + i) * kUnits + lane) * kBlock;
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
        if (there) load_keys(smem + Lay::kKeys + ks * kKeyStage + lane * kQ8HalfBytes, &map, p.h, at, key_full + ks);
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
                   a.pages + (static_cast<int64_t>(at) * a.Hkv + p.h) * kQ8UnitBytes + kQ8HalfBytes, kRest,
                   value_full + vs);
        ++gv;
      }
    }
    // No copy may outlive the CTA, whatever the other warps met.
    for (int j = max(gk - Lay::kK, 0); j < gk; ++j) (void)mbar_wait(key_full + j % Lay::kK, (j / Lay::kK) & 1);
    for (int j = max(gv - Lay::kV, 0); j < gv; ++j) (void)mbar_wait(value_full + j % Lay::kV, (j / Lay::kV) & 1);
  } else if (warp == kOutWarp) {
    // ---- outputs' products.  (Two warps issue products: while one waits the other's
    // run.)
    //
    // No loop of the two ends by what a thread finds, and sizes go through a warp's
    // reduction: so all that the descriptors are made of is known to be the warp's
    // alike and stays in uniform registers, where the instruction wants it.  After a
    // wait that ran out a segment's loop runs on, on this CTA's memory alone; the call
    // has failed, and what the products then find is not used.
    const uint32_t lead = elected();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = reached(bar, parity);
    };
    const uint64_t v_desc = smem_desc_plain(smem_u32(smem + Lay::kHalves), 4096, 128);
    int g = 0;                             // tiles so far
    uint32_t buffer = 0, parity = 0;       // of the next job
    for (int segments = 0;; ++segments) {
      wait(plan_full + segments % kPlans, segments / kPlans & 1);
      const volatile Plan& plan = plans[segments % kPlans];
      const int n = __reduce_max_sync(0xffffffffu, ok ? plan.n : 0);
      const bool two = kTiles == 2 && __reduce_max_sync(0xffffffffu, plan.rows) > kTile;
      plan_read(segments);
      if (n == 0) break;
      // A tile's jobs: of the streams in turn, the even or the odd tokens, each in
      // the buffer that follows the last one's.
      const int jobs = two ? 4 : 2;
      for (int i = 0; i < n; ++i, ++g) {
        const uint32_t st = g % Lay::kC;
        wait(half_full + st, (g / Lay::kC) & 1);
#pragma unroll 1
        for (int j = 0; j < jobs; ++j) {
          const uint32_t odd = two ? j >> 1 : j;
          const uint64_t v = v_desc + st * (kHalfStage >> 4) + odd * (2048 >> 4);
          const uint32_t to = kOutAt + (j & 1) * 128, from = buffer * 64;
          wait(p_full + buffer, parity);
          fence_after();
#pragma unroll
          for (int s = 0; s < 4; ++s)  // the even or odd tokens of two units a step
            mma_ts<kOutInstr>(to, from + s * 8, v + s * (8192 >> 4), i > 0 || j > 1 || s > 0, lead);
          mma_commit(o_done + buffer, lead);
          parity ^= buffer == 2;
          buffer = buffer == 2 ? 0 : buffer + 1;
        }
        mma_commit(half_empty + st, lead);
      }
    }
    // No product may outlive its operands and accumulators, either.
    mma_commit(drain, elected());
    (void)mbar_wait(drain, 0);
  } else if (warp == kScoreWarp) {
    // ---- scores' products
    const uint32_t lead = elected();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = reached(bar, parity);
    };
    const uint64_t q_desc = smem_desc(smem_u32(smem + Lay::kQ), 16);
    const uint64_t k_desc = smem_desc(smem_u32(smem + Lay::kKeys), 16, 2048);
    const uint64_t qs_desc = smem_desc_plain(smem_u32(smem + Lay::kQueryScale), 0, 128);
    const uint64_t ks_desc = smem_desc_plain(smem_u32(smem + Lay::kKeyScale), 0, 128);
    int g = 0;
    uint32_t buffer = 0, parity = 0;
    for (int segments = 0;; ++segments) {
      wait(plan_full + segments % kPlans, segments / kPlans & 1);
      const volatile Plan& plan = plans[segments % kPlans];
      const int n = __reduce_max_sync(0xffffffffu, ok ? plan.n : 0);
      const bool two = kTiles == 2 && __reduce_max_sync(0xffffffffu, plan.rows) > kTile;
      plan_read(segments);
      if (n == 0) break;
      wait(q_ready, segments & 1);
      fence_after();
#pragma unroll
      for (int t = 0; t < kTiles; ++t) load_scales(kQueryScaleAt + 4 * t, qs_desc + t * (512 >> 4), lead);
      auto tile = [&](auto streams) {
        constexpr int kStreams = decltype(streams)::value;
        const uint32_t st = g % Lay::kK, sc = g % Lay::kC;
        wait(key_full + st, (g / Lay::kK) & 1);
        wait(scale_full + sc, (g / Lay::kC) & 1);
        fence_after();
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
          load_scales(kKeyScaleAt + (2 * sc + odd) * 4, ks_desc + (2 * sc + odd) * (512 >> 4), lead);
#pragma unroll
        for (int j = 0; j < 2 * kStreams; ++j) {
          const uint32_t t = kStreams == 2 ? j & 1 : 0, odd = j / kStreams;
          const uint64_t q = q_desc + t * kTerms * (kTerm >> 4);
          const uint64_t k = k_desc + st * (kKeyStage >> 4) + odd * (1024 >> 4);
          const uint32_t scale = kKeyScaleAt + (2 * sc + odd) * 4;
          wait(o_done + buffer, parity ^ 1);  // (at once for the first three)
          fence_after();
#pragma unroll
          for (int term = 0; term < kTerms; ++term)
#pragma unroll
            for (int s = 0; s < 4; ++s)  // 32 dims a step
              mma_ss_scaled<kScoreInstr>(buffer * 64, q + term * (kTerm >> 4) + s * 2, k + (s ^ 2 * odd) * 2,
                                         kQueryScaleAt + 4 * t, scale, term > 0 || s > 0, lead);
          mma_commit(s_full + buffer, lead);
          parity ^= buffer == 2;
          buffer = buffer == 2 ? 0 : buffer + 1;
        }
        mma_commit(key_empty + st, lead);
      };
      if (two)
        for (int i = 0; i < n; ++i, ++g) tile(std::integral_constant<int, 2>{});
      else
        for (int i = 0; i < n; ++i, ++g) tile(std::integral_constant<int, 1>{});
    }
    mma_commit(drain + 1, elected());
    (void)mbar_wait(drain + 1, 0);
  } else if (warp >= kConvertWarp) {
    // ---- values to fp16: a thread a dim
    const int d = tid - kSoftmaxThreads, unit = d >> 4, j = d & 15;
    const int* valid_s = reinterpret_cast<const int*>(smem + Lay::kValid);
    int2* seen = reinterpret_cast<int2*>(smem + Lay::kConvert);
    uint16_t* half_scale = reinterpret_cast<uint16_t*>(smem + Lay::kHalfScale);
    int g = 0;
    for (int k = 0; ok; ++k) {
      ok = all_of<kConvertThreads>(2, plan_there(k));
      if (!ok) break;
      const Plan& plan = plans[k % kPlans];
      const int n = plan.n, base = plan.base, first = plan.first;
      plan_read(k);
      if (n == 0) break;
      int U = 0;         // the largest exponent byte so far
      uint64_t nan = 0;  // nodes whose value of dim d is NaN
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++g) {
        const int vs = g % Lay::kV, st = g % Lay::kC, t0 = (first + i) * kTile;
        // (One warp waits for all: polls take the place of others' instructions.)
        if (warp == kConvertWarp)
          ok = reached(value_full + vs, (g / Lay::kV) & 1) &&
               (g < Lay::kC || reached(half_empty + st, (g / Lay::kC - 1) & 1));
        ok = all_of<kConvertThreads>(2, ok);
        if (!ok) break;
        uint8_t* raw = smem + Lay::kValues + vs * kValueStage;
        // First a thread a token.
        const bool valid = j < valid_s[vs * kUnits + unit];
        const int ke = valid ? raw[unit * kRest + kQ8HalfBytes + j] : 0;
        const int ve = valid ? raw[unit * kRest + kQ8HalfBytes + kBlock + j] : 0;
        const int top = __reduce_max_sync(0xffffffffu, ve);
        const int low = __reduce_min_sync(0xffffffffu, valid ? ve : 255);
        const uint32_t have_s = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) seen[warp - kConvertWarp] = make_int2(have_s == ~0u ? top : top - 1024, low);
        named_barrier<2, kConvertThreads>();
        bool all_valid = true;
        int least = 255;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int2 s = seen[w];
          all_valid = all_valid && s.x >= 0;
          U = max(U, s.x >= 0 ? s.x : s.x + 1024);
          least = min(least, s.y);
        }
        // 2^(e - U + 6), as two factors where fp16 does not hold it.  In a tile that
        // rows see parts of, U may come from tokens that a row does not see.  If some
        // are more than 2^kReach below it the tile is wide: all keep their bits, as
        // codes times 2^(max(e - U, -kReach) + 6), and the rows' weights take the rest.
        const bool seen_by_all = all_valid && t0 + kTile <= base, far = U - least > kReach;
        const int up = ve - U + kValueUp;
        const int place = unit * kBlock + (j & 1) * 8 + (j >> 1);  // even tokens, then odd ones
        half_scale[place] = valid ? pow2h(max(up, -14)) : 0;
        half_scale[kTile + place] = pow2h(min(up + 14, 0));
        const int column = unit * 8 + (j >> 1);                    // of the scores of its kind
        reinterpret_cast<uint32_t*>(smem + Lay::kKeyScale)[st * 256 + (j & 1) * 128 + (column & 31) * 4 + (column >> 5)] =
            (valid ? ke : 127) * 0x01010101u;
        if (far && !seen_by_all) (smem + Lay::kExps)[st * kTile + (j & 1) * 64 + column] = static_cast<uint8_t>(ve);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (d == 0)
          reinterpret_cast<int4*>(smem + Lay::kInfo)[2 * st] = make_int4(t0, seen_by_all, U, far && !seen_by_all);
        if (lane == 0) reinterpret_cast<uint32_t*>(smem + Lay::kInfo)[st * 8 + 4 + warp - kConvertWarp] = have_s;
        named_barrier<2, kConvertThreads>();
        if (lane == 0) mbar_arrive(scale_full + st);
        // Then a thread a dim.
        const bool small = far && seen_by_all, tail = t0 + kTile > base;
        uint8_t* to = smem + Lay::kHalves + st * kHalfStage + d * 16;
        if (!all_valid || tail) {
          // A NaN code times a zero weight is NaN.  So codes past the end are
          // cleared where they lie, and so are NaN codes of nodes, whose NaN is given
          // to the rows that see them at the end.
#pragma unroll 1
          for (int b = 0; b < kTile / 4; ++b) {  // four tokens
            uint32_t* at = reinterpret_cast<uint32_t*>(raw + (b >> 2) * kRest + d * 16 + (b & 3) * 4);
            const int have = valid_s[vs * kUnits + (b >> 2)] - 4 * (b & 3), node = t0 + 4 * b - base;
            uint32_t w = *at & (have >= 4 ? ~0u : have <= 0 ? 0u : (1u << (8 * have)) - 1u);
            if (node + 3 >= 0) {
              uint32_t bad = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
              if (node < 0) bad &= ~0u << (8 * -node);
              w &= ~bad;
              for (; bad; bad &= bad - 1) nan |= 1ull << (node + ((__ffs(bad) - 1) >> 3));
            }
            *at = w;
          }
        }
#pragma unroll 2
        for (int u = 0; u < kUnits; ++u) {
          const uint4 w = *reinterpret_cast<const uint4*>(raw + u * kRest + d * 16);
          const uint4 f0 = *reinterpret_cast<const uint4*>(half_scale + u * kBlock);
          const uint4 f1 = *reinterpret_cast<const uint4*>(half_scale + u * kBlock + 8);
          const uint32_t f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
          const uint32_t sorted[4] = {__byte_perm(w.x, w.y, 0x6420), __byte_perm(w.z, w.w, 0x6420),
                                      __byte_perm(w.x, w.y, 0x7531), __byte_perm(w.z, w.w, 0x7531)};
          uint32_t o[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t v = q8_unpack2(sorted[b >> 1] >> (16 * (b & 1)));
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
        if (i == n - 1) {
          const int ring = g % (Lay::kC + 1);
          reinterpret_cast<uint64_t*>(smem + Lay::kNan)[ring * kHeadDim + d] = nan;
          const int any = __any_sync(0xffffffffu, nan != 0);
          if (lane == 0) reinterpret_cast<int*>(smem + Lay::kNanFlag)[ring * 4 + warp - kConvertWarp] = any;
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
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16, o_at = lanes + kOutAt;
    int buffer = t, parity = 0;  // of the stream's next job; they take turns
    // The same of its last one, two buffers before.
    auto last_done = [&]() {
      return reached(o_done + (buffer == 2 ? 0 : buffer + 1), buffer == 2 ? parity : parity ^ 1);
    };
    float* factor = reinterpret_cast<float*>(smem + Lay::kFactor);
    float4* stat = reinterpret_cast<float4*>(smem + Lay::kStat);
    const uint8_t* exps = smem + Lay::kExps;
    int g = 0;                   // tiles so far
    for (int k = 0;; ++k) {
      ok = plan_there(k);
      const volatile Plan& plan = plans[k % kPlans];
      const int n = ok ? plan.n : 0, rows = plan.rows;
      const bool two = kTiles == 2 && rows > kTile;
      // The segment's queries: eight lanes a row, the next ones on their way.  (The
      // last ones' products are done: every stream has waited for its own.)
      if (n > 0) {
        const T* q_row = static_cast<const T*>(a.q) + plan.query + (lane & 7) * 16;
        const int row0 = plan.row0;
        constexpr int kStep = 4 * kSoftmaxWarps;
        struct Part {
          uint4 lo, hi;
        };
        auto load = [&](int row) {
          const int at = row0 + row, node = static_cast<int>(at * a.over_G >> 16);
          const uint4* p =
              reinterpret_cast<const uint4*>(q_row + (node * a.Hq + at - node * a.G) * static_cast<int64_t>(kHeadDim));
          return row < rows ? Part{__ldg(p), __ldg(p + 1)} : Part{};
        };
        int row = warp * 4 + (lane >> 3);
        Part v = load(row), next = load(row + kStep);
#pragma unroll 1
        for (; row < (rows + 31) / 32 * 32; row += kStep) {  // (others' weights are not formed)
          const uint32_t w[8] = {v.lo.x, v.lo.y, v.lo.z, v.lo.w, v.hi.x, v.hi.y, v.hi.z, v.hi.w};
          v = next;
          next = load(row + 2 * kStep);
          float x[16];
          uint32_t amax = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 y = kTerms == 2 ? make_float2(bf16lo(w[i]), bf16hi(w[i]))
                                         : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
            amax = max(amax, max(__float_as_uint(y.x) & 0x7fffffffu, __float_as_uint(y.y) & 0x7fffffffu));
          }
#pragma unroll
          for (int off = 4; off; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
          const bool finite_row = amax < 0x7f800000u;
          const int e = q8_exponent(finite_row ? amax : 0, -126);
          if ((lane & 7) == 0) {
            reinterpret_cast<uint32_t*>(smem + Lay::kQueryScale)[(row >> 7) * 128 + (row & 31) * 4 + (row >> 5 & 3)] =
                (e + 127) * 0x01010101u;
            // (Held above 0: -inf times a factor has to stay.)
            factor[row] = finite_row ? fmaxf(a.scale_log2, 0x1p-126f) : __int_as_float(0x7fffffff);
          }
          const float down = pow2f(-e);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= down;
          uint8_t* tile = smem + Lay::kQ + (row >> 7) * kTerms * kTerm + (row & 127) * 128 +
                          (((lane & 7) ^ (row & 7)) << 4);
#pragma unroll
          for (int term = 0; term < kTerms; ++term) {
            uint32_t code[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              code[i] = q8_pack4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
#pragma unroll
              for (int j = 0; j < 2; ++j) {  // what is left, exactly
                const uint32_t y = q8_unpack2(j ? code[i] >> 16 : code[i] & 0xffffu);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y));
                x[4 * i + 2 * j] -= f.x;
                x[4 * i + 2 * j + 1] -= f.y;
              }
            }
            *reinterpret_cast<uint4*>(tile + term * kTerm) = make_uint4(code[0], code[1], code[2], code[3]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      ok = all_of<kSoftmaxThreads>(1, ok);
      if (!ok || n == 0) break;  // every warp alike
      if (lane == 0) mbar_arrive(q_ready);
      const int row = (two ? t * kTile : 0) + rr;  // of the block
      const bool busy = __any_sync(0xffffffffu, row < rows);
      const float f = factor[row];
      // Which node the row is of, and what it sees.
      auto word_of = [&]() {
        uint64_t word = 0;
        if (row < rows) {
          word = __ldg(a.words + static_cast<int64_t>(plan.r) * a.N + static_cast<int>((plan.row0 + row) * a.over_G >> 16));
          const int nodes = plan.nodes;
          if (nodes < 64) word &= (1ull << nodes) - 1;
        }
        return word;
      };

      float m = -INFINITY, l = 0.f;
      int U = 0;
      const int jobs = two ? 2 * n : n;
#pragma unroll 1
      for (int i = 0; i < jobs; ++i) {
        const int st = g % Lay::kC, odd = two ? i & 1 : t;
        const uint32_t at = lanes + buffer * 64;
        ok = reached(scale_full + st, (g / Lay::kC) & 1);  // (before its scores)
        const int4 info = reinterpret_cast<const int4*>(smem + Lay::kInfo)[2 * st];
        const bool all_seen = info.y != 0;
        bool look = !all_seen || U != info.z || !__all_sync(0xffffffffu, m > -INFINITY);
        ok = ok && reached(s_full + buffer, parity);
        if (!ok) break;
        fence_after();
        if (busy) {
          uint32_t see[2];
          if (!all_seen) {
            // Which of the tokens the row sees: those there are, before the tree
            // or named by its word; of them the even or the odd ones.
            const uint64_t word = word_of();
            const int to_tree = plan.base - info.x;  // tokens of the tile before the first node (under 0: nodes before it)
            see[0] = see[1] = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int left = to_tree - 32 * w;  // the same of these 32 tokens
              uint32_t bits = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1;
              if (left <= 0 && left > -64) bits = static_cast<uint32_t>(word >> -left);
              if (left > 0 && left < 32) bits |= static_cast<uint32_t>(word) << left;
              bits &= reinterpret_cast<const uint32_t*>(smem + Lay::kInfo)[st * 8 + 4 + w];
              see[w >> 1] |= even_bits(bits >> odd) << (16 * (w & 1));
            }
          }
          float x[64];
          auto scores = [&]() {
            tmem_ld32(at, x);
            tmem_ld32(at + 32, x + 32);
            tmem_wait_ld();
            if (!all_seen) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (!(see[c >> 5] >> (c & 31) & 1)) x[c] = -INFINITY;
            }
          };
          // The weights are formed with the maximum as it is, without a look at
          // the tile's own: they are right unless one passes 2^15, which their
          // sum tells.  Then, and where there is no maximum yet or not all is
          // seen, the maximum comes first, and the outputs follow it.
          uint32_t w[32];
          float sum;
          for (;;) {
            scores();
            if (look) {
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 64; c += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j) mx[j] = fmax3(mx[j], x[c + 2 * j], x[c + 2 * j + 1]);
              const float to = fmaxf(fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * f, m);
              float alpha = m == -INFINITY ? 0.f : ex2(m - to);
              m = to;
              l *= alpha;
              // A row's U: the tile's, but no more than kReach above what the row sees.
              int to_U = info.z;
              if (!all_seen) {
                if ((see[0] | see[1]) == 0) {
                  to_U = U;
                } else if (info.w) {
                  int most = 0;
#pragma unroll 1
                  for (uint64_t left = see[0] | static_cast<uint64_t>(see[1]) << 32; left; left &= left - 1)
                    most = max(most, exps[st * kTile + odd * 64 + __ffsll(static_cast<long long>(left)) - 1]);
                  to_U = max(U, min(to_U, most + kReach));
                }
              }
              alpha *= pow2_held(U - to_U);
              U = to_U;
              if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                // (The last job's product may still run: only that of the one before
                // was issued ahead of these scores.)
                ok = last_done();
                fence_after();
#pragma unroll 1
                for (int d = 0; d < 128; d += 16) {
                  float o[16];
                  tmem_ld16(o_at + t * 128 + d, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] *= alpha;
                  tmem_st16(o_at + t * 128 + d, reinterpret_cast<const uint32_t*>(o));
                }
              }
            }
            const float off = kWeight - finite_or_0(m);
            const uint64_t f2 = f2pack(f, f), off2 = f2pack(off, off);
            uint64_t sums[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float* y = x + c;
              f2unpack(ffma2(f2pack(y[0], y[1]), f2, off2), y[0], y[1]);
              y[0] = ex2(y[0]);
              y[1] = ex2(y[1]);
              sums[c >> 1 & 1] = fadd2(sums[c >> 1 & 1], f2pack(y[0], y[1]));
              w[c >> 1] = pack_f16x2(y[0], y[1]);
            }
            sum = f2sum(fadd2(sums[0], sums[1]));
            if (look || __all_sync(0xffffffffu, sum <= kMostSum)) break;
            look = true;
          }
          if (!ok) break;
          l += sum;
          tmem_st32(at, w);
          tmem_wait_st();
          if (info.w) {
            // A wide tile: 2^(min(the tile's U, e + kReach) - the row's U), at most 1 where
            // the row sees the token.
#pragma unroll 1
            for (int c = 0; c < 32; c += 16) {
              float o[16];
              tmem_ld16(at + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint8_t* e = exps + st * kTile + odd * 64 + 2 * (c + j);
                const uint32_t f2 = pow2h(min(min(info.z, e[0] + kReach) - U, 0)) |
                                    static_cast<uint32_t>(pow2h(min(min(info.z, e[1] + kReach) - U, 0))) << 16;
                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&o[j]), *reinterpret_cast<const __half2*>(&f2));
                o[j] = *reinterpret_cast<const float*>(&y);
              }
              tmem_st16(at + c, reinterpret_cast<const uint32_t*>(o));
            }
            tmem_wait_st();
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + buffer);
        parity ^= buffer > 0;
        buffer = buffer == 0 ? 2 : buffer - 1;
        g += !two || odd;
      }
      if (ok) ok = last_done();
      stat[t * kTile + rr] = make_float4(m, l, __int_as_float(U), 0.f);
      fence_before();
      ok = all_of<kSoftmaxThreads>(1, ok);
      if (!ok) break;
      fence_after();

      // The rows' outputs, averages in units of 2^8: of this stream's row, or of
      // half the dims of both streams' shares of it.
      if (busy) {
        const bool both = !two;
        const float4 s0 = stat[(two ? t : 0) * kTile + rr];
        const float4 s1 = both ? stat[kTile + rr] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        const float mx = fmaxf(s0.x, s1.x);
        float c0 = scale_of(s0.x, mx), c1 = scale_of(s1.x, mx);
        const float sum = s0.y * c0 + s1.y * c1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        c0 *= inv;
        c1 *= inv;
        const float p0 = pow2_held(__float_as_int(s0.z) - 127 - kValueUp - 8);
        const float p1 = pow2_held(__float_as_int(s1.z) - 127 - kValueUp - 8);
        const int ring = (g - 1) % (Lay::kC + 1);
        const int4 flags = reinterpret_cast<const int4*>(smem + Lay::kNanFlag)[ring];
        const bool some_nan = (flags.x | flags.y | flags.z | flags.w) != 0;
        const uint64_t* nan = reinterpret_cast<const uint64_t*>(smem + Lay::kNan) + ring * kHeadDim;
        const uint64_t word = some_nan ? word_of() : 0;
        const bool whole = plan.whole;
        const int64_t share = plan.share + row;
        const int at = plan.row0 + row, node = static_cast<int>(at * a.over_G >> 16);
        const int64_t to_row = plan.query + (node * a.Hq + at - node * a.G) * static_cast<int64_t>(kHeadDim);
        if (!whole && row < rows && (two || t == 0)) a.stat[share] = make_float2(mx, sum);
#pragma unroll 1
        for (int d = two ? 0 : t * 64; d < (two ? 128 : t * 64 + 64); d += 16) {
          float o[16], o1[16];
          tmem_ld16(o_at + (two ? t * 128 : 0) + d, o);
          if (both) tmem_ld16(o_at + 128 + d, o1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j] = o[j] * c0 * p0;
            if (both) o[j] += o1[j] * c1 * p1;
          }
          if (some_nan) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (nan[d + j] & word) o[j] = __int_as_float(0x7fffffff);
          }
          if (row < rows) {
            if (!whole || a.out_fp32) {
              float* to = whole ? static_cast<float*>(a.out) + to_row : a.part + share * kHeadDim;
              const float up = whole ? 256.f : 1.f;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                store4_finite(to + d + 4 * j,
                              make_float4(o[4 * j] * up, o[4 * j + 1] * up, o[4 * j + 2] * up, o[4 * j + 3] * up));
            } else {
              T* to = static_cast<T*>(a.out) + to_row + d;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  w[b] = pack2_finite(to, o[8 * j + 2 * b] * 256.f, o[8 * j + 2 * b + 1] * 256.f);
                *reinterpret_cast<uint4*>(to + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        fence_before();
      }
      plan_read(k);
    }
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout);
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kScoreWarp) tmem_free(0, 512);
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
