// prefix.cu -- attention of a whole batch over the prefix it shares.
//
// The queries of all requests that read one KV head are the rows of one
// matrix (row (r * S + s) * G + gi), so the prefix is read once, and with
// many requests the work is two matrix products: 4 * 128 operations a row and
// token against 512 bytes a token, bound by the tensor cores from about 300
// rows on (below, by HBM).
//
// One CTA per 128 or 256 rows, KV head and share of the prefix: warps 0..7
// are the softmax of two tiles of 128 rows, one thread a row; warp 8 brings
// tiles of 128 tokens (TMA, 128-byte swizzle, a ring of four 32 KiB stages
// that holds keys and values in turn); one thread of warp 9 issues the
// products (tcgen05, M = N = 128).  Scores and outputs stay in tensor memory
// (512 columns: two tiles of 128 + 128); the weights go back there as bf16
// over the scores they came from and are the second product's A operand.
// While one tile's weights are formed the other's products run.  The running
// maximum is only moved when a row's grows by more than 2^8, so the outputs
// are seldom rescaled.
//
// Each share writes its rows' unnormalised outputs, maxima and sums, as the
// attention over the requests' own pages does.  Three launches that overlap:
// this one; the pages' share, bound by latency and memory, on the SMs that
// are idle or get free; the join, a warp a row.
#include "q8.cuh"
#include "q8.h"
#include "tcgen05.cuh"

namespace oasis {
namespace {

constexpr int kTile = 128;                                 // rows, tokens
constexpr int kHalfTile = kTile * 128;                     // 64 dims of a tile: 16 KiB
constexpr int kStageBytes = 2 * kHalfTile;                 // 32 KiB
constexpr int kRingStages = 4;
constexpr float kLazy = 8.f;                               // growth of a maximum let pass (log2)

template <int kTiles>
struct PrefixLayout {
  static constexpr int kThreads = kTiles * 128 + 64;
  static constexpr int kQ = 0;
  static constexpr int kRing = kTiles * kStageBytes;
  static constexpr int kBars = kRing + kRingStages * kStageBytes;
  static constexpr int kRows = kBars + 256;                // where a row's query begins
  static constexpr int kBytes = kRows + kTiles * kTile * 4 + 1024;  // + alignment
  static constexpr int kColumns = kTiles * 256;            // tensor memory
};

// bf16 x bf16 -> fp32, M = N = 128; B's columns are contiguous in kInstrBt.
constexpr uint32_t kInstr = kMmaF32 | kMmaBf16A | kMmaBf16B | mma_shape(128, 128);
constexpr uint32_t kInstrBt = kInstr | kMmaTransposeB;

// 64 dims of 8 blocks' keys (z = 0) or values (z = 1).
__device__ __forceinline__ void load_blocks(void* dst, const CUtensorMap* map, int x, int z, int block,
                                            int head, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(z), "r"(block), "r"(head),
      "r"(smem_u32(bar))
      : "memory");
}

template <int kTiles>
__global__ void __launch_bounds__(PrefixLayout<kTiles>::kThreads, 1)
    prefix_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap map) {
  using Lay = PrefixLayout<kTiles>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBars);
  uint64_t* full = bars;                       // [4] a stage has landed
  uint64_t* empty = bars + kRingStages;        // [4] its products are done
  uint64_t* s_full = bars + 2 * kRingStages;   // [2] scores of a tile
  uint64_t* p_half = s_full + 2;               // [2] its first 64 tokens' weights (four warps)
  uint64_t* p_full = p_half + 2;               // [2] all its weights
  uint64_t* o_done = p_full + 2;               // [2] its outputs
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_tile = blockIdx.x % a.row_tiles;
  const int h = (blockIdx.x / a.row_tiles) % a.Hkv;
  const int split = blockIdx.x / a.row_tiles / a.Hkv;
  const int per_request = a.S * a.G;
  const int rows = a.R * per_request;
  const int row0 = row_tile * kTiles * kTile;
  const int all_tiles = (a.prefix_len + kTile - 1) / kTile;
  const int tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * split / a.splits);
  const int n = static_cast<int>(static_cast<int64_t>(all_tiles) * (split + 1) / a.splits) - tile0;

  // The loading thread sets the barriers up and starts at once: the first
  // tiles come in while the queries are placed.  Stage 2 i is tile i's keys,
  // 2 i + 1 its values.
  const bool loader = threadIdx.x == kTiles * 128;
  auto load = [&](int j) {
    const int st = j % kRingStages;
    uint8_t* dst = smem + Lay::kRing + st * kStageBytes;
    const int block = (tile0 + (j >> 1)) * (kTile / kBlock);
    mbar_arrive_expect_tx(&full[st], kStageBytes);
    load_blocks(dst, &map, 0, j & 1, block, h, &full[st]);
    load_blocks(dst + kHalfTile, &map, 64, j & 1, block, h, &full[st]);
  };
  int loaded = 0;
  previous_done();
  // (Not before: a kernel ahead that takes tensor memory after it has let its
  // dependents begin would wait for this one's.)
  if (warp == kTiles * 4 + 1) tmem_alloc(tmem_s, Lay::kColumns);
  next_may_begin();  // the pages' share takes the SMs this leaves idle
  if (loader) {
    prefetch_tensormap(&map);
    for (int i = 0; i < 2 * kRingStages + 2; ++i) mbar_init(&bars[i], 1);  // to s_full
    for (int i = 0; i < 4; ++i) mbar_init(&p_half[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&o_done[i], 1);
    mbar_init(drain, 1);
    fence_barrier_init();
    for (; loaded < 2 * n && loaded < kRingStages; ++loaded) load(loaded);
  }
  // The query rows: where each begins (one division a row), then half a warp a
  // row, all of a thread's loads in flight, to where the swizzle has them.
  int* begin = reinterpret_cast<int*>(smem + Lay::kRows);
  for (int rr = threadIdx.x; rr < kTiles * kTile; rr += Lay::kThreads) {
    const int row = row0 + rr, r = row / per_request, c = row - r * per_request, s = c / a.G;
    begin[rr] = row < rows ? (s * a.R + r) * a.Hq + h * a.G + c - s * a.G : -1;
  }
  __syncthreads();
  {
    constexpr int kStep = Lay::kThreads / 16, kLoads = (kTiles * kTile + kStep - 1) / kStep;
    const int ch = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    uint4 v[kLoads];
#pragma unroll
    for (int b = 0; b < kLoads; ++b) {
      const int rr = r0 + b * kStep;
      const int at = rr < kTiles * kTile ? begin[rr] : -1;
      v[b] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) v[b] = static_cast<const uint4*>(a.q)[static_cast<int64_t>(at) * 16 + ch];
    }
#pragma unroll
    for (int b = 0; b < kLoads; ++b) {
      const int rr = r0 + b * kStep;
      if (rr < kTiles * kTile) {
        uint8_t* tile = smem + Lay::kQ + (rr / kTile) * kStageBytes + (ch >> 3) * kHalfTile;
        *reinterpret_cast<uint4*>(tile + (rr % kTile) * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v[b];
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_s, 0);

  bool ok = true;
  if (warp == kTiles * 4) {
    // ---- loads
    if (loader) {
      for (; loaded < 2 * n && ok; ++loaded) {
        const int st = loaded % kRingStages;
        ok = mbar_wait(&empty[st], (loaded / kRingStages - 1) & 1, a.wait_limit);
        if (!ok) break;
        load(loaded);
      }
      // No copy may outlive the CTA, whatever the other warps met.
      for (int j = max(loaded - kRingStages, 0); j < loaded; ++j)
        (void)mbar_wait(&full[j % kRingStages], (j / kRingStages) & 1);
    }
  } else if (warp == kTiles * 4 + 1) {
    // ---- products
    const uint32_t lead = elected();
    auto reached = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_limit)) != 0;
    };
    auto landed = [&](int j) { return reached(&full[j % kRingStages], (j / kRingStages) & 1); };
    const uint64_t q_desc = smem_desc(smem_u32(smem + Lay::kQ), 16);
    const uint64_t k_desc = smem_desc(smem_u32(smem + Lay::kRing), 16);
    const uint64_t v_desc = smem_desc(smem_u32(smem + Lay::kRing), kHalfTile);
    constexpr uint64_t kStep = kStageBytes >> 4;  // between tiles and stages, in a descriptor
    auto scores = [&](int t, int i) {
      const uint64_t q = q_desc + t * kStep, k = k_desc + (2 * i) % kRingStages * kStep;
#pragma unroll
      for (int s = 0; s < 8; ++s) {  // 16 dims a step
        constexpr int kHalf = kHalfTile >> 4;
        const uint32_t off = (s >> 2) * kHalf + (s & 3) * 2;
        mma_ss<kInstr>(tmem + t * 128, q + off, k + off, s > 0, lead);
      }
      mma_commit(&s_full[t], lead);
      if (t == kTiles - 1) mma_commit(&empty[(2 * i) % kRingStages], lead);
    };
    ok = landed(0);
    if (ok) {
      fence_after();
#pragma unroll
      for (int t = 0; t < kTiles; ++t) scores(t, 0);
    }
    for (int i = 0; i < n && ok; ++i) {
      ok = landed(2 * i + 1);
      const uint64_t v = v_desc + (2 * i + 1) % kRingStages * kStep;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && reached(half ? &p_full[t] : &p_half[t], i & 1);
          if (!ok) break;
          fence_after();
#pragma unroll
          for (int s = half * 4; s < half * 4 + 4; ++s)  // 16 tokens a step
            mma_ts<kInstrBt>(tmem + kTiles * 128 + t * 128, tmem + t * 128 + s * 8, v + s * (16 * 128 >> 4),
                             i > 0 || s > 0, lead);
        }
        if (!ok) break;
        mma_commit(&o_done[t], lead);
        if (t == kTiles - 1) mma_commit(&empty[(2 * i + 1) % kRingStages], lead);
        if (i + 1 < n) {
          if (t == 0) ok = landed(2 * i + 2);
          if (!ok) break;
          scores(t, i + 1);
        }
      }
    }
    // No product may outlive its operands and accumulators, either.
    mma_commit(drain, lead);
    (void)mbar_wait(drain, 0);
  } else {
    // ---- softmax of row `lane` of this warp's quarter of tile t
    const int t = warp >> 2;
    const int rr = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + kTiles * 128 + t * 128;
    const float sc = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], i & 1, a.wait_limit));
      if (!ok) break;
      fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, s + c * 32);
      tmem_wait_ld();
      const int valid = a.prefix_len - (tile0 + i) * kTile;
      if (valid < kTile) {
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c >= valid) s[c] = -INFINITY;
        if (t == 0) {
          // Values past the end may be anything, and 0 * NaN is NaN: clear them.
          ok = __all_sync(0xffffffffu, mbar_wait(&full[(2 * i + 1) % kRingStages],
                                                 ((2 * i + 1) / kRingStages) & 1, a.wait_limit));
          if (!ok) break;
          if (rr >= valid) {
            uint8_t* at = smem + Lay::kRing + ((2 * i + 1) % kRingStages) * kStageBytes + rr * 128;
#pragma unroll
            for (int c = 0; c < 16; ++c)
              *reinterpret_cast<uint4*>(at + (c >> 3) * kHalfTile + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 124; c += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmax3(mx[j], s[c + 2 * j], s[c + 2 * j + 1]);
      mx[0] = fmax3(mx[0], s[124], s[125]);
      mx[1] = fmax3(mx[1], s[126], s[127]);
      const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sc;
      float alpha = 1.f;
      if (top > m + kLazy || m == -INFINITY) {
        const float to = fmaxf(top, m);
        alpha = m == -INFINITY ? 0.f : ex2(m - to);
        m = to;
      }
      if (__any_sync(0xffffffffu, alpha != 1.f) && i > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (i - 1) & 1, a.wait_limit));
        if (!ok) break;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[32];
          tmem_ld32(o_at + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] *= alpha;
          tmem_st32(o_at + c * 32, reinterpret_cast<const uint32_t*>(o));
        }
      }
      l *= alpha;
      const float off = m == -INFINITY ? 0.f : -m;
      const uint64_t sc2 = f2pack(sc, sc), off2 = f2pack(off, off);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float p0, p1;
          f2unpack(ffma2(f2pack(s[c * 64 + 2 * j], s[c * 64 + 2 * j + 1]), sc2, off2), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          sum[j & 1] = fadd2(sum[j & 1], f2pack(p0, p1));
          w[j] = pack_bf16x2(p0, p1);
        }
        tmem_st32(s_at + c * 32, w);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c ? &p_full[t] : &p_half[t]);  // one a warp: arrivals queue
      }
      l += f2sum(fadd2(sum[0], sum[1]));
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t], (n - 1) & 1, a.wait_limit));
    if (ok) {
      fence_after();
      const int row = row0 + t * kTile + rr;
      const int64_t at = (static_cast<int64_t>(split) * a.Hkv + h) * rows + row;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld32(o_at + c * 32, o);
        tmem_wait_ld();
        if (row < rows) {
          float* dst = a.part + at * kHeadDim + c * 32;
#pragma unroll
          for (int j = 0; j < 4; ++j) store8(dst + j * 8, o + j * 8);
        }
      }
      if (row < rows) a.stat[at] = make_float2(m, l);
    }
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout);
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kTiles * 4 + 1) tmem_free(tmem, Lay::kColumns);
}

// The shares' rows joined: a warp a row.
template <typename T>
__global__ void __launch_bounds__(128) join_kernel(const PrefixArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int per_request = a.S * a.G;
  const int64_t rows = static_cast<int64_t>(a.Hkv) * a.R * per_request;
  if (row >= rows) return;
  const int c = static_cast<int>(row % per_request), s = c / a.G;
  const int64_t hr = row / per_request;
  const int h = static_cast<int>(hr / a.R), r = static_cast<int>(hr % a.R);
  T* out = static_cast<T*>(a.out) +
           ((static_cast<int64_t>(s) * a.R + r) * a.Hq + h * a.G + c - s * a.G) * kHeadDim + lane * 4;
  previous_done();
  next_may_begin();
  float sum;
  const float4 acc = join_shares(reinterpret_cast<const float4*>(a.part) + row * 32, a.stat + row, rows,
                                 a.splits + 1, lane, sum);
  store4(out, make_float4(acc.x / sum, acc.y / sum, acc.z / sum, acc.w / sum));
}

}  // namespace

PrefixShape prefix_shape(int R, int S, int G, int Hkv, int prefix_len) {
  PrefixShape p{};
  const int64_t rows = static_cast<int64_t>(R) * S * G;
  p.rows = rows;
  p.tiles = rows > kTile ? 2 : 1;
  p.row_tiles = static_cast<int>((rows + p.tiles * kTile - 1) / (p.tiles * kTile));
  const int64_t units = static_cast<int64_t>(p.row_tiles) * Hkv;
  const int all = (prefix_len + kTile - 1) / kTile;
  // As many shares as give every SM a CTA, but no more than shorten the
  // longest: the SMs left over are the pages' share's.
  int64_t splits = units > 0 ? 152 / units : 1;
  if (splits > all) splits = all;
  if (splits < 1) splits = 1;
  if (all > 0) {
    const int64_t longest = (all + splits - 1) / splits;
    splits = (all + longest - 1) / longest;
  }
  p.splits = static_cast<int>(splits);
  const int64_t vectors = (p.splits + 1) * static_cast<int64_t>(Hkv) * rows;
  p.part_bytes = static_cast<size_t>(vectors) * kHeadDim * 4;
  p.bytes = p.part_bytes + static_cast<size_t>(vectors) * 8;
  return p;
}

cudaError_t launch_prefix(const PrefixArgs& a, int tiles, const CUtensorMap& map, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.row_tiles) * a.Hkv * a.splits;
  return tiles == 2
             ? launch_early(prefix_kernel<2>, grid, PrefixLayout<2>::kThreads, PrefixLayout<2>::kBytes, s, 0, a, map)
             : launch_early(prefix_kernel<1>, grid, PrefixLayout<1>::kThreads, PrefixLayout<1>::kBytes, s, 0, a, map);
}

cudaError_t launch_join(const PrefixArgs& a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.Hkv) * a.R * a.S * a.G;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  return launch_early(a.out_fp32 ? join_kernel<float> : join_kernel<__nv_bfloat16>, grid, 128, 0, s, 0, a);
}

cudaError_t preload_prefix_kernels() {
  cudaError_t e = cudaFuncSetAttribute(prefix_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PrefixLayout<1>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prefix_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PrefixLayout<2>::kBytes);
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, join_kernel<float>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, join_kernel<__nv_bfloat16>);
  return e;
}

}  // namespace oasis
