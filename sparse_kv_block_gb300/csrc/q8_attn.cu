// q8_attn.cu -- attention of a request's one to four queries over its 8-bit
// pages (memory bound: 258 bytes a token and KV head, read once for all the
// queries of that head).
//
// One CTA, or one cluster of CTAs where there are few (request, KV head)
// pairs, per pair; or, given scratch, as many CTAs a request as its length
// asks for, joined by a second launch.  Every warp takes groups of 64 tokens
// (four units) through a ring of its own, two bulk copies per unit (its keys;
// its values and exponents).  The two products run on mma.sync m16n8k16 with
// tokens, then dims, as M and up to 16 query columns (query s, head gi: column
// s * G + gi) as N.  Codes become fp16 exactly;
// which token stands for which matrix row is chosen so that a lane's 16-byte
// loads are whole fragments and the transposed weights (movmatrix) meet the
// value codes as they lie:
//   S step i (0..3), row g:      token 4 i + (g & 1) of unit g / 2
//                    row g + 8:  token 4 i + 2 + (g & 1) of unit g / 2
//   so a lane of the transposed weights holds tokens 4 i .. 4 i + 3 of unit t,
//   which is word i of a dim's 16 codes.
//
// Powers of two stay out of the roundings: a query row is scaled by its own
// (its largest value at 2^13, so bf16 keeps all bits in fp16), a key's is
// multiplied into the score, and a value's is added to the score's logarithm:
// with x the score (base 2) and e the value's exponent the weight is
//   w = 2^(x + e - M + 14),  M the running maximum of x + e,
// the output is 2^(M - 14 - L) sum w code / sum 2^(x - L), L the running
// maximum of x.  The largest w is 2^14: fp16 keeps all bits of weights down to
// 2^-28 of it, and rounds those below by at most 2^-39 of it.  (One sum of
// w 2^-e would lose tokens whose values are 2^-140 of others', rows of zeros
// among them; the second power costs nothing here.)
#include "q8.cuh"
#include "q8.h"

namespace oasis {
namespace {

constexpr int kGroupUnits = 4;
constexpr int kGroupTokens = kGroupUnits * kBlock;           // 64
constexpr int kGroupBytes = kGroupUnits * kQ8UnitBytes;      // 16512
constexpr float kWeightLog2 = 14.f;
// Sums of weighted values are kept in units of 2^22 once in the sum's units: a
// request has up to 2^21 tokens of up to 448 * 2^120, and 2^21 * 2^129 / 2^22
// is in fp32's range, as the output is, an average.  (A power of two, so no
// bits change.)
constexpr float kSumDown = 0x1p-22f, kSumUp = 0x1p22f;
constexpr int kSplitRequests = 128;  // requests of a batch that can be cut into parts
constexpr int kLeastGroups = 4;      // of a part's warp

template <int W, int kNT>
struct Layout {
  static constexpr int kCols = 8 * kNT;
  static constexpr int kRing = W * kGroupBytes;              // one group a warp
  static constexpr int kPartial = kCols * kHeadDim * 4;      // one warp's partial output
  static_assert(W * kPartial + (W > 1 ? kPartial + 3 * kCols * 4 : 0) <= kRing, "the partial outputs reuse the ring");
  static constexpr int kMerged = W * kPartial;               // (W > 1) the CTA's [kCols][d], [kCols] M, L, sums
  static constexpr int kBars = kRing;                        // keys' and values' barrier a warp
  static constexpr int kValid = kBars + W * 16;              // int4 for even and odd groups
  static constexpr int kStat = kValid + W * 32;              // [W][kCols] M, L, sums
  static constexpr int kFactor = kStat + 3 * W * kCols * 4;  // of a column's scores
  static constexpr int kQuery = kFactor + kCols * 4;         // [kNT][8][32 lanes] fragments
  static constexpr int kBytes = kQuery + kNT * 8 * 32 * 8;
};

// 16 bytes of shared memory.  (An ordinary load: the compiler may move it,
// but not across the barrier waits, which clobber memory.)
__device__ __forceinline__ uint4 lds128(const uint8_t* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Four codes -> two half pairs.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// The output of sums in units of 2^22; what a query sees nothing of is 0.
__device__ __forceinline__ float4 average(const float4& acc, float sum) {
  if (sum == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(acc.x / sum * kSumUp, acc.y / sum * kSumUp, acc.z / sum * kSumUp, acc.w / sum * kSumUp);
}

// Which part of which request a CTA of column `col` takes.  A part is up to W *
// m groups, m the least number with which no more than a.columns parts come
// out; every warp finds it from all lengths (up to 128, four a lane).
template <int W>
__device__ __forceinline__ bool part_of(const Q8AttnArgs& a, int col, int warp, int lane, int& r, int& rank,
                                        int& parts, int& len) {
  int lens[kSplitRequests / 32], groups[kSplitRequests / 32];
  int total = 0, longest = 0;
#pragma unroll
  for (int j = 0; j < kSplitRequests / 32; ++j)
    lens[j] = j * 32 + lane < a.R ? __ldcg(a.len + j * 32 + lane) : 0;
#pragma unroll
  for (int j = 0; j < kSplitRequests / 32; ++j) {
    groups[j] = (min(max(lens[j], 0), a.max_blocks * kBlock) + kGroupTokens - 1) / kGroupTokens;
    total += groups[j];
    longest = max(longest, groups[j]);
  }
  total = __reduce_add_sync(0xffffffffu, total);
  longest = __reduce_max_sync(0xffffffffu, longest);
  int lo = max((total + W * a.columns - 1) / (W * a.columns), kLeastGroups);
  int hi = max((longest + W - 1) / W, lo);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int n = 0;
#pragma unroll
    for (int j = 0; j < kSplitRequests / 32; ++j) n += (groups[j] + W * mid - 1) / (W * mid);
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, n)) <= a.columns) hi = mid;
    else lo = mid + 1;
  }
  bool found = false;
  int before = 0;
#pragma unroll
  for (int j = 0; j < kSplitRequests / 32; ++j) {
    if (j * 32 >= a.R) break;
    const int n = (groups[j] + W * lo - 1) / (W * lo);
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const int from = before + incl - n;
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0 && j * 32 + lane <= a.R) a.plan[j * 32 + lane] = from;
    before += __shfl_sync(0xffffffffu, incl, 31);
    const unsigned here = __ballot_sync(0xffffffffu, col >= from && col < from + n);
    if (here) {
      const int src = __ffs(here) - 1;
      found = true;
      r = j * 32 + src;
      rank = col - __shfl_sync(0xffffffffu, from, src);
      parts = __shfl_sync(0xffffffffu, n, src);
      len = __shfl_sync(0xffffffffu, lens[j], src);
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0 && lane == 0) a.plan[a.R] = before;
  return found;
}

template <typename T, int W, int kNT>
__global__ void __launch_bounds__(W * 32, (kNT == 1 ? 12 : 8) / W)
    attn_kernel(const Q8AttnArgs a, int most, int each) {
  using Lay = Layout<W, kNT>;
  constexpr int kCols = Lay::kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  // A prefix's share of pages needs nothing of the launch ahead, the prefix's
  // own, which has itself waited for what came before.  (This grid has not:
  // it reads past L1, which may hold what was there before.)
  const bool beside = a.part && !a.plan;
  if (!beside) previous_done();
  next_may_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int r, h, rank, parts = 0, len;
  if (a.plan) {
    h = static_cast<int>(blockIdx.x % a.Hkv);
    if (!part_of<W>(a, static_cast<int>(blockIdx.x / a.Hkv), warp, lane, r, rank, parts, len)) return;
  } else {
    const int pair = blockIdx.x / most;
    rank = static_cast<int>(most == 1 ? 0u : cluster_rank());
    r = pair / a.Hkv;
    h = pair - r * a.Hkv;
    len = __ldcg(a.len + r);
  }
  const int col0 = blockIdx.y * kCols;                 // first column of this CTA
  const int cols = min(a.S * a.G - col0, kCols);

  uint8_t* ring = smem + warp * kGroupBytes;
  uint64_t* key_bar = reinterpret_cast<uint64_t*>(smem + Lay::kBars) + warp * 2;
  uint64_t* value_bar = key_bar + 1;
  int* valid_s = reinterpret_cast<int*>(smem + Lay::kValid) + warp * 8;
  if (lane == 0) {
    mbar_init(key_bar, 1);
    mbar_init(value_bar, 1);
    fence_barrier_init();
  }
  __syncwarp();

  // Loads that need nothing else, in flight together: the length, the first
  // group's pages (rows of the table are readable throughout) and the queries.
  const int first = rank * W + warp;
  const int32_t* row = a.table + static_cast<int64_t>(r) * a.max_blocks;
  int step = 0;  // groups between a warp's, once the length is known
  auto page_of = [&](int k) {
    const int64_t b = (first + static_cast<int64_t>(k) * step) * kGroupUnits + lane;
    return lane < kGroupUnits && b < a.max_blocks ? __ldcg(row + b) : -1;
  };
  int page = page_of(0);
  uint4 qv[4];  // warp nt < kNT: of column 8 nt + g, dims 64 (j / 2) + 16 t + 8 (j % 2) .. + 7
  {
    const int c = col0 + warp * 8 + g;
    if (warp < kNT && warp * 8 + g < cols) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const T*>(a.q) +
          ((static_cast<int64_t>(c / a.G) * a.R + r) * a.Hq + h * a.G + c % a.G) * kHeadDim);
#pragma unroll
      for (int j = 0; j < 4; ++j) qv[j] = __ldcg(src + (j >> 1) * 8 + t * 2 + (j & 1));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) qv[j] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  len = max(len, 0);
  if (len > a.max_blocks * kBlock) {
    if (threadIdx.x == 0) raise_error(a.err, kErrBadBlock);
    len = a.max_blocks * kBlock;
  }
  const int groups = (len + kGroupTokens - 1) / kGroupTokens;
  // A request takes as many of the cluster's CTAs as have `each` groups a warp
  // (one for a short one); the others leave at once, though their room is kept
  // until the whole cluster has ended.
  const int cluster = parts ? parts : min(most, max((groups + W * each - 1) / (W * each), 1));
  if (rank >= cluster) {
    if (beside && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) previous_done();  // see the end
    return;
  }
  step = cluster * W;
  const int count = groups > first ? (groups - first + step - 1) / step : 0;

  // Lanes 0..3 fetch a group's pages (the table's entries a turn ahead) and
  // issue its copies: the keys as soon as the last group's have been used, so
  // that they come in beside its second half; then the values and exponents.
  const uint8_t* src = nullptr;  // this lane's unit of the group issued last, if it has one
  auto issue_keys = [&](int k) {
    const int b = (first + k * step) * kGroupUnits + lane;
    const bool inside = lane < kGroupUnits && b * kBlock < len;
    const bool ok = inside && page >= 0 && page < a.num_pages;
    if (inside && !ok) raise_error(a.err, kErrBadBlock);
    src = ok ? a.pages + (static_cast<int64_t>(page) * a.Hkv + h) * kQ8UnitBytes : nullptr;
    const unsigned oks = __ballot_sync(0xffffffffu, ok);
    if (lane < kGroupUnits) valid_s[(k & 1) * 4 + lane] = ok ? min(len - b * kBlock, kBlock) : 0;
    if (lane == 0) mbar_arrive_expect_tx(key_bar, __popc(oks) * kQ8HalfBytes);
    __syncwarp();
    if (ok) bulk_g2s(ring + lane * kQ8UnitBytes, src, kQ8HalfBytes, key_bar);
    page = page_of(k + 1);
  };
  auto issue_values = [&]() {
    const unsigned oks = __ballot_sync(0xffffffffu, src != nullptr);
    constexpr int kRest = kQ8UnitBytes - kQ8HalfBytes;
    if (lane == 0) mbar_arrive_expect_tx(value_bar, __popc(oks) * kRest);
    __syncwarp();
    if (src) bulk_g2s(ring + lane * kQ8UnitBytes + kQ8HalfBytes, src + kQ8HalfBytes, kRest, value_bar);
  };
  if (count > 0) {
    issue_keys(0);
    issue_values();
  }

  // Query columns as B fragments, in shared memory (registers for them would
  // cost a third of the CTAs an SM holds): warp nt makes those of tile nt.
  // Step (j, w) of the contraction covers, for lane t, dims 64 j + 16 t + 4 w
  // .. + 3.
  float* factor = reinterpret_cast<float*>(smem + Lay::kFactor);
  uint2* query = reinterpret_cast<uint2*>(smem + Lay::kQuery);
  if (warp < kNT) {
    float x[32];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      T e[8];
      memcpy(e, &qv[j], 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[j * 8 + i] = as_float(e[i]);
        const float b = fabsf(x[j * 8 + i]);
        if (b < INFINITY) amax = fmaxf(amax, b);
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 13, -100);
    const float down = pow2f(-e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      query[(warp * 8 + i) * 32 + lane] = make_uint2(pack_f16x2(x[4 * i] * down, x[4 * i + 1] * down),
                                                     pack_f16x2(x[4 * i + 2] * down, x[4 * i + 3] * down));
    if (t == 0) factor[warp * 8 + g] = a.scale_log2 * pow2f(e);
  }
  __syncthreads();
  float f0[kNT], f1[kNT];        // score factors of columns 2 t, 2 t + 1
  int lim0[kNT], lim1[kNT];      // tokens those columns see
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    f0[nt] = factor[nt * 8 + 2 * t];
    f1[nt] = factor[nt * 8 + 2 * t + 1];
    const int c0 = col0 + nt * 8 + 2 * t;
    lim0[nt] = a.causal ? len - (a.S - 1 - c0 / a.G) : len;
    lim1[nt] = a.causal ? len - (a.S - 1 - (c0 + 1) / a.G) : len;
  }
  const int all_see = a.causal ? len - (a.S - 1) : len;  // tokens every query sees

  float o[kNT][8][4];
  // Columns 2 t, 2 t + 1: M (the warp's), L and the sum (this lane's tokens).
  float m0[kNT], m1[kNT], ml0[kNT], ml1[kNT], l0[kNT], l1[kNT];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    m0[nt] = m1[nt] = ml0[nt] = ml1[nt] = -INFINITY;
    l0[nt] = l1[nt] = 0.f;
  }

  const uint32_t key_lane = (g >> 1) * kQ8UnitBytes + (g & 1) * kHeadDim + t * 16;
  const uint32_t value_lane = t * kQ8UnitBytes + kQ8HalfBytes + g * kBlock;
  const int odd = (g & 1) * 8;  // shift of this lane's even / odd token in a word
  int k = 0;
  bool keys_late = false, values_late = false;
  const uint8_t* sb = ring;
  for (; k < count; ++k) {
    if (!__all_sync(0xffffffffu, mbar_wait(key_bar, k & 1, a.wait_limit))) {
      keys_late = true;
      break;
    }
    const int base = (first + k * step) * kGroupTokens;  // position of the group's first token
    const int4 valid = *reinterpret_cast<const int4*>(valid_s + (k & 1) * 4);
    const bool whole = min(min(valid.x, valid.y), min(valid.z, valid.w)) == kBlock &&
                       base + kGroupTokens <= all_see;

    // Scores: S^T (64 tokens x columns), four steps of 16 tokens.  The steps go
    // side by side, so that neighbouring products do not wait on one another.
    float s[kNT][4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) s[nt][i][0] = s[nt][i][1] = s[nt][i][2] = s[nt][i][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* at = sb + key_lane + ((j ^ (g & 1)) << 6) + i * 4 * kHeadDim;
        lo[i] = lds128(at);
        hi[i] = lds128(at + 2 * kHeadDim);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint2 q[kNT];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) q[nt] = query[(nt * 8 + j * 4 + w) * 32 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          unpack4(word(lo[i], w), a0, a2);
          unpack4(word(hi[i], w), a1, a3);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma_f16_16816(s[nt][i], a0, a1, a2, a3, q[nt].x, q[nt].y);
        }
      }
    }

    __syncwarp();
    if (k + 1 < count) issue_keys(k + 1);
    if (!__all_sync(0xffffffffu, mbar_wait(value_bar, k & 1, a.wait_limit))) {
      values_late = true;
      break;
    }

    // x, masked, and the maximum of x + e; the tokens of rows g, g + 8 of step i are bytes odd, odd
    // + 2 of word i of unit g / 2's exponents.
    const uint8_t* ex = sb + (g >> 1) * kQ8UnitBytes + kQ8ExpOffset;
    const uint4 ke = lds128(ex), ve = lds128(ex + kBlock);
    const int mine = g < 4 ? (g < 2 ? valid.x : valid.y) : (g < 6 ? valid.z : valid.w);
    const int pos = base + (g >> 1) * kBlock + (g & 1);
    float t0[kNT], t1[kNT], u0[kNT], u1[kNT], vl[4][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      t0[nt] = t1[nt] = -INFINITY;
      u0[nt] = ml0[nt];
      u1[nt] = ml1[nt];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int up = 0; up < 2; ++up) {  // rows g, g + 8
        const uint32_t kb = (word(ke, i) >> (odd + 16 * up)) & 255u, vb = (word(ve, i) >> (odd + 16 * up)) & 255u;
        const float ks = __uint_as_float(kb << 23);
        vl[i][up] = static_cast<float>(static_cast<int>(vb) - 127);
        const int tok = 4 * i + 2 * up;
        const bool in = tok + (g & 1) < mine;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float& x0 = s[nt][i][2 * up];
          float& x1 = s[nt][i][2 * up + 1];
          x0 *= ks * f0[nt];
          x1 *= ks * f1[nt];
          if (!whole) {
            if (!in || pos + tok >= lim0[nt]) x0 = -INFINITY;
            if (!in || pos + tok >= lim1[nt]) x1 = -INFINITY;
          }
          u0[nt] = fmaxf(u0[nt], x0);
          u1[nt] = fmaxf(u1[nt], x1);
          t0[nt] = fmaxf(t0[nt], x0 + vl[i][up]);
          t1[nt] = fmaxf(t1[nt], x1 + vl[i][up]);
        }
      }
    }

    uint32_t pb[kNT][4][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        t0[nt] = fmaxf(t0[nt], __shfl_xor_sync(0xffffffffu, t0[nt], off));
        t1[nt] = fmaxf(t1[nt], __shfl_xor_sync(0xffffffffu, t1[nt], off));
      }
      const float n0 = fmaxf(m0[nt], t0[nt]), n1 = fmaxf(m1[nt], t1[nt]);
      // What has seen nothing keeps a maximum of -inf; its weights are 2^-inf.
      const float b0 = finite_or_0(n0) - kWeightLog2, b1 = finite_or_0(n1) - kWeightLog2;
      const float c0 = finite_or_0(u0[nt]), c1 = finite_or_0(u1[nt]);
      const float al0 = ex2(m0[nt] - kWeightLog2 - b0), al1 = ex2(m1[nt] - kWeightLog2 - b1);
      l0[nt] *= ex2(ml0[nt] - c0);
      l1[nt] *= ex2(ml1[nt] - c1);
      m0[nt] = n0;
      m1[nt] = n1;
      ml0[nt] = u0[nt];
      ml1[nt] = u1[nt];
      if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[nt][mt][0] *= al0;
          o[nt][mt][1] *= al1;
          o[nt][mt][2] *= al0;
          o[nt][mt][3] *= al1;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float w[4];
#pragma unroll
        for (int up = 0; up < 2; ++up) {
          const float x0 = s[nt][i][2 * up], x1 = s[nt][i][2 * up + 1];
          w[2 * up] = ex2(x0 + vl[i][up] - b0);
          w[2 * up + 1] = ex2(x1 + vl[i][up] - b1);
          l0[nt] += ex2(x0 - c0);
          l1[nt] += ex2(x1 - c1);
        }
        pb[nt][i][0] = transposed(pack_f16x2(w[0], w[1]));
        pb[nt][i][1] = transposed(pack_f16x2(w[2], w[3]));
      }
    }

    // A NaN code times a zero weight is NaN.  So in a group with an end, codes
    // past it are cleared in place, and so are NaN codes of tokens that only
    // some queries see, whose NaN is given to the queries that see them below
    // (bits 3 mt + token - all_see of nan_lo, nan_hi: dims 16 mt + g, + 8).
    // Each lane treats the codes that it reads as fragments.
    uint32_t nan_lo = 0, nan_hi = 0;
    if (!whole) {
      const int v = t < 2 ? (t == 0 ? valid.x : valid.y) : (t == 2 ? valid.z : valid.w);
      const int seen = all_see - base - t * kBlock;  // of unit t, by every query
      auto bytes = [](int n) { return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u; };
      uint32_t keep[4], some[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        keep[j] = bytes(v - 4 * j);
        some[j] = keep[j] & ~bytes(seen - 4 * j);
      }
      const bool tail = (some[0] | some[1] | some[2] | some[3]) != 0;
      if (v < kBlock || tail) {
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 4) {  // dims 8 i + g, four at a time
          uint4* at = reinterpret_cast<uint4*>(ring + value_lane + i0 * 8 * kBlock);
          uint32_t w[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(w[i]) = at[i * 8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t bad = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (tail) {
                uint32_t b = __vcmpeq4(w[i][j] & 0x7f7f7f7fu, 0x7f7f7f7fu) & some[j];
                w[i][j] &= ~b;
                for (; b; b &= b - 1) bad |= 1u << (4 * j + ((__ffs(b) - 1) >> 3) - seen);
              }
              w[i][j] &= keep[j];
            }
            at[i * 8] = *reinterpret_cast<const uint4*>(w[i]);
            const int mt = (i0 + i) >> 1;
            if (i & 1) nan_hi |= bad << (3 * mt);
            else nan_lo |= bad << (3 * mt);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        nan_lo |= __shfl_xor_sync(0xffffffffu, nan_lo, off);
        nan_hi |= __shfl_xor_sync(0xffffffffu, nan_hi, off);
      }
    }

    // Outputs: O^T (128 dims x columns) += V^T P^T.
#pragma unroll
    for (int mt = 0; mt < 8; mt += 2) {
      uint4 lo[2], hi[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        lo[b] = lds128(sb + value_lane + (mt + b) * 16 * kBlock);
        hi[b] = lds128(sb + value_lane + (mt + b) * 16 * kBlock + 8 * kBlock);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t a0, a1, a2, a3;
          unpack4(word(lo[b], i), a0, a2);
          unpack4(word(hi[b], i), a1, a3);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
            mma_f16_16816(o[nt][mt + b], a0, a1, a2, a3, pb[nt][i][0], pb[nt][i][1]);
        }
      }
    }
    if (__any_sync(0xffffffffu, (nan_lo | nan_hi) != 0)) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const int lo = all_see + __ffs((nan_lo >> (3 * mt)) & 7) - 1;  // first such token
        const int hi = all_see + __ffs((nan_hi >> (3 * mt)) & 7) - 1;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          if (lo >= all_see && lo < lim0[nt]) o[nt][mt][0] = __int_as_float(0x7fffffff);
          if (lo >= all_see && lo < lim1[nt]) o[nt][mt][1] = __int_as_float(0x7fffffff);
          if (hi >= all_see && hi < lim0[nt]) o[nt][mt][2] = __int_as_float(0x7fffffff);
          if (hi >= all_see && hi < lim1[nt]) o[nt][mt][3] = __int_as_float(0x7fffffff);
        }
      }
    }
    __syncwarp();
    if (k + 1 < count) issue_values();
  }
  if (keys_late || values_late) {
    if (lane == 0) raise_error(a.err, kErrTimeout);
    // Wait for the copies still in flight before their memory is used again.
    if (keys_late) (void)mbar_wait(key_bar, k & 1);
    (void)mbar_wait(value_bar, k & 1);
    if (values_late && k + 1 < count) (void)mbar_wait(key_bar, (k + 1) & 1);
  }

  // Join the warps, then the cluster's CTAs.
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      join_sum(ml0[nt], l0[nt], __shfl_xor_sync(0xffffffffu, ml0[nt], off),
               __shfl_xor_sync(0xffffffffu, l0[nt], off));
      join_sum(ml1[nt], l1[nt], __shfl_xor_sync(0xffffffffu, ml1[nt], off),
               __shfl_xor_sync(0xffffffffu, l1[nt], off));
    }
  }
  __syncthreads();  // every stage has been read: its memory holds partial outputs now
  float* part = reinterpret_cast<float*>(smem);                    // [W][kCols][d]
  float* pm = reinterpret_cast<float*>(smem + Lay::kStat);         // [W][kCols]
  float* pml = pm + W * kCols;
  float* pl = pml + W * kCols;
  float* merged = reinterpret_cast<float*>(smem + Lay::kMerged);   // [kCols][d]
  float* mm = merged + kCols * kHeadDim;                           // [kCols]
  float* mml = mm + kCols;
  float* ml = mml + kCols;
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int c0 = nt * 8 + 2 * t;
    float* p0 = part + (warp * kCols + c0) * kHeadDim;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      p0[mt * 16 + g] = o[nt][mt][0];
      p0[kHeadDim + mt * 16 + g] = o[nt][mt][1];
      p0[mt * 16 + g + 8] = o[nt][mt][2];
      p0[kHeadDim + mt * 16 + g + 8] = o[nt][mt][3];
    }
    if (g == 0) {
      pm[warp * kCols + c0] = m0[nt];
      pm[warp * kCols + c0 + 1] = m1[nt];
      pml[warp * kCols + c0] = ml0[nt];
      pml[warp * kCols + c0 + 1] = ml1[nt];
      pl[warp * kCols + c0] = l0[nt];
      pl[warp * kCols + c0 + 1] = l1[nt];
    }
  }
  __syncthreads();
  // A column's parts, four dims a lane: of this CTA's warps, then of the
  // cluster's CTAs, whose warps share the columns out.
  auto of_warps = [&](int c, float4& acc, float& mx, float& msum, float& sum) {
#pragma unroll
    for (int w = 0; w < W; ++w) mx = fmaxf(mx, pm[w * kCols + c]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      add4(acc, scale_of(pm[w * kCols + c], mx),
           *reinterpret_cast<const float4*>(part + (w * kCols + c) * kHeadDim + lane * 4));
      join_sum(msum, sum, pml[w * kCols + c], pl[w * kCols + c]);
    }
  };
  const int gang = parts ? 1 : cluster;  // CTAs that join here
  if (gang > 1) {
    for (int c = warp; c < cols; c += W) {
      float mx = -INFINITY, msum = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      of_warps(c, acc, mx, msum, sum);
      *reinterpret_cast<float4*>(merged + c * kHeadDim + lane * 4) = acc;
      if (lane == 0) {
        mm[c] = mx;
        mml[c] = msum;
        ml[c] = sum;
      }
    }
    cluster_sync();
  }
  constexpr int kMine = (kCols + W - 1) / W;  // columns of a warp at most
  float4 acc[kMine];
  float sum[kMine], msum[kMine];
  auto column = [&](int j) { return (j * gang + (gang > 1 ? rank : 0)) * W + warp; };
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int c = column(j);
    acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    sum[j] = 0.f;
    msum[j] = -INFINITY;
    if (c >= cols) continue;
    float mx = -INFINITY;
    if (gang == 1) {
      of_warps(c, acc[j], mx, msum[j], sum[j]);
    } else {
      for (int i = 0; i < gang; ++i) mx = fmaxf(mx, load_remote(mm + c, i));
      for (int i = 0; i < gang; ++i) {
        add4(acc[j], scale_of(load_remote(mm + c, i), mx), load_remote4(merged + c * kHeadDim + lane * 4, i));
        join_sum(msum[j], sum[j], load_remote(mml + c, i), load_remote(ml + c, i));
      }
    }
    // From units of 2^(M - 14) to the sum's (2^22 of them; a prefix's shares
    // are joined in single ones).
    if (mx > -INFINITY) scale4(acc[j], ex2(mx - kWeightLog2 - msum[j]) * (beside ? 1.f : kSumDown));
  }
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int c = column(j);
    if (c >= cols) continue;
    if (a.part) {  // a share among others, joined later
      const int64_t at =
          (parts ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(h) * a.R + r) * (a.S * a.G) + col0 + c;
      store4(a.part + at * kHeadDim + lane * 4, acc[j]);
      if (lane == 0) a.stat[at] = make_float2(msum[j], sum[j]);
      continue;
    }
    const int s = (col0 + c) / a.G, gi = (col0 + c) % a.G;
    const int64_t at = ((static_cast<int64_t>(s) * a.R + r) * a.Hq + h * a.G + gi) * kHeadDim + lane * 4;
    const float4 v = average(acc[j], sum[j]);
    if (a.out_fp32) store4_finite(static_cast<float*>(a.out) + at, v);
    else store4_finite(static_cast<T*>(a.out) + at, v);
  }
  // Beside another launch that writes shares: who waits for this grid has to
  // have waited for that one.  One CTA does it for all (others would keep SMs
  // from the CTAs behind them).
  if (beside && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)
    previous_done();
  if (gang == 1) return;
  cluster_sync();  // no CTA leaves while another still reads its shared memory
}
template <typename T, int W, int kNT>
cudaError_t configure() {
  return cudaFuncSetAttribute(attn_kernel<T, W, kNT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<W, kNT>::kBytes);
}

template <typename T, int W, int kNT>
cudaError_t launch_t(const Q8AttnArgs& a, int col_groups, cudaStream_t s) {
  const int64_t ctas = static_cast<int64_t>(a.R) * a.Hkv * col_groups;
  const int groups = (a.max_blocks + kGroupUnits - 1) / kGroupUnits;
  // CTAs of a pair, by the longest context that the table can hold.  While
  // all fit the card at once: as many as have a group for every warp (latency
  // counts: one request of 4096 tokens takes 27.6, 17.0, 11.1, 8.3 us with
  // one, two, four, eight).  Beyond that, where every warp keeps eight groups
  // to spread its start and join over: up to three rounds of CTAs, or one and
  // a half with two column tiles (two CTAs an SM), so that long requests do
  // not run on alone.  GB300, us with one, two, four, eight: 64 requests x 8
  // heads x 16384 tokens 402, 338, 316, 338; 24 ragged ones up to 9001, four
  // queries 94, 71, 71, 87; 10 x 16 heads up to 20000 129, 96, 65, 72; but 32
  // even ones of 8192 89, 111, 98, 104.  Short contexts stay whole: 64 up to
  // 2000 33, 39, 45, 56.
  // In rounds a request takes only as many of its cluster's CTAs as leave each
  // of their warps `each` groups, six: 64 up to 8192 of which nine in ten have
  // under 1024 tokens 60 us, with one group 64, with twelve 66 (all lengths
  // alike, to 8192: 115, 115, 117).
  const int64_t slots = 152 * ((kNT == 1 ? 12 : 8) / W);
  const int64_t enough = kNT == 1 ? 3 * slots : slots * 3 / 2;
  int cluster = 1, each = 1;
  while (W > 1 && cluster < 8 && ctas * cluster * 2 <= slots && 2 * cluster * W <= groups) cluster *= 2;
  while (W > 1 && cluster < 8 && ctas * cluster < enough && 2 * cluster * W * 8 <= groups) {
    cluster *= 2;
    each = ctas * cluster > slots ? 6 : 1;
  }
  return launch_early(attn_kernel<T, W, kNT>,
                      dim3(static_cast<unsigned>(a.R) * a.Hkv * cluster, col_groups), W * 32,
                      Layout<W, kNT>::kBytes, s, cluster, a, cluster, each);
}

template <typename T>
cudaError_t launch_n(const Q8AttnArgs& a, cudaStream_t s) {
  // Warps a CTA: four; where there are more pairs than the card holds such
  // CTAs, two for contexts up to 512 tokens and (one column tile) one up to
  // 256: a warp's start and join, some 5 us, are then spread over more of its
  // 1.4 us groups.  GB300, us with four, two, one: 128 requests x 8 heads x 256
  // tokens 15.7, 15.5, 13.3; 300 x 16 x 100 66, 41, 37; 128 ragged ones up to
  // 500 23.3, 23.1, 24.4; with two tiles, 128 up to 300 40, 33; but 64 up to
  // 1000 19.8, 23.8.
  // More than eight columns: a tile of eight a CTA where all is small, or where
  // contexts are short and it leaves a pair as many CTAs, although the pages
  // are then read again (from the L2): a warp's chain is shorter and the card
  // is not full.  Four queries x four heads, us with two tiles a CTA
  // and with one: 300 tokens x 8 heads 11.7, 9.8; 8 x 300 12.0, 9.6; 40 x 300
  // 19.3, 16.7; 8000 18.8, 16.3; but 16 x 1000 16.4, 16.8; 8 x 2000 15.8, 17.5;
  // 4 x 4000 16.3, 18.7.  As many CTAs: 20 x 777 17.6, 14.9; 24 x 1500 25.4, 22.6;
  // 12 x 2000 21.1, 18.6.
  const int cols = a.S * a.G, groups = (a.max_blocks + kGroupUnits - 1) / kGroupUnits;
  const int64_t pairs = static_cast<int64_t>(a.R) * a.Hkv;
  auto cluster = [](int64_t ctas, int64_t fit) {
    int c = 1;
    while (c < 8 && ctas * c * 2 <= fit) c *= 2;
    return c;
  };
  const int64_t single = pairs * ((cols + 7) / 8);  // CTAs of one tile
  if (cols <= 8 || pairs * groups <= 1600 ||
      (groups <= 32 && single <= 3 * 152 &&
       cluster(single, 3 * 152) >= cluster(pairs * ((cols + 15) / 16), 2 * 152))) {
    const int col_groups = (cols + 7) / 8;
    if (pairs * col_groups <= 3 * 152 || groups > 8) return launch_t<T, 4, 1>(a, col_groups, s);
    return groups > 4 ? launch_t<T, 2, 1>(a, col_groups, s) : launch_t<T, 1, 1>(a, col_groups, s);
  }
  const int col_groups = (cols + 15) / 16;
  if (pairs * col_groups <= 2 * 152 || groups > 8) return launch_t<T, 4, 2>(a, col_groups, s);
  return launch_t<T, 2, 2>(a, col_groups, s);
}

// The parts of each request joined: a warp a row of out.
template <typename T>
__global__ void __launch_bounds__(128) join_parts(const Q8AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.S) * a.R * a.Hq) return;
  const int hq = static_cast<int>(row % a.Hq), r = static_cast<int>(row / a.Hq % a.R);
  const int s = static_cast<int>(row / a.Hq / a.R), h = hq / a.G;
  const int cols = a.S * a.G, c = s * a.G + hq - h * a.G;
  previous_done();
  next_may_begin();
  const int first = __ldcg(a.plan + r), parts = __ldcg(a.plan + r + 1) - first;
  const int64_t at = (static_cast<int64_t>(first) * a.Hkv + h) * cols + c;  // of the first part
  float sum;
  const float4 acc = join_shares(reinterpret_cast<const float4*>(a.part) + at * 32, a.stat + at,
                                 static_cast<int64_t>(a.Hkv) * cols, parts, lane, sum);
  const float4 v = average(acc, sum);
  if (a.out_fp32) store4_finite(static_cast<float*>(a.out) + row * kHeadDim + lane * 4, v);
  else store4_finite(static_cast<T*>(a.out) + row * kHeadDim + lane * 4, v);
}

template <typename T, int W, int kNT>
cudaError_t launch_split(const Q8AttnArgs& a, cudaStream_t s) {
  const cudaError_t e =
      launch_early(attn_kernel<T, W, kNT>,
                   dim3(static_cast<unsigned>(a.columns) * a.Hkv, (a.S * a.G + 8 * kNT - 1) / (8 * kNT)), W * 32,
                   Layout<W, kNT>::kBytes, s, 0, a, 1, 1);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.S) * a.R * a.Hq;
  return launch_early(a.out_fp32 ? join_parts<float> : join_parts<T>, static_cast<unsigned>((rows + 3) / 4), 128, 0,
                      s, 0, a);
}

template <typename T>
cudaError_t launch_split(const Q8AttnArgs& a, int warps, cudaStream_t s) {
  if (a.S * a.G <= 8) return launch_split<T, 4, 1>(a, s);
  return warps == 2 ? launch_split<T, 2, 2>(a, s) : launch_split<T, 4, 2>(a, s);
}

}  // namespace

// Cutting requests into parts costs some 5 us (the parts' sizes, a second
// launch) and gains where lengths differ or pairs are few: one round of CTAs of
// about one size fills the card, where a cluster ends at eight CTAs and keeps
// the room of those that a short request leaves idle.  So: where the card holds
// at least 1.7 CTAs a pair (of two warps with two column tiles), and in
// clusters of one round a warp of the longest request has seven groups or more
// (of a single one, eight more than in parts).  GB300, us
// without and with (8 KV heads of four query heads, lengths uniform up to the
// given one; in brackets four queries): 2 x 131072 118, 84 [157, 87]; 2 x 32000
// 34, 25 [46, 32]; 5 x 30000 32, 27 [38, 35.5]; 24 x 9001 51.5, 49.5 [74, 61];
// 38 x 8192 [94, 80]; 16 x 4000 25.5, 22 [32, 30]; 24 x 3000 [39, 28]; 6 x 8000
// [31, 25]; one of 131072 104, 57 [140, 59], of 32768 30, 22 [43, 26].  But, not
// cut, 8 x 4000 16, 18 [21, 25]; 24 x 2000 17.5, 19.5; where rounds are needed
// 100 x 4000 81, 83 [111, 121].  Equal lengths lose near the bound (16 x 4000
// 29, 32 [34, 41]) and nothing further on (24 x 3000 [42, 43]).  Rounds are
// taken with two column tiles, up to two of them, from 48 groups on: [64 x 16384
// 239, 200; equal 371, 379]; below it is [64 x 8192 131, 130; equal 197, 221].
Q8Split q8_split(int R, int S, int G, int Hkv, int max_blocks) {
  Q8Split p{};
  if (R < 1 || R > kSplitRequests) return p;
  const int cols = S * G, col_groups = (cols + 15) / 16, CTAs = cols <= 8 ? 3 : 2;
  const int64_t pairs = static_cast<int64_t>(R) * Hkv * col_groups;
  const int64_t groups = (max_blocks + kGroupUnits - 1) / kGroupUnits;
  const int64_t fit = 152 * CTAs;  // CTAs of four warps that the card holds
  // Groups of a warp at the longest in clusters that fit the card at once: an
  // estimate (launch_t goes on to more rounds of larger clusters, and to no
  // more CTAs than there are groups), which the bounds below were measured with.
  int64_t cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= fit) cluster *= 2;
  const int64_t whole = groups / (cluster * 4);
  int64_t slots;
  if (pairs * 17 <= fit * (cols > 8 ? 20 : 10)) {
    // Two warps a CTA with two column tiles where parts of four would be a
    // quarter of a pair or more: 24 x 9001 65, 61 us with four, two; 40 x 4000
    // 64, 56; but 5 x 30000 35, 38, one of 131072 59, 66.
    p.warps = cols > 8 && pairs * 4 > fit ? 2 : 4;
    slots = fit * 4 / p.warps;
    const int64_t part = pairs * groups / (slots * p.warps);
    if (whole < (R > 1 ? 7 : (part > kLeastGroups ? part : kLeastGroups) + 8)) return p;
  } else {
    // In rounds.
    if (cols <= 8 || pairs > 2 * fit || whole < 48) return p;
    p.warps = 4;
    slots = fit * ((2 * pairs + fit - 1) / fit);
  }
  p.columns = static_cast<int>(slots / (static_cast<int64_t>(Hkv) * col_groups));
  const int64_t rows = static_cast<int64_t>(p.columns) * Hkv * cols;
  auto up = [](int64_t n) { return static_cast<size_t>((n + 255) / 256 * 256); };
  p.part_bytes = up(rows * kHeadDim * 4);
  p.stat_bytes = up(rows * 8);
  p.bytes = p.part_bytes + p.stat_bytes + up((R + 1) * 4);
  return p;
}

cudaError_t launch_q8_attn(const Q8AttnArgs& a, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  if (a.plan)
    return a.type == kBf16 ? launch_split<__nv_bfloat16>(a, a.warps, s) : launch_split<__half>(a, a.warps, s);
  return a.type == kBf16 ? launch_n<__nv_bfloat16>(a, s) : launch_n<__half>(a, s);
}

namespace {
template <typename T>
cudaError_t configure_all() {
  cudaError_t e = configure<T, 4, 1>();
  if (e == cudaSuccess) e = configure<T, 2, 1>();
  if (e == cudaSuccess) e = configure<T, 1, 1>();
  if (e == cudaSuccess) e = configure<T, 4, 2>();
  if (e == cudaSuccess) e = configure<T, 2, 2>();
  cudaFuncAttributes at;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, join_parts<T>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, join_parts<float>);
  return e;
}
}  // namespace

// Their code and shared memory on the current device.
cudaError_t preload_q8_attn_kernels() {
  const cudaError_t e = configure_all<__nv_bfloat16>();
  return e == cudaSuccess ? configure_all<__half>() : e;
}

}  // namespace oasis
