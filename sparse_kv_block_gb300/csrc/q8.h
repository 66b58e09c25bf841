// q8.h -- host-side launchers of the quantised-cache kernels and of the
// draft verification.  Plain C++ structs; used by the C ABI in q8_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace oasis {

enum Q8Type { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

constexpr int kQ8MaxGroup = 8;     // query heads per KV head
constexpr int kQ8MaxQueries = 4;   // queries per request
constexpr int kVerifyMaxDrafts = 64;
constexpr int kTreeMaxNodes = 64;  // bits of a node's word
constexpr int kLogprobsMaxTop = 32;

struct Q8WriteArgs {
  const void* k;             // [T][Hkv][d], token stride in elements
  const void* v;
  int64_t k_stride, v_stride;
  const int64_t* slots;      // [T]: page * 16 + token in the page, < 0 skips
  uint8_t* pages;            // [num_pages][Hkv][unit]
  uint32_t* err;
  int64_t num_slots;         // num_pages * 16
  int T, Hkv, type;
};

struct AppendArgs {
  Q8WriteArgs kv;            // keys (to be turned), values and where they go
  const void* q;             // [T][Hq][d], token stride in elements
  void* out;                 // turned queries
  int64_t q_stride, out_stride;
  const int64_t* positions;  // [axes][T]
  int Hq;                    // 0: keys alone
  int half, interleaved;     // pairs; (2 i, 2 i + 1) in place of (i, i + half)
  float scale;               // of cos and sin
  int chunk, chunks;         // heads of a warp (the launcher's)
  uint64_t turn[64];         // of a pair: turns a position, in units of 2^-64
  uint8_t axis[64];
};

struct KeepArgs {
  uint8_t* pages;
  const int32_t* table;      // [R][max_blocks]
  const int32_t* len;        // [R], the tree's nodes included
  const int32_t* size;       // [R] or null: N
  const int32_t* nodes;      // [R][M]
  const int32_t* keep;       // [R]
  uint32_t* err;
  int R, N, M, Hkv, num_pages, max_blocks;
};

struct TreeArgs {
  const void* q;             // [R][N][Hq][d]
  void* out;
  const uint8_t* pages;
  const uint64_t* words;     // [R][N]: bit j of node i's: it sees node j
  const int32_t* table;      // [R][max_blocks]
  const int32_t* len;        // [R], the tree's nodes included
  const int32_t* size;       // [R] or null: N
  uint32_t* err;
  int R, N, Hq, Hkv, G, num_pages, max_blocks;
  int type, out_fp32;
  float scale_log2;
  long long wait_limit;
  // Shares of pairs that several CTAs have: average (in units of 2^8), (m, sum).
  float* part;               // [2 ctas][part_rows][d]: of the pair that a CTA finds begun, and of its last one
  float2* stat;
  int4* info;                // [ctas]: the pair that begins there and goes on (r, h, block, shares), r -1: none
  int ctas, part_rows;
  uint32_t over_G;           // 2^16 / G + 1: row / G is row * over_G >> 16 (exact for the rows of 64 nodes, G to 8)
};

// Launch and scratch of the tree attention.
struct TreeShape {
  int tiles;                 // of 128 rows a CTA, 1 or 2
  int ctas, rows;
  size_t part_bytes, stat_bytes, bytes;
};

struct LogprobsArgs {
  const void* logits;        // rows of V, stride elements apart
  int64_t stride;
  const int32_t* tokens;     // [rows] or null
  float* logprobs;           // [rows] or null
  float* entropy;            // [rows] or null
  int32_t* top_ids;          // [rows][k]
  float* top_logprobs;
  int rows, V, k, type;
};

struct Q8ReadArgs {
  const uint8_t* pages;
  const int32_t* table;      // [R][max_blocks]
  const int32_t* len;        // [R]
  void* out;                 // [R][Hkv][out_blocks][2][B][d]
  uint32_t* err;
  int R, Hkv, num_pages, max_blocks, out_blocks, type;
};

struct Q8AttnArgs {
  const void* q;             // [S][R][Hq][d]
  void* out;                 // [S][R][Hq][d]
  const uint8_t* pages;
  const int32_t* table;      // [R][max_blocks]
  const int32_t* len;        // [R]
  uint32_t* err;
  int R, S, Hq, Hkv, G, num_pages, max_blocks;
  int causal, type, out_fp32;
  float scale_log2;          // softmax scale * log2(e)
  long long wait_limit;
  // Set: the outputs go here instead, as one share of a softmax: row (h * R +
  // r) * S * G + s * G + gi [d] in units of 2^m, and (m, sum).
  float* part;
  float2* stat;
  // Set too: requests are cut into parts by their lengths.  Row (CTA * S * G +
  // s * G + gi) of the above; plan[r]: the parts before request r's.
  int* plan;                 // [R + 1]
  int columns, warps;        // of Q8Split
};

// Parts of a batch's requests, of about one length, and their scratch.
struct Q8Split {
  int columns;               // parts over all requests, at most (a CTA each and KV head); 0: not cut
  int warps;                 // of a CTA
  size_t part_bytes, stat_bytes, bytes;
};

// Shares and row tiles of the prefix attention, and its scratch.
struct PrefixShape {
  int64_t rows;      // R * S * G
  int tiles;         // 128-row tiles a CTA, 1 or 2
  int row_tiles;     // CTAs over the rows
  int splits;        // shares of the prefix; one more is the requests' own pages
  size_t part_bytes, bytes;
};

struct PrefixArgs {
  const void* q;             // [S][R][Hq][d] bf16
  void* out;                 // [S][R][Hq][d] bf16 or fp32
  float* part;               // [splits + 1][Hkv][rows][d]
  float2* stat;              // [splits + 1][Hkv][rows]
  uint32_t* err;
  int R, S, Hq, Hkv, G, prefix_len, row_tiles, splits;
  int out_fp32;
  float scale_log2;
  long long wait_limit;
};

struct VerifyArgs {
  const void* target;        // [R][n + 1] rows of V probabilities
  const void* draft;         // [R][n] rows, or null: the drafts are certain
  int64_t target_stride, draft_stride;  // elements between rows
  const int32_t* tokens;     // [R][n]
  const int32_t* n_drafts;   // [R] or null
  const float* u_accept;     // [R][n]
  const float* u_sample;     // [R]
  int32_t* out_tokens;       // [R][n + 1]
  int32_t* n_accept;         // [R]
  int R, n, V, type;
};

// A launch that may begin before the one ahead of it in the stream has ended
// (programmatic dependent launch).  Its kernel waits for that one, with
// previous_done(), before it touches memory; only the launches of one prefix
// attention wait later, where they say so.  In a loop of small calls this
// hides most of a launch.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         int cluster, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_q8_write(const Q8WriteArgs& a, cudaStream_t s);
cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s);
cudaError_t launch_q8_attn(const Q8AttnArgs& a, cudaStream_t s);
Q8Split q8_split(int R, int S, int G, int Hkv, int max_blocks);
PrefixShape prefix_shape(int R, int S, int G, int Hkv, int prefix_len);
// The map covers the prefix [Hkv][blocks][2][B][d] with boxes of 8 blocks'
// keys or values, 64 dims.
// Then launch_q8_attn with `part` set (it may run beside this one), then
// launch_join, which waits for both.
cudaError_t launch_prefix(const PrefixArgs& a, int tiles, const CUtensorMap& map, cudaStream_t s);
cudaError_t launch_join(const PrefixArgs& a, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);
cudaError_t launch_q8_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_q8_keep(const KeepArgs& a, cudaStream_t s);
TreeShape tree_shape(int R, int N, int G, int Hkv, int max_blocks, int type);
// The map covers the pages' keys, [pages][Hkv][2 (even, odd tokens)][8][128 bytes], with boxes of one unit's.
cudaError_t launch_q8_tree(const TreeArgs& a, int tiles, const CUtensorMap& map, cudaStream_t s);
cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t s);

// Load the kernels' code (and set their shared memory) on the current device.
cudaError_t preload_q8_cache_kernels();
cudaError_t preload_q8_attn_kernels();
cudaError_t preload_prefix_kernels();
cudaError_t preload_verify_kernels();
cudaError_t preload_append_kernels();
cudaError_t preload_tree_kernels();
cudaError_t preload_logprobs_kernels();

}  // namespace oasis
