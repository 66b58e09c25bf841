// q8_api.cu -- the C ABI of decoding over the 8-bit cache (include/oasis.h):
// argument checks, the handle and the launches.
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/oasis.h"
#include "common.cuh"
#include "q8.cuh"
#include "q8.h"

using namespace oasis;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int type_bytes(int type) { return type == OASIS_FP32 ? 4 : 2; }
bool any_type(int type) { return type == OASIS_BF16 || type == OASIS_FP16 || type == OASIS_FP32; }

const char* config_error(const oasis_q8_config* c) {
  if (!c) return "null config";
  if (c->num_pages <= 0 || c->num_pages > (1 << 27)) return "num_pages must be in 1..2^27";
  if (c->max_blocks <= 0 || c->max_blocks > 131072) return "max_blocks must be in 1..131072";
  if (c->num_kv_heads <= 0 || c->num_q_heads <= 0) return "head counts must be > 0";
  if (c->num_kv_heads > 65535) return "num_kv_heads must be <= 65535";
  if (c->num_q_heads % c->num_kv_heads != 0) return "num_q_heads must be a multiple of num_kv_heads";
  if (c->num_q_heads / c->num_kv_heads > kQ8MaxGroup) return "query heads per KV head must be <= 8";
  if (c->head_dim != kHeadDim) return "head_dim must be 128";
  if (c->block_size != kBlock) return "block_size must be 16";
  if (!(c->softmax_scale >= 0.f) || std::isinf(c->softmax_scale * kLog2e))
    return "softmax_scale must be >= 0 and finite, also times log2(e)";
  if (c->out_fp32 != 0 && c->out_fp32 != 1) return "out_fp32 must be 0 or 1";
  if (c->device < 0) return "device must be >= 0";
  return nullptr;
}

// The call's device, and the caller's again afterwards.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    e_ = cudaGetDevice(&was_);
    if (e_ == cudaSuccess && was_ != device) {
      e_ = cudaSetDevice(device);
      moved_ = e_ == cudaSuccess;
    }
  }
  ~OnDevice() {
    if (moved_) cudaSetDevice(was_);
  }
  cudaError_t error() const { return e_; }

 private:
  int was_ = 0;
  bool moved_ = false;
  cudaError_t e_;
};

}  // namespace

struct oasis_q8 {
  oasis_q8_config cfg{};
  int G = 0;
  float scale_log2 = 0.f;
  uint8_t* pages = nullptr;
  uint32_t* err = nullptr;
  long long wait_limit = kWaitLimitCycles;
  char last_error[256] = "";

  int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(last_error, sizeof last_error, fmt, ap);
    va_end(ap);
    return code;
  }
  int cuda(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return OASIS_OK;
    return fail(OASIS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  }
};

OASIS_API const char* oasis_q8_config_error(const oasis_q8_config* cfg) { return config_error(cfg); }

OASIS_API int oasis_q8_query_sizes(const oasis_q8_config* cfg, oasis_q8_sizes* out) {
  if (config_error(cfg) || !out) return OASIS_EINVAL;
  out->pages_bytes = static_cast<size_t>(cfg->num_pages) * cfg->num_kv_heads * kQ8UnitBytes;
  out->workspace_bytes = 256;
  return OASIS_OK;
}

OASIS_API int oasis_q8_init(const oasis_q8_config* cfg, void* pages, void* workspace,
                            oasis_q8** out) {
  if (!out) return OASIS_EINVAL;
  *out = nullptr;
  if (config_error(cfg) || !pages || !workspace) return OASIS_EINVAL;
  if (!aligned(pages, 16) || !aligned(workspace, 256)) return OASIS_EINVAL;
  OnDevice dev(cfg->device);
  if (dev.error() != cudaSuccess) return OASIS_ECUDA;
  if (preload_q8_cache_kernels() != cudaSuccess || preload_q8_attn_kernels() != cudaSuccess ||
      preload_prefix_kernels() != cudaSuccess)
    return OASIS_ECUDA;
  // The caller's memory may still be written by what it was used for before.
  if (cudaDeviceSynchronize() != cudaSuccess) return OASIS_ECUDA;
  // (A memset may return early; the caller's streams need not wait for it.)
  if (cudaMemset(workspace, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return OASIS_ECUDA;
  oasis_q8* q = new (std::nothrow) oasis_q8;
  if (!q) return OASIS_ENOMEM;
  q->cfg = *cfg;
  q->G = cfg->num_q_heads / cfg->num_kv_heads;
  const float scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.f / std::sqrt(static_cast<float>(kHeadDim));
  q->scale_log2 = scale * kLog2e;
  q->pages = static_cast<uint8_t*>(pages);
  q->err = static_cast<uint32_t*>(workspace);
  *out = q;
  return OASIS_OK;
}

OASIS_API int oasis_q8_destroy(oasis_q8* q8) {
  delete q8;
  return OASIS_OK;
}

OASIS_API const char* oasis_q8_last_error(const oasis_q8* q8) {
  return q8 ? q8->last_error : "null handle";
}

OASIS_API int oasis_q8_sync(oasis_q8* q8, uint32_t* device_bits) {
  if (!q8) return OASIS_EINVAL;
  OnDevice dev(q8->cfg.device);
  if (int rc = q8->cuda(dev.error(), "cudaSetDevice")) return rc;
  if (int rc = q8->cuda(cudaDeviceSynchronize(), "cudaDeviceSynchronize")) return rc;
  uint32_t bits = 0;
  if (int rc = q8->cuda(cudaMemcpy(&bits, q8->err, sizeof bits, cudaMemcpyDeviceToHost),
                        "read device error word"))
    return rc;
  if (device_bits) *device_bits = bits;
  if (!bits) return OASIS_OK;
  if (int rc = q8->cuda(cudaMemset(q8->err, 0, sizeof bits), "clear device error word")) return rc;
  // A later call's bits on a stream of the caller's must come after it.
  if (int rc = q8->cuda(cudaDeviceSynchronize(), "cudaDeviceSynchronize")) return rc;
  return q8->fail(OASIS_EDEVICE, "device error bits 0x%x", bits);
}

OASIS_API int oasis_q8_set_wait_limit(oasis_q8* q8, long long cycles) {
  if (!q8) return OASIS_EINVAL;
  q8->wait_limit = cycles > 0 ? cycles : kWaitLimitCycles;
  return OASIS_OK;
}

OASIS_API int oasis_q8_write(oasis_q8* q8, const void* k, const void* v, int type,
                             int64_t k_stride, int64_t v_stride, const int64_t* slots,
                             int num_tokens, void* stream) {
  if (!q8) return OASIS_EINVAL;
  if (!any_type(type)) return q8->fail(OASIS_EINVAL, "q8_write: bad type %d", type);
  if (num_tokens < 0) return q8->fail(OASIS_EINVAL, "q8_write: num_tokens must be >= 0");
  if (static_cast<int64_t>(num_tokens) * q8->cfg.num_kv_heads > (1ll << 33))
    return q8->fail(OASIS_EINVAL, "q8_write: num_tokens * num_kv_heads must be <= 2^33");
  if (num_tokens == 0) return OASIS_OK;
  if (!k || !v || !slots) return q8->fail(OASIS_EINVAL, "q8_write: null pointer");
  const int b = type_bytes(type);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || k_stride < 0 || v_stride < 0 ||
      k_stride * b % 16 || v_stride * b % 16)
    return q8->fail(OASIS_EINVAL, "q8_write: k, v and their strides must be 16-byte aligned, the strides >= 0");
  OnDevice dev(q8->cfg.device);
  if (int rc = q8->cuda(dev.error(), "cudaSetDevice")) return rc;
  Q8WriteArgs a{};
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.pages = q8->pages;
  a.err = q8->err;
  a.num_slots = static_cast<int64_t>(q8->cfg.num_pages) * kBlock;
  a.T = num_tokens;
  a.Hkv = q8->cfg.num_kv_heads;
  a.type = type;
  return q8->cuda(launch_q8_write(a, static_cast<cudaStream_t>(stream)), "q8_write launch");
}

OASIS_API int oasis_q8_read(oasis_q8* q8, int num_requests, const int32_t* page_table,
                            const int32_t* seq_len, void* out, int type, int out_blocks,
                            void* stream) {
  if (!q8) return OASIS_EINVAL;
  if (!any_type(type)) return q8->fail(OASIS_EINVAL, "q8_read: bad type %d", type);
  if (num_requests < 0 || num_requests > 65535)
    return q8->fail(OASIS_EINVAL, "q8_read: num_requests must be in 0..65535");
  if (out_blocks < 1) return q8->fail(OASIS_EINVAL, "q8_read: out_blocks must be >= 1");
  const int blocks = out_blocks < q8->cfg.max_blocks ? out_blocks : q8->cfg.max_blocks;
  if (static_cast<int64_t>(num_requests) * blocks * q8->cfg.num_kv_heads > (1ll << 33))
    return q8->fail(OASIS_EINVAL, "q8_read: num_requests * blocks * num_kv_heads must be <= 2^33");
  if (num_requests == 0) return OASIS_OK;
  if (!page_table || !seq_len || !out) return q8->fail(OASIS_EINVAL, "q8_read: null pointer");
  if (!aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_len, 4))
    return q8->fail(OASIS_EINVAL, "q8_read: misaligned pointer (out: 16 bytes)");
  OnDevice dev(q8->cfg.device);
  if (int rc = q8->cuda(dev.error(), "cudaSetDevice")) return rc;
  Q8ReadArgs a{};
  a.pages = q8->pages;
  a.table = page_table;
  a.len = seq_len;
  a.out = out;
  a.err = q8->err;
  a.R = num_requests;
  a.Hkv = q8->cfg.num_kv_heads;
  a.num_pages = q8->cfg.num_pages;
  a.max_blocks = q8->cfg.max_blocks;
  a.out_blocks = out_blocks;
  a.type = type;
  return q8->cuda(launch_q8_read(a, static_cast<cudaStream_t>(stream)), "q8_read launch");
}

namespace {

// The checks and arguments that both attention calls share.
int attn_args(oasis_q8* q8, const char* who, int R, int S, int causal, const void* q, int type,
              const int32_t* table, const int32_t* len, void* out, Q8AttnArgs* a) {
  if (type != OASIS_BF16 && type != OASIS_FP16)
    return q8->fail(OASIS_EINVAL, "%s: queries must be bf16 or fp16", who);
  if (R < 0 || R > 65535) return q8->fail(OASIS_EINVAL, "%s: num_requests must be in 0..65535", who);
  if (S < 1 || S > kQ8MaxQueries) return q8->fail(OASIS_EINVAL, "%s: num_queries must be in 1..4", who);
  if (static_cast<int64_t>(S) * R * q8->cfg.num_q_heads > 0x7fffffff)
    return q8->fail(OASIS_EINVAL, "%s: too many query vectors", who);
  if (R > 0) {
    if (!q || !table || !len || !out) return q8->fail(OASIS_EINVAL, "%s: null pointer", who);
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(len, 4))
      return q8->fail(OASIS_EINVAL, "%s: misaligned pointer (q, out: 16 bytes)", who);
  }
  a->q = q;
  a->out = out;
  a->pages = q8->pages;
  a->table = table;
  a->len = len;
  a->err = q8->err;
  a->R = R;
  a->S = S;
  a->Hq = q8->cfg.num_q_heads;
  a->Hkv = q8->cfg.num_kv_heads;
  a->G = q8->G;
  a->num_pages = q8->cfg.num_pages;
  a->max_blocks = q8->cfg.max_blocks;
  a->causal = causal != 0;
  a->type = type;
  a->out_fp32 = q8->cfg.out_fp32;
  a->scale_log2 = q8->scale_log2;
  a->wait_limit = q8->wait_limit;
  return OASIS_OK;
}

// A map of a prefix [Hkv][blocks][2][B][d] with boxes of 8 blocks' keys or
// values, 64 dims: 128 tokens of 128 bytes.  Blocks past the end read as 0.
int prefix_map(oasis_q8* q8, const void* kv, int blocks, CUtensorMap* map) {
  static const auto encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  if (!encode) return q8->fail(OASIS_ECUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[5] = {kHeadDim, kBlock, 2, static_cast<cuuint64_t>(blocks),
                              static_cast<cuuint64_t>(q8->cfg.num_kv_heads)};
  const cuuint64_t strides[4] = {kHeadDim * 2, kBlock * kHeadDim * 2, kUnitBytes,
                                 static_cast<cuuint64_t>(blocks) * kUnitBytes};
  const cuuint32_t box[5] = {64, kBlock, 1, 8, 1}, one[5] = {1, 1, 1, 1, 1};
  if (encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(kv), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return q8->fail(OASIS_ECUDA, "prefix_attn: tensor map encode failed");
  return OASIS_OK;
}

}  // namespace

OASIS_API int oasis_q8_attn_workspace(const oasis_q8* q8, int num_requests, int num_queries, size_t* bytes) {
  if (!q8 || !bytes || num_requests < 0 || num_requests > 65535 || num_queries < 1 || num_queries > kQ8MaxQueries)
    return OASIS_EINVAL;
  *bytes = q8_split(num_requests, num_queries, q8->G, q8->cfg.num_kv_heads, q8->cfg.max_blocks).bytes;
  return OASIS_OK;
}

OASIS_API int oasis_q8_attn(oasis_q8* q8, int num_requests, int num_queries, int causal,
                            const void* q, int type, const int32_t* page_table,
                            const int32_t* seq_len, void* out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!q8) return OASIS_EINVAL;
  Q8AttnArgs a{};
  if (int rc = attn_args(q8, "q8_attn", num_requests, num_queries, causal, q, type, page_table,
                         seq_len, out, &a))
    return rc;
  if (workspace && !aligned(workspace, 256))
    return q8->fail(OASIS_EINVAL, "q8_attn: workspace not 256-byte aligned");
  if (num_requests == 0) return OASIS_OK;
  if (workspace) {
    const Q8Split sp = q8_split(num_requests, num_queries, q8->G, q8->cfg.num_kv_heads, q8->cfg.max_blocks);
    if (workspace_bytes < sp.bytes)
      return q8->fail(OASIS_EINVAL, "q8_attn: workspace under %zu bytes", sp.bytes);
    if (sp.columns) {
      uint8_t* ws = static_cast<uint8_t*>(workspace);
      a.part = reinterpret_cast<float*>(ws);
      a.stat = reinterpret_cast<float2*>(ws + sp.part_bytes);
      a.plan = reinterpret_cast<int*>(ws + sp.part_bytes + sp.stat_bytes);
      a.columns = sp.columns;
      a.warps = sp.warps;
    }
  }
  OnDevice dev(q8->cfg.device);
  if (int rc = q8->cuda(dev.error(), "cudaSetDevice")) return rc;
  return q8->cuda(launch_q8_attn(a, static_cast<cudaStream_t>(stream)), "q8_attn launch");
}

OASIS_API int oasis_prefix_workspace(const oasis_q8* q8, int num_requests, int num_queries,
                                     int prefix_len, size_t* bytes) {
  if (!q8 || !bytes || num_requests < 0 || num_requests > 65535 || num_queries < 1 ||
      num_queries > kQ8MaxQueries || prefix_len < 0)
    return OASIS_EINVAL;
  *bytes = num_requests > 0 && prefix_len > 0
               ? prefix_shape(num_requests, num_queries, q8->G, q8->cfg.num_kv_heads, prefix_len).bytes
               : 0;
  return OASIS_OK;
}

OASIS_API int oasis_prefix_attn(oasis_q8* q8, int num_requests, int num_queries, int causal,
                                const void* q, int type, const void* prefix_kv,
                                int prefix_blocks, int prefix_len, const int32_t* page_table,
                                const int32_t* seq_len, void* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!q8) return OASIS_EINVAL;
  Q8AttnArgs a{};
  if (int rc = attn_args(q8, "prefix_attn", num_requests, num_queries, causal, q, type, page_table,
                         seq_len, out, &a))
    return rc;
  if (type != OASIS_BF16) return q8->fail(OASIS_EINVAL, "prefix_attn: queries must be bf16");
  if (prefix_blocks < 0 || prefix_blocks > 131072 || prefix_len < 0 ||
      prefix_len > static_cast<int64_t>(prefix_blocks) * kBlock)
    return q8->fail(OASIS_EINVAL, "prefix_attn: prefix_len must be in 0..16 * prefix_blocks, prefix_blocks <= 131072");
  if (prefix_len > 0 && (!prefix_kv || !aligned(prefix_kv, 16)))
    return q8->fail(OASIS_EINVAL, "prefix_attn: prefix_kv null or not 16-byte aligned");
  size_t need = 0;
  oasis_prefix_workspace(q8, num_requests, num_queries, prefix_len, &need);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return q8->fail(OASIS_EINVAL, "prefix_attn: workspace null, misaligned (256 bytes) or under %zu bytes", need);
  if (num_requests == 0) return OASIS_OK;
  OnDevice dev(q8->cfg.device);
  if (int rc = q8->cuda(dev.error(), "cudaSetDevice")) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prefix_len == 0) return q8->cuda(launch_q8_attn(a, st), "prefix_attn launch");
  const PrefixShape sh = prefix_shape(num_requests, num_queries, q8->G, q8->cfg.num_kv_heads, prefix_len);
  CUtensorMap map;
  if (int rc = prefix_map(q8, prefix_kv, prefix_blocks, &map)) return rc;
  PrefixArgs p{};
  p.q = q;
  p.out = out;
  p.part = static_cast<float*>(workspace);
  p.stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + sh.part_bytes);
  p.err = q8->err;
  p.R = num_requests;
  p.S = num_queries;
  p.Hq = q8->cfg.num_q_heads;
  p.Hkv = q8->cfg.num_kv_heads;
  p.G = q8->G;
  p.prefix_len = prefix_len;
  p.row_tiles = sh.row_tiles;
  p.splits = sh.splits;
  p.out_fp32 = q8->cfg.out_fp32;
  p.scale_log2 = q8->scale_log2;
  p.wait_limit = q8->wait_limit;
  const int64_t share = static_cast<int64_t>(sh.splits) * p.Hkv * sh.rows;  // the pages' share
  a.part = p.part + share * kHeadDim;
  a.stat = p.stat + share;
  if (int rc = q8->cuda(launch_prefix(p, sh.tiles, map, st), "prefix_attn launch")) return rc;
  if (int rc = q8->cuda(launch_q8_attn(a, st), "prefix_attn launch (pages)")) return rc;
  return q8->cuda(launch_join(p, st), "prefix_attn launch (join)");
}

OASIS_API const char* oasis_verify_error(const oasis_verify_args* a) {
  if (!a) return "null arguments";
  if (a->num_requests < 0 || a->num_requests > (1 << 20)) return "num_requests must be in 0..2^20";
  if (a->num_drafts < 0 || a->num_drafts > kVerifyMaxDrafts) return "num_drafts must be in 0..64";
  if (a->vocab < 1 || a->vocab > (1 << 20)) return "vocab must be in 1..2^20";
  if (!any_type(a->type)) return "type must be OASIS_BF16, OASIS_FP16 or OASIS_FP32";
  if (a->device < 0) return "device must be >= 0";
  if (a->num_requests == 0) return nullptr;
  if (!a->target || !a->u_sample || !a->out_tokens || !a->n_accept) return "null pointer";
  if (a->num_drafts > 0 && (!a->tokens || !a->u_accept)) return "null pointer (tokens or u_accept)";
  if (a->target_stride < a->vocab) return "target_stride must be >= vocab";
  if (a->draft && a->num_drafts > 0 && a->draft_stride < a->vocab) return "draft_stride must be >= vocab";
  const size_t b = type_bytes(a->type);
  if (!aligned(a->target, b) || (a->draft && !aligned(a->draft, b)) || !aligned(a->tokens, 4) ||
      !aligned(a->n_drafts, 4) || !aligned(a->u_accept, 4) || !aligned(a->u_sample, 4) ||
      !aligned(a->out_tokens, 4) || !aligned(a->n_accept, 4))
    return "a pointer is not aligned to its type";
  return nullptr;
}

OASIS_API int oasis_verify_drafts(const oasis_verify_args* a, void* stream) {
  if (oasis_verify_error(a)) return OASIS_EINVAL;
  if (a->num_requests == 0) return OASIS_OK;
  OnDevice dev(a->device);
  if (dev.error() != cudaSuccess) return OASIS_ECUDA;
  VerifyArgs v{};
  v.target = a->target;
  v.draft = a->num_drafts > 0 ? a->draft : nullptr;
  v.target_stride = a->target_stride;
  v.draft_stride = a->draft_stride;
  v.tokens = a->tokens;
  v.n_drafts = a->n_drafts;
  v.u_accept = a->u_accept;
  v.u_sample = a->u_sample;
  v.out_tokens = a->out_tokens;
  v.n_accept = a->n_accept;
  v.R = a->num_requests;
  v.n = a->num_drafts;
  v.V = a->vocab;
  v.type = a->type;
  // Load the kernels on a device's first call, so that it may be inside a
  // stream capture.
  static std::atomic<uint64_t> loaded{0};
  const uint64_t bit = a->device < 64 ? 1ull << a->device : 0;
  if (!(loaded.load(std::memory_order_acquire) & bit)) {
    if (preload_verify_kernels() != cudaSuccess) return OASIS_ECUDA;
    loaded.fetch_or(bit, std::memory_order_release);
  }
  return launch_verify(v, static_cast<cudaStream_t>(stream)) == cudaSuccess ? OASIS_OK : OASIS_ECUDA;
}
