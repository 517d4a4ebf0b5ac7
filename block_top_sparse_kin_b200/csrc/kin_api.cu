// kin_api.cu -- the extern "C" boundary of libkin.so: argument checks,
// workspace layout, launch-shape heuristics and launches.
// Semantics of every call are documented in include/kin.h.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <cmath>

#include "kin_internal.cuh"

#define KIN_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using namespace kin;

constexpr int kTargetSMs = 148;  // B200 SM count, used only to shape grids
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

int nbcap_of(const kin_dims& d) { return (d.max_seq_len + d.block_size - 1) / d.block_size; }
int pairs_of(const kin_dims& d) { return d.batch * d.num_kv_heads; }

#ifndef KIN_ATTN_CHUNK_TOKENS
#define KIN_ATTN_CHUNK_TOKENS 768
#endif

// Kept blocks per attention CTA: KIN_ATTN_CHUNK_TOKENS tokens (768 -> 384 KB
// of K+V), fewer when the grid would hold fewer than 2 CTAs per SM.
int attn_chunk_blocks(const kin_dims& d, int k) {
  const int k_eff = k < nbcap_of(d) ? k : nbcap_of(d);
  const int by_tokens = KIN_ATTN_CHUNK_TOKENS / d.block_size > 0 ? KIN_ATTN_CHUNK_TOKENS / d.block_size : 1;
  const int64_t by_grid = (int64_t)k_eff * pairs_of(d) / (2 * kTargetSMs);
  int ch = by_tokens;
  if (by_grid < ch) ch = by_grid > 0 ? (int)by_grid : 1;
  const int cap = kMaxItemTiles / (d.block_size / kTileTokens);  // tiles per item <= 64
  return ch < cap ? ch : cap;
}

int attn_max_chunks(const kin_dims& d, int k) {
  const int k_eff = k < nbcap_of(d) ? k : nbcap_of(d);
  const int ch = attn_chunk_blocks(d, k);
  return (k_eff + ch - 1) / ch;
}

struct WsLayout {
  size_t attn_counters, scores, partials, total;
};

WsLayout ws_layout(const kin_dims& d, int k) {
  WsLayout w;
  const size_t pairs = (size_t)pairs_of(d);
  const size_t g = (size_t)(d.num_q_heads / d.num_kv_heads);
  size_t off = 0;
  w.attn_counters = off;
  off = align_up(off + pairs * sizeof(uint32_t));
  w.scores = off;
  off = align_up(off + pairs * (size_t)nbcap_of(d) * sizeof(float));
  w.partials = off;
  off = align_up(off + pairs * (size_t)attn_max_chunks(d, k) * g * kPartStride * sizeof(float));
  w.total = off;
  return w;
}

kin_status check_ws(const kin_dims& d, int k, void* ws, size_t ws_bytes, WsLayout* out) {
  *out = ws_layout(d, k);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return KIN_ERR_WORKSPACE;
  if (ws_bytes < out->total) return KIN_ERR_WORKSPACE;
  return KIN_OK;
}

kin_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KIN_OK : KIN_ERR_CUDA; }

PageTable contiguous() {
  PageTable pt;
  pt.table = nullptr;
  pt.max_blocks = 0;
  pt.num_pages = 0;
  return pt;
}

// A page pool [num_pages][Hkv][bs][D] bf16 and its table [B][ceil(Lcap / bs)].
kin_status check_pages(const kin_dims& d, const void* pool, int32_t num_pages, const int32_t* table,
                       PageTable* out) {
  if (!pool || !table || num_pages < 1) return KIN_ERR_INVALID_ARG;
  if (!aligned16(pool)) return KIN_ERR_INVALID_ARG;
  out->table = table;
  out->max_blocks = nbcap_of(d);
  out->num_pages = num_pages;
  return KIN_OK;
}

}  // namespace

namespace kin {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

kin_status check_dims(const kin_dims* d) {
  if (!d) return KIN_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_kv_heads < 1 || d->num_q_heads < 1 || d->max_seq_len < 1)
    return KIN_ERR_INVALID_ARG;
  if (d->num_q_heads % d->num_kv_heads != 0) return KIN_ERR_INVALID_ARG;
  if (d->head_dim != kHeadDim) return KIN_ERR_INVALID_ARG;
  const int bs = d->block_size;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return KIN_ERR_INVALID_ARG;
  if (d->num_q_heads / d->num_kv_heads > kMaxGroup) return KIN_ERR_CAPACITY;
  if ((d->max_seq_len + bs - 1) / bs > kMaxBlocksPerSeq) return KIN_ERR_CAPACITY;
  if ((int64_t)d->batch * d->num_kv_heads * d->max_seq_len >= (int64_t)1 << 31) return KIN_ERR_CAPACITY;
  return KIN_OK;
}

constexpr int kMaxDevices = 64;
constexpr int kSmemSlots = 24;

int device_sm_count() {
  // per device, written once with the same value by whichever thread gets there first
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return kTargetSMs;
  int n = dev < kMaxDevices ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return kTargetSMs;
    if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaError_t ensure_smem_limit(const void* kernel, int slot, size_t bytes) {
  // slot: a small per-kernel index.  The kernel's limit only ever grows: it
  // is read and raised under one lock, so a thread never lowers it under
  // another thread's launch, and the cache (the limit last seen, per slot and
  // device) never exceeds the limit in force.
  // slots in use: 0, 2, 3, then 8, 9, 10, then 12, 13, 14 block top-k (256,
  // 512, 1024 threads; plain, refining, refining per page), 1 attention, 4
  // means update, 5 token top-k, 6 token logits, 7 and 11 eviction select, 16..19
  // attention over a cache of either format
  static std::atomic<size_t> done[kSmemSlots][kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices && slot >= 0 && slot < kSmemSlots;
  if (cached && done[slot][dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mu);
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  size_t limit = attr.maxDynamicSharedSizeBytes > 0 ? (size_t)attr.maxDynamicSharedSizeBytes : 0;
  if (limit < bytes) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    limit = bytes;
  }
  if (cached) done[slot][dev].store(limit, std::memory_order_release);
  return cudaSuccess;
}

}  // namespace kin

KIN_EXPORT const char* kin_status_string(kin_status s) {
  switch (s) {
    case KIN_OK: return "KIN_OK";
    case KIN_ERR_INVALID_ARG: return "KIN_ERR_INVALID_ARG";
    case KIN_ERR_WORKSPACE: return "KIN_ERR_WORKSPACE";
    case KIN_ERR_CAPACITY: return "KIN_ERR_CAPACITY";
    case KIN_ERR_CUDA: return "KIN_ERR_CUDA";
    case KIN_ERR_DEVICE_DATA: return "KIN_ERR_DEVICE_DATA";
    case KIN_ERR_TIMEOUT: return "KIN_ERR_TIMEOUT";
  }
  return "KIN_ERR_UNKNOWN";
}

KIN_EXPORT size_t kin_workspace_bytes(const kin_dims* dims, int32_t k_blocks) {
  if (check_dims(dims) != KIN_OK || k_blocks < 2) return 0;
  return ws_layout(*dims, k_blocks).total;
}

KIN_EXPORT size_t kin_dual_means_bytes(const kin_dims* dims) {
  if (check_dims(dims) != KIN_OK) return 0;
  const int64_t rows = (int64_t)dims->batch * dims->num_kv_heads * nbcap_of(*dims);
  return (size_t)rows * (kHeadDim * 4 + kHeadDim * 2 + 4);
}

KIN_EXPORT size_t kin_dual_page_means_bytes(const kin_dims* dims, int32_t num_pages) {
  if (check_dims(dims) != KIN_OK || num_pages < 1) return 0;
  const int64_t rows = (int64_t)num_pages * dims->num_kv_heads;
  return (size_t)rows * (kHeadDim * 4 + kHeadDim * 2 + 4);
}

namespace {

kin_status means_build(const kin_dims* dims, const void* k_rows, const PageTable& pt, const int32_t* seq_lens,
                       void* block_means, int means_bf16, int32_t* dev_status, void* stream, int per_page = 0) {
  MeansBuildParams p{};  // every field not set below is zero or null
  p.means_per_page = per_page;
  p.k_cache = static_cast<const __nv_bfloat16*>(k_rows);
  p.seq_lens = seq_lens;
  p.means = block_means;
  p.means_bf16 = means_bf16;
  p.dev_status = dev_status;
  p.pages = pt;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Lcap = dims->max_seq_len;
  p.bs = dims->block_size;
  p.nbcap = nbcap_of(*dims);
  p.mean_rows = per_page ? (int64_t)pt.num_pages * p.Hkv : (int64_t)p.B * p.Hkv * p.nbcap;
  return from_cuda(launch_means_build(p, static_cast<cudaStream_t>(stream)));
}

kin_status means_update(const kin_dims* dims, void* k_rows, void* v_rows, const PageTable& pt,
                        void* block_means, int means_bf16, int32_t* seq_lens, const void* k_new,
                        const void* v_new, int32_t n_new, int32_t* dev_status, void* stream, int per_page = 0) {
  MeansUpdateParams p{};
  p.means_per_page = per_page;
  p.k_cache = static_cast<__nv_bfloat16*>(k_rows);
  p.v_cache = static_cast<__nv_bfloat16*>(v_rows);
  p.means = block_means;
  p.means_bf16 = means_bf16;
  p.seq_lens = seq_lens;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.dev_status = dev_status;
  p.pages = pt;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Lcap = dims->max_seq_len;
  p.bs = dims->block_size;
  p.nbcap = nbcap_of(*dims);
  p.mean_rows = per_page ? (int64_t)pt.num_pages * p.Hkv : (int64_t)p.B * p.Hkv * p.nbcap;
  p.n_new = n_new;
  return from_cuda(launch_means_update(p, static_cast<cudaStream_t>(stream)));
}

kin_status check_update_count(const kin_dims* dims, int32_t n_new) {
  if (n_new < 0) return KIN_ERR_INVALID_ARG;
  if (n_new > dims->max_seq_len) return KIN_ERR_CAPACITY;
  return KIN_OK;
}

kin_status check_update_args(const void* k_rows, const void* v_rows, const void* block_means,
                             const int32_t* seq_lens, const void* k_new, const void* v_new) {
  if (!k_rows || !v_rows || !block_means || !seq_lens || !k_new || !v_new) return KIN_ERR_INVALID_ARG;
  if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(block_means) || !aligned16(k_new) ||
      !aligned16(v_new))
    return KIN_ERR_INVALID_ARG;
  return KIN_OK;
}

}  // namespace

KIN_EXPORT kin_status kin_block_means_build(const kin_dims* dims, const void* k_cache,
                                            const int32_t* seq_lens, float* block_means,
                                            int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  if (!k_cache || !seq_lens || !block_means) return KIN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(block_means)) return KIN_ERR_INVALID_ARG;
  return means_build(dims, k_cache, contiguous(), seq_lens, block_means, 0, dev_status, stream);
}

KIN_EXPORT kin_status kin_block_means_build_paged(const kin_dims* dims, const void* k_pages, int32_t num_pages,
                                                  const int32_t* block_table, const int32_t* seq_lens,
                                                  float* block_means, int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  PageTable pt;
  st = check_pages(*dims, k_pages, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  if (!seq_lens || !block_means || !aligned16(block_means)) return KIN_ERR_INVALID_ARG;
  return means_build(dims, k_pages, pt, seq_lens, block_means, 0, dev_status, stream);
}

KIN_EXPORT kin_status kin_block_means_update(const kin_dims* dims, void* k_cache, void* v_cache,
                                             float* block_means, int32_t* seq_lens,
                                             const void* k_new, const void* v_new, int32_t n_new,
                                             int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  st = check_update_count(dims, n_new);
  if (st != KIN_OK || n_new == 0) return st;
  st = check_update_args(k_cache, v_cache, block_means, seq_lens, k_new, v_new);
  if (st != KIN_OK) return st;
  return means_update(dims, k_cache, v_cache, contiguous(), block_means, 0, seq_lens, k_new, v_new, n_new,
                      dev_status, stream);
}

KIN_EXPORT kin_status kin_block_means_update_paged(const kin_dims* dims, void* k_pages, void* v_pages,
                                                   int32_t num_pages, const int32_t* block_table,
                                                   float* block_means, int32_t* seq_lens, const void* k_new,
                                                   const void* v_new, int32_t n_new, int32_t* dev_status,
                                                   void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  st = check_update_count(dims, n_new);
  if (st != KIN_OK || n_new == 0) return st;
  PageTable pt;
  st = check_pages(*dims, k_pages, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  st = check_update_args(k_pages, v_pages, block_means, seq_lens, k_new, v_new);
  if (st != KIN_OK) return st;
  return means_update(dims, k_pages, v_pages, pt, block_means, 0, seq_lens, k_new, v_new, n_new, dev_status,
                      stream);
}

namespace {

kin_status topk_select(const kin_dims* dims, const void* q, const void* block_means, int means_bf16,
                       const int32_t* seq_lens, int32_t k_blocks, int32_t* sel_idx, int32_t* sel_cnt,
                       void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream,
                       const PageTable* mpages = nullptr) {
  if (k_blocks < 2) return KIN_ERR_INVALID_ARG;
  if (!q || !block_means || !seq_lens || !sel_idx || !sel_cnt) return KIN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(block_means)) return KIN_ERR_INVALID_ARG;
  WsLayout w;
  kin_status st = check_ws(*dims, k_blocks, workspace, ws_bytes, &w);
  if (st != KIN_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SelectParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.means = block_means;
  p.means_bf16 = means_bf16;
  p.refine = 0;
  p.means_f32 = nullptr;
  p.radii = nullptr;
  if (means_bf16 == 2) {  // dual: scan the bf16 rows, rescore from the fp32 rows
    const int64_t rows = mpages ? (int64_t)mpages->num_pages * dims->num_kv_heads
                                : (int64_t)dims->batch * dims->num_kv_heads * nbcap_of(*dims);
    const float* f = static_cast<const float*>(block_means);
    p.means = f + rows * kHeadDim;
    p.means_bf16 = 1;
    p.refine = 1;
    p.means_f32 = f;
    p.radii = f + rows * (kHeadDim + kHeadDim / 2);
  }
  p.mpages = mpages ? *mpages : contiguous();
  p.seq_lens = seq_lens;
  p.sel_idx = sel_idx;
  p.sel_cnt = sel_cnt;
  p.scores = reinterpret_cast<float*>(ws + w.scores);
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Hq = dims->num_q_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.bs = dims->block_size;
  p.Lcap = dims->max_seq_len;
  p.nbcap = nbcap_of(*dims);
  p.k = k_blocks;
  p.score_scale = 1.0f / std::sqrt((float)kHeadDim);
  return from_cuda(launch_select(p, static_cast<cudaStream_t>(stream)));
}

// means_dtype as a kernel flag (0 fp32, 1 bf16, 2 dual); -1 for an unknown value
int means_flag(int32_t means_dtype) {
  const int32_t t = means_dtype & ~KIN_MEANS_PER_PAGE;
  return t == KIN_MEANS_F32 ? 0 : t == KIN_MEANS_BF16 ? 1 : t == KIN_MEANS_DUAL ? 2 : -1;
}
int per_page_flag(int32_t means_dtype) { return (means_dtype & KIN_MEANS_PER_PAGE) ? 1 : 0; }

// A NULL table selects the contiguous cache (num_pages ignored).
kin_status layout_of(const kin_dims& d, const void* k_rows, int32_t num_pages, const int32_t* block_table,
                     PageTable* pt) {
  if (!block_table) {
    *pt = contiguous();
    return KIN_OK;
  }
  return check_pages(d, k_rows, num_pages, block_table, pt);
}

}  // namespace

KIN_EXPORT kin_status kin_block_topk_select(const kin_dims* dims, const void* q, const float* block_means,
                                            const int32_t* seq_lens, int32_t k_blocks, int32_t* sel_idx,
                                            int32_t* sel_cnt, void* workspace, size_t ws_bytes,
                                            int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  return topk_select(dims, q, block_means, 0, seq_lens, k_blocks, sel_idx, sel_cnt, workspace, ws_bytes,
                     dev_status, stream);
}

KIN_EXPORT kin_status kin_block_topk_select_ex(const kin_dims* dims, const void* q, const void* block_means,
                                               int32_t means_dtype, const int32_t* seq_lens, int32_t k_blocks,
                                               int32_t* sel_idx, int32_t* sel_cnt, void* workspace,
                                               size_t ws_bytes, int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  const int bf = means_flag(means_dtype);
  if (bf < 0 || per_page_flag(means_dtype)) return KIN_ERR_INVALID_ARG;  // per-page means need the table
  return topk_select(dims, q, block_means, bf, seq_lens, k_blocks, sel_idx, sel_cnt, workspace, ws_bytes,
                     dev_status, stream);
}

KIN_EXPORT kin_status kin_block_topk_select_paged(const kin_dims* dims, const void* q, const void* page_means,
                                                  int32_t means_dtype, int32_t num_pages,
                                                  const int32_t* block_table, const int32_t* seq_lens,
                                                  int32_t k_blocks, int32_t* sel_idx, int32_t* sel_cnt,
                                                  void* workspace, size_t ws_bytes, int32_t* dev_status,
                                                  void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  const int bf = means_flag(means_dtype);
  if (bf < 0) return KIN_ERR_INVALID_ARG;
  PageTable pt;
  st = check_pages(*dims, page_means, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  return topk_select(dims, q, page_means, bf, seq_lens, k_blocks, sel_idx, sel_cnt, workspace, ws_bytes,
                     dev_status, stream, &pt);
}

KIN_EXPORT kin_status kin_block_means_build_ex(const kin_dims* dims, const void* k_rows, int32_t num_pages,
                                               const int32_t* block_table, const int32_t* seq_lens,
                                               void* block_means, int32_t means_dtype, int32_t* dev_status,
                                               void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  const int bf = means_flag(means_dtype);
  if (bf < 0) return KIN_ERR_INVALID_ARG;
  if (!k_rows || !seq_lens || !block_means) return KIN_ERR_INVALID_ARG;
  if (!aligned16(k_rows) || !aligned16(block_means)) return KIN_ERR_INVALID_ARG;
  PageTable pt;
  st = layout_of(*dims, k_rows, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  const int pp = per_page_flag(means_dtype);
  if (pp && !block_table) return KIN_ERR_INVALID_ARG;
  return means_build(dims, k_rows, pt, seq_lens, block_means, bf, dev_status, stream, pp);
}

KIN_EXPORT kin_status kin_block_means_update_ex(const kin_dims* dims, void* k_rows, void* v_rows,
                                                int32_t num_pages, const int32_t* block_table,
                                                void* block_means, int32_t means_dtype, int32_t* seq_lens,
                                                const void* k_new, const void* v_new, int32_t n_new,
                                                int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  const int bf = means_flag(means_dtype);
  if (bf < 0) return KIN_ERR_INVALID_ARG;
  st = check_update_count(dims, n_new);
  if (st != KIN_OK || n_new == 0) return st;
  st = check_update_args(k_rows, v_rows, block_means, seq_lens, k_new, v_new);
  if (st != KIN_OK) return st;
  PageTable pt;
  st = layout_of(*dims, k_rows, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  const int pp = per_page_flag(means_dtype);
  if (pp && !block_table) return KIN_ERR_INVALID_ARG;
  return means_update(dims, k_rows, v_rows, pt, block_means, bf, seq_lens, k_new, v_new, n_new, dev_status,
                      stream, pp);
}

namespace {

kin_status sparse_decode_attn(const kin_dims* dims, const void* q, const void* k_rows, const void* v_rows,
                              const PageTable& pt, const int32_t* seq_lens, const int32_t* sel_idx,
                              const int32_t* sel_cnt, int32_t k_blocks, float softmax_scale, void* out,
                              float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (k_blocks < 2) return KIN_ERR_INVALID_ARG;
  if (!q || !k_rows || !v_rows || !seq_lens || !sel_idx || !sel_cnt || !out) return KIN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_rows) || !aligned16(v_rows) || !aligned16(out)) return KIN_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale)) return KIN_ERR_INVALID_ARG;
  WsLayout w;
  kin_status st = check_ws(*dims, k_blocks, workspace, ws_bytes, &w);
  if (st != KIN_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const __nv_bfloat16*>(k_rows);
  p.v_cache = static_cast<const __nv_bfloat16*>(v_rows);
  p.seq_lens = seq_lens;
  p.sel_idx = sel_idx;
  p.sel_cnt = sel_cnt;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.partials = reinterpret_cast<float*>(ws + w.partials);
  p.counters = reinterpret_cast<uint32_t*>(ws + w.attn_counters);
  p.dev_status = dev_status;
  p.pages = pt;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Hq = dims->num_q_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.bs = dims->block_size;
  p.Lcap = dims->max_seq_len;
  p.k = k_blocks;
  p.chunk_blocks = attn_chunk_blocks(*dims, k_blocks);
  p.max_chunks = attn_max_chunks(*dims, k_blocks);
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)kHeadDim);
  p.scale_log2 = scale * 1.4426950408889634f;
  const int num_items = pairs_of(*dims) * p.max_chunks;
  return from_cuda(launch_attn(p, num_items, static_cast<cudaStream_t>(stream)));
}

}  // namespace

KIN_EXPORT kin_status kin_sparse_decode_attn(const kin_dims* dims, const void* q, const void* k_cache,
                                             const void* v_cache, const int32_t* seq_lens,
                                             const int32_t* sel_idx, const int32_t* sel_cnt,
                                             int32_t k_blocks, float softmax_scale, void* out, float* lse,
                                             void* workspace, size_t ws_bytes, int32_t* dev_status,
                                             void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  return sparse_decode_attn(dims, q, k_cache, v_cache, contiguous(), seq_lens, sel_idx, sel_cnt, k_blocks,
                            softmax_scale, out, lse, workspace, ws_bytes, dev_status, stream);
}

KIN_EXPORT kin_status kin_sparse_decode_attn_paged(const kin_dims* dims, const void* q, const void* k_pages,
                                                   const void* v_pages, int32_t num_pages,
                                                   const int32_t* block_table, const int32_t* seq_lens,
                                                   const int32_t* sel_idx, const int32_t* sel_cnt,
                                                   int32_t k_blocks, float softmax_scale, void* out,
                                                   float* lse, void* workspace, size_t ws_bytes,
                                                   int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  PageTable pt;
  st = check_pages(*dims, k_pages, num_pages, block_table, &pt);
  if (st != KIN_OK) return st;
  return sparse_decode_attn(dims, q, k_pages, v_pages, pt, seq_lens, sel_idx, sel_cnt, k_blocks,
                            softmax_scale, out, lse, workspace, ws_bytes, dev_status, stream);
}

// ------------------------------------------------------------ token top-k
namespace {

constexpr int kTokenKeyCap = 32768;  // the token top-k keeps keys in shared memory up to this length

struct TokenWs {
  size_t logits, keys, sel, cnt, total;
};

TokenWs token_ws_layout(const kin_dims& d, int kt) {
  const size_t rows = (size_t)d.batch * d.num_q_heads;
  TokenWs w;
  size_t off = 0;
  w.logits = off;
  off = align_up(off + rows * (size_t)d.max_seq_len * sizeof(float));
  w.keys = off;
  if (d.max_seq_len > kTokenKeyCap) off = align_up(off + rows * (size_t)d.max_seq_len * sizeof(uint32_t));
  w.sel = off;
  off = align_up(off + rows * (size_t)kt * sizeof(int32_t));
  w.cnt = off;
  off = align_up(off + rows * sizeof(int32_t));
  w.total = off;
  return w;
}

}  // namespace

KIN_EXPORT size_t kin_token_topk_workspace_bytes(const kin_dims* dims, int32_t k_tokens) {
  if (check_dims(dims) != KIN_OK || k_tokens < 1) return 0;
  return token_ws_layout(*dims, k_tokens).total;
}

KIN_EXPORT kin_status kin_token_topk_decode_attn(const kin_dims* dims, const void* q, const void* k_cache,
                                                 const void* v_cache, const int32_t* seq_lens, int32_t k_tokens,
                                                 float softmax_scale, void* out, float* lse, int32_t* sel_tokens,
                                                 void* workspace, size_t ws_bytes, int32_t* dev_status,
                                                 void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  if (k_tokens < 1) return KIN_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !seq_lens || !out) return KIN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return KIN_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale)) return KIN_ERR_INVALID_ARG;
  if ((int64_t)dims->batch * dims->num_q_heads * dims->max_seq_len >= (int64_t)1 << 31) return KIN_ERR_CAPACITY;
  const TokenWs w = token_ws_layout(*dims, k_tokens);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0 || ws_bytes < w.total)
    return KIN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TokenParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  p.seq_lens = seq_lens;
  p.logits = reinterpret_cast<float*>(ws + w.logits);
  p.key_scratch = reinterpret_cast<uint32_t*>(ws + w.keys);
  p.sel = sel_tokens ? sel_tokens : reinterpret_cast<int32_t*>(ws + w.sel);
  p.cnt = reinterpret_cast<int32_t*>(ws + w.cnt);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Hq = dims->num_q_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.Lcap = dims->max_seq_len;
  p.kt = k_tokens;
  p.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)kHeadDim);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_token_logits(p, s);
  if (e == cudaSuccess) e = launch_token_topk(p, s);
  if (e == cudaSuccess) e = launch_token_attn(p, s);
  return from_cuda(e);
}

// ------------------------------------------------- KV caches of either format
namespace {

// A cache descriptor against dims: format, pointers, pages.
kin_status kv_view(const kin_dims& d, const kin_kv* kv, KvView* out) {
  if (!kv || (kv->format != KIN_KV_BF16 && kv->format != KIN_KV_INT4)) return KIN_ERR_INVALID_ARG;
  const bool int4 = kv->format == KIN_KV_INT4;
  if (!kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return KIN_ERR_INVALID_ARG;
  if (int4 && (!kv->k_scales || !kv->v_scales || !aligned16(kv->k_scales) || !aligned16(kv->v_scales)))
    return KIN_ERR_INVALID_ARG;
  *out = KvView{};
  out->pages = contiguous();
  if (kv->block_table) {
    kin_status st = check_pages(d, kv->k, kv->num_pages, kv->block_table, &out->pages);
    if (st != KIN_OK) return st;
    // rows are numbered in 32 bits
    if ((int64_t)kv->num_pages * d.num_kv_heads * d.block_size >= (int64_t)1 << 31) return KIN_ERR_CAPACITY;
  }
  out->k = static_cast<uint8_t*>(kv->k);
  out->v = static_cast<uint8_t*>(kv->v);
  out->ks = int4 ? static_cast<uint16_t*>(kv->k_scales) : nullptr;
  out->vs = int4 ? static_cast<uint16_t*>(kv->v_scales) : nullptr;
  out->int4 = int4;
  out->Lcap = d.max_seq_len;
  return KIN_OK;
}

// Optional block means written beside a cache: their layout, and the row
// stride of the dual form.
kin_status means_layout(const kin_dims& d, const KvView& kv, const void* means, int32_t dtype, int* flag, int* per_page,
                        int64_t* rows) {
  *flag = means_flag(dtype);
  *per_page = per_page_flag(dtype);
  *rows = 0;
  if (!means) return KIN_OK;
  if (*flag < 0 || !aligned16(means)) return KIN_ERR_INVALID_ARG;
  if (*per_page && !kv.pages.table) return KIN_ERR_INVALID_ARG;
  *rows = *per_page ? (int64_t)kv.pages.num_pages * d.num_kv_heads : (int64_t)pairs_of(d) * nbcap_of(d);
  return KIN_OK;
}

// The two share a buffer, a page pool included.
bool same_cache(const KvView& a, const KvView& b) { return a.k == b.k || a.v == b.v || a.k == b.v || a.v == b.k; }

// n bytes at a and m bytes at b share one.
bool meet(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + m && y < x + n;
}

size_t kv_rows(const kin_dims& d, const KvView& v) {
  return v.pages.table ? (size_t)v.pages.num_pages * d.num_kv_heads * d.block_size : (size_t)pairs_of(d) * d.max_seq_len;
}

// n bytes at a and the cache's rows or scales share one.
bool meets_cache(const void* a, size_t n, const kin_dims& d, const KvView& v) {
  const size_t rows = kv_rows(d, v), codes = rows * (v.int4 ? kCodeBytes : kHeadDim * 2), scales = rows * kGroups * 2;
  return meet(a, n, v.k, codes) || meet(a, n, v.v, codes) || meet(a, n, v.ks, scales) || meet(a, n, v.vs, scales);
}

bool caches_meet(const kin_dims& da, const KvView& a, const kin_dims& db, const KvView& b) {
  const size_t rows = kv_rows(da, a), codes = rows * (a.int4 ? kCodeBytes : kHeadDim * 2), scales = rows * kGroups * 2;
  return meets_cache(a.k, codes, db, b) || meets_cache(a.v, codes, db, b) || meets_cache(a.ks, scales, db, b) ||
         meets_cache(a.vs, scales, db, b);
}

// How the attention cuts the (pair, kept block) slots into ranges of `per`
// blocks, one per CTA.  A pair's slots are padded to `stride`: a multiple of
// per (aligned: no range crosses a pair), or k itself (ranges that run on into
// the next pair, so that every resident CTA gets the same).
// fit, in a dense call whose ranges all are resident at once: the kernel, which
// knows the lengths, cuts each pair into ranges of fit (32 tiles, chosen so
// that short sequences leave few partials; not swept) to per blocks.  8 pairs, 8 heads,
// a cache of 128K tokens that holds 8K: 17.1 us, 31.9 with the capacity's
// ranges; 128 pairs, 2000 of 8192 tokens: 17.6 for 28.8; calls of a few short
// sequences take 0.2 us more.  (These and the times below were taken with a
// build whose 4-bit tiles took 2 to 4% less than now, on either side alike.)
struct KvSplit {
  int per, stride, fit;
};

// Chosen by an estimate in microseconds, from timings of 4-bit caches; bf16
// tiles take two and a half times as long and are cut alike (16 x 8 pairs of
// 8192 such tokens: 84.0 us, 83.5 in shorter ranges):
// a range takes 4, or 5 where ranges of a pair are merged, and a tile 0.109,
// 0.149 or 0.216 with one, two or three CTAs on an SM.  256 pairs of 256
// tiles: 42.5 with one range each, 52.9 with two, 41.8 with even ranges over
// the pairs' borders; 256 pairs of 32 tiles: 8.7 with one range each, 17.7
// with even ranges.
KvSplit kv_split(const kin_dims& d, int k, bool dense) {
  const int tpb = d.block_size / kTileTokens;
  const int64_t pairs = pairs_of(d);
  const int most = (dense ? kKvItemTiles / 2 : kKvItemTiles) / tpb;  // dense: lengths unknown here, ranges may be empty
  const int least = (8 + tpb - 1) / tpb;                             // a step of each warp
  const int64_t wave = (int64_t)kTargetSMs * kKvCtasPerSm;
  auto range_us = [&](int64_t tiles, int64_t per_sm, bool merged) {
    return (double)tiles * (per_sm <= 1 ? 0.109 : per_sm == 2 ? 0.149 : 0.216) + (merged ? 5.0 : 4.0);
  };
  KvSplit best{0, 0, 0};
  double best_us = 0;
  auto consider = [&](int per) {
    const int64_t n = pairs * ((k + per - 1) / per), full = n / wave, rest = n % wave;
    double us = (double)full * range_us((int64_t)per * tpb, kKvCtasPerSm, per < k);
    if (rest) us += range_us((int64_t)per * tpb, (rest + kTargetSMs - 1) / kTargetSMs, per < k);
    if (!best.per || us < best_us) {
      best = KvSplit{per, (k + per - 1) / per * per, 0};
      best_us = us;
    }
  };
  const int c0 = (k + most - 1) / most;
  for (int c = c0; c < c0 + 64; ++c) {
    const int per = (k + c - 1) / c;
    if (c > c0 && per < least) break;
    consider(per);
  }
  // dense: longer ranges where one wave holds them all, none waits for another
  // (8 pairs of 128K tokens, 8 heads: 50 us, 72 in ranges of 128 tiles or less;
  // 128 pairs of 8192: 42 for 46.5)
  if (dense && pairs <= wave) {
    const int c = (int)(wave / pairs), per = (k + c - 1) / c;
    if (per > most && per <= kKvItemTiles / tpb) consider(per);
  }
  // even ranges: whole waves of them; one may run over several short pairs
  const int64_t slots = pairs * k, cap = k <= most ? slots : most;
  const int64_t waves = (slots + wave * cap - 1) / (wave * cap);
  const int64_t per = (slots + wave * waves - 1) / (wave * waves);
  if (!dense && per >= least && per != k && per < 2 * k) {
    const double us = (double)waves * (range_us(per * tpb, kKvCtasPerSm, true) + 5.0 * (double)((per - 1) / k + 1));
    if (us < best_us) best = KvSplit{(int)per, k, 0};
  }
  if (dense && pairs * (best.stride / best.per) <= wave) best.fit = std::min(best.per, (32 + tpb - 1) / tpb);
  return best;
}

// The slots of the kept blocks of a pair: at most k_blocks, at most all.
int kv_slots(const kin_dims& d, int k_blocks) {
  const int nb = nbcap_of(d);
  return k_blocks == 0 || k_blocks > nb ? nb : k_blocks;
}

// CTAs whose ranges a pair's slots may meet.
int kv_max_chunks(int k, const KvSplit& s) {
  return s.stride % s.per == 0 ? s.stride / s.per : (k + s.per - 2) / s.per + 1;
}

struct KvWs {
  size_t counters, partials, z, lse2, total;
};

// The select's regions first (its counters' place is this call's too), so
// that one buffer serves both.
KvWs kv_ws_layout(const kin_dims& d, int k_blocks, const KvSplit& split, bool acc) {
  KvWs w;
  const size_t pairs = (size_t)pairs_of(d), g = (size_t)(d.num_q_heads / d.num_kv_heads);
  const int k = kv_slots(d, k_blocks);
  size_t off = 0;
  w.counters = 0;
  off = k_blocks >= 2 ? ws_layout(d, k_blocks).total : align_up(pairs * sizeof(uint32_t));
  w.partials = off;
  off = align_up(off + pairs * (size_t)kv_max_chunks(k, split) * g * kPartStride * sizeof(float));
  w.z = off;
  if (acc) off = align_up(off + pairs * (size_t)k * d.block_size * g * sizeof(float));
  w.lse2 = off;
  if (acc) off = align_up(off + pairs * g * sizeof(float));
  w.total = off;
  return w;
}

}  // namespace

KIN_EXPORT kin_status kin_kv4_store(const kin_dims* dims, const kin_kv* src, const kin_kv* dst,
                                    const int32_t* seq_lens, void* block_means, int32_t means_dtype,
                                    int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  KvView s, d;
  if ((st = kv_view(*dims, src, &s)) != KIN_OK || (st = kv_view(*dims, dst, &d)) != KIN_OK) return st;
  if (s.int4 || !d.int4 || !seq_lens) return KIN_ERR_INVALID_ARG;
  if (caches_meet(*dims, s, *dims, d)) return KIN_ERR_INVALID_ARG;  // rows are read in no order
  Kv4WriteParams p{};
  st = means_layout(*dims, d, block_means, means_dtype, &p.means_flag, &p.means_per_page, &p.mean_rows);
  if (st != KIN_OK) return st;
  p.dst = d;
  p.k_src = s.k;
  p.v_src = s.v;
  p.src_pages = s.pages;
  p.seq_lens = seq_lens;
  p.means = block_means;
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.bs = dims->block_size;
  p.nbcap = nbcap_of(*dims);
  p.span = p.nbcap;
  return from_cuda(launch_kv4_write(p, static_cast<cudaStream_t>(stream)));
}

KIN_EXPORT kin_status kin_kv4_append(const kin_dims* dims, const kin_kv* kv, void* block_means, int32_t means_dtype,
                                     const int32_t* seq_lens, int32_t* new_lens, const void* k_new, const void* v_new,
                                     int32_t n_new, int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  if ((st = check_update_count(dims, n_new)) != KIN_OK) return st;
  KvView d;
  if ((st = kv_view(*dims, kv, &d)) != KIN_OK) return st;
  if (!d.int4 || !seq_lens || !new_lens || !k_new || !v_new) return KIN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new)) return KIN_ERR_INVALID_ARG;
  const size_t lens_bytes = (size_t)dims->batch * sizeof(int32_t);
  if (new_lens != seq_lens && meet(new_lens, lens_bytes, seq_lens, lens_bytes)) return KIN_ERR_INVALID_ARG;
  Kv4WriteParams p{};
  st = means_layout(*dims, d, block_means, means_dtype, &p.means_flag, &p.means_per_page, &p.mean_rows);
  if (st != KIN_OK) return st;
  if (n_new == 0 && new_lens == seq_lens) return KIN_OK;
  p.dst = d;
  p.k_src = static_cast<const uint8_t*>(k_new);
  p.v_src = static_cast<const uint8_t*>(v_new);
  p.src_pages = contiguous();
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.means = n_new ? block_means : nullptr;
  p.dev_status = dev_status;
  p.append = 1;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.bs = dims->block_size;
  p.nbcap = nbcap_of(*dims);
  p.n_new = n_new;
  p.span = n_new ? (n_new + p.bs - 2) / p.bs + 1 : 1;  // blocks that n_new rows can touch
  return from_cuda(launch_kv4_write(p, static_cast<cudaStream_t>(stream)));
}

KIN_EXPORT kin_status kin_kv4_load(const kin_dims* dims, const kin_kv* kv, const int32_t* seq_lens,
                                   const int32_t* starts, int32_t n, void* k_out, void* v_out, int32_t* dev_status,
                                   void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  if (n < 0) return KIN_ERR_INVALID_ARG;
  if (n > dims->max_seq_len) return KIN_ERR_CAPACITY;
  KvView s;
  if ((st = kv_view(*dims, kv, &s)) != KIN_OK) return st;
  if (!s.int4 || !seq_lens || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return KIN_ERR_INVALID_ARG;
  if (n == 0) return KIN_OK;
  const size_t out_bytes = (size_t)pairs_of(*dims) * n * kHeadDim * 2;
  if (meet(k_out, out_bytes, v_out, out_bytes) || meets_cache(k_out, out_bytes, *dims, s) ||
      meets_cache(v_out, out_bytes, *dims, s))
    return KIN_ERR_INVALID_ARG;
  Kv4LoadParams p{};
  p.src = s;
  p.seq_lens = seq_lens;
  p.starts = starts;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.bs = dims->block_size;
  p.n = n;
  return from_cuda(launch_kv4_load(p, static_cast<cudaStream_t>(stream)));
}

KIN_EXPORT size_t kin_kv_attn_workspace_bytes(const kin_dims* dims, int32_t k_blocks, int32_t with_acc) {
  if (check_dims(dims) != KIN_OK || k_blocks < 0 || k_blocks == 1) return 0;
  const KvSplit split = kv_split(*dims, kv_slots(*dims, k_blocks), k_blocks == 0);
  return kv_ws_layout(*dims, k_blocks, split, with_acc != 0).total;
}

KIN_EXPORT kin_status kin_kv_decode_attn(const kin_dims* dims, const void* q, const kin_kv* kv, const int32_t* seq_lens,
                                         const int32_t* sel_idx, const int32_t* sel_cnt, int32_t k_blocks,
                                         float softmax_scale, void* out, float* lse, float* acc, void* workspace,
                                         size_t ws_bytes, int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK) return st;
  // no selection: every block (k_blocks 0); else both arrays and a budget
  if (k_blocks < 0 || k_blocks == 1 || (k_blocks == 0) != (sel_idx == nullptr) || (k_blocks == 0) != (sel_cnt == nullptr))
    return KIN_ERR_INVALID_ARG;
  KvAttnParams p{};
  if ((st = kv_view(*dims, kv, &p.kv)) != KIN_OK) return st;
  if (!q || !seq_lens || !out || !aligned16(q) || !aligned16(out)) return KIN_ERR_INVALID_ARG;
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale)) return KIN_ERR_INVALID_ARG;
  const KvSplit split = kv_split(*dims, kv_slots(*dims, k_blocks), k_blocks == 0);
  const KvWs w = kv_ws_layout(*dims, k_blocks, split, acc != nullptr);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0 || ws_bytes < w.total)
    return KIN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.seq_lens = seq_lens;
  p.sel_idx = sel_idx;
  p.sel_cnt = sel_cnt;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  p.z = reinterpret_cast<float*>(ws + w.z);
  p.acc = acc;
  p.partials = reinterpret_cast<float*>(ws + w.partials);
  p.counters = reinterpret_cast<uint32_t*>(ws + w.counters);
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.Hq = dims->num_q_heads;
  p.g = dims->num_q_heads / dims->num_kv_heads;
  p.bs = dims->block_size;
  p.k_row = k_blocks;
  p.k = kv_slots(*dims, k_blocks);
  p.per = split.per;
  p.stride = split.stride;
  p.fit = split.fit;
  if ((int64_t)pairs_of(*dims) * p.stride >= (int64_t)1 << 31) return KIN_ERR_CAPACITY;
  p.slots = pairs_of(*dims) * p.stride;
  p.max_chunks = kv_max_chunks(p.k, split);
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)kHeadDim);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.two24 = 1u << 24;
  return from_cuda(launch_kv_attn(p, static_cast<cudaStream_t>(stream)));
}

namespace {

struct EvictWs {
  size_t sel, keys, total;
};

EvictWs evict_ws_layout(const kin_dims& d, int n_keep) {
  EvictWs w;
  const size_t pairs = (size_t)pairs_of(d);
  size_t off = 0;
  w.sel = off;
  off = align_up(off + pairs * (size_t)n_keep * sizeof(int32_t));
  w.keys = off;
  if (d.max_seq_len > kTokenKeyCap) off = align_up(off + pairs * (size_t)d.max_seq_len * sizeof(uint32_t));
  w.total = off;
  return w;
}

}  // namespace

KIN_EXPORT size_t kin_kv_evict_workspace_bytes(const kin_dims* dims, int32_t n_keep) {
  if (check_dims(dims) != KIN_OK || n_keep < 1 || n_keep > dims->max_seq_len) return 0;
  return evict_ws_layout(*dims, n_keep).total;
}

KIN_EXPORT kin_status kin_kv_evict(const kin_dims* dims, const kin_kv* kv, const float* acc, const int32_t* seq_lens,
                                   int32_t n_keep, int32_t n_sink, int32_t n_recent, const kin_dims* dst_dims,
                                   const kin_kv* dst, float* dst_acc, int32_t* dst_lens, void* block_means,
                                   int32_t means_dtype, int32_t* sel_tokens, void* workspace, size_t ws_bytes,
                                   int32_t* dev_status, void* stream) {
  KIN_NVTX_RANGE();
  kin_status st = check_dims(dims);
  if (st != KIN_OK || (st = check_dims(dst_dims)) != KIN_OK) return st;
  if (n_keep < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > n_keep) return KIN_ERR_INVALID_ARG;
  if (n_keep > dims->max_seq_len || n_keep > dst_dims->max_seq_len) return KIN_ERR_CAPACITY;
  if (dst_dims->batch != dims->batch || dst_dims->num_kv_heads != dims->num_kv_heads ||
      dst_dims->num_q_heads != dims->num_q_heads || dst_dims->block_size != dims->block_size)
    return KIN_ERR_INVALID_ARG;
  EvictParams p{};
  if ((st = kv_view(*dims, kv, &p.src)) != KIN_OK || (st = kv_view(*dst_dims, dst, &p.dst)) != KIN_OK) return st;
  if (p.src.int4 != p.dst.int4 || !acc || !seq_lens || !dst_lens) return KIN_ERR_INVALID_ARG;
  // every head's tokens move at once: the two caches are two buffers, or
  // disjoint pages of one pool
  if (same_cache(p.src, p.dst) && !(p.src.pages.table && p.dst.pages.table && p.src.k == p.dst.k && p.src.v == p.dst.v))
    return KIN_ERR_INVALID_ARG;
  if (p.src.pages.table && p.src.pages.table == p.dst.pages.table && p.src.k == p.dst.k) return KIN_ERR_INVALID_ARG;
  if (!(p.src.pages.table && p.dst.pages.table) && caches_meet(*dims, p.src, *dst_dims, p.dst)) return KIN_ERR_INVALID_ARG;
  const size_t acc_bytes = (size_t)pairs_of(*dims) * sizeof(float), lens_bytes = (size_t)dims->batch * sizeof(int32_t);
  if (meet(acc, acc_bytes * dims->max_seq_len, dst_acc, acc_bytes * dst_dims->max_seq_len) ||
      meet(seq_lens, lens_bytes, dst_lens, lens_bytes))
    return KIN_ERR_INVALID_ARG;
  st = means_layout(*dst_dims, p.dst, block_means, means_dtype, &p.means_flag, &p.means_per_page, &p.mean_rows);
  if (st != KIN_OK) return st;
  const EvictWs w = evict_ws_layout(*dims, n_keep);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0 || ws_bytes < w.total)
    return KIN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.acc = acc;
  p.dst_acc = dst_acc;
  p.seq_lens = seq_lens;
  p.dst_lens = dst_lens;
  p.sel = sel_tokens ? sel_tokens : reinterpret_cast<int32_t*>(ws + w.sel);
  p.key_scratch = reinterpret_cast<uint32_t*>(ws + w.keys);
  p.means = block_means;
  p.dev_status = dev_status;
  p.B = dims->batch;
  p.Hkv = dims->num_kv_heads;
  p.bs = dims->block_size;
  p.nbcap_dst = nbcap_of(*dst_dims);
  p.n_keep = n_keep;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_evict_select(p, s);
  if (e == cudaSuccess) e = launch_evict_move(p, s);
  return from_cuda(e);
}
