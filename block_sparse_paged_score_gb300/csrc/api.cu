// api.cu -- the C ABI of libbsp (declared in include/bsp.h): argument
// validation on the host, the split plans, and the kernel launches.  Nothing
// here allocates, synchronises or reads device memory.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/bsp.h"
#include "common.cuh"
#include "kernels.h"

using namespace bsp;

namespace {

std::atomic<int32_t> g_last_cuda_error{0};
std::atomic<int64_t> g_launches{0};

std::atomic<int> g_sms[kMaxDevices];

int device_sms() {
  return cached_per_device(g_sms, [] {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                  cudaSuccess || n <= 0)
      n = 148;
    return n;
  });
}

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool valid_dtype(int32_t d) { return d == BSP_BF16 || d == BSP_FP8_E4M3 || d == BSP_MXFP4; }
bool valid_group(int32_t g) { return g == 1 || g == 2 || g == 4 || g == 8 || g == 16; }

bsp_status cuda_status(cudaError_t e) {
  if (e != cudaSuccess) {
    g_last_cuda_error.store(static_cast<int32_t>(e));
    return BSP_ERR_CUDA;
  }
  return BSP_OK;
}

int64_t index_field(int32_t dtype) {
  return dtype == BSP_BF16 ? kBf16IndexField : (dtype == BSP_FP8_E4M3 ? kFp8IndexField : kMxField);
}

bsp_status check_kv(const bsp_kv_cache* kv) {
  if (!kv || !valid_dtype(kv->dtype) || kv->num_kv_heads < 1 || !kv->k_base || !kv->v_base) return BSP_ERR_INVALID_ARG;
  if (!al(kv->k_base, 16) || !al(kv->v_base, 16) || kv->id_stride_bytes <= 0 || kv->id_stride_bytes % 16)
    return BSP_ERR_INVALID_ARG;
  const int64_t page = kv->dtype == BSP_BF16 ? 4096 : 2048;
  if (kv->dtype == BSP_MXFP4 ? kv->id_stride_bytes < 2LL * kv->num_kv_heads * kMxField
                             : kv->id_stride_bytes < kv->num_kv_heads * page)
    return BSP_ERR_INVALID_ARG;
  if (kv->num_ids < 0 || kv->num_blocks < 0) return BSP_ERR_INVALID_ARG;
  return BSP_OK;
}

bsp_status check_idx(const bsp_index_cache* idx) {
  if (!idx || !valid_dtype(idx->dtype) || idx->num_heads < 1 || !idx->base || !al(idx->base, 16))
    return BSP_ERR_INVALID_ARG;
  if (idx->block_stride_bytes < idx->num_heads * index_field(idx->dtype) || idx->block_stride_bytes % 16 ||
      idx->num_blocks < 0)
    return BSP_ERR_INVALID_ARG;
  return BSP_OK;
}

}  // namespace

extern "C" {

int64_t bsp_kv_block_bytes(int32_t dtype, int32_t num_kv_heads) {
  if (!valid_dtype(dtype) || num_kv_heads < 1) return -1;
  if (dtype == BSP_MXFP4) return 2LL * num_kv_heads * kMxField;
  return 16LL * num_kv_heads * (dtype == BSP_BF16 ? 4096 : 2048);
}

int64_t bsp_index_field_bytes(int32_t dtype) { return valid_dtype(dtype) ? index_field(dtype) : -1; }

bsp_status bsp_kv_cache_interleaved(int32_t dtype, int32_t num_kv_heads, void* base, int64_t num_blocks,
                                    float k_scale, float v_scale, bsp_kv_cache* out) {
  if (!out || !valid_dtype(dtype) || num_kv_heads < 1 || !base || !al(base, 16) || num_blocks < 1)
    return BSP_ERR_INVALID_ARG;
  out->dtype = dtype;
  out->num_kv_heads = num_kv_heads;
  out->k_base = base;
  out->num_blocks = num_blocks;
  out->k_scale = k_scale;
  out->v_scale = v_scale;
  if (dtype == BSP_MXFP4) {
    out->id_stride_bytes = 2LL * num_kv_heads * kMxField;
    out->v_base = static_cast<uint8_t*>(base) + static_cast<int64_t>(num_kv_heads) * kMxField;
    out->num_ids = 8 * num_blocks;
  } else {
    out->id_stride_bytes = static_cast<int64_t>(num_kv_heads) * (dtype == BSP_BF16 ? 4096 : 2048);
    out->v_base = static_cast<uint8_t*>(base) + 8 * out->id_stride_bytes;
    out->num_ids = 16 * num_blocks - 8;
  }
  return BSP_OK;
}

bsp_status bsp_index_cache_packed(int32_t dtype, int32_t num_heads, void* base, int64_t num_blocks,
                                  bsp_index_cache* out) {
  if (!out || !valid_dtype(dtype) || num_heads < 1 || !base || !al(base, 16) || num_blocks < 1)
    return BSP_ERR_INVALID_ARG;
  out->dtype = dtype;
  out->num_heads = num_heads;
  out->base = base;
  out->block_stride_bytes = num_heads * index_field(dtype);
  out->num_blocks = num_blocks;
  return BSP_OK;
}

bsp_status bsp_kv_page_write(const bsp_kv_cache* kv, const bsp_index_cache* idx, const void* k, const void* v,
                             const void* idx_k, const int64_t* slot, int32_t num_tokens, int32_t* dev_err,
                             bsp_stream_t stream) {
  bsp_status st = check_kv(kv);
  if (st != BSP_OK) return st;
  if (num_tokens < 0) return BSP_ERR_INVALID_ARG;
  if (num_tokens == 0) return BSP_OK;
  if (!k || !v || !slot || !al(k, 16) || !al(v, 16) || !al(slot, 8)) return BSP_ERR_INVALID_ARG;
  if (idx_k && !idx) return BSP_ERR_INVALID_ARG;
  if (idx_k) {
    if ((st = check_idx(idx)) != BSP_OK) return st;
    if (!al(idx_k, 16)) return BSP_ERR_INVALID_ARG;
  }
  KvWriteParams p{};
  p.kv_dtype = kv->dtype;
  p.hkv = kv->num_kv_heads;
  p.k_base = static_cast<uint8_t*>(kv->k_base);
  p.v_base = static_cast<uint8_t*>(kv->v_base);
  p.id_stride = kv->id_stride_bytes;
  p.num_blocks = kv->num_blocks;
  p.k_scale = kv->k_scale;
  p.v_scale = kv->v_scale;
  if (idx_k) {
    p.idx_dtype = idx->dtype;
    p.hidx = idx->num_heads;
    p.idx_base = static_cast<uint8_t*>(idx->base);
    p.idx_block_stride = idx->block_stride_bytes;
    p.idx_num_blocks = idx->num_blocks;
  }
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.idx_k = static_cast<const uint16_t*>(idx_k);
  p.slot = slot;
  p.num_tokens = num_tokens;
  p.err = dev_err;
  st = cuda_status(launch_kv_page_write(p, reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_cast_e4m3(const void* x, void* out, int64_t n, bsp_stream_t stream) {
  if (n < 0) return BSP_ERR_INVALID_ARG;
  if (n == 0) return BSP_OK;
  if (!x || !out || !al(x, 16) || !al(out, 8)) return BSP_ERR_INVALID_ARG;
  bsp_status st = cuda_status(launch_cast_e4m3(static_cast<const uint16_t*>(x), static_cast<uint8_t*>(out), n,
                                               reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_row_lengths_decode(const int32_t* seq_lens, int32_t num_seqs, int32_t q_len, int32_t num_heads,
                                  int32_t* row_seq, int32_t* row_len, bsp_stream_t stream) {
  if (num_seqs < 0 || q_len < 1 || num_heads < 1) return BSP_ERR_INVALID_ARG;
  if (num_seqs == 0) return BSP_OK;
  if (!seq_lens || !row_seq || !row_len) return BSP_ERR_INVALID_ARG;
  bsp_status st = cuda_status(launch_row_lengths_decode(seq_lens, num_seqs, q_len, num_heads, row_seq, row_len,
                                                        reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_row_lengths_prefill(const int32_t* query_req_id, const int32_t* query_abs_pos, int32_t num_tokens,
                                   int32_t num_heads, int32_t* row_seq, int32_t* row_len, bsp_stream_t stream) {
  if (num_tokens < 0 || num_heads < 1) return BSP_ERR_INVALID_ARG;
  if (num_tokens == 0) return BSP_OK;
  if (!query_req_id || !query_abs_pos || !row_seq || !row_len) return BSP_ERR_INVALID_ARG;
  bsp_status st = cuda_status(launch_row_lengths_prefill(query_req_id, query_abs_pos, num_tokens, num_heads, row_seq,
                                                         row_len, reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

// the decode scorer's argument checks (also run by the decode step before its
// first launch)
static bsp_status index_score_check(const bsp_index_cache* idx, const void* idx_q, int32_t q_dtype,
                                    const int32_t* block_table, int32_t bt_stride, const int32_t* row_seq,
                                    const int32_t* row_len, int32_t num_rows, int32_t q_group, int32_t max_pages,
                                    const float* scores) {
  bsp_status st = check_idx(idx);
  if (st != BSP_OK) return st;
  if (num_rows < 0 || max_pages < 1 || bt_stride < 1) return BSP_ERR_INVALID_ARG;
  if (q_dtype != BSP_BF16 && q_dtype != BSP_FP8_E4M3) return BSP_ERR_UNSUPPORTED;
  if (q_group < 1 || q_group > 8) return BSP_ERR_UNSUPPORTED;
  if (num_rows % idx->num_heads) return BSP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) > static_cast<int64_t>(bt_stride) * 8) return BSP_ERR_INVALID_ARG;
  if (num_rows == 0) return BSP_OK;
  if (!idx_q || !block_table || !row_seq || !row_len || !scores || !al(idx_q, 8)) return BSP_ERR_INVALID_ARG;
  return BSP_OK;
}

// seq_is_group: the decode step's own rows, where query group g is sequence g
static bsp_status index_score_impl(const bsp_index_cache* idx, const void* idx_q, int32_t q_dtype,
                                   const int32_t* block_table, int32_t bt_stride, const int32_t* row_seq,
                                   const int32_t* row_len, int32_t num_rows, int32_t q_group, int32_t max_pages,
                                   float* scores, int32_t* dev_err, bsp_stream_t stream, int32_t seq_is_group,
                                   const TopkParams* sel = nullptr, int32_t* sel_counters = nullptr) {
  bsp_status st = index_score_check(idx, idx_q, q_dtype, block_table, bt_stride, row_seq, row_len, num_rows,
                                    q_group, max_pages, scores);
  if (st != BSP_OK || num_rows == 0) return st;
  IndexScoreParams p{};
  p.idx_dtype = idx->dtype;
  p.hidx = idx->num_heads;
  p.idx_base = static_cast<const uint8_t*>(idx->base);
  p.block_stride = idx->block_stride_bytes;
  p.num_blocks = idx->num_blocks;
  p.q = idx_q;
  p.q_dtype = q_dtype;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.row_seq = row_seq;
  p.row_len = row_len;
  p.num_rows = num_rows;
  p.num_tokens = num_rows / idx->num_heads;
  p.q_group = q_group;
  p.max_pages = max_pages;
  p.scores = scores;
  p.err = dev_err;
  p.seq_is_group = seq_is_group;
  if (sel) {
    p.sel = *sel;
    p.sel_counters = sel_counters;
  }
  st = cuda_status(launch_index_score(p, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_index_score(const bsp_index_cache* idx, const void* idx_q, int32_t q_dtype,
                           const int32_t* block_table, int32_t bt_stride, const int32_t* row_seq,
                           const int32_t* row_len, int32_t num_rows, int32_t q_group, int32_t max_pages,
                           float* scores, int32_t* dev_err, bsp_stream_t stream) {
  return index_score_impl(idx, idx_q, q_dtype, block_table, bt_stride, row_seq, row_len, num_rows, q_group,
                          max_pages, scores, dev_err, stream, 0);
}

bsp_status bsp_index_score_prefill(const bsp_index_cache* idx, const void* idx_q, int32_t q_dtype,
                                   const int32_t* block_table, int32_t bt_stride, const int32_t* row_seq,
                                   const int32_t* row_len, int32_t num_rows, const int32_t* cu_tokens,
                                   int32_t num_chunks, int32_t max_tiles, int32_t max_pages, float* scores,
                                   int32_t* dev_err, bsp_stream_t stream) {
  bsp_status st = check_idx(idx);
  if (st != BSP_OK) return st;
  const bool mx = idx->dtype == BSP_MXFP4;
  if ((idx->dtype != BSP_FP8_E4M3 && !mx) || q_dtype != BSP_FP8_E4M3 || idx->num_heads != 1)
    return BSP_ERR_UNSUPPORTED;
  if (idx->block_stride_bytes % (mx ? 64 : 128)) return BSP_ERR_UNSUPPORTED;
  if (num_rows < 0 || max_pages < 1 || bt_stride < 1 || num_chunks < 0 || max_tiles < 0) return BSP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) > static_cast<int64_t>(bt_stride) * 8) return BSP_ERR_INVALID_ARG;
  if (num_rows == 0 || num_chunks == 0 || max_tiles == 0) return BSP_OK;
  if (!idx_q || !block_table || !row_seq || !row_len || !scores || !cu_tokens || !al(idx_q, 16))
    return BSP_ERR_INVALID_ARG;
  PrefillScoreParams p{};
  p.idx_base = static_cast<const uint8_t*>(idx->base);
  p.block_stride = idx->block_stride_bytes;
  p.num_blocks = idx->num_blocks;
  p.q = static_cast<const uint8_t*>(idx_q);
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.row_seq = row_seq;
  p.row_len = row_len;
  p.num_rows = num_rows;
  p.cu_tokens = cu_tokens;
  p.num_chunks = num_chunks;
  p.max_tiles = max_tiles;
  p.max_pages = max_pages;
  p.scores = scores;
  p.err = dev_err;
  cudaError_t e = mx ? launch_index_score_prefill_mx(p, reinterpret_cast<cudaStream_t>(stream))
                     : launch_index_score_prefill(p, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return BSP_ERR_UNSUPPORTED;
  st = cuda_status(e);
  if (st == BSP_OK) ++g_launches;
  return st;
}

// The selector's parameters, checked.  rows_per_seq > 0: row r belongs to
// sequence r / rows_per_seq (the decode step's own rows).
static bsp_status topk_params(const float* scores, int32_t num_rows, int32_t max_pages, const int32_t* row_seq,
                              const int32_t* row_len, const int32_t* block_table, int32_t bt_stride, int32_t kv_dtype,
                              int32_t k_pages, int32_t flags, int32_t* topk_idx, int32_t* sparse_bt,
                              int32_t* sparse_ctx, int32_t rows_per_seq, TopkParams& p) {
  if (num_rows < 0 || max_pages < 1 || bt_stride < 1 || k_pages < 1 || !valid_dtype(kv_dtype))
    return BSP_ERR_INVALID_ARG;
  if (k_pages > 2048 || max_pages > 65536) return BSP_ERR_UNSUPPORTED;
  if ((flags & BSP_SELECT_BLOCKS) && k_pages < kPagesPerSide) return BSP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) > static_cast<int64_t>(bt_stride) * 8) return BSP_ERR_INVALID_ARG;
  if (num_rows > 0 &&
      (!scores || !row_seq || !row_len || !block_table || !topk_idx || !sparse_bt || !sparse_ctx || !al(scores, 16)))
    return BSP_ERR_INVALID_ARG;
  p = TopkParams{};
  p.scores = scores;
  p.num_rows = num_rows;
  p.max_pages = max_pages;
  p.row_seq = row_seq;
  p.row_len = row_len;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.id_mul = kv_dtype == BSP_MXFP4 ? 8 : 16;
  p.k_pages = k_pages;
  p.force_tail = (flags & BSP_FORCE_TAIL) ? 1 : 0;
  p.topk_idx = topk_idx;
  p.sparse_bt = sparse_bt;
  p.sparse_ctx = sparse_ctx;
  p.rows_per_seq = rows_per_seq;
  p.blocks = (flags & BSP_SELECT_BLOCKS) ? 1 : 0;
  return BSP_OK;
}

static bsp_status topk_impl(const float* scores, int32_t num_rows, int32_t max_pages, const int32_t* row_seq,
                            const int32_t* row_len, const int32_t* block_table, int32_t bt_stride, int32_t kv_dtype,
                            int32_t k_pages, int32_t flags, int32_t* topk_idx, int32_t* sparse_bt,
                            int32_t* sparse_ctx, bsp_stream_t stream, int32_t rows_per_seq) {
  TopkParams p;
  bsp_status st = topk_params(scores, num_rows, max_pages, row_seq, row_len, block_table, bt_stride, kv_dtype, k_pages,
                              flags, topk_idx, sparse_bt, sparse_ctx, rows_per_seq, p);
  if (st != BSP_OK || num_rows == 0) return st;
  st = cuda_status(launch_topk_select(p, reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_topk_select(const float* scores, int32_t num_rows, int32_t max_pages, const int32_t* row_seq,
                           const int32_t* row_len, const int32_t* block_table, int32_t bt_stride, int32_t kv_dtype,
                           int32_t k_pages, int32_t flags, int32_t* topk_idx, int32_t* sparse_bt, int32_t* sparse_ctx,
                           bsp_stream_t stream) {
  return topk_impl(scores, num_rows, max_pages, row_seq, row_len, block_table, bt_stride, kv_dtype, k_pages, flags,
                   topk_idx, sparse_bt, sparse_ctx, stream, 0);
}

size_t bsp_sparse_pa_decode_workspace_bytes(int32_t num_rows, int32_t k_pages, int32_t group) {
  (void)group;
  if (num_rows <= 0 || k_pages <= 0) return 0;
  // the largest of the three KV formats' plans (the query has no format)
  size_t need = 0;
  for (int32_t kv : {BSP_BF16, BSP_FP8_E4M3, BSP_MXFP4})
    need = std::max(need, sparse_pa_ws_bytes(num_rows, sparse_pa_plan(kv, num_rows, k_pages, device_sms())));
  return need;
}

int32_t bsp_sparse_pa_decode_splits(int32_t kv_dtype, int32_t num_rows, int32_t k_pages) {
  if (!valid_dtype(kv_dtype) || num_rows < 1 || k_pages < 1) return 0;
  return sparse_pa_plan(kv_dtype, num_rows, k_pages, device_sms()).nsplit;
}

}  // extern "C"

namespace bsp {

bsp_status sparse_pa_check_args(const bsp_kv_cache* kv, const void* q, int32_t q_dtype, int32_t num_q_heads,
                                const int32_t* sparse_bt, const int32_t* sparse_ctx, int32_t num_rows,
                                int32_t k_pages, const void* out) {
  bsp_status st = check_kv(kv);
  if (st != BSP_OK) return st;
  if (num_rows < 0 || k_pages < 1 || num_q_heads < 1) return BSP_ERR_INVALID_ARG;
  if (num_q_heads % kv->num_kv_heads || num_rows % kv->num_kv_heads) return BSP_ERR_INVALID_ARG;
  if (!valid_group(num_q_heads / kv->num_kv_heads)) return BSP_ERR_UNSUPPORTED;
  if (q_dtype != BSP_BF16 && q_dtype != BSP_FP8_E4M3) return BSP_ERR_UNSUPPORTED;
  if (num_rows == 0) return BSP_OK;
  if (!q || !sparse_bt || !sparse_ctx || !out || !al(out, 16) || !al(q, 16)) return BSP_ERR_INVALID_ARG;
  return BSP_OK;
}

size_t sparse_pa_decode_ws_need(int32_t kv_dtype, int32_t num_rows, int32_t k_pages) {
  if (num_rows <= 0 || k_pages <= 0) return 0;
  return sparse_pa_ws_bytes(num_rows, sparse_pa_plan(kv_dtype, num_rows, k_pages, device_sms()));
}

}  // namespace bsp

namespace {

// whether [a, a + an) and [b, b + bn) share a byte
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an > 0 && bn > 0 && x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

// whether [a, a + an) shares a byte with one of the pieces [b + i * step, + bn), i < n
bool overlap_pieces(const void* a, int64_t an, const void* b, int64_t bn, int64_t step, int64_t n) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  if (!a || !b || an <= 0 || bn <= 0 || n <= 0 || x + static_cast<uintptr_t>(an) <= y) return false;
  // the last piece that starts before the range ends
  const auto i = std::min<uintptr_t>((x + static_cast<uintptr_t>(an) - 1 - y) / static_cast<uintptr_t>(step),
                                     static_cast<uintptr_t>(n - 1));
  return x < y + i * static_cast<uintptr_t>(step) + static_cast<uintptr_t>(bn);
}

// whether a range shares a byte with what a cache's blocks hold
bool overlap_cache(const void* a, int64_t an, const bsp_kv_cache* kv) {
  if (!kv) return false;
  const int64_t heads = kv->num_kv_heads;
  if (kv->dtype == BSP_MXFP4)
    return overlap_pieces(a, an, kv->k_base, heads * kMxField, kv->id_stride_bytes, kv->num_blocks) ||
           overlap_pieces(a, an, kv->v_base, heads * kMxField, kv->id_stride_bytes, kv->num_blocks);
  const int64_t page = heads * (kv->dtype == BSP_BF16 ? 4096 : 2048), step = 16 * kv->id_stride_bytes;
  for (int j = 0; j < 8; ++j)
    if (overlap_pieces(a, an, static_cast<const uint8_t*>(kv->k_base) + j * kv->id_stride_bytes, page, step,
                       kv->num_blocks) ||
        overlap_pieces(a, an, static_cast<const uint8_t*>(kv->v_base) + j * kv->id_stride_bytes, page, step,
                       kv->num_blocks))
      return true;
  return false;
}
bool overlap_cache(const void* a, int64_t an, const bsp_index_cache* idx) {
  return idx && overlap_pieces(a, an, idx->base, idx->num_heads * index_field(idx->dtype), idx->block_stride_bytes,
                               idx->num_blocks);
}

// the cache fields of a writer or reader
void set_caches(KvWriteParams& p, const bsp_kv_cache* kv, const bsp_index_cache* idx) {
  if (kv) {
    p.kv_dtype = kv->dtype;
    p.hkv = kv->num_kv_heads;
    p.k_base = static_cast<uint8_t*>(kv->k_base);
    p.v_base = static_cast<uint8_t*>(kv->v_base);
    p.id_stride = kv->id_stride_bytes;
    p.num_blocks = kv->num_blocks;
    p.k_scale = kv->k_scale;
    p.v_scale = kv->v_scale;
  }
  if (idx) {
    p.idx_dtype = idx->dtype;
    p.hidx = idx->num_heads;
    p.idx_base = static_cast<uint8_t*>(idx->base);
    p.idx_block_stride = idx->block_stride_bytes;
    p.idx_num_blocks = idx->num_blocks;
  }
}

}  // namespace

extern "C" {

bsp_status bsp_step_tables(const bsp_step_tables_args* a, bsp_stream_t stream) {
  if (!a || a->num_seqs < 0 || a->bt_stride < 1 || a->num_free < 0 || a->token_capacity < 0 || a->num_blocks < 0)
    return BSP_ERR_INVALID_ARG;
  if (a->num_seqs > 65536) return BSP_ERR_UNSUPPORTED;
  if (!a->cu_tokens || !a->blocks_taken) return BSP_ERR_INVALID_ARG;
  if (a->num_seqs && (!a->context_lens || !a->new_lens || !a->block_table || !a->seq_lens)) return BSP_ERR_INVALID_ARG;
  if (a->num_free && !a->free_blocks) return BSP_ERR_INVALID_ARG;
  if (a->token_capacity && (!a->slot || !a->query_req_id || !a->query_abs_pos)) return BSP_ERR_INVALID_ARG;
  const int64_t n = a->num_seqs, cap = a->token_capacity;
  struct Range {
    const void* p;
    int64_t bytes, align;
  };
  const Range in[] = {{a->context_lens, 4 * n, 4}, {a->new_lens, 4 * n, 4}, {a->free_blocks, 4LL * a->num_free, 4},
                      {a->free_head, 4, 4}};
  const Range out[] = {{a->block_table, 4 * n * a->bt_stride, 4}, {a->seq_lens, 4 * n, 4}, {a->cu_tokens, 4 * (n + 1), 4},
                       {a->blocks_taken, 4, 4}, {a->slot, 8 * cap, 8}, {a->query_req_id, 4 * cap, 4},
                       {a->query_abs_pos, 4 * cap, 4}, {a->dev_err, 4, 4}};
  for (const Range& r : in)
    if (!al(r.p, r.align)) return BSP_ERR_INVALID_ARG;
  for (const Range& o : out) {
    if (!al(o.p, o.align)) return BSP_ERR_INVALID_ARG;
    for (const Range& r : in)
      if (overlap(o.p, o.bytes, r.p, r.bytes)) return BSP_ERR_INVALID_ARG;
    for (const Range& r : out)
      if (&r != &o && overlap(o.p, o.bytes, r.p, r.bytes)) return BSP_ERR_INVALID_ARG;
  }
  StepTablesParams p{};
  p.context_lens = a->context_lens;
  p.new_lens = a->new_lens;
  p.num_seqs = a->num_seqs;
  p.block_table = a->block_table;
  p.bt_stride = a->bt_stride;
  p.free_blocks = a->free_blocks;
  p.free_head = a->free_head;
  p.num_free = a->num_free;
  p.num_blocks = a->num_blocks;
  p.token_capacity = a->token_capacity;
  p.seq_lens = a->seq_lens;
  p.cu_tokens = a->cu_tokens;
  p.blocks_taken = a->blocks_taken;
  p.slot = a->slot;
  p.query_req_id = a->query_req_id;
  p.query_abs_pos = a->query_abs_pos;
  p.err = a->dev_err;
  const bsp_status st = cuda_status(launch_step_tables(p, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_norm_rope_write(const bsp_norm_rope_args* a, bsp_stream_t stream) {
  if (!a || a->num_tokens < 0) return BSP_ERR_INVALID_ARG;
  bsp_status st;
  if (a->kv && (st = check_kv(a->kv)) != BSP_OK) return st;
  if (a->idx && (st = check_idx(a->idx)) != BSP_OK) return st;
  if ((a->q_out && a->q_out_dtype != BSP_BF16 && a->q_out_dtype != BSP_FP8_E4M3) ||
      (a->idx_q_out && a->idx_q_out_dtype != BSP_BF16 && a->idx_q_out_dtype != BSP_FP8_E4M3))
    return BSP_ERR_UNSUPPORTED;
  if (a->rot_dim < 0 || a->rot_dim > kDim || a->rot_dim % 16) return BSP_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.f) || !(a->weight_offset == a->weight_offset)) return BSP_ERR_INVALID_ARG;
  // each input has somewhere to go, and each output comes from somewhere
  if (!a->q != !a->q_out || !a->idx_q != !a->idx_q_out || !a->idx_k != !a->idx) return BSP_ERR_INVALID_ARG;
  if ((a->kv && (!a->k || !a->v)) || (a->k_out && !a->k) || (a->k && !a->kv && !a->k_out) || (a->v && !a->kv))
    return BSP_ERR_INVALID_ARG;
  if ((a->kv && a->num_kv_heads != a->kv->num_kv_heads) || (a->idx && a->num_idx_heads != a->idx->num_heads))
    return BSP_ERR_INVALID_ARG;
  if (a->num_tokens == 0) return BSP_OK;
  if ((a->kv || a->idx) && (!a->slot || !al(a->slot, 8))) return BSP_ERR_INVALID_ARG;
  if (a->rot_dim && (!a->rope_table || !al(a->rope_table, 16) || a->rope_rows < 1 || !a->positions))
    return BSP_ERR_INVALID_ARG;
  if (a->positions && !al(a->positions, 4)) return BSP_ERR_INVALID_ARG;
  const int64_t T = a->num_tokens;
  NormRopeParams p{};
  const void* src[kHeadTypes] = {a->q, a->k, a->v, a->idx_q, a->idx_k};
  const int64_t stride[kHeadTypes] = {a->q_stride, a->k_stride, a->v_stride, a->idx_q_stride, a->idx_k_stride};
  const int32_t heads[kHeadTypes] = {a->num_q_heads, a->num_kv_heads, a->num_kv_heads, a->num_idx_heads,
                                     a->num_idx_heads};
  const void* weight[kHeadTypes] = {a->q_weight, a->k_weight, nullptr, a->idx_q_weight, a->idx_k_weight};
  void* out[kHeadTypes] = {a->q_out, a->k_out, nullptr, a->idx_q_out, nullptr};
  const int32_t out_dtype[kHeadTypes] = {a->q_out_dtype, BSP_BF16, 0, a->idx_q_out_dtype, 0};
  for (int i = 0; i < kHeadTypes; ++i) {
    if (!src[i]) continue;
    const int64_t row = static_cast<int64_t>(heads[i]) * kDim;
    if (heads[i] < 1 || stride[i] < row || stride[i] % 8 || !al(src[i], 16) || !al(weight[i], 16) || !al(out[i], 16))
      return BSP_ERR_INVALID_ARG;
    if (heads[i] > (1 << 16) || stride[i] > (int64_t{1} << 32)) return BSP_ERR_UNSUPPORTED;
    p.src[i] = static_cast<const uint16_t*>(src[i]);
    p.stride[i] = stride[i];
    p.heads[i] = heads[i];
    p.weight[i] = static_cast<const uint16_t*>(weight[i]);
    p.out[i] = out[i];
    p.out_dtype[i] = out_dtype[i];
  }
  // no output on an input or another output, but a bf16 one in place
  struct Range {
    const void* p;
    int64_t bytes;
  };
  Range in[2 * kHeadTypes + 3], out_of[kHeadTypes + 1];
  for (int i = 0; i < kHeadTypes; ++i) {
    in[i] = {p.src[i], p.src[i] ? ((T - 1) * stride[i] + p.heads[i] * kDim) * 2 : 0};
    in[kHeadTypes + i] = {p.weight[i], 2 * kDim};
    out_of[i] = {p.out[i], p.out[i] ? T * p.heads[i] * kDim * (p.out_dtype[i] == BSP_BF16 ? 2 : 1) : 0};
  }
  in[2 * kHeadTypes] = {a->positions, 4 * T};
  in[2 * kHeadTypes + 1] = {a->kv || a->idx ? a->slot : nullptr, 8 * T};
  in[2 * kHeadTypes + 2] = {a->rot_dim ? a->rope_table : nullptr, 4 * a->rope_rows * a->rot_dim};
  out_of[kHeadTypes] = {a->dev_err, 4};
  for (int i = 0; i <= kHeadTypes; ++i) {
    const Range& o = out_of[i];
    if (!o.p) continue;
    for (int j = 0; j < 2 * kHeadTypes + 3; ++j) {
      const bool in_place = i < kHeadTypes && j == i && o.p == in[j].p && p.out_dtype[i] == BSP_BF16 &&
                            stride[i] == p.heads[i] * kDim;
      if (!in_place && overlap(o.p, o.bytes, in[j].p, in[j].bytes)) return BSP_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(o.p, o.bytes, out_of[j].p, out_of[j].bytes)) return BSP_ERR_INVALID_ARG;
    if (overlap_cache(o.p, o.bytes, a->kv) || overlap_cache(o.p, o.bytes, a->idx)) return BSP_ERR_INVALID_ARG;
  }
  for (const Range& r : in)
    if (overlap_cache(r.p, r.bytes, a->kv) || overlap_cache(r.p, r.bytes, a->idx)) return BSP_ERR_INVALID_ARG;
  p.weight_offset = a->weight_offset;
  p.eps = a->eps;
  p.rope = a->rope_table;
  p.rope_rows = a->rope_rows;
  p.rot_dim = a->rot_dim;
  p.rope_pairs = a->rope_pairs ? 1 : 0;
  p.positions = a->positions;
  p.slot = a->slot;
  p.num_tokens = a->num_tokens;
  set_caches(p.cache, a->kv, a->idx);
  p.err = a->dev_err;
  if (!a->q && !a->k && !a->idx_q && !a->idx_k) return BSP_OK;
  st = cuda_status(launch_norm_rope(p, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_kv_page_read(const bsp_kv_cache* kv, const bsp_index_cache* idx, const int64_t* slot,
                            int32_t num_tokens, void* k, void* v, void* idx_k, int32_t* dev_err, bsp_stream_t stream) {
  if (num_tokens < 0 || !k != !v) return BSP_ERR_INVALID_ARG;
  bsp_status st;
  if (k && (st = check_kv(kv)) != BSP_OK) return st;
  if (idx_k && (st = check_idx(idx)) != BSP_OK) return st;
  if (num_tokens == 0 || (!k && !idx_k)) return BSP_OK;
  if (!slot || !al(slot, 8) || !al(k, 16) || !al(v, 16) || !al(idx_k, 16)) return BSP_ERR_INVALID_ARG;
  const int64_t units = (k ? kv->num_kv_heads : 0) + (idx_k ? idx->num_heads : 0);
  if ((static_cast<int64_t>(num_tokens) + 15) / 16 * units > INT32_MAX) return BSP_ERR_UNSUPPORTED;
  KvReadParams p{};
  set_caches(p.cache, k ? kv : nullptr, idx_k ? idx : nullptr);
  p.cache.slot = slot;
  p.cache.num_tokens = num_tokens;
  p.cache.err = dev_err;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.idx_k = static_cast<uint16_t*>(idx_k);
  st = cuda_status(launch_kv_page_read(p, reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

size_t bsp_dense_pa_workspace_bytes(int32_t num_rows, int32_t num_kv_heads, int32_t group, int32_t q_group) {
  if (num_rows <= 0 || num_kv_heads < 1 || num_rows % num_kv_heads || !valid_group(group) || q_group < 1 || q_group > 8)
    return 0;
  return dense_pa_ws_bytes(num_rows, num_kv_heads, group, q_group, device_sms());
}

bsp_status bsp_dense_pa_decode(const bsp_kv_cache* kv, const void* q, int32_t q_dtype, int32_t num_q_heads,
                               const int32_t* block_table, int32_t bt_stride, const int32_t* row_seq,
                               const int32_t* row_len, int32_t num_rows, int32_t q_group, float sm_scale, void* out,
                               void* ws, size_t ws_bytes, int32_t* dev_err, bsp_stream_t stream) {
  bsp_status st = check_kv(kv);
  if (st != BSP_OK) return st;
  if (kv->dtype != BSP_MXFP4 || (q_dtype != BSP_BF16 && q_dtype != BSP_FP8_E4M3)) return BSP_ERR_UNSUPPORTED;
  if (num_rows < 0 || num_q_heads < 1 || bt_stride < 1) return BSP_ERR_INVALID_ARG;
  if (num_q_heads % kv->num_kv_heads || num_rows % kv->num_kv_heads) return BSP_ERR_INVALID_ARG;
  const int32_t group = num_q_heads / kv->num_kv_heads;
  if (!valid_group(group) || q_group < 1 || q_group > 8) return BSP_ERR_UNSUPPORTED;
  // the keys' 4-bit tensor copies
  if (!al(kv->k_base, 32) || kv->id_stride_bytes % 32) return BSP_ERR_UNSUPPORTED;
  if (!(sm_scale - sm_scale == 0.f)) return BSP_ERR_INVALID_ARG;  // infinite or NaN
  if (num_rows == 0) return BSP_OK;
  if (!q || !block_table || !row_seq || !row_len || !out || !al(q, 16) || !al(out, 16) || !al(block_table, 4) ||
      !al(row_seq, 4) || !al(row_len, 4))
    return BSP_ERR_INVALID_ARG;
  const size_t need = dense_pa_ws_bytes(num_rows, kv->num_kv_heads, group, q_group, device_sms());
  if (need && (!ws || ws_bytes < need || !al(ws, 16))) return BSP_ERR_WORKSPACE;
  DensePaParams p{};
  p.k_base = static_cast<const uint8_t*>(kv->k_base);
  p.v_base = static_cast<const uint8_t*>(kv->v_base);
  p.id_stride = kv->id_stride_bytes;
  p.num_blocks = kv->num_blocks;
  p.hkv = kv->num_kv_heads;
  p.group = group;
  p.q = q;
  p.q_dtype = q_dtype;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.row_seq = row_seq;
  p.row_len = row_len;
  p.num_rows = num_rows;
  p.q_group = q_group;
  p.sm_scale = sm_scale;
  p.out = out;
  p.ws = ws;
  p.err = dev_err;
  int launches = 0;
  st = cuda_status(launch_dense_pa(p, device_sms(), reinterpret_cast<cudaStream_t>(stream), &launches));
  g_launches += launches;
  return st;
}

}  // extern "C"

namespace {

bsp_status check_scaled(const bsp_kv_cache* kv, const bsp_kv_scales* scales) {
  const bsp_status st = check_kv(kv);
  if (st != BSP_OK) return st;
  if (kv->dtype != BSP_FP8_E4M3) return BSP_ERR_UNSUPPORTED;
  if (!scales || !scales->k || !scales->v || !al(scales->k, 4) || !al(scales->v, 4)) return BSP_ERR_INVALID_ARG;
  if (kv->num_kv_heads > (1 << 16)) return BSP_ERR_UNSUPPORTED;
  return BSP_OK;
}

struct Span {
  const void* p;
  int64_t bytes;
};
// whether one of `out` shares a byte with one of `in`, with another of `out` or with the cache
template <size_t NO, size_t NI>
bool spans_collide(const Span (&out)[NO], const Span (&in)[NI], const bsp_kv_cache* kv) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    if (overlap_cache(out[i].p, out[i].bytes, kv)) return true;
  }
  return false;
}

int64_t row_span(int64_t rows, int64_t stride, int64_t heads) { return rows ? ((rows - 1) * stride + heads * kDim) * 2 : 0; }

}  // namespace

extern "C" {

bsp_status bsp_kv_scaled_write(const bsp_kv_cache* kv, const bsp_kv_scales* scales, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int64_t* slot, int32_t num_tokens,
                               int32_t* dev_err, bsp_stream_t stream) {
  bsp_status st = check_scaled(kv, scales);
  if (st != BSP_OK) return st;
  if (num_tokens < 0) return BSP_ERR_INVALID_ARG;
  if (kv->num_kv_heads > 65535) return BSP_ERR_UNSUPPORTED;  // (a grid dimension)
  const int64_t heads = kv->num_kv_heads, T = num_tokens;
  if (k_stride < heads * kDim || v_stride < heads * kDim || k_stride % 8 || v_stride % 8) return BSP_ERR_INVALID_ARG;
  if (k_stride > (int64_t{1} << 32) || v_stride > (int64_t{1} << 32)) return BSP_ERR_UNSUPPORTED;
  if (num_tokens == 0) return BSP_OK;
  if (!k || !v || !slot || !al(k, 16) || !al(v, 16) || !al(slot, 8) || !al(dev_err, 4)) return BSP_ERR_INVALID_ARG;
  const Span in[] = {{k, row_span(T, k_stride, heads)}, {v, row_span(T, v_stride, heads)}, {slot, 8 * T}};
  const Span out[] = {{scales->k, 4 * kv->num_blocks * heads}, {scales->v, 4 * kv->num_blocks * heads}, {dev_err, 4}};
  if (spans_collide(out, in, kv)) return BSP_ERR_INVALID_ARG;
  for (const Span& i : in)
    if (overlap_cache(i.p, i.bytes, kv)) return BSP_ERR_INVALID_ARG;
  KvScaledWriteParams p{};
  p.base[0] = static_cast<uint8_t*>(kv->k_base);
  p.base[1] = static_cast<uint8_t*>(kv->v_base);
  p.scales[0] = scales->k;
  p.scales[1] = scales->v;
  p.src[0] = static_cast<const uint16_t*>(k);
  p.src[1] = static_cast<const uint16_t*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.id_stride = kv->id_stride_bytes;
  p.num_blocks = kv->num_blocks;
  p.hkv = kv->num_kv_heads;
  p.slot = slot;
  p.num_tokens = num_tokens;
  p.err = dev_err;
  st = cuda_status(launch_kv_scaled_write(p, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

bsp_status bsp_kv_scaled_read(const bsp_kv_cache* kv, const bsp_kv_scales* scales, const int64_t* slot,
                              int32_t num_tokens, void* k, void* v, int32_t* dev_err, bsp_stream_t stream) {
  bsp_status st = check_scaled(kv, scales);
  if (st != BSP_OK) return st;
  if (num_tokens < 0) return BSP_ERR_INVALID_ARG;
  if (num_tokens == 0) return BSP_OK;
  if (!slot || !k || !v || !al(slot, 8) || !al(k, 16) || !al(v, 16) || !al(dev_err, 4)) return BSP_ERR_INVALID_ARG;
  const int64_t heads = kv->num_kv_heads, T = num_tokens;
  if ((T + 15) / 16 * heads > INT32_MAX) return BSP_ERR_UNSUPPORTED;
  const Span in[] = {{slot, 8 * T}, {scales->k, 4 * kv->num_blocks * heads}, {scales->v, 4 * kv->num_blocks * heads}};
  const Span out[] = {{k, T * heads * kDim * 2}, {v, T * heads * kDim * 2}, {dev_err, 4}};
  if (spans_collide(out, in, kv)) return BSP_ERR_INVALID_ARG;
  KvReadParams p{};
  set_caches(p.cache, kv, nullptr);
  p.cache.slot = slot;
  p.cache.num_tokens = num_tokens;
  p.cache.err = dev_err;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.k_scales = scales->k;
  p.v_scales = scales->v;
  st = cuda_status(launch_kv_page_read(p, reinterpret_cast<cudaStream_t>(stream)));
  if (st == BSP_OK) ++g_launches;
  return st;
}

size_t bsp_dense_pa_fp8_workspace_bytes(int32_t num_rows, int32_t num_kv_heads, int32_t group, int32_t q_group) {
  if (num_rows <= 0 || num_kv_heads < 1 || num_rows % num_kv_heads || !valid_group(group) || q_group < 1 || q_group > 8)
    return 0;
  return dense_pa_fp8_ws_bytes(num_rows, num_kv_heads, group, q_group, device_sms());
}

bsp_status bsp_dense_pa_decode_fp8(const bsp_kv_cache* kv, const bsp_kv_scales* scales, const void* q, int32_t q_dtype,
                                   int32_t num_q_heads, const int32_t* block_table, int32_t bt_stride,
                                   const int32_t* row_seq, const int32_t* row_len, int32_t num_rows, int32_t q_group,
                                   float sm_scale, void* out, void* ws, size_t ws_bytes, int32_t* dev_err,
                                   bsp_stream_t stream) {
  bsp_status st = scales ? check_scaled(kv, scales) : check_kv(kv);
  if (st != BSP_OK) return st;
  if (kv->dtype != BSP_FP8_E4M3 || (q_dtype != BSP_BF16 && q_dtype != BSP_FP8_E4M3)) return BSP_ERR_UNSUPPORTED;
  if (num_rows < 0 || num_q_heads < 1 || bt_stride < 1) return BSP_ERR_INVALID_ARG;
  if (num_q_heads % kv->num_kv_heads || num_rows % kv->num_kv_heads) return BSP_ERR_INVALID_ARG;
  const int32_t group = num_q_heads / kv->num_kv_heads;
  if (!valid_group(group) || q_group < 1 || q_group > 8) return BSP_ERR_UNSUPPORTED;
  if (!(sm_scale - sm_scale == 0.f)) return BSP_ERR_INVALID_ARG;  // infinite or NaN
  if (num_rows == 0) return BSP_OK;
  if (!q || !block_table || !row_seq || !row_len || !out || !al(q, 16) || !al(out, 16) || !al(block_table, 4) ||
      !al(row_seq, 4) || !al(row_len, 4) || !al(dev_err, 4))
    return BSP_ERR_INVALID_ARG;
  const size_t need = dense_pa_fp8_ws_bytes(num_rows, kv->num_kv_heads, group, q_group, device_sms());
  if (need && (!ws || ws_bytes < need || !al(ws, 16))) return BSP_ERR_WORKSPACE;
  const int64_t heads = kv->num_kv_heads, n = num_rows, qn = n * group * kDim;
  const Span in[] = {{q, qn * (q_dtype == BSP_BF16 ? 2 : 1)}, {row_seq, 4 * n}, {row_len, 4 * n},
                     {scales ? scales->k : nullptr, 4 * kv->num_blocks * heads},
                     {scales ? scales->v : nullptr, 4 * kv->num_blocks * heads}};
  const Span outs[] = {{out, qn * 2}, {need ? ws : nullptr, static_cast<int64_t>(need)}, {dev_err, 4}};
  if (spans_collide(outs, in, kv)) return BSP_ERR_INVALID_ARG;
  DensePaFp8Params p{};
  p.a.k_base = static_cast<const uint8_t*>(kv->k_base);
  p.a.v_base = static_cast<const uint8_t*>(kv->v_base);
  p.a.id_stride = kv->id_stride_bytes;
  p.a.num_blocks = kv->num_blocks;
  p.a.hkv = kv->num_kv_heads;
  p.a.group = group;
  p.a.q = q;
  p.a.q_dtype = q_dtype;
  p.a.block_table = block_table;
  p.a.bt_stride = bt_stride;
  p.a.row_seq = row_seq;
  p.a.row_len = row_len;
  p.a.num_rows = num_rows;
  p.a.q_group = q_group;
  p.a.sm_scale = sm_scale;
  p.a.out = out;
  p.a.ws = ws;
  p.a.err = dev_err;
  p.k_scales = scales ? scales->k : nullptr;
  p.v_scales = scales ? scales->v : nullptr;
  p.k_scale = kv->k_scale;
  p.v_scale = kv->v_scale;
  int launches = 0;
  st = cuda_status(launch_dense_pa_fp8(p, device_sms(), reinterpret_cast<cudaStream_t>(stream), &launches));
  g_launches += launches;
  return st;
}

size_t bsp_prompt_attention_workspace_bytes(int32_t num_tokens, int32_t num_seqs, int32_t num_kv_heads, int32_t group) {
  if (num_tokens < 1 || num_seqs < 1 || num_kv_heads < 1 || !valid_group(group)) return 0;
  return prompt_ws_bytes(num_tokens, num_seqs, num_kv_heads, group, device_sms());
}

bsp_status bsp_prompt_attention(const bsp_prompt_attention_args* a, bsp_stream_t stream) {
  if (!a || a->num_tokens < 0 || a->num_keys < 0 || a->num_seqs < 0 || a->num_q_heads < 1 || a->num_kv_heads < 1 ||
      a->num_q_heads % a->num_kv_heads)
    return BSP_ERR_INVALID_ARG;
  const int32_t group = a->num_q_heads / a->num_kv_heads;
  if (!valid_group(group)) return BSP_ERR_UNSUPPORTED;
  const int64_t hq = a->num_q_heads, hkv = a->num_kv_heads, T = a->num_tokens, K = a->num_keys, n = a->num_seqs;
  // (int32 tile counts, and the copies' strides)
  if (hq > (1 << 16) || n > (1 << 20) || (T + n) * hq > INT32_MAX) return BSP_ERR_UNSUPPORTED;
  for (int64_t st : {a->q_stride, a->k_stride, a->v_stride})
    if (st % 8) return BSP_ERR_INVALID_ARG;
  if (a->q_stride < hq * kDim || a->k_stride < hkv * kDim || a->v_stride < hkv * kDim) return BSP_ERR_INVALID_ARG;
  if (a->q_stride > (int64_t{1} << 32) || a->k_stride > (int64_t{1} << 32) || a->v_stride > (int64_t{1} << 32))
    return BSP_ERR_UNSUPPORTED;
  if (!(a->sm_scale - a->sm_scale == 0.f)) return BSP_ERR_INVALID_ARG;  // infinite or NaN
  if (T == 0 || n == 0) return BSP_OK;
  if (!a->q || !a->out || !a->cu_q || !a->cu_k || !al(a->q, 16) || !al(a->out, 16) || !al(a->cu_q, 4) ||
      !al(a->cu_k, 4) || !al(a->dev_err, 4))
    return BSP_ERR_INVALID_ARG;
  if (K && (!a->k || !a->v || !al(a->k, 16) || !al(a->v, 16))) return BSP_ERR_INVALID_ARG;
  const size_t need = prompt_ws_bytes(a->num_tokens, a->num_seqs, a->num_kv_heads, group, device_sms());
  if (need && (!a->ws || a->ws_bytes < need || !al(a->ws, 16))) return BSP_ERR_WORKSPACE;
  const Span in[] = {{a->q, row_span(T, a->q_stride, hq)}, {a->k, row_span(K, a->k_stride, hkv)},
                     {a->v, row_span(K, a->v_stride, hkv)}, {a->cu_q, 4 * (n + 1)}, {a->cu_k, 4 * (n + 1)}};
  const Span out[] = {{a->out, T * hq * kDim * 2}, {need ? a->ws : nullptr, static_cast<int64_t>(need)},
                      {a->dev_err, 4}};
  if (spans_collide(out, in, nullptr)) return BSP_ERR_INVALID_ARG;
  PromptParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.num_tokens = a->num_tokens;
  p.num_keys = a->num_keys;
  p.hkv = a->num_kv_heads;
  p.group = group;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.num_seqs = a->num_seqs;
  p.sm_scale = a->sm_scale;
  p.out = static_cast<uint16_t*>(a->out);
  p.ws = a->ws;
  p.err = a->dev_err;
  int launches = 0;
  const bsp_status st = cuda_status(launch_prompt(p, device_sms(), reinterpret_cast<cudaStream_t>(stream), &launches));
  g_launches += launches;
  return st;
}

}  // extern "C"

extern "C" {

static bsp_status sparse_pa_common(const bsp_kv_cache* kv, const void* q, int32_t q_dtype, int32_t num_q_heads,
                                   const int32_t* sparse_bt, const int32_t* sparse_ctx, int32_t num_rows,
                                   int32_t k_pages, float sm_scale, void* out, void* ws, size_t ws_bytes,
                                   int32_t* dev_err, bsp_stream_t stream, bool decode, bool q_early = false) {
  bsp_status st = sparse_pa_check_args(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, num_rows, k_pages, out);
  if (st != BSP_OK || num_rows == 0) return st;
  const int32_t group = num_q_heads / kv->num_kv_heads;
  SparsePaParams p{};
  p.kv_dtype = kv->dtype;
  p.hkv = kv->num_kv_heads;
  p.k_base = static_cast<const uint8_t*>(kv->k_base);
  p.v_base = static_cast<const uint8_t*>(kv->v_base);
  p.id_stride = kv->id_stride_bytes;
  p.num_ids = kv->num_ids;
  p.k_scale = kv->k_scale;
  p.v_scale = kv->v_scale;
  p.q = q;
  p.q_dtype = q_dtype;
  p.group = group;
  p.sparse_bt = sparse_bt;
  p.sparse_ctx = sparse_ctx;
  p.num_rows = num_rows;
  p.k_pages = k_pages;
  p.sm_scale = sm_scale;
  p.out = out;
  p.err = dev_err;
  p.q_early = q_early;
  if (decode) {
    const PaPlan plan = sparse_pa_plan(kv->dtype, num_rows, k_pages, device_sms());
    p.nsplit = plan.nsplit;
    p.pages_per_split = plan.pages_per_split;
    p.cluster = plan.cluster;
    p.ring = plan.ring;
    const size_t need = sparse_pa_ws_bytes(num_rows, plan);
    if (need) {
      if (!ws || ws_bytes < need || !al(ws, 16)) return BSP_ERR_WORKSPACE;
      p.ws = static_cast<float*>(ws);
    }
  } else {
    const PaPlan plan = sparse_pa_prefill_plan(kv->dtype, k_pages);
    p.nsplit = plan.nsplit;
    p.pages_per_split = plan.pages_per_split;
    p.ring = plan.ring;
  }
  int launches = 0;
  st = cuda_status(launch_sparse_pa(p, reinterpret_cast<cudaStream_t>(stream), &launches));
  g_launches += launches;
  return st;
}

// the decode attention's workspace check (also run by the decode step before
// its first launch): a plan that merges through the workspace needs `need`
// bytes of it, 16-byte aligned
static bsp_status sparse_pa_ws_check(int32_t kv_dtype, int32_t num_rows, int32_t k_pages, const void* ws,
                                     size_t ws_bytes) {
  const size_t need = sparse_pa_decode_ws_need(kv_dtype, num_rows, k_pages);
  return need && (!ws || ws_bytes < need || !al(ws, 16)) ? BSP_ERR_WORKSPACE : BSP_OK;
}

bsp_status bsp_sparse_pa_decode(const bsp_kv_cache* kv, const void* q, int32_t q_dtype, int32_t num_q_heads,
                                const int32_t* sparse_bt, const int32_t* sparse_ctx, int32_t num_rows,
                                int32_t k_pages, float sm_scale, void* out, void* ws, size_t ws_bytes,
                                int32_t* dev_err, bsp_stream_t stream) {
  return sparse_pa_common(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, num_rows, k_pages, sm_scale, out, ws,
                          ws_bytes, dev_err, stream, true);
}

bsp_status bsp_sparse_pa_prefill(const bsp_kv_cache* kv, const void* q, int32_t q_dtype, int32_t num_q_heads,
                                 const int32_t* sparse_bt, const int32_t* sparse_ctx, int32_t num_rows,
                                 int32_t k_pages, float sm_scale, void* out, int32_t* dev_err, bsp_stream_t stream) {
  return sparse_pa_common(kv, q, q_dtype, num_q_heads, sparse_bt, sparse_ctx, num_rows, k_pages, sm_scale, out,
                          nullptr, 0, dev_err, stream, false);
}

bsp_status bsp_sparse_decode_step(const bsp_decode_step_args* a, bsp_event_t* events, bsp_stream_t stream) {
  if (!a || !a->kv) return BSP_ERR_INVALID_ARG;
  const bool reuse = (a->flags & BSP_REUSE_SELECTION) != 0;
  if (!reuse && !a->idx) return BSP_ERR_INVALID_ARG;
  const int32_t hkv = a->kv->num_kv_heads;
  const int32_t hidx = reuse ? 0 : a->idx->num_heads;
  if (!reuse && hidx != hkv) return BSP_ERR_UNSUPPORTED;  // rows are shared by the scorer and the attention
  if (a->num_seqs < 0 || a->q_len < 1 || a->q_len > 8) return BSP_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a->num_seqs) * a->q_len * hkv > INT32_MAX) return BSP_ERR_UNSUPPORTED;  // int32 rows
  const int32_t tokens = a->num_seqs * a->q_len;
  const int32_t rows = tokens * hkv;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto mark = [&](int i) {
    if (events) cudaEventRecord(reinterpret_cast<cudaEvent_t>(events[i]), s);
  };
  bsp_status st = check_kv(a->kv);
  if (st != BSP_OK) return st;
  if (!reuse && (st = check_idx(a->idx)) != BSP_OK) return st;
  if (a->num_new_tokens < 0 || a->num_q_heads < 1) return BSP_ERR_INVALID_ARG;
  if (a->num_new_tokens && (!a->k_new || !a->v_new || !a->slot || !al(a->k_new, 16) || !al(a->v_new, 16) ||
                            !al(a->slot, 8) || (!reuse && (!a->idx_k_new || !al(a->idx_k_new, 16)))))
    return BSP_ERR_INVALID_ARG;
  if (!a->q || !al(a->q, 16)) return BSP_ERR_INVALID_ARG;
  if (reuse ? (!a->sparse_bt || !a->sparse_ctx)
            : (!a->idx_q || !al(a->idx_q, 16) || !a->seq_lens || !a->row_seq || !a->row_len))
    return BSP_ERR_INVALID_ARG;
  const bool cast_q = a->q_dtype == BSP_FP8_E4M3, cast_iq = !reuse && a->idx_q_dtype == BSP_FP8_E4M3;
  if ((cast_q && (!a->q_cast || !al(a->q_cast, 16))) || (cast_iq && (!a->idx_q_cast || !al(a->idx_q_cast, 16))))
    return BSP_ERR_INVALID_ARG;
  // the queries the scorer and the attention read
  const void* q = cast_q ? a->q_cast : a->q;
  const void* iq = cast_iq ? a->idx_q_cast : a->idx_q;
  // The step's rows are decode-ordered (row_seq = token / q_len, as the prep
  // kernel writes it): the scorer and the selector find a row's sequence
  // without reading row_seq first.  With sel_counters the scorer's last CTA
  // of each query group selects the group's rows (no selector launch).
  const int32_t topk_flags = a->flags & (BSP_FORCE_TAIL | BSP_SELECT_BLOCKS);
  const bool fused = !reuse && a->sel_counters &&
                     index_score_can_select(a->idx->dtype, a->idx_q_dtype, a->max_pages,
                                            (a->flags & BSP_SELECT_BLOCKS) != 0);
  // every later stage's checks too, so that an invalid step enqueues nothing
  TopkParams sel;
  if (!reuse) {
    if (fused && !al(a->sel_counters, 4)) return BSP_ERR_INVALID_ARG;
    if ((st = index_score_check(a->idx, iq, a->idx_q_dtype, a->block_table, a->bt_stride, a->row_seq, a->row_len,
                                rows, a->q_len, a->max_pages, a->scores)) != BSP_OK ||
        (st = topk_params(a->scores, rows, a->max_pages, a->row_seq, a->row_len, a->block_table, a->bt_stride,
                          a->kv->dtype, a->k_pages, topk_flags, a->topk_idx, a->sparse_bt, a->sparse_ctx,
                          a->q_len * hkv, sel)) != BSP_OK)
      return st;
  }
  if ((st = sparse_pa_check_args(a->kv, q, a->q_dtype, a->num_q_heads, a->sparse_bt, a->sparse_ctx, rows, a->k_pages,
                                 a->out)) != BSP_OK ||
      (st = sparse_pa_ws_check(a->kv->dtype, rows, a->k_pages, a->ws, a->ws_bytes)) != BSP_OK)
    return st;
  mark(0);
  // write + e4m3 casts + row lengths: one launch
  DecodePrepParams pp{};
  KvWriteParams& w = pp.write;
  w.kv_dtype = a->kv->dtype;
  w.hkv = hkv;
  w.k_base = static_cast<uint8_t*>(a->kv->k_base);
  w.v_base = static_cast<uint8_t*>(a->kv->v_base);
  w.id_stride = a->kv->id_stride_bytes;
  w.num_blocks = a->kv->num_blocks;
  w.k_scale = a->kv->k_scale;
  w.v_scale = a->kv->v_scale;
  w.hidx = hidx;  // 0: no index-key write
  if (!reuse) {
    w.idx_dtype = a->idx->dtype;
    w.idx_base = static_cast<uint8_t*>(a->idx->base);
    w.idx_block_stride = a->idx->block_stride_bytes;
    w.idx_num_blocks = a->idx->num_blocks;
    w.idx_k = static_cast<const uint16_t*>(a->idx_k_new);
  }
  w.k = static_cast<const uint16_t*>(a->k_new);
  w.v = static_cast<const uint16_t*>(a->v_new);
  w.slot = a->slot;
  w.num_tokens = a->num_new_tokens;
  w.err = a->dev_err;
  if (cast_q) {
    pp.cast_src[0] = static_cast<const uint16_t*>(a->q);
    pp.cast_dst[0] = static_cast<uint8_t*>(a->q_cast);
    pp.cast_n[0] = static_cast<int64_t>(tokens) * a->num_q_heads * kDim;
  }
  if (cast_iq) {
    pp.cast_src[1] = static_cast<const uint16_t*>(a->idx_q);
    pp.cast_dst[1] = static_cast<uint8_t*>(a->idx_q_cast);
    pp.cast_n[1] = static_cast<int64_t>(tokens) * hidx * kDim;
  }
  if (!reuse) {  // the selection's rows; nothing to compute when it is reused
    pp.seq_lens = a->seq_lens;
    pp.num_seqs = a->num_seqs;
    pp.q_len = a->q_len;
    pp.heads = hkv;
    pp.row_seq = a->row_seq;
    pp.row_len = a->row_len;
  }
  if ((st = cuda_status(launch_decode_prep(pp, s))) != BSP_OK) return st;
  ++g_launches;
  mark(1);
  if (!reuse &&
      (st = index_score_impl(a->idx, iq, a->idx_q_dtype, a->block_table, a->bt_stride, a->row_seq, a->row_len, rows,
                             a->q_len, a->max_pages, a->scores, a->dev_err, stream, 1, fused ? &sel : nullptr,
                             fused ? a->sel_counters : nullptr)) != BSP_OK)
    return st;
  mark(2);
  if (!reuse && !fused &&
      (st = topk_impl(a->scores, rows, a->max_pages, a->row_seq, a->row_len, a->block_table, a->bt_stride,
                      a->kv->dtype, a->k_pages, topk_flags, a->topk_idx, a->sparse_bt, a->sparse_ctx, stream,
                      a->q_len * hkv)) != BSP_OK)
    return st;
  mark(3);
  // the attention's queries were written two launches back (or are the
  // caller's bf16 input) unless the prep kernel right before it cast them
  const bool q_early = !(reuse && a->q_dtype == BSP_FP8_E4M3);
  if ((st = sparse_pa_common(a->kv, q, a->q_dtype, a->num_q_heads, a->sparse_bt, a->sparse_ctx, rows, a->k_pages,
                             a->sm_scale, a->out, a->ws, a->ws_bytes, a->dev_err, stream, true, q_early)) != BSP_OK)
    return st;
  mark(4);
  return BSP_OK;
}

const char* bsp_status_str(bsp_status s) {
  switch (s) {
    case BSP_OK:
      return "ok";
    case BSP_ERR_INVALID_ARG:
      return "invalid argument";
    case BSP_ERR_UNSUPPORTED:
      return "unsupported size or dtype";
    case BSP_ERR_WORKSPACE:
      return "workspace too small";
    case BSP_ERR_CUDA:
      return "CUDA error";
  }
  return "unknown status";
}

int32_t bsp_last_cuda_error(void) { return g_last_cuda_error.load(); }
int64_t bsp_launch_count(void) { return g_launches.load(); }
int32_t bsp_version(void) { return 110; }

}  // extern "C"
