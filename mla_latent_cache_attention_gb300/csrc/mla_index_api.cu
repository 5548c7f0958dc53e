// mla_index_api.cu -- the C ABI of the selector in front of sparse attention: argument checks,
// tensor maps, workspace carving and launches.  Host code only.
#include <cuda.h>

#include "mla.h"
#include "mla_host.h"
#include "mla_index.h"

using namespace mla;

namespace {

bool index_format(mla_cache_format fmt) { return fmt == MLA_CACHE_BF16 || fmt == MLA_CACHE_FP8; }

// Shared checks of an index cache and its scales.
int check_index_cache(const void* cache, mla_cache_format fmt, int64_t num_blocks, int64_t block_stride,
                      int64_t entry_stride, const float* scales, int64_t scale_stride, int32_t block_size) {
  const int64_t bytes = fmt == MLA_CACHE_BF16 ? 2 * kIndexDim : kIndexDim;
  if (!cache) return fail(MLA_ERR_INVALID, "index_cache is NULL");
  if (block_size < 1 || num_blocks < 1) return fail(MLA_ERR_INVALID, "bad cache geometry");
  if (num_blocks >= (int64_t(1) << 31)) return fail(MLA_ERR_UNSUPPORTED, "num_blocks must be below 2^31");
  if (entry_stride < bytes || entry_stride % 16 || block_stride % 16 || block_stride < entry_stride * block_size ||
      !aligned(cache, 16))
    return fail(MLA_ERR_INVALID, "index keys need 16-byte alignment and non-overlapping strides");
  if (fmt == MLA_CACHE_BF16) {
    if (scales) return fail(MLA_ERR_INVALID, "index_scales are only for the fp8 index cache");
  } else {
    if (!scales) return fail(MLA_ERR_INVALID, "the fp8 index cache needs index_scales");
    if (scale_stride < block_size || scale_stride % 4 || !aligned(scales, 16))
      return fail(MLA_ERR_INVALID, "index_scales need 16-byte aligned blocks that do not overlap");
  }
  return MLA_OK;
}

int check_table(const int32_t* table, int64_t bt_stride, int64_t bt_cols, int64_t rows) {
  if (!table) return fail(MLA_ERR_INVALID, "block_table is NULL");
  if (bt_cols < 1 || (rows > 1 && bt_stride < bt_cols)) return fail(MLA_ERR_INVALID, "bad block_table geometry");
  if (!aligned(table, 4)) return fail(MLA_ERR_INVALID, "block_table must be 4-byte aligned");
  return MLA_OK;
}

int check_rows(int32_t B, int32_t T, const int32_t* cu_q) {
  if (B < 0 || T < 0) return fail(MLA_ERR_INVALID, "bad shape B=%d T=%d", B, T);
  if (!cu_q && T > B) return fail(MLA_ERR_INVALID, "without cu_q_lens every row is a request: T=%d exceeds B=%d", T, B);
  return MLA_OK;
}

}  // namespace

extern "C" int mla_index_q_cache_insert(const void* q, int64_t q_s0, int64_t q_s1, const void* k, int64_t k_s0,
                                        const float* weights, int64_t w_s0, float weight_scale, void* q_out,
                                        float* w_out, void* index_cache, mla_cache_format fmt, int64_t num_blocks,
                                        int64_t block_stride_bytes, int64_t entry_stride_bytes, float* index_scales,
                                        int64_t scale_block_stride, int32_t block_size, const int64_t* slot_mapping,
                                        const int64_t* positions, const float* cos_sin_cache, int64_t max_position,
                                        int32_t T, int32_t Hi, cudaStream_t stream) {
  if (!index_format(fmt)) return fail(MLA_ERR_INVALID, "the index cache is bf16 or fp8 (format %d)", static_cast<int>(fmt));
  if (T < 0) return fail(MLA_ERR_INVALID, "bad shape T=%d", T);
  if (Hi < 1 || Hi > 64) return fail(MLA_ERR_UNSUPPORTED, "Hi must be in [1, 64], got %d", Hi);
  if (T == 0) return ok();
  if (!q || !k || !weights || !q_out || !w_out || !slot_mapping) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (q_s1 < kIndexDim || q_s0 < static_cast<int64_t>(Hi - 1) * q_s1 + kIndexDim || k_s0 < kIndexDim || w_s0 < Hi)
    return fail(MLA_ERR_INVALID, "activation strides overlap rows");
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(weights, 4) || !aligned(w_out, 4) || !aligned(q_out, 16))
    return fail(MLA_ERR_INVALID, "misaligned tensors (q_out needs 16 bytes)");
  if (int rc = check_index_cache(index_cache, fmt, num_blocks, block_stride_bytes, entry_stride_bytes, index_scales,
                                 scale_block_stride, block_size))
    return rc;
  if ((positions == nullptr) != (cos_sin_cache == nullptr))
    return fail(MLA_ERR_INVALID, "positions and cos_sin_cache must be given together");
  if (positions && max_position < 1) return fail(MLA_ERR_INVALID, "max_position must be >= 1");
  if (!aligned(cos_sin_cache, 16)) return fail(MLA_ERR_INVALID, "cos_sin_cache must be 16-byte aligned");
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  IndexInsertParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_s0 = q_s0;
  p.q_s1 = q_s1;
  p.k = static_cast<const uint16_t*>(k);
  p.k_s0 = k_s0;
  p.w = weights;
  p.w_s0 = w_s0;
  p.weight_scale = weight_scale;
  p.q_out = q_out;
  p.w_out = w_out;
  p.cache = static_cast<uint8_t*>(index_cache);
  p.num_blocks = num_blocks;
  p.block_stride = block_stride_bytes;
  p.entry_stride = entry_stride_bytes;
  p.scales = index_scales;
  p.sc_stride = scale_block_stride;
  p.block_size = block_size;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.cos_sin = cos_sin_cache;
  p.max_position = max_position;
  p.T = T;
  p.Hi = Hi;
  p.vec = aligned(q, 16) && aligned(k, 16) && q_s0 % 8 == 0 && q_s1 % 8 == 0 && k_s0 % 8 == 0;
  p.err = d->err;
  if (launch_index_insert(fmt == MLA_CACHE_BF16, p, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "index insert launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

extern "C" int mla_index_gather(const void* index_cache, mla_cache_format fmt, int64_t num_blocks,
                                int64_t block_stride_bytes, int64_t entry_stride_bytes, const float* index_scales,
                                int64_t scale_block_stride, int32_t block_size, const int32_t* block_table,
                                int64_t bt_stride, int64_t bt_cols, const int32_t* cu_seq_lens,
                                const int32_t* seq_starts, int32_t batch, int64_t num_tokens, void* dst,
                                int64_t dst_row_stride, cudaStream_t stream) {
  if (!index_format(fmt)) return fail(MLA_ERR_INVALID, "the index cache is bf16 or fp8 (format %d)", static_cast<int>(fmt));
  if (batch < 0 || num_tokens < 0) return fail(MLA_ERR_INVALID, "bad shape batch=%d num_tokens=%lld", batch, static_cast<long long>(num_tokens));
  if (num_tokens >= (int64_t(1) << 31)) return fail(MLA_ERR_UNSUPPORTED, "num_tokens must be below 2^31");
  if (batch == 0 || num_tokens == 0) return ok();
  if (int rc = check_index_cache(index_cache, fmt, num_blocks, block_stride_bytes, entry_stride_bytes, index_scales,
                                 scale_block_stride, block_size))
    return rc;
  if (int rc = check_table(block_table, bt_stride, bt_cols, batch)) return rc;
  if (!cu_seq_lens || !dst) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (dst_row_stride < kIndexDim || !aligned(dst, 2)) return fail(MLA_ERR_INVALID, "bad dst rows");
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  IndexGatherParams p{};
  p.cache = static_cast<const uint8_t*>(index_cache);
  p.num_blocks = num_blocks;
  p.block_stride = block_stride_bytes;
  p.entry_stride = entry_stride_bytes;
  p.scales = index_scales;
  p.sc_stride = scale_block_stride;
  p.block_size = block_size;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.cu = cu_seq_lens;
  p.starts = seq_starts;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.dst = static_cast<uint16_t*>(dst);
  p.dst_row = dst_row_stride;
  p.vec = aligned(dst, 16) && dst_row_stride % 8 == 0;
  p.err = d->err;
  if (launch_index_gather(fmt == MLA_CACHE_BF16, p, d->sms, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "index gather launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

extern "C" int mla_index_scores(const void* q, int64_t q_s0, int64_t q_s1, const float* weights, int64_t w_s0,
                                const void* index_cache, mla_cache_format fmt, int64_t num_blocks,
                                int64_t block_stride_bytes, int64_t entry_stride_bytes, const float* index_scales,
                                int64_t scale_block_stride, int32_t block_size, const int32_t* block_table,
                                int64_t bt_stride, int64_t bt_cols, const int32_t* seq_lens, const int32_t* cu_q_lens,
                                int32_t B, int32_t T, int32_t Hi, int32_t block_tokens, float* scores, int64_t s_stride,
                                int64_t width, cudaStream_t stream) {
  if (!index_format(fmt)) return fail(MLA_ERR_INVALID, "the index cache is bf16 or fp8 (format %d)", static_cast<int>(fmt));
  if (int rc = check_rows(B, T, cu_q_lens)) return rc;
  if (Hi < 1 || Hi > 64) return fail(MLA_ERR_UNSUPPORTED, "Hi must be in [1, 64], got %d", Hi);
  if (block_tokens != 1 && block_tokens != 16 && block_tokens != 32 && block_tokens != 64 && block_tokens != 128)
    return fail(MLA_ERR_UNSUPPORTED, "block_tokens must be 1, 16, 32, 64 or 128, got %d", block_tokens);
  if (width < 0) return fail(MLA_ERR_INVALID, "width must be >= 0");
  if (B == 0 || T == 0 || width == 0) return ok();
  if (int rc = check_index_cache(index_cache, fmt, num_blocks, block_stride_bytes, entry_stride_bytes, index_scales,
                                 scale_block_stride, block_size))
    return rc;
  const int rows = tma_rows_for(block_size);
  if (rows == 0)
    return fail(MLA_ERR_UNSUPPORTED, "block_size must be 16, 32, 64, 128 or a multiple of 128, got %d", block_size);
  if (int rc = check_table(block_table, bt_stride, bt_cols, B)) return rc;
  if (!q || !weights || !seq_lens || !scores) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  const int e = fmt == MLA_CACHE_BF16 ? 2 : 1;
  if (!aligned(q, 16) || (q_s0 * e) % 16 || (q_s1 * e) % 16 || q_s1 < kIndexDim ||
      q_s0 < static_cast<int64_t>(Hi - 1) * q_s1 + kIndexDim)
    return fail(MLA_ERR_INVALID, "q needs 16-byte alignment and non-overlapping strides");
  if (w_s0 < Hi || !aligned(weights, 4)) return fail(MLA_ERR_INVALID, "bad weights rows");
  if (s_stride < width || !aligned(scores, 4)) return fail(MLA_ERR_INVALID, "bad scores rows");
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  const int hp = Hi <= 8 ? 8 : Hi <= 16 ? 16 : Hi <= 32 ? 32 : 64;
  CUtensorMap tk, tq;
  const uint64_t kd[3] = {static_cast<uint64_t>(kIndexDim * e), static_cast<uint64_t>(block_size), static_cast<uint64_t>(num_blocks)};
  const uint64_t ks[2] = {static_cast<uint64_t>(entry_stride_bytes), static_cast<uint64_t>(block_stride_bytes)};
  const uint32_t kb[3] = {128, static_cast<uint32_t>(rows), 1};
  if (int rc = tmap_3d(index_cache, kd, ks, kb, &tk)) return rc;
  // a box of hp heads x 256 / hp rows; heads and rows past the tensor read as zeros
  const uint64_t qd[3] = {static_cast<uint64_t>(kIndexDim * e), static_cast<uint64_t>(Hi), static_cast<uint64_t>(T)};
  const uint64_t qs[2] = {static_cast<uint64_t>(q_s1 * e), static_cast<uint64_t>(q_s0 * e)};
  const uint32_t qb[3] = {128, static_cast<uint32_t>(hp), static_cast<uint32_t>(256 / hp)};
  if (int rc = tmap_3d(q, qd, qs, qb, &tq)) return rc;
  IndexScoresParams p{};
  p.weights = weights;
  p.w_stride = w_s0;
  p.key_scales = index_scales;
  p.ks_stride = scale_block_stride;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.B = B;
  p.T = T;
  p.Hi = Hi;
  p.num_blocks = static_cast<int>(num_blocks);
  p.block_size = block_size;
  p.BR = rows;
  p.block_tokens = block_tokens;
  constexpr int64_t kMostKeys = (int64_t(1) << 31) - 1024;      // positions and tile edges stay in 32 bits
  p.cap = width > kMostKeys / block_tokens ? kMostKeys : width * block_tokens;
  p.scores = scores;
  p.s_stride = s_stride;
  p.err = d->err;
  if (launch_index_scores(fmt == MLA_CACHE_BF16, hp, p, &tk, &tq, d->sms, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "index scores launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

extern "C" int mla_index_select(const float* scores, int64_t s_stride, int64_t width, const int32_t* seq_lens,
                                const int32_t* cu_q_lens, int32_t B, int32_t T, int32_t block_tokens, int32_t topk,
                                int32_t first, int32_t last, int32_t* blocks, int64_t b_stride, int32_t* slots,
                                int64_t sl_stride, const int32_t* block_table, int64_t bt_stride, int64_t bt_cols,
                                int32_t page_size, int64_t num_blocks, cudaStream_t stream) {
  if (int rc = check_rows(B, T, cu_q_lens)) return rc;
  if (block_tokens < 1) return fail(MLA_ERR_INVALID, "block_tokens must be >= 1, got %d", block_tokens);
  if (topk < 1) return fail(MLA_ERR_INVALID, "topk must be >= 1, got %d", topk);
  if (topk > kSelectMaxTopk) return fail(MLA_ERR_UNSUPPORTED, "topk must be <= %d, got %d", kSelectMaxTopk, topk);
  if (first < 0 || last < 0 || static_cast<int64_t>(first) + last > topk)
    return fail(MLA_ERR_INVALID, "first and last must be >= 0 and fit in topk");
  if (width < 0 || width >= (int64_t(1) << 30)) return fail(MLA_ERR_UNSUPPORTED, "width must be in [0, 2^30)");
  if (B == 0 || T == 0) return ok();
  // (without a column no score and no page is looked at: every row is a list of none)
  if ((!scores && width > 0) || !seq_lens || !blocks) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (s_stride < width || !aligned(scores, 4)) return fail(MLA_ERR_INVALID, "bad scores rows");
  if (b_stride < topk || !aligned(blocks, 4)) return fail(MLA_ERR_INVALID, "bad blocks rows");
  if (slots) {
    const int64_t n = static_cast<int64_t>(topk) * block_tokens;
    if (n >= (int64_t(1) << 31)) return fail(MLA_ERR_UNSUPPORTED, "topk * block_tokens must be below 2^31");
    if (sl_stride < n || !aligned(slots, 4)) return fail(MLA_ERR_INVALID, "bad slots rows");
    if (width > 0)
      if (int rc = check_table(block_table, bt_stride, bt_cols, B)) return rc;
    if (page_size < 1 || num_blocks < 1) return fail(MLA_ERR_INVALID, "slots need page_size and num_blocks");
    if (num_blocks >= (int64_t(1) << 31) || num_blocks * page_size >= (int64_t(1) << 31))
      return fail(MLA_ERR_UNSUPPORTED, "num_blocks * page_size must be below 2^31");
  }
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  IndexSelectParams p{};
  p.scores = scores;
  p.s_stride = s_stride;
  p.width = width;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.B = B;
  p.T = T;
  p.block_tokens = block_tokens;
  p.topk = topk;
  p.first = first;
  p.last = last;
  p.blocks = blocks;
  p.b_stride = b_stride;
  p.slots = slots;
  p.sl_stride = sl_stride;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.page_size = page_size;
  p.num_blocks = num_blocks;
  p.err = d->err;
  if (launch_index_select(p, d->sms, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "index select launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

// The page table [T, topk] and lengths [T] of the selected pages, then the decode's own scratch.
static size_t selected_list_bytes(int32_t T, int32_t topk) {
  const size_t lens = (static_cast<size_t>(T) * 4 + 255) & ~size_t(255);
  const size_t table = (static_cast<size_t>(T) * topk * 4 + 255) & ~size_t(255);
  return lens + table;
}

namespace {

// The SM count of a workspace query: as given, or the current device's (0: no size).
int query_sms(int32_t T, int32_t topk, int32_t block_size, int32_t H, int32_t num_sms) {
  if (T <= 0 || topk <= 0 || block_size <= 0 || H <= 0) return 0;
  if (static_cast<int64_t>(topk) * block_size >= (1 << 30)) return 0;
  if (num_sms > 0) return num_sms;
  DevInfo* d = nullptr;
  return dev_info(&d) == MLA_OK ? d->sms : 0;
}

}  // namespace

extern "C" size_t mla_selected_decode_workspace_size(mla_cache_format fmt, int32_t T, int32_t topk, int32_t block_size,
                                                     int32_t H, int32_t num_sms) {
  const int sms = query_sms(T, topk, block_size, H, num_sms);
  if (sms == 0) return 0;
  if (fmt == MLA_CACHE_MXFP4) return selected_list_bytes(T, topk) + fp4_workspace_bytes(1, H, sms);
  const SelectedPlan sp = plan_selected(fmt, T, H, static_cast<int64_t>(topk) * block_size, sms);
  return selected_list_bytes(T, topk) + workspace_bytes_for(sp.rows, H, sp.main) + workspace_bytes_for(T - sp.rows, H, sp.tail);
}

extern "C" size_t mla_selected_decode_workspace_bound(mla_cache_format fmt, int32_t max_T, int32_t topk,
                                                      int32_t block_size, int32_t H, int32_t num_sms) {
  const int sms = query_sms(max_T, topk, block_size, H, num_sms);
  if (sms == 0) return 0;
  if (fmt == MLA_CACHE_MXFP4) return selected_list_bytes(max_T, topk) + fp4_workspace_bytes(1, H, sms);
  return selected_list_bytes(max_T, topk) + selected_partials_bound(fmt, max_T, H, static_cast<int64_t>(topk) * block_size, sms);
}

extern "C" int mla_selected_decode(const void* q, int64_t q_s0, int64_t q_s1, const void* kv_cache,
                                   mla_cache_format fmt, int64_t num_blocks, int64_t block_stride_bytes,
                                   int64_t entry_stride_bytes, int32_t block_size, const int32_t* block_table,
                                   int64_t bt_stride, int64_t bt_cols, const int32_t* seq_lens,
                                   const int32_t* cu_q_lens, const int32_t* blocks, int64_t b_stride, int32_t topk,
                                   int32_t B, int32_t T, int32_t H, float softmax_scale, float q_scale, float k_scale,
                                   void* out, int64_t o_s0, int64_t o_s1, float* lse, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  if (int rc = check_rows(B, T, cu_q_lens)) return rc;
  if (topk < 1 || block_size < 1) return fail(MLA_ERR_INVALID, "bad shape topk=%d block_size=%d", topk, block_size);
  if (static_cast<int64_t>(topk) * block_size >= (1 << 30))
    return fail(MLA_ERR_UNSUPPORTED, "topk * block_size must be below 2^30");
  if (B == 0 || T == 0) return ok();
  if (!seq_lens || !blocks) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (b_stride < topk || !aligned(blocks, 4)) return fail(MLA_ERR_INVALID, "bad blocks rows");
  if (H < 1 || H > 128) return fail(MLA_ERR_UNSUPPORTED, "H must be in [1, 128], got %d", H);
  if (int rc = check_table(block_table, bt_stride, bt_cols, B)) return rc;
  const size_t lists = selected_list_bytes(T, topk);
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  const bool fp4 = fmt == MLA_CACHE_MXFP4;
  const SelectedPlan sp = fp4 ? SelectedPlan{T, {1, 0}, {1, 0}} : plan_selected(fmt, T, H, static_cast<int64_t>(topk) * block_size, d->sms);
  // (the work items of the decode: at most 8 column groups a row and split)
  if (static_cast<int64_t>(T) * 8 * (sp.main.n_splits > sp.tail.n_splits ? sp.main.n_splits : sp.tail.n_splits) >= (int64_t(1) << 31))
    return fail(MLA_ERR_UNSUPPORTED, "too many rows");
  const int32_t rows = static_cast<int32_t>(sp.rows), more = T - rows;
  const size_t part = workspace_bytes_for(rows, H, sp.main), need = lists + (fp4 ? fp4_workspace_bytes(1, H, d->sms) : part + workspace_bytes_for(more, H, sp.tail));
  if (!workspace || workspace_bytes < need)
    return fail(MLA_ERR_INVALID, "workspace too small: need %zu bytes, got %zu", need, workspace_bytes);
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID, "workspace must be 256-byte aligned");
  const int32_t ctx = topk * block_size;
  uint8_t* rest = static_cast<uint8_t*>(workspace) + lists;
  // the decode's own checks, before the lists are launched
  if (int rc = check_paged_decode(q, q_s0, q_s1, kv_cache, fmt, num_blocks, block_stride_bytes, entry_stride_bytes,
                                  block_size, block_table, topk, seq_lens, T, 1, H, ctx, out, o_s0, o_s1, lse))
    return rc;
  PageListParams p{};
  p.blocks = blocks;
  p.b_stride = b_stride;
  p.topk = topk;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.B = B;
  p.T = T;
  p.block_size = block_size;
  p.lens = static_cast<int32_t*>(workspace);
  p.table = p.lens + ((static_cast<size_t>(T) * 4 + 255) & ~size_t(255)) / 4;
  p.sched[0] = sched_word(rest, rows, H, sp.main);
  p.sched[1] = sched_word(rest + part, more, H, sp.tail);
  p.err = d->err;
  if (launch_page_list(p, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "page list launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  if (fp4)
    return run_fp4_decode(q, q_s0, q_s1, kv_cache, num_blocks, block_stride_bytes, entry_stride_bytes, block_size, p.table, topk, p.lens, T, 1,
                          H, softmax_scale, out, o_s0, o_s1, lse, rest, workspace_bytes - lists, stream);
  if (int rc = run_paged_decode(q, q_s0, q_s1, kv_cache, fmt, num_blocks, block_stride_bytes, entry_stride_bytes, block_size,
                                p.table, topk, p.lens, rows, 1, H, ctx, softmax_scale, q_scale, k_scale, out, o_s0, o_s1, lse,
                                rest, part, sp.main, true, stream))
    return rc;
  if (more == 0) return ok();
  const int64_t qe = fmt == MLA_CACHE_FP8 ? 1 : 2;
  return run_paged_decode(static_cast<const uint8_t*>(q) + rows * q_s0 * qe, q_s0, q_s1, kv_cache, fmt, num_blocks,
                          block_stride_bytes, entry_stride_bytes, block_size, p.table + static_cast<int64_t>(rows) * topk, topk,
                          p.lens + rows, more, 1, H, ctx, softmax_scale, q_scale, k_scale,
                          static_cast<uint8_t*>(out) + rows * o_s0 * 2, o_s0, o_s1,
                          lse ? lse + static_cast<int64_t>(rows) * H : nullptr, rest + part, need - lists - part, sp.tail, true,
                          stream);
}
