// mla_index.h -- parameter blocks and launchers of the selector in front of sparse attention: the
// index cache (insert, gather), the scores, the selection and the selected pages (not part of the
// public C ABI).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mla {

constexpr int kSelectMaxTopk = 8192;
constexpr int kIndexDim = 128;    // values of an index query or key: [nope (64) | rope (64)]

// Decode / prefill epilogue of the selector: index queries and keys rotated, quantised, inserted.
struct IndexInsertParams {
  const uint16_t* q;       // bf16 [T, Hi, 128]
  int64_t q_s0, q_s1;
  const uint16_t* k;       // bf16 [T, 128]
  int64_t k_s0;
  const float* w;          // [T, Hi]
  int64_t w_s0;
  float weight_scale;
  void* q_out;             // bf16 or E4M3 [T, Hi, 128] contiguous
  float* w_out;            // [T, Hi] contiguous
  uint8_t* cache;
  int64_t num_blocks, block_stride, entry_stride;    // bytes
  float* scales;           // [num_blocks, block_size], fp8 only
  int64_t sc_stride;
  int block_size;
  const int64_t* slot_mapping;
  const int64_t* positions;
  const float* cos_sin;
  int64_t max_position;
  int T, Hi;
  int vec;                 // q and k rows 16-byte aligned, the rope table's too
  uint32_t* err;
};

struct IndexGatherParams {
  const uint8_t* cache;
  int64_t num_blocks, block_stride, entry_stride;
  const float* scales;
  int64_t sc_stride;
  int block_size;
  const int32_t* block_table;
  int64_t bt_stride, bt_cols;
  const int32_t* cu;       // [batch + 1]
  const int32_t* starts;   // [batch] or null
  int batch;
  int64_t num_tokens;
  uint16_t* dst;           // bf16 rows
  int64_t dst_row;         // elements
  int vec;                 // dst rows 16-byte aligned
  uint32_t* err;
};

struct IndexScoresParams {
  const float* weights;    // [T, Hi]
  int64_t w_stride;
  const float* key_scales; // [num_blocks, block_size], fp8 only
  int64_t ks_stride;
  const int32_t* block_table;
  int64_t bt_stride, bt_cols;
  const int32_t* seq_lens; // [B]
  const int32_t* cu_q;     // [B + 1] or null: one row per request
  int B, T, Hi;
  int num_blocks, block_size, BR;
  int block_tokens;
  int64_t cap;             // keys that have a column: width * block_tokens
  float* scores;
  int64_t s_stride;
  uint32_t* err;
};

struct IndexSelectParams {
  const float* scores;
  int64_t s_stride;
  int64_t width;           // columns of scores
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int B, T;
  int block_tokens, topk, first, last;
  int32_t* blocks;         // [T, topk]
  int64_t b_stride;
  int32_t* slots;          // [T, topk * block_tokens] or null
  int64_t sl_stride;
  const int32_t* block_table;
  int64_t bt_stride, bt_cols;
  int page_size;
  int64_t num_blocks;
  uint32_t* err;
};

// Page lists of the selected blocks of each row, as a block table and lengths for the paged decode.
struct PageListParams {
  const int32_t* blocks;   // [T, topk]
  int64_t b_stride;
  int topk;
  const int32_t* block_table;
  int64_t bt_stride, bt_cols;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  int B, T, block_size;
  int32_t* table;          // [T, topk]
  int32_t* lens;           // [T]
  uint32_t* sched[2];      // scheduler words of the decode's launches, zeroed here, or null
  uint32_t* err;
};

cudaError_t launch_index_insert(int bf16, const IndexInsertParams& p, cudaStream_t stream);
cudaError_t launch_index_gather(int bf16, const IndexGatherParams& p, int sms, cudaStream_t stream);
// hp: heads padded to 8, 16, 32 or 64; tk / tq point to CUtensorMaps of the cache and the queries
cudaError_t launch_index_scores(int bf16, int hp, const IndexScoresParams& p, const void* tk, const void* tq, int grid,
                                cudaStream_t stream);
cudaError_t launch_index_select(const IndexSelectParams& p, int sms, cudaStream_t stream);
cudaError_t launch_page_list(const PageListParams& p, cudaStream_t stream);

// Request of row t and the keys the row sees (seq_len - rows of the request + its place + 1), for a
// whole warp: a 32-way search over cu_q (null: row t is request t).  A row of no request gives -1.
__device__ __forceinline__ int row_request(const int32_t* cu_q, const int32_t* seq_lens, int B, int t, int64_t* visible) {
  int b = t, place = 0, n = 1;
  if (cu_q) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = B + 1;         // the last entry at or below t is in cu_q[lo .. lo + len)
    bool found = true;
    while (len > 1) {
      const int step = (len + 31) / 32, i = lo + lane * step;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane * step < len && cu_q[i < B ? i : B] <= t);
      if (m == 0) {
        found = false;
        break;
      }
      const int last = 31 - __clz(m);
      lo += last * step;
      len = min(step, len - last * step);
    }
    if (!found || lo >= B) return -1;
    b = lo;
    const int first = cu_q[b];
    if (t < first) return -1;
    place = t - first;
    n = cu_q[b + 1] - first;
    if (place >= n) return -1;
  } else if (t >= B) {
    return -1;
  }
  const int64_t v = static_cast<int64_t>(max(seq_lens[b], 0)) - n + place + 1;
  *visible = v > 0 ? v : 0;
  return b;
}

}  // namespace mla
