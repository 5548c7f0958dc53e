// mla_host.h -- host-side helpers of the C ABI's translation units: error returns, per-device
// lookups, tensor maps.
#pragma once
#include <cuda.h>
#include <cstdint>
#include <cuda_runtime.h>

namespace mla {

struct DevInfo {
  bool ready = false;
  int sms = 0;
  uint32_t* err = nullptr;
};

// Set the message of mla_last_error() and return `code`; clear it and return MLA_OK.
int fail(int code, const char* fmt, ...);
int ok();
// SM count and device error word of the current device (looked up once per device).
int dev_info(DevInfo** out);
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Rows per TMA box for a block size, or 0 when the page kernels do not serve it: the box rows must
// divide the 128-key tile (block_size 16..128 a power of two) or be a whole 128-row slice of a
// larger block.
int tma_rows_for(int block_size, int keys_per_tile = 128);
// 3-D uint8 tensor map (128-byte swizzle, or none): dims {x bytes, y, z}, strides {y, z} in bytes.
int tmap_3d(const void* base, const uint64_t (&dims)[3], const uint64_t (&strides)[2], const uint32_t (&box)[3],
            CUtensorMap* out, bool swizzle = true);

// The argument checks of mla_paged_decode (MLA_OK, or its error with the message set).
int check_paged_decode(const void* q, int64_t q_s0, int64_t q_s1, const void* kv_cache, int fmt, int64_t num_blocks,
                       int64_t block_stride_bytes, int64_t entry_stride_bytes, int32_t block_size,
                       const int32_t* block_table, int64_t bt_stride, const int32_t* seq_lens, int32_t B,
                       int32_t q_len, int32_t H, int32_t max_context, const void* out, int64_t o_s0, int64_t o_s1,
                       const float* lse);


// Split-K plan of a paged decode: n_splits parts of `chunk` keys.
struct SplitPlan {
  int n_splits;
  int64_t chunk;
};
// Plan of a decode over selected pages: rows [0, rows) in one launch, the rest (if any) in another.
struct SelectedPlan {
  int64_t rows;
  SplitPlan main, tail;
};
SelectedPlan plan_selected(int fmt, int64_t T, int H, int64_t context, int sms);
// The largest workspace_bytes_for of the parts of plan_selected over 1 .. T rows.
size_t selected_partials_bound(int fmt, int64_t T, int H, int64_t context, int sms);
// Workspace of a plan, and the address of its scheduler word there (null without splits).
size_t workspace_bytes_for(int64_t n_rows, int H, const SplitPlan& sp);
uint32_t* sched_word(void* workspace, int64_t n_rows, int H, const SplitPlan& sp);
// mla_paged_decode after its checks, with a plan; sched_ready: the scheduler word is zeroed by earlier
// work of the stream.
int run_paged_decode(const void* q, int64_t q_s0, int64_t q_s1, const void* kv_cache, int cache_fmt, int64_t num_blocks,
                     int64_t block_stride_bytes, int64_t entry_stride_bytes, int32_t block_size,
                     const int32_t* block_table, int64_t bt_stride, const int32_t* seq_lens, int32_t B, int32_t q_len,
                     int32_t H, int32_t max_context, float softmax_scale, float q_scale, float k_scale, void* out,
                     int64_t o_s0, int64_t o_s1, float* lse, void* workspace, size_t workspace_bytes,
                     const SplitPlan& sp, bool sched_ready, cudaStream_t stream);

// Workspace of an mxfp4 decode, and that decode after its checks (check_paged_decode).
size_t fp4_workspace_bytes(int q_len, int H, int sms);
int run_fp4_decode(const void* q, int64_t q_s0, int64_t q_s1, const void* kv_cache, int64_t num_blocks,
                   int64_t block_stride_bytes, int64_t entry_stride_bytes, int32_t block_size, const int32_t* block_table,
                   int64_t bt_stride, const int32_t* seq_lens, int32_t B, int32_t q_len, int32_t H, float softmax_scale,
                   void* out, int64_t o_s0, int64_t o_s1, float* lse, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream);

}  // namespace mla
