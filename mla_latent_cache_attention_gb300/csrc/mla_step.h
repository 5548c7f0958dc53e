// mla_step.h -- parameter blocks of the step around the attention: rotary positions and the planned
// blocks and slots (mla_rope.cu, mla_plan.cu; entry points in mla_step_api.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace mla {

struct RopeTensor {
  const uint8_t* in;
  uint8_t* out;
  int64_t i_s0, i_s1, o_s0, o_s1;      // bytes
  int H, D, at;                        // heads, width, first rotated value
  int units;                           // work units of a head (launch_rope)
};

struct RopeParams {
  RopeTensor x[2];                     // the second with H = 0 where there is none
  const int64_t* positions;
  const float* cos_sin;                // [max_position][R]: cosines, then sines
  int64_t max_position;
  int T, R;
  int inverse;
  int joint;                           // the heads of both are one run of the same shape (launch_rope)
  uint32_t* err;
};

// type: 0 bf16, 1 fp16, 2 fp32; half: pairs (i, i + R / 2), else (2 i, 2 i + 1); vec: 16-byte accesses are possible
cudaError_t launch_rope(int type, bool half, bool vec, bool copy, RopeParams p, cudaStream_t stream);

constexpr int kRopeMaxHalf = 256;
struct RopeTableParams {
  float* out;
  int64_t n;                           // positions
  int R;
  double scale;                        // of every cosine and sine
  double freq[kRopeMaxHalf];           // angle of a pair per position
};
cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream);

constexpr int kPlanKept = 1024;          // requests whose sums are kept on chip
constexpr int kPlanMost = 0x7FFFFFFF - 8 * kPlanKept;      // requests or rows: one more round of all threads still counts in 32 bits
struct PlanParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  const uint8_t* finished;             // [B] truth values, or null
  int32_t* table;
  int64_t t_stride;
  int32_t* free_blocks;
  int64_t capacity;                    // entries of free_blocks
  const int32_t* num_free;
  int32_t* seq_out;
  int32_t* num_free_out;
  uint8_t* served;                     // [B]; null: not wanted (B <= kPlanKept)
  int32_t* cu;                         // [B + 1]
  int64_t* slots;                      // [T]
  int64_t* positions;                  // [T]
  int B, cols, T, block_size;
  uint32_t* err;
};
cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream);

}  // namespace mla
