// mla_step_api.cu -- entry points of the step around the attention: rotary positions and the planned blocks and slots.
// Host code only.
#include <cmath>

#include "mla.h"
#include "mla_host.h"
#include "mla_step.h"

using namespace mla;

namespace {

// One past the last byte of a [T, H, D] tensor (strides in bytes).
const uint8_t* end_of(const uint8_t* p, int64_t s0, int64_t s1, int T, int H, int64_t row) {
  return p + (T - 1) * s0 + (H - 1) * s1 + row;
}

// A tensor of mla_rope into x; vec and copy are narrowed to what it allows and needs.
int rope_tensor(const char* name, const void* in, int64_t i_s0, int64_t i_s1, void* out, int64_t o_s0, int64_t o_s1, int32_t T, int32_t H,
                int32_t D, int32_t at, int32_t R, int bytes, bool half, RopeTensor* x, bool* vec, bool* inplace) {
  if (H < 1 || D < R || at < 0 || at > D - R) return fail(MLA_ERR_INVALID, "%s: bad shape H=%d D=%d at=%d R=%d", name, H, D, at, R);
  if (D > 1024) return fail(MLA_ERR_UNSUPPORTED, "%s: D must be <= 1024, got %d", name, D);
  // (a token's values are counted in 32 bits)
  if (static_cast<int64_t>(H) * D >= (int64_t(1) << 31)) return fail(MLA_ERR_UNSUPPORTED, "%s: a token of %d heads is too large", name, H);
  if (!in || !out) return fail(MLA_ERR_INVALID, "%s: a required pointer is NULL", name);
  if (!aligned(in, bytes) || !aligned(out, bytes)) return fail(MLA_ERR_INVALID, "%s must be aligned to its type", name);
  if (i_s1 < D || i_s0 < static_cast<int64_t>(H) * i_s1 || o_s1 < D || o_s0 < static_cast<int64_t>(H) * o_s1)
    return fail(MLA_ERR_INVALID, "%s: strides overlap rows", name);
  *x = RopeTensor{static_cast<const uint8_t*>(in), static_cast<uint8_t*>(out), i_s0 * bytes, i_s1 * bytes, o_s0 * bytes, o_s1 * bytes, H, D, at, 0};
  *inplace = in == out && i_s0 == o_s0 && i_s1 == o_s1;
  if (!*inplace && x->in < end_of(x->out, x->o_s0, x->o_s1, T, H, D * bytes) && x->out < end_of(x->in, x->i_s0, x->i_s1, T, H, D * bytes))
    return fail(MLA_ERR_INVALID, "%s: the output meets the input without being the same tensor", name);
  const int W = 16 / bytes;
  *vec = *vec && aligned(in, 16) && aligned(out, 16) && i_s0 % W == 0 && i_s1 % W == 0 && o_s0 % W == 0 && o_s1 % W == 0 && D % W == 0 &&
         at % W == 0 && R % (half ? 2 * W : W) == 0;
  return MLA_OK;
}

}  // namespace

extern "C" int mla_rope(int32_t type, const void* q, int64_t q_s0, int64_t q_s1, void* q_out, int64_t qo_s0, int64_t qo_s1, int32_t H,
                        int32_t D, int32_t q_at, const void* k, int64_t k_s0, int64_t k_s1, void* k_out, int64_t ko_s0, int64_t ko_s1,
                        int32_t Hk, int32_t Dk, int32_t k_at, const int64_t* positions, const float* cos_sin, int64_t max_position,
                        int32_t R, int32_t half, int32_t inverse, int32_t T, cudaStream_t stream) {
  if (type != MLA_TYPE_BF16 && type != MLA_TYPE_FP16 && type != MLA_TYPE_FP32) return fail(MLA_ERR_INVALID, "unknown element type %d", type);
  if (T < 0) return fail(MLA_ERR_INVALID, "T must be >= 0");
  if (R < 2 || R % 2) return fail(MLA_ERR_INVALID, "the rotated width must be even and positive, got %d", R);
  if (R > 2 * kRopeMaxHalf) return fail(MLA_ERR_UNSUPPORTED, "the rotated width must be <= %d, got %d", 2 * kRopeMaxHalf, R);
  if ((k == nullptr) != (k_out == nullptr)) return fail(MLA_ERR_INVALID, "k and k_out must be given together");
  if (T == 0) return ok();
  if (!positions || !cos_sin) return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (max_position < 1) return fail(MLA_ERR_INVALID, "max_position must be >= 1");
  if (!aligned(positions, 8) || !aligned(cos_sin, 4)) return fail(MLA_ERR_INVALID, "positions and cos_sin must be aligned to their types");
  const int bytes = type == MLA_TYPE_FP32 ? 4 : 2;
  RopeParams p{};
  // whole pieces of 16 bytes, and of their pairs' cosines and sines
  bool vec = aligned(cos_sin, 16) && R % 8 == 0, in0 = false, in1 = false;
  if (int rc = rope_tensor("q", q, q_s0, q_s1, q_out, qo_s0, qo_s1, T, H, D, q_at, R, bytes, half != 0, &p.x[0], &vec, &in0)) return rc;
  if (k) {
    if (int rc = rope_tensor("k", k, k_s0, k_s1, k_out, ko_s0, ko_s1, T, Hk, Dk, k_at, R, bytes, half != 0, &p.x[1], &vec, &in1)) return rc;
    if (in0 != in1) return fail(MLA_ERR_INVALID, "q and k are rotated in place both or neither");
  }
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.T = T;
  p.R = R;
  p.inverse = inverse != 0;
  p.err = d->err;
  if (launch_rope(type, half != 0, vec, !in0, p, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "rope launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

extern "C" int mla_rope_table(float* out, int64_t max_position, int32_t R, double base, int32_t scaling, double factor, int64_t original,
                              double beta_fast, double beta_slow, double attn_scale, cudaStream_t stream) {
  if (R < 2 || R % 2) return fail(MLA_ERR_INVALID, "the rotated width must be even and positive, got %d", R);
  if (R > 2 * kRopeMaxHalf) return fail(MLA_ERR_UNSUPPORTED, "the rotated width must be <= %d, got %d", 2 * kRopeMaxHalf, R);
  if (max_position < 0) return fail(MLA_ERR_INVALID, "max_position must be >= 0");
  if (max_position > (int64_t(1) << 40) / R) return fail(MLA_ERR_UNSUPPORTED, "the table is too large");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(MLA_ERR_INVALID, "base must be above 1");
  if (scaling < MLA_ROPE_PLAIN || scaling > MLA_ROPE_YARN) return fail(MLA_ERR_INVALID, "unknown scaling %d", scaling);
  if (scaling != MLA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return fail(MLA_ERR_INVALID, "factor must be positive");
  if (scaling == MLA_ROPE_NTK && R <= 2) return fail(MLA_ERR_INVALID, "the ntk scaling needs a rotated width above 2");
  if (scaling == MLA_ROPE_YARN && (original < 1 || !(beta_fast > 0.0) || !(beta_slow > 0.0)))
    return fail(MLA_ERR_INVALID, "the yarn scaling needs original >= 1 and positive betas");
  if (!std::isfinite(attn_scale)) return fail(MLA_ERR_INVALID, "attn_scale must be finite");
  if (max_position == 0) return ok();
  if (!out || !aligned(out, 4)) return fail(MLA_ERR_INVALID, "bad out");
  RopeTableParams p{};
  p.out = out;
  p.n = max_position;
  p.R = R;
  p.scale = attn_scale;
  const double pi = 3.14159265358979323846;
  const double b = scaling == MLA_ROPE_NTK ? base * std::pow(factor, static_cast<double>(R) / (R - 2)) : base;
  auto turns = [&](double beta) { return R * std::log(static_cast<double>(original) / (2.0 * pi * beta)) / (2.0 * std::log(base)); };
  double lo = 0, hi = 1;
  if (scaling == MLA_ROPE_YARN) {
    lo = std::fmax(std::floor(turns(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(turns(beta_slow)), R - 1.0);
    if (hi <= lo) hi = lo + 0.001;
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(b, -2.0 * i / R);
    if (scaling == MLA_ROPE_LINEAR) f /= factor;
    if (scaling == MLA_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f = f * (1.0 - r) + f / factor * r;
    }
    p.freq[i] = f;
  }
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  if (launch_rope_table(p, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "rope table launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}

extern "C" int mla_plan_step(const int32_t* seq_lens, const int32_t* new_lens, const uint8_t* finished, int32_t* block_table,
                             int64_t t_stride, int32_t cols, int32_t* free_blocks, int64_t capacity, const int32_t* num_free,
                             int32_t* seq_out, int32_t* num_free_out, uint8_t* served, int32_t* cu_q_lens, int64_t* slots,
                             int64_t* positions, int32_t B, int32_t T, int32_t block_size, cudaStream_t stream) {
  if (B < 1 || T < 0) return fail(MLA_ERR_INVALID, "bad shape B=%d T=%d", B, T);
  if (B > kPlanMost || T > kPlanMost) return fail(MLA_ERR_UNSUPPORTED, "B and T must be <= %d, got %d and %d", kPlanMost, B, T);
  if (block_size < 1) return fail(MLA_ERR_INVALID, "block_size must be >= 1");
  if (cols < 1 || t_stride < cols) return fail(MLA_ERR_INVALID, "bad block table: %d columns, row stride %lld", cols, static_cast<long long>(t_stride));
  if (capacity < 0 || capacity > 0x7FFFFFFF) return fail(MLA_ERR_INVALID, "bad capacity of the free blocks");
  if (!seq_lens || !new_lens || !block_table || (capacity > 0 && !free_blocks) || !num_free || !seq_out || !num_free_out ||
      (!served && B > kPlanKept) || !cu_q_lens || (T > 0 && (!slots || !positions)))
    return fail(MLA_ERR_INVALID, "a required pointer is NULL");
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) || !aligned(num_free, 4) ||
      !aligned(seq_out, 4) || !aligned(num_free_out, 4) || !aligned(cu_q_lens, 4) || !aligned(slots, 8) || !aligned(positions, 8))
    return fail(MLA_ERR_INVALID, "tensors must be aligned to their types");
  DevInfo* d = nullptr;
  if (int rc = dev_info(&d)) return rc;
  PlanParams p{};
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.finished = finished;
  p.table = block_table;
  p.t_stride = t_stride;
  p.free_blocks = free_blocks;
  p.capacity = capacity;
  p.num_free = num_free;
  p.seq_out = seq_out;
  p.num_free_out = num_free_out;
  p.served = served;
  p.cu = cu_q_lens;
  p.slots = slots;
  p.positions = positions;
  p.B = B;
  p.cols = cols;
  p.T = T;
  p.block_size = block_size;
  p.err = d->err;
  if (launch_plan(p, stream) != cudaSuccess)
    return fail(MLA_ERR_CUDA, "plan launch failed: %s", cudaGetErrorString(cudaGetLastError()));
  return ok();
}
