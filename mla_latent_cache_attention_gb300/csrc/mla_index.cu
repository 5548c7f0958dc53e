// mla_index.cu -- the memory-bound kernels of the selector in front of sparse attention:
//   * index queries and keys rotated, quantised and inserted into the paged index cache;
//   * cached index keys read back as bf16;
//   * the exact selection of the topk best-scored blocks of every row;
//   * the page lists of selected blocks for the paged decode.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "mla_index.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace {

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t bf16_rn(float x) {
  __nv_bfloat16 b = __float2bfloat16_rn(x);
  return *reinterpret_cast<uint16_t*>(&b);
}

// k, the least integer with amax <= 448 * 2^k = 1.75 * 2^(8 + k), from the bits of amax; at least
// -126, and 0 for amax = 0.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0;
  const int e = static_cast<int>(u >> 23);
  if (e == 0) return -126;
  const int k = e - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return k < -126 ? -126 : k;
}

// 8 consecutive bf16 values as fp32
__device__ __forceinline__ void load_bf16x8(const uint16_t* __restrict__ src, bool vec, float (&x)[8]) {
  if (vec) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf16_value(__ldg(src + i));
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = bf16_rn(x[2 * i]) | (bf16_rn(x[2 * i + 1]) << 16);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// ------------------------------------------------------------------------------------------
// Insert.  y = [nope | rope(pe)] in fp32 (GPT-J pairs, the table's cos and sin, one product
// rounded before the fused sum, as the latent epilogue); E4M3: scale 2^k from the vector's largest
// magnitude, codes e4m3(y / 2^k), the query's scale folded into its weight; bf16: y rounded once.
//
// Bound by memory: one read of every query and one write.  A half-warp owns a vector (8 values a
// lane: a 16-byte load, an 8- or 16-byte store), the four butterflies of the maximum stay inside
// it.  Vector Hi of a token is its key.
constexpr int kInsVec = 2;      // vectors of a half-warp, their loads in flight together

template <bool kBf16>
__global__ void __launch_bounds__(128) mla_index_insert_kernel(const IndexInsertParams p) {
  // a kernel launched next as a programmatic dependent may be scheduled now
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15, d0 = 8 * l;
  const int v0 = (blockIdx.y * 8 + hw) * kInsVec;
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  if (v0 > p.Hi) return;
  float x[kInsVec][8];
#pragma unroll
  for (int u = 0; u < kInsVec; ++u) {
    const int v = v0 + u;
    if (v <= p.Hi) load_bf16x8((v < p.Hi ? p.q + t * p.q_s0 + v * p.q_s1 : p.k + t * p.k_s0) + d0, p.vec != 0, x[u]);
  }
  const int64_t slot = p.Hi < v0 + kInsVec ? p.slot_mapping[t] : -1;
  if (p.positions) {
    int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) {
      if (l == 0 && p.Hi < v0 + kInsVec) set_device_error(p.err, 8u);
      pos = pos < 0 ? 0 : p.max_position - 1;
    }
    if (l >= 8) {      // the rotated half: lane l holds pairs 4 (l - 8) .. 4 (l - 8) + 3
      const float* cs = p.cos_sin + pos * 64 + 4 * (l - 8);
      float c[4], s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __ldg(cs + i), s[i] = __ldg(cs + 32 + i);
#pragma unroll
      for (int u = 0; u < kInsVec; ++u) {
        if (v0 + u > p.Hi) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[u][2 * i], b = x[u][2 * i + 1];
          x[u][2 * i] = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
          x[u][2 * i + 1] = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kInsVec; ++u) {
    const int v = v0 + u;
    if (v > p.Hi) break;
    uint8_t* ent = nullptr;
    int64_t blk = 0, off = 0;
    if (v == p.Hi && slot >= 0) {
      blk = slot / p.block_size;
      off = slot - blk * p.block_size;
      if (blk < p.num_blocks)
        ent = p.cache + blk * p.block_stride + off * p.entry_stride;
      else if (l == 0)
        set_device_error(p.err, 4u);
    }
    const int64_t o = (t * p.Hi + v) * kIndexDim + d0;
    if (kBf16) {
      const uint4 y = pack_bf16x8(x[u]);
      if (v < p.Hi) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + o) = y;
        if (l == 0) p.w_out[t * p.Hi + v] = p.w[t * p.w_s0 + v] * p.weight_scale;
      } else if (ent) {
        *reinterpret_cast<uint4*>(ent + 2 * d0) = y;
      }
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[u][i]));
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, m));
    const int k = scale_exponent(amax);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);      // 2^-k, exact
    const float sc = k < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = static_cast<uint32_t>(
          __nv_cvt_float2_to_fp8x2(make_float2(x[u][2 * i] * inv, x[u][2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3));
      c[i >> 1] |= two << (16 * (i & 1));
    }
    if (v < p.Hi) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q_out) + o) = make_uint2(c[0], c[1]);
      if (l == 0) p.w_out[t * p.Hi + v] = p.w[t * p.w_s0 + v] * p.weight_scale * sc;
    } else if (ent) {
      *reinterpret_cast<uint2*>(ent + d0) = make_uint2(c[0], c[1]);
      if (l == 0) p.scales[blk * p.sc_stride + off] = sc;
    }
  }
}

// ------------------------------------------------------------------------------------------
// Gather: row r of request b (cu[b] <= r < cu[b+1]) is position starts[b] + r - cu[b], as
// bf16(code * scale).  A half-warp writes a 256-byte row, 8 values a lane.
template <bool kBf16>
__global__ void __launch_bounds__(128) mla_index_gather_kernel(const IndexGatherParams p) {
  const int l = threadIdx.x & 15, d0 = 8 * l;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 4);
  if (r >= p.num_tokens || r >= p.cu[p.batch] || r < p.cu[0]) return;
  int lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const int64_t pos = static_cast<int64_t>(p.starts ? p.starts[lo] : 0) + (r - p.cu[lo]);
  const int64_t col = pos >= 0 ? pos / p.block_size : -1;
  const int64_t blk = col >= 0 && col < p.bt_cols ? p.block_table[lo * p.bt_stride + col] : -1;
  uint4 y = make_uint4(0, 0, 0, 0);
  if (blk < 0 || blk >= p.num_blocks) {
    if (l == 0) set_device_error(p.err, 2u);
  } else {
    const int64_t off = pos % p.block_size;
    const uint8_t* ent = p.cache + blk * p.block_stride + off * p.entry_stride;
    if (kBf16) {
      y = __ldg(reinterpret_cast<const uint4*>(ent + 2 * d0));
    } else {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(ent + d0));
      const float s = __ldg(p.scales + blk * p.sc_stride + off);
      const uint32_t w[2] = {c.x, c.y};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));      // exact
        x[2 * i] = f.x * s;
        x[2 * i + 1] = f.y * s;
      }
      y = pack_bf16x8(x);
    }
  }
  uint16_t* dst = p.dst + r * p.dst_row + d0;
  if (p.vec) {
    *reinterpret_cast<uint4*>(dst) = y;
  } else {
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

// ------------------------------------------------------------------------------------------
// Selection.  A score becomes a 32-bit key whose unsigned order is the scores' (0 = never taken:
// -inf and NaN; all ones: a forced block), so the k-th largest key is found digit by digit
// (11 + 11 + 10 bits) from histograms of the keys that match the digits so far.  A last pass in
// index order takes every larger key and the first ones of those that equal it: ties go to the
// lowest index, the list comes out ascending, and nothing depends on the order of atomics.
constexpr int kSelThreads = 1024;

struct SelRow {
  const float* x;
  int64_t n;               // visible blocks
  int64_t lo, hi;          // forced: below lo, from hi on
};

__device__ __forceinline__ uint32_t select_key(const SelRow& r, int64_t i) {
  if (i >= r.n) return 0u;
  if (i < r.lo || i >= r.hi) return 0xFFFFFFFFu;
  const float f = r.x[i] + 0.f;          // -0 and +0 are equal
  const uint32_t u = __float_as_uint(f);
  const uint32_t key = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return (f != f || key < 0x00800000u) ? 0u : min(key, 0xFFFFFFFEu);
}

__global__ void __launch_bounds__(kSelThreads) mla_index_select_kernel(const IndexSelectParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t wsum[32];
  __shared__ int64_t srow[2];
  __shared__ uint32_t sdig[3];       // digit, keys above it, keys in it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x;
  if (tid == 0) {
    int64_t vis = 0;
    srow[0] = row_request(p.cu_q, p.seq_lens, p.B, t, &vis);
    srow[1] = vis;
  }
  __syncthreads();
  const int b = static_cast<int>(srow[0]);
  const int64_t vis = srow[1];
  if (b < 0) return;
  SelRow r;
  r.x = p.scores + t * p.s_stride;
  r.n = min((vis + p.block_tokens - 1) / p.block_tokens, p.width);
  r.lo = p.first;
  r.hi = r.n - p.last;
  int32_t* out = p.blocks + t * p.b_stride;
  int32_t* out_slots = p.slots ? p.slots + t * p.sl_stride : nullptr;

  // ---- the k-th largest key: keys above `thr` are taken, and the first `ties` that equal it
  uint32_t thr = 0, ties = 0;
  if (r.n > p.topk) {
    uint32_t left = p.topk, prefix = 0;
    for (int d = 0; d < 3; ++d) {
      const int bits = d < 2 ? 11 : 10, shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = 1 << bits;
      const int above = shift + bits;            // the digits found so far
      for (int i = tid; i < bins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int64_t i = tid; i < r.n; i += kSelThreads) {
        const uint32_t key = select_key(r, i);
        if (d == 0 || (key >> above) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // suffix sums, two bins a thread from the top: thread q holds bins - 1 - 2q and the next
      const int hi_bin = bins - 1 - 2 * tid;
      const uint32_t c0 = hi_bin >= 0 ? hist[hi_bin] : 0, c1 = hi_bin > 0 ? hist[hi_bin - 1] : 0;
      uint32_t inc = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      uint32_t base = 0;
      for (int w = 0; w < warp; ++w) base += wsum[w];
      const uint32_t upto = base + inc, before = upto - c0 - c1;
      if (before < left && left <= upto) {       // exactly one thread
        const bool first = left <= before + c0;
        sdig[0] = static_cast<uint32_t>(first ? hi_bin : hi_bin - 1);
        sdig[1] = first ? before : before + c0;
        sdig[2] = first ? c0 : c1;
      }
      __syncthreads();
      prefix = (prefix << bits) | sdig[0];
      left -= sdig[1];
    }
    thr = prefix;
    ties = left;
    if (thr == 0) ties = 0;      // fewer candidates than topk: keys of 0 are never taken
  }

  // ---- in index order: positions by prefix sums over (larger, equal)
  uint32_t gt0 = 0, eq0 = 0;     // taken before this chunk
  for (int64_t c0 = 0; c0 < r.n; c0 += kSelThreads) {
    const int64_t i = c0 + tid;
    const uint32_t key = select_key(r, i);
    const bool gt = key > thr, eq = key == thr && thr != 0;
    const uint32_t bg = __ballot_sync(0xFFFFFFFFu, gt), be = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) wsum[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    const uint32_t lt = (1u << lane) - 1;
    const uint32_t g = gt0 + (before & 0xFFFF) + __popc(bg & lt);
    const uint32_t e = eq0 + (before >> 16) + __popc(be & lt);
    if (gt || (eq && e < ties)) out[g + min(e, ties)] = static_cast<int32_t>(i);
    gt0 += all & 0xFFFF;
    eq0 += all >> 16;
    __syncthreads();
  }
  const int taken = static_cast<int>(gt0 + min(eq0, ties));
  for (int i = taken + tid; i < p.topk; i += kSelThreads) out[i] = -1;
  if (!out_slots) return;
  // ---- token slots of the taken blocks through the block table
  __syncthreads();
  const int64_t total = static_cast<int64_t>(p.topk) * p.block_tokens;
  for (int64_t i = tid; i < total; i += kSelThreads) {
    const int j = static_cast<int>(i / p.block_tokens);
    int32_t slot = -1;
    if (j < taken) {
      const int64_t pos = static_cast<int64_t>(out[j]) * p.block_tokens + i % p.block_tokens;
      if (pos < vis) {
        const int64_t col = pos / p.page_size;
        const int64_t id = col < p.bt_cols ? p.block_table[b * p.bt_stride + col] : -1;
        if (id < 0 || id >= p.num_blocks)
          set_device_error(p.err, 2u);
        else
          slot = static_cast<int32_t>(id * p.page_size + pos % p.page_size);
      }
    }
    out_slots[i] = slot;
  }
}

// ------------------------------------------------------------------------------------------
// Page lists.  One warp per row keeps the visible pages of its list in order and puts the partly
// visible one (the row's newest page, when its last tokens are hidden or unwritten) last, so that
// a length alone says which tokens the row attends: full pages x block_size + the part.
__global__ void __launch_bounds__(128) mla_page_list_kernel(const PageListParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= p.T) return;
  int64_t vis = 0;
  const int b = row_request(p.cu_q, p.seq_lens, p.B, t, &vis);
  if (b < 0) {
    if (lane == 0) p.lens[t] = 0;
    return;
  }
  const int64_t full = vis / p.block_size;         // pages below this one are wholly visible
  const int part = static_cast<int>(vis % p.block_size);
  const int32_t* src = p.blocks + t * p.b_stride;
  int32_t* dst = p.table + static_cast<int64_t>(t) * p.topk;
  int count = 0;
  bool partly = false;
  uint32_t errbits = 0;
  auto page = [&](int64_t c) -> int32_t {           // a page past the table: an id that the decode reports
    return c < p.bt_cols ? p.block_table[b * p.bt_stride + c] : -1;
  };
  for (int c0 = 0; c0 < p.topk; c0 += 32) {
    const int c = c0 + lane < p.topk ? src[c0 + lane] : -1;
    const bool is_part = part > 0 && c == full;
    const bool ok = c >= 0 && c < full;
    if (c >= 0 && !ok && !is_part) errbits |= 1u;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, ok);
    const int n_part = __popc(__ballot_sync(0xFFFFFFFFu, is_part));
    if (n_part > (partly ? 0 : 1)) errbits |= 1u;   // it can be attended once only
    partly |= n_part > 0;
    if (ok) dst[count + __popc(m & ((1u << lane) - 1))] = page(c);
    count += __popc(m);
  }
  if (lane == 0) {
    if (partly) dst[count] = page(full);
    p.lens[t] = count * p.block_size + (partly ? part : 0);
  }
  errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
  if (lane == 0 && errbits) set_device_error(p.err, errbits);
}

}  // namespace

cudaError_t launch_index_insert(int bf16, const IndexInsertParams& p, cudaStream_t stream) {
  const dim3 grid(p.T, (p.Hi + 1 + 8 * kInsVec - 1) / (8 * kInsVec));
  if (bf16)
    mla_index_insert_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    mla_index_insert_kernel<false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_index_gather(int bf16, const IndexGatherParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.num_tokens + 7) / 8);
  if (bf16)
    mla_index_gather_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    mla_index_gather_kernel<false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_index_select(const IndexSelectParams& p, int sms, cudaStream_t stream) {
  (void)sms;
  mla_index_select_kernel<<<p.T, kSelThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_page_list(const PageListParams& p, cudaStream_t stream) {
  mla_page_list_kernel<<<(p.T + 3) / 4, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
