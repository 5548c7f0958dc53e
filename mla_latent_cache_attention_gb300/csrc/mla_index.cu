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
// Selection.  A score becomes a 32-bit key whose unsigned order is the scores'; all ones is a forced
// block, and -inf and NaN, which are never taken, have none.  Every score is read once: a CTA streams
// its row (or its part of it) in index order and keeps those above the topk-th largest so far in a
// list in shared memory.  An equal score later in the row has the higher index and loses the tie, so
// "above" is enough.  When a chunk might not fit, the list is cut to its exact topk, which raises the
// bound; of n scores in random order about topk (1 + ln(n / topk)) enter the list, and an ascending
// row, the worst one, only costs more cuts.  The list keeps the row's order, so it comes out
// ascending, and no result depends on the order of atomics.
//
// The cut finds the topk-th largest key from histograms of 2048 bins that divide the keys' own
// range evenly: bins by leading bits would put scores of similar size into a few of them.
//
// Long rows in small batches are shared by a cluster: every CTA takes a part, the histograms of the
// last cut are summed over the cluster, and every CTA writes its part's share.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelPer = 8;                               // scores a thread takes from a chunk
constexpr int kSelChunk = kSelThreads * kSelPer;
constexpr int kSelBins = 2048;
constexpr int kSelFixed = kSelBins * 4 + 512;
constexpr uint32_t kForced = 0xFFFFFFFFu;

// Shared memory of a row with topk: the list (topk + a chunk), a copy of topk entries for the cut.
__host__ __device__ constexpr int64_t select_smem(int64_t topk) { return kSelFixed + (2 * topk + kSelChunk) * 8; }

__device__ __forceinline__ uint32_t score_key(float f) {        // f neither NaN nor -inf
  const uint32_t u = __float_as_uint(f + 0.f);                  // -0 and +0 are equal
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

struct SelShared {
  uint32_t* hist;          // [kSelBins]
  uint32_t* wsum;          // [2][kSelWarps]
  uint32_t* stat;          // [4] smallest key, largest key, count of this CTA's list; spare
  uint32_t* found;         // [4] bin, keys above it, keys in it
};

// The value at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(p, rank)) : "memory");
  return v;
}

// Keys above *thr are the list's k largest unforced ones, together with the first *ties that equal
// it.  With ranks > 1 the list is that of all CTAs of the cluster.
__device__ void find_threshold(const uint32_t* keys, int m, uint32_t k, int ranks, const SelShared& s, uint32_t* thr,
                               uint32_t* ties) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t lo = kForced, hi = 0, n = 0;
  for (int i = tid; i < m; i += kSelThreads) {
    const uint32_t key = keys[i];
    if (key != kForced) {
      lo = min(lo, key);
      hi = max(hi, key);
      ++n;
    }
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  if (tid == 0) s.stat[0] = kForced, s.stat[1] = 0, s.stat[2] = 0;
  __syncthreads();
  if (lane == 0) {
    atomicMin(&s.stat[0], lo);
    atomicMax(&s.stat[1], hi);
    atomicAdd(&s.stat[2], n);
  }
  __syncthreads();
  if (ranks == 1) {
    lo = s.stat[0], hi = s.stat[1], n = s.stat[2];
  } else {
    cluster_sync();
    lo = kForced, hi = 0, n = 0;
    for (int r = 0; r < ranks; ++r) {
      lo = min(lo, ld_cluster_u32(&s.stat[0], r));
      hi = max(hi, ld_cluster_u32(&s.stat[1], r));
      n += ld_cluster_u32(&s.stat[2], r);
    }
  }
  *ties = 0;
  if (n <= k) {
    *thr = 0;
    if (ranks > 1) cluster_sync();      // the others have read stat
    return;
  }
  uint32_t left = k, range = hi - lo;
  if (k == 0) {
    *thr = hi;
    if (ranks > 1) cluster_sync();
    return;
  }
  for (;;) {
    const int bits = 32 - __clz(range), shift = bits > 11 ? bits - 11 : 0;
    reinterpret_cast<uint4*>(s.hist)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t d = keys[i] - lo;
      if (keys[i] >= lo && d <= range && keys[i] != kForced) atomicAdd(&s.hist[d >> shift], 1u);
    }
    __syncthreads();
    // counts from the top: thread q has bins 2047 - 4 q .. 2044 - 4 q
    uint4 c = make_uint4(0, 0, 0, 0);
    if (ranks == 1) {
      c = reinterpret_cast<const uint4*>(s.hist)[kSelThreads - 1 - tid];
    } else {
      cluster_sync();
      for (int r = 0; r < ranks; ++r) {
        const uint4 v = ld_cluster_v4(mapa_shared(s.hist + 4 * (kSelThreads - 1 - tid), r));
        c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
      }
    }
    const uint32_t own = c.x + c.y + c.z + c.w;
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s.wsum[warp] = inc;
    __syncthreads();
    uint32_t before = inc - own;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
      if (w < warp) before += s.wsum[w];
    if (before < left && left <= before + own) {       // exactly one thread
      uint32_t bin = kSelBins - 1 - 4 * tid, cnt = c.w;
      if (left > before + cnt) before += cnt, --bin, cnt = c.z;
      if (left > before + cnt) before += cnt, --bin, cnt = c.y;
      if (left > before + cnt) before += cnt, --bin, cnt = c.x;
      s.found[0] = bin;
      s.found[1] = before;
      s.found[2] = cnt;
    }
    __syncthreads();
    if (ranks > 1) cluster_sync();      // the others have read hist (and stat)
    left -= s.found[1];
    lo += s.found[0] << shift;
    if (s.found[2] == left) {           // the whole bin is taken
      *thr = lo - 1;
      return;
    }
    if (shift == 0) {
      *thr = lo;
      *ties = left;
      return;
    }
    range = (1u << shift) - 1;
  }
}

// In list order: put(position, entry) for every taken entry, positions from (g0 larger, e0 equal) on;
// returns the list's own counts (larger | equal << 16).
template <class Put>
__device__ __forceinline__ uint32_t take_in_order(const uint32_t* keys, int m, uint32_t thr, uint32_t ties, uint32_t* wsum,
                                                  uint32_t g0, uint32_t e0, bool count_only, Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = ((m + kSelWarps - 1) / kSelWarps + 31) & ~31, from = warp * span, to = min(m, from + span);
  uint32_t cnt = 0;
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < to ? keys[i] : 0u;
    cnt += __popc(__ballot_sync(0xFFFFFFFFu, i < to && key > thr)) | (__popc(__ballot_sync(0xFFFFFFFFu, i < to && key == thr)) << 16);
  }
  if (lane == 0) wsum[warp] = cnt;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t v = wsum[w];
    if (w < warp) before += v;
    all += v;
  }
  if (!count_only) {
    uint32_t g = g0 + (before & 0xFFFFu), e = e0 + (before >> 16);
    const uint32_t lt = (1u << lane) - 1;
    for (int i0 = from; i0 < to; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t key = i < to ? keys[i] : 0u;
      const bool gt = i < to && key > thr, eq = i < to && key == thr;
      const uint32_t bg = __ballot_sync(0xFFFFFFFFu, gt), be = __ballot_sync(0xFFFFFFFFu, eq);
      const uint32_t eb = e + __popc(be & lt);
      if (gt || (eq && eb < ties)) put(static_cast<int>(g + __popc(bg & lt) + min(eb, ties)), i);
      g += __popc(bg);
      e += __popc(be);
    }
  }
  __syncthreads();
  return all;
}

__global__ void __launch_bounds__(kSelThreads, 3) mla_index_select_kernel(const IndexSelectParams p, int ranks) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  SelShared s;
  s.hist = sel_smem;
  s.wsum = s.hist + kSelBins;
  s.stat = s.wsum + 2 * kSelWarps;
  s.found = s.stat + 4;
  int64_t* srow = reinterpret_cast<int64_t*>(s.found + 4);       // [2]
  uint32_t* keys = sel_smem + kSelFixed / 4;
  uint32_t* idx = keys + p.topk + kSelChunk;
  uint32_t* copy = idx + p.topk + kSelChunk;                     // [2][topk]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  if (tid == 0) {
    int64_t vis = 0;
    srow[0] = row_request(p.cu_q, p.seq_lens, p.B, t, &vis);
    srow[1] = vis;
  }
  __syncthreads();
  const int b = static_cast<int>(srow[0]);
  const int64_t vis = srow[1];
  if (b < 0) return;       // every CTA of the cluster
  const float* __restrict__ x = p.scores + t * p.s_stride;
  const int n = static_cast<int>(min((vis + p.block_tokens - 1) / p.block_tokens, p.width));
  const int f_lo = min(p.first, n), f_hi = max(f_lo, n - p.last);      // forced: below f_lo, from f_hi on
  const uint32_t kk = p.topk - (f_lo + n - f_hi);                // places of the others
  const int part = ((n + ranks - 1) / ranks + 3) & ~3;
  const int from = min(n, rank * part), to = min(n, from + part);
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;

  // ---- stream: a warp takes 32 * kSelPer neighbouring scores of a chunk, 4 a lane and load
  float cur[kSelPer], nxt[kSelPer];
  auto load = [&](int c0, float (&v)[kSelPer]) {
#pragma unroll
    for (int j = 0; j < kSelPer / 4; ++j) {
      const int i = c0 + warp * 32 * kSelPer + j * 128 + 4 * lane;
      if (vec && i + 3 < to) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(x + i));
        v[4 * j] = w.x, v[4 * j + 1] = w.y, v[4 * j + 2] = w.z, v[4 * j + 3] = w.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] = i + e < to ? __ldg(x + i + e) : CUDART_NAN_F;
      }
    }
  };
  int m = 0, flip = 0;
  float bound = -CUDART_INF_F;
  load(from, cur);
  for (int c0 = from; c0 < to; c0 += kSelChunk) {
    load(c0 + kSelChunk, nxt);
    const bool forced_here = c0 < f_lo || c0 + kSelChunk > f_hi;
    for (;;) {
      // scores above the bound; NaN is not, and -inf is above nothing
      uint32_t take = 0;
#pragma unroll
      for (int j = 0; j < kSelPer; ++j) take |= (cur[j] > bound ? 1u : 0u) << j;
      if (forced_here) {
#pragma unroll
        for (int j = 0; j < kSelPer; ++j) {
          const int i = c0 + warp * 32 * kSelPer + (j >> 2) * 128 + 4 * lane + (j & 3);
          if (i < to && (i < f_lo || i >= f_hi)) take |= 1u << j;
        }
      }
      // ranks in row order: load by load, lane by lane, then the lane's four
      uint32_t at[kSelPer / 4], cnt = 0;
#pragma unroll
      for (int j = 0; j < kSelPer / 4; ++j) {
        const uint32_t mine = (take >> (4 * j)) & 15u;
        uint32_t inc = __popc(mine);
        if (__any_sync(0xFFFFFFFFu, inc)) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
          }
          at[j] = cnt + inc - __popc(mine);
          cnt += __shfl_sync(0xFFFFFFFFu, inc, 31);
        } else {
          at[j] = cnt;
        }
      }
      uint32_t* ws = s.wsum + flip * kSelWarps;
      flip ^= 1;
      if (lane == 0) ws[warp] = cnt;
      __syncthreads();
      uint32_t before = m, all = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) {
        const uint32_t v = ws[w];
        if (w < warp) before += v;
        all += v;
      }
      if (m + static_cast<int>(all) <= p.topk + kSelChunk) {
#pragma unroll
        for (int j = 0; j < kSelPer; ++j) {
          if (!((take >> j) & 1u)) continue;
          const int i = c0 + warp * 32 * kSelPer + (j >> 2) * 128 + 4 * lane + (j & 3);
          const uint32_t pos = before + at[j >> 2] + __popc((take >> (4 * (j >> 2))) & ((1u << (j & 3)) - 1));
          keys[pos] = i < f_lo || i >= f_hi ? kForced : score_key(cur[j]);
          idx[pos] = i;
        }
        m += all;
        break;
      }
      // cut the list to its topk, then take the chunk again
      __syncthreads();
      uint32_t thr, ties;
      find_threshold(keys, m, kk, 1, s, &thr, &ties);
      const uint32_t got = take_in_order(keys, m, thr, ties, s.wsum, 0, 0, false, [&](int pos, int i) {
        copy[pos] = keys[i];
        copy[p.topk + pos] = idx[i];
      });
      m = static_cast<int>((got & 0xFFFFu) + min(got >> 16, ties));
      for (int i = tid; i < m; i += kSelThreads) {
        keys[i] = copy[i];
        idx[i] = copy[p.topk + i];
      }
      // everything kept equals the bound or is above it (thr itself when ties were cut, else the next
      // key): a later score has to be above thr
      bound = thr == 0 ? bound : kk == 0 ? CUDART_INF_F : key_score(thr);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) cur[j] = nxt[j];
  }
  __syncthreads();

  // ---- the last cut, over the row
  uint32_t thr, ties;
  find_threshold(keys, m, kk, ranks, s, &thr, &ties);
  int32_t* out = p.blocks + t * p.b_stride;
  int32_t* out_slots = p.slots ? p.slots + t * p.sl_stride : nullptr;
  const bool one = p.block_tokens == 1;
  auto slot_of = [&](int64_t pos) -> int32_t {
    if (pos >= vis) return -1;
    const int64_t col = pos / p.page_size;
    const int64_t id = col < p.bt_cols ? p.block_table[b * p.bt_stride + col] : -1;
    if (id < 0 || id >= p.num_blocks) {
      set_device_error(p.err, 2u);
      return -1;
    }
    return static_cast<int32_t>(id * p.page_size + pos % p.page_size);
  };
  uint32_t g0 = 0, e0 = 0, g_all = 0, e_all = 0;
  auto put = [&](int pos, int i) {
    const int32_t c = static_cast<int32_t>(idx[i]);
    out[pos] = c;
    if (out_slots && one) out_slots[pos] = slot_of(c);
    if (out_slots && !one)
      for (int u = 0; u < p.block_tokens; ++u)
        out_slots[static_cast<int64_t>(pos) * p.block_tokens + u] = slot_of(static_cast<int64_t>(c) * p.block_tokens + u);
  };
  if (ranks > 1) {
    const uint32_t mine = take_in_order(keys, m, thr, ties, s.wsum, 0, 0, true, put);
    if (tid == 0) s.stat[3] = mine;
    cluster_sync();
    for (int r = 0; r < ranks; ++r) {
      const uint32_t v = ld_cluster_u32(&s.stat[3], r);
      if (r < rank) g0 += v & 0xFFFFu, e0 += v >> 16;
      g_all += v & 0xFFFFu, e_all += v >> 16;
    }
    cluster_sync();       // no CTA leaves while another may read its counts
    take_in_order(keys, m, thr, ties, s.wsum, g0, e0, false, put);
  } else {
    const uint32_t v = take_in_order(keys, m, thr, ties, s.wsum, 0, 0, false, put);
    g_all = v & 0xFFFFu, e_all = v >> 16;
  }
  // ---- -1 after the list
  const int taken = static_cast<int>(g_all + min(e_all, ties));
  for (int i = taken + rank * kSelThreads + tid; i < p.topk; i += ranks * kSelThreads) out[i] = -1;
  if (out_slots) {
    const int64_t all = static_cast<int64_t>(p.topk) * p.block_tokens;
    for (int64_t i = static_cast<int64_t>(taken) * p.block_tokens + rank * kSelThreads + tid; i < all; i += ranks * kSelThreads)
      out_slots[i] = -1;
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

static_assert(select_smem(kSelectMaxTopk) <= 227 * 1024, "shared memory budget");

cudaError_t launch_index_select(const IndexSelectParams& p, int sms, cudaStream_t stream) {
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mla_index_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  // CTAs that share a row: while the batch leaves SMs idle and a part keeps two chunks
  int ranks = 1;
  while (ranks < 8 && static_cast<int64_t>(p.T) * ranks * 2 <= 2 * sms && p.width / (ranks * 2) >= 2 * kSelChunk) ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T) * ranks);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(select_smem(p.topk));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_index_select_kernel, p, ranks);
}

cudaError_t launch_page_list(const PageListParams& p, cudaStream_t stream) {
  mla_page_list_kernel<<<(p.T + 3) / 4, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
