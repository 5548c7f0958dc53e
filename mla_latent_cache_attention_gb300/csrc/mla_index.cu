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

#include <cmath>

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

// 8 consecutive bf16 values, as stored and as fp32
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* __restrict__ src, bool vec) {
  if (vec) return __ldcs(reinterpret_cast<const uint4*>(src));      // read once
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __ldg(src + 2 * i) | static_cast<uint32_t>(__ldg(src + 2 * i + 1)) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void bf16x8_values(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
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
// it, and it has kVec vectors' loads in flight.  The first CTA of a token also inserts its key.
// Measured: 8191 tokens of 64 heads (211 MB) 41.6 us, 5.1 TB/s, issuing 71 % of the time; the stores are marked
// as streaming (42.9 us without).
// The rotated half of a vector: lane l >= 8 holds pairs 4 (l - 8) .. 4 (l - 8) + 3.
__device__ __forceinline__ void rotate_vector(float (&x)[8], const float4 c4, const float4 s4, bool on) {
  if (!on) return;
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = __fmaf_rn(a, c[i], -__fmul_rn(b, s[i]));
    x[2 * i + 1] = __fmaf_rn(b, c[i], __fmul_rn(a, s[i]));
  }
}

// Scale exponent and codes of a half-warp's vector.
__device__ __forceinline__ uint2 quantise_vector(const float (&x)[8], uint32_t half, float& scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half, amax, m));
  const int k = scale_exponent(amax);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);      // 2^-k, exact
  scale = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = static_cast<uint32_t>(
        __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3));
    c[i >> 1] |= two << (16 * (i & 1));
  }
  return make_uint2(c[0], c[1]);
}

template <bool kBf16, int kVec>
__global__ void __launch_bounds__(128) mla_index_insert_kernel(const IndexInsertParams p) {
  // a kernel launched next as a programmatic dependent may be scheduled now
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15, d0 = 8 * l;
  const int v0 = blockIdx.y * 8 * kVec + hw;      // vectors v0, v0 + 8, ...
  const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
  const bool keyed = blockIdx.y == 0 && hw == 7;
  const int64_t slot = keyed ? p.slot_mapping[t] : -1;
  const float* cs = nullptr;
  if (p.positions) {
    int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) {
      if (l == 0 && keyed) set_device_error(p.err, 8u);
      pos = pos < 0 ? 0 : p.max_position - 1;
    }
    cs = p.cos_sin + pos * 64 + 4 * (l & 7);
  }
  uint4 raw[kVec];
  const uint16_t* q = p.q + t * p.q_s0 + d0;
#pragma unroll
  for (int u = 0; u < kVec; ++u)
    if (v0 + 8 * u < p.Hi) raw[u] = load_bf16x8(q + (v0 + 8 * u) * p.q_s1, p.vec != 0);
  uint4 raw_k = make_uint4(0, 0, 0, 0);
  if (keyed) raw_k = load_bf16x8(p.k + t * p.k_s0 + d0, p.vec != 0);
  float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
  if (cs) c = __ldg(reinterpret_cast<const float4*>(cs)), s = __ldg(reinterpret_cast<const float4*>(cs + 32));
  float w[kVec];
  if (l == 0)
#pragma unroll
    for (int u = 0; u < kVec; ++u)
      if (v0 + 8 * u < p.Hi) w[u] = __ldg(p.w + t * p.w_s0 + v0 + 8 * u);
#pragma unroll
  for (int u = 0; u < kVec; ++u) {
    const int v = v0 + 8 * u;
    if (v >= p.Hi) break;
    float x[8];
    bf16x8_values(raw[u], x);
    rotate_vector(x, c, s, cs && l >= 8);
    const int64_t o = (t * p.Hi + v) * kIndexDim + d0;
    if (kBf16) {
      __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + o), pack_bf16x8(x));
      if (l == 0) p.w_out[t * p.Hi + v] = w[u] * p.weight_scale;
    } else {
      float sc;
      __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q_out) + o), quantise_vector(x, half, sc));
      if (l == 0) p.w_out[t * p.Hi + v] = w[u] * p.weight_scale * sc;
    }
  }
  if (!keyed || slot < 0) return;
  const int64_t blk = slot / p.block_size, off = slot - blk * p.block_size;
  if (blk >= p.num_blocks) {
    if (l == 0) set_device_error(p.err, 4u);
    return;
  }
  uint8_t* ent = p.cache + blk * p.block_stride + off * p.entry_stride;
  float k[8];
  bf16x8_values(raw_k, k);
  rotate_vector(k, c, s, cs && l >= 8);
  if (kBf16) {
    *reinterpret_cast<uint4*>(ent + 2 * d0) = pack_bf16x8(k);
  } else {
    float sc;
    *reinterpret_cast<uint2*>(ent + d0) = quantise_vector(k, half, sc);
    if (l == 0) p.scales[blk * p.sc_stride + off] = sc;
  }
}

// ------------------------------------------------------------------------------------------
// Gather: row r of request b (cu[b] <= r < cu[b+1]) is position starts[b] + r - cu[b], as
// bf16(code * scale).  A warp takes kRows neighbouring rows at a time: each lane finds one row's key (the
// search over cu, the page, the scale: five dependent loads), then half-warps write the 256-byte rows, 8
// values a lane, with those addresses.  The next rows' keys are found while this step's values are on
// their way (without that 512000 rows took 42 us instead of 35).  Stores are marked as streaming: 242000 rows 21.3
// -> 18.1 us.  Measured past L2: 256000 keys of 8 requests (100 MB) 16.5 us, 6.0 TB/s, where a row by a half-warp
// that finds it itself took 34 us.
template <bool kBf16, int kRows>
__global__ void __launch_bounds__(128) mla_index_gather_kernel(const IndexGatherParams p) {
  const int lane = threadIdx.x & 31, d0 = 8 * (lane & 15);
  const int64_t end = min(p.num_tokens, static_cast<int64_t>(p.cu[p.batch])), first = p.cu[0];
  const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * kRows;
  // lane u < kRows: the key and scale of row r0 + u (no key: zeros)
  auto lookup = [&](int64_t r0, const uint8_t*& ent, float& scale) {
    ent = nullptr;
    scale = 0.f;
    const int64_t r = r0 + lane;
    if (lane >= kRows || r >= end || r < first) return;
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const int64_t pos = static_cast<int64_t>(p.starts ? p.starts[lo] : 0) + (r - p.cu[lo]);
    const int64_t col = pos >= 0 ? static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.block_size) : -1;      // below 2^32
    const int64_t blk = col >= 0 && col < p.bt_cols ? p.block_table[lo * p.bt_stride + col] : -1;
    if (blk < 0 || blk >= p.num_blocks) {
      set_device_error(p.err, 2u);
    } else {
      const int64_t off = pos - col * p.block_size;
      ent = p.cache + blk * p.block_stride + off * p.entry_stride;
      if (!kBf16) scale = __ldg(p.scales + blk * p.sc_stride + off);
    }
  };
  int64_t r0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)) * kRows;
  const uint8_t* ent;
  float scale;
  lookup(r0, ent, scale);
  for (; r0 < end; r0 += step) {
    uint4 raw[kRows / 2];
    float s[kRows / 2];
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const int src = 2 * i + (lane >> 4);
      const uint8_t* e = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(ent), src));
      s[i] = __shfl_sync(0xFFFFFFFFu, scale, src);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (kBf16) {
        if (e) raw[i] = __ldg(reinterpret_cast<const uint4*>(e + 2 * d0));
      } else if (e) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(e + d0));
        raw[i].x = c.x, raw[i].y = c.y;
      }
    }
    if (r0 + step < end) lookup(r0 + step, ent, scale);       // while the keys are on their way
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const int64_t r = r0 + 2 * i + (lane >> 4);
      if (r >= end || r < first) continue;
      uint4 y = raw[i];
      if (!kBf16) {
        const uint32_t w[2] = {y.x, y.y};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));      // exact
          x[2 * j] = f.x * s[i];
          x[2 * j + 1] = f.y * s[i];
        }
        y = pack_bf16x8(x);
      }
      uint16_t* dst = p.dst + r * p.dst_row + d0;
      if (p.vec) {
        __stcs(reinterpret_cast<uint4*>(dst), y);
      } else {
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// Selection.  A score becomes a 32-bit key whose unsigned order is the scores'.  A row is streamed
// once: a bound, taken from 4096 scores spread over the row so that it almost surely lies a little
// below the topk-th largest, lets some topk (1 + a few standard deviations of the sample's rank) of
// them into a list in shared memory.  The exact cut is made in the list.  Its scores are counted in bins
// that divide the range above the bound evenly; the bin of the topk-th holds a few of them, which are
// ranked directly, an equal score with a lower index before.  Where no bound was taken (a short row) or a
// bin holds many (equal scores), the cut is the topk-th largest key, from histograms of 2048 bins that
// divide the keys' own range evenly (bins by leading bits would put scores of similar size into a few of
// them), and among keys that equal it the lowest indices, by the same search over the indices.  The
// taken indices then become bits of a map of the row, whose prefix counts give their ascending
// positions.  No result depends on the order of atomics.
//
// Where the bound lets in too few or too many, the row is streamed once more with the sample's rank that the
// count now gives for the middle of the list's room: a row whose neighbours resemble one another misses its
// place more often than its sample's size says (1024 rows of 65536 scores, without this: a moving mean of 32
// 149 instead of 97 us, blocks of 16 equal ones and a little noise 162 instead of 105).  Where that does not
// help (equal scores, a row that repeats with the sample's stride) it is streamed in order, and whenever the
// list is full it is cut to its exact topk, which raises the bound; a later equal score has the higher index,
// so "above the bound" is enough.
//
// Long rows in small batches are shared by a cluster: every CTA streams a part and keeps a list of its
// own; the counts are summed over the cluster, and the few keys in the bin of the cut are read by all.
// (Before, every CTA read the others' lists and cut the whole: 20.3 -> 17.0 us for the 32 rows below.)
//
// Measured (GB300): 4096 rows of up to 65536 scores, topk 2048: 271 us, 4.0 TB/s (1.07 GB read once;
// a row's sample waits for its 512 sectors behind the other rows' streams), 313 us with their slots (divisions and
// two dependent loads for each of 8 million);
// 32 rows of up to 131072 with their slots: 17 us; 128 rows of up to 512 blocks, topk 32: 7.7 us.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelSample = 4096;
constexpr int kSelChunk = 2048;                          // scores of an ordered round
constexpr int kSelBins = 2048;
constexpr int kSelNear = 128;                            // keys of the cut's bin that are ranked directly
constexpr int kSelFixed = kSelBins * 4 + kSelNear * 8 + 512;

// Entries of the list: topk and room beyond it, for an ordered round or for what the bound lets in: the
// score of rank rho = r + 6 sqrt(r) + 8 of a sample of 4096, r = topk 4096 / n, lets in n / 4096 times
// rho +- sqrt(rho) of n; six of those are kept (with 3.5, one of 4096 rows overflowed, and its ordered
// pass took 40 us longer than the others).  What shared memory leaves of an SM is L1, and loads in flight
// take place there: with 25 KB a row more the same kernel took 352 us instead of 290 us for 4096 rows of 65536.
inline int select_capacity(int64_t topk, int64_t width) {
  const double per = static_cast<double>(width) / kSelSample, r = topk / per;
  const double rho = r + 6.0 * sqrt(r) + 8.0, most = (200 * 1024 - kSelFixed) / 8.0 - topk;
  const double want = per * (rho + 6.0 * sqrt(rho)) - topk, room = want < most ? want : most;
  return static_cast<int>(topk + (room > kSelChunk ? room : kSelChunk));
}

__device__ __forceinline__ uint32_t score_key(float f) {        // f neither NaN nor -inf: at least 0x00800000
  const uint32_t u = __float_as_uint(f + 0.f);                  // -0 and +0 are equal
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kForcedKey = 0xFFFFFFFFu;

struct SelShared {
  uint32_t hist[kSelBins];        // histogram, or the map of 65536 indices
  uint32_t wsum[32];              // totals of the warps; the last keys of a cut
  uint32_t stat[4];               // smallest key, largest key, their number, entries taken
  uint32_t found[4];              // bin, keys above it, keys in it
  uint32_t count;                 // entries of the list
  float again, tried;             // factor of the sample's rank (1 at first), the bound before
  uint32_t nears;                 // entries of near
  int64_t row[2];                 // request and visible keys
  uint2 near[kSelNear];           // this CTA's (key, index) in the bin of the cut
};
static_assert(sizeof(SelShared) <= kSelFixed, "shared memory layout");

// The value at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld_cluster_v2(uint32_t cluster_addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_addr) : "memory");
  return v;
}

// Every CTA's value at p: lane r has that of CTA r of the cluster (0 from `ranks` on).
__device__ __forceinline__ uint32_t ld_ranks(const uint32_t* p, int ranks) {
  const int lane = threadIdx.x & 31;
  return lane < ranks ? ld_cluster_u32(p, lane) : 0u;
}

// Exclusive prefix of `own` over the threads of the CTA (two barriers).
__device__ __forceinline__ uint32_t block_prefix(uint32_t own, uint32_t* wsum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  uint32_t w = lane < warp ? wsum[lane & (kSelWarps - 1)] : 0u;       // warp <= 15
  w = __reduce_add_sync(0xFFFFFFFFu, w);
  __syncthreads();
  return w + inc - own;
}

struct Cut {
  uint32_t thr, ties;      // keys above thr, and `ties` of those that equal it
};

// The k largest of the keys val(0) .. val(m - 1) (0: none); with ranks > 1 of all CTAs' together.
template <class Val>
__device__ Cut find_cut(int m, uint32_t k, int ranks, SelShared& s, Val val) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t lo = 0xFFFFFFFFu, hi = 0, n = 0;
  for (int i = tid; i < m; i += kSelThreads) {
    const uint32_t key = val(i);
    if (key) {
      lo = min(lo, key);
      hi = max(hi, key);
      ++n;
    }
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  __syncthreads();
  if (tid == 0) s.stat[0] = 0xFFFFFFFFu, s.stat[1] = 0, s.stat[2] = 0;
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
    lo = 0xFFFFFFFFu, hi = 0, n = 0;
    for (int r = 0; r < ranks; ++r) {
      lo = min(lo, ld_cluster_u32(&s.stat[0], r));
      hi = max(hi, ld_cluster_u32(&s.stat[1], r));
      n += ld_cluster_u32(&s.stat[2], r);
    }
    cluster_sync();      // every CTA has read the others'
  }
  if (n <= k) return Cut{0u, 0u};
  if (k == 0) return Cut{hi, 0u};
  uint32_t left = k, range = hi - lo;
  for (;;) {
    const int bits = 32 - __clz(range), shift = bits > 11 ? bits - 11 : 0;
    reinterpret_cast<uint4*>(s.hist)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t key = val(i);
      if (key >= lo && key - lo <= range) atomicAdd(&s.hist[(key - lo) >> shift], 1u);
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
    uint32_t before = block_prefix(own, s.wsum);
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
    if (ranks > 1) cluster_sync();      // every CTA has read the others' histogram
    left -= s.found[1];
    lo += s.found[0] << shift;
    if (s.found[2] == left) return Cut{lo - 1, 0u};       // the whole bin
    if (shift == 0) return Cut{lo, left};
    range = (1u << shift) - 1;
    const bool few = ranks == 1 && s.found[2] <= 32;
    __syncthreads();                    // found has been read
    if (few) {                          // a warp ranks the bin's keys
      if (tid == 0) s.found[3] = 0;
      __syncthreads();
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t key = val(i);
        if (key >= lo && key - lo <= range) s.wsum[atomicAdd(&s.found[3], 1u)] = key;
      }
      __syncthreads();
      if (tid < 32) {
        const int cnt = static_cast<int>(s.found[3]);
        const uint32_t key = lane < cnt ? s.wsum[lane] : 0u;
        uint32_t above = 0, same = 0;
        for (int i = 0; i < cnt; ++i) {
          const uint32_t o = __shfl_sync(0xFFFFFFFFu, key, i);
          above += o > key ? 1u : 0u;
          same += o == key ? 1u : 0u;
        }
        if (lane < cnt && above < left && left <= above + same) {      // every lane that holds the key agrees
          s.found[0] = left == above + same ? key - 1 : key;
          s.found[1] = left == above + same ? 0u : left - above;
        }
      }
      __syncthreads();
      return Cut{s.found[0], s.found[1]};
    }
  }
}

// Bins of the scores that a bound lets in: evenly from the bound on, the last one for what lies past it.
// Scores in order are in bins in order, whatever the roundings.
struct Bins {
  float from, scale;          // scale 0: not counted
  __device__ __forceinline__ uint32_t of(float v) const {
    return min(static_cast<uint32_t>(__float2int_rz((v - from) * scale)), static_cast<uint32_t>(kSelBins - 1));
  }
};

// Adds the entries of a warp's `take` bits (bit j: index i0 + 128 (j / 4) + 4 lane + j % 4 of x)
// to the list; those past its end are dropped, which the count shows.
__device__ __forceinline__ void append(uint2* list, uint32_t cap, uint32_t* count, uint32_t take, const float* __restrict__ x,
                                       int i0, bool as_key, int f_lo, int f_hi) {
  if (!__any_sync(0xFFFFFFFFu, take)) return;
  const int lane = threadIdx.x & 31;
  const uint32_t mine = __popc(take);
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t w = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += w;
  }
  uint32_t base = 0;
  if (lane == 31) base = atomicAdd(count, inc);
  base = __shfl_sync(0xFFFFFFFFu, base, 31);
  uint32_t pos = base + inc - mine;
  // few are taken: their values are read again (from L1) instead of picked out of registers
  while (__any_sync(0xFFFFFFFFu, take)) {
    if (take) {
      const int j = __ffs(take) - 1, i = i0 + (j >> 2) * 128 + 4 * lane + (j & 3);
      take &= take - 1;
      const float v = __ldg(x + i);
      uint32_t bits = __float_as_uint(v);
      if (as_key) bits = i < f_lo || i >= f_hi ? kForcedKey : score_key(v);
      if (pos < cap) list[pos] = make_uint2(bits, static_cast<uint32_t>(i));
      ++pos;
    }
  }
}

// Four of the sample's scores: half g % 2 of one of 512 groups of eight neighbours (a sector) spread over the n.
__device__ __forceinline__ int sample_at(int g, int n) { return (static_cast<int>((static_cast<int64_t>(g >> 1) * n) >> 9) & ~7) + 4 * (g & 1); }

__device__ __forceinline__ int select_blocks_of(const IndexSelectParams& p, int64_t vis) {
  return static_cast<int>(min((vis + p.block_tokens - 1) / p.block_tokens, p.width));
}

// A lane's four scores at i .. i + 3 of x; NaN from `to` on.
__device__ __forceinline__ void load_scores(const float* __restrict__ x, bool vec, int i, int to, float* v) {
  if (vec && i + 3 < to) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(x + i));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < to ? __ldg(x + i + e) : CUDART_NAN_F;
  }
}

// Bits of a warp's scores at i0 + 128 (j / 4) + 4 lane + j % 4 that are forced.
__device__ __forceinline__ uint32_t forced_bits(int i0, int loads, int to, int f_lo, int f_hi) {
  uint32_t f = 0;
  for (int j = 0; j < 4 * loads; ++j) {
    const int i = i0 + (j >> 2) * 128 + 4 * (threadIdx.x & 31) + (j & 3);
    if (i < to && (i < f_lo || i >= f_hi)) f |= 1u << j;
  }
  return f;
}

// The list of a part in the ordered way: rounds in index order, the list cut to its kk largest whenever it
// is full.  Returns its length.  Out of line, so that the usual way keeps its registers.
__device__ __noinline__ int ordered_list(const float* __restrict__ x, bool vec, int from, int to, int f_lo, int f_hi, uint32_t kk,
                                         uint32_t cap, SelShared& s, uint2* list) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int m = 0;
  float bound = -CUDART_INF_F;
  for (int c0 = from; c0 < to; c0 += kSelChunk) {
    const int i0 = c0 + warp * 128;
    float v[4];
    load_scores(x, vec, i0 + 4 * lane, to, v);
    for (;;) {
      if (tid == 0) s.count = m;
      __syncthreads();
      uint32_t take = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) take |= (v[j] > bound ? 1u : 0u) << j;
      if (i0 < f_lo || i0 + 128 > f_hi) take |= forced_bits(i0, 1, to, f_lo, f_hi);
      append(list, cap, &s.count, take, x, i0, true, f_lo, f_hi);
      __syncthreads();
      const int now = static_cast<int>(s.count);
      __syncthreads();
      if (now <= static_cast<int>(cap)) {
        m = now;
        break;
      }
      // the list of the rounds before this one, cut; then the round again
      const Cut c = find_cut(m, kk, 1, s, [&](int i) { return list[i].x == kForcedKey ? 0u : list[i].x; });
      uint32_t first = 0;
      if (c.ties) first = find_cut(m, c.ties, 1, s, [&](int i) { return list[i].x == c.thr ? ~list[i].y : 0u; }).thr;
      if (tid == 0) s.count = 0;
      __syncthreads();
      for (int i1 = 0; i1 < m; i1 += kSelThreads) {      // to the front, which has been read
        const uint2 e = i1 + tid < m ? list[i1 + tid] : make_uint2(0u, 0u);
        __syncthreads();
        if (i1 + tid < m && (e.x > c.thr || (c.ties && e.x == c.thr && ~e.y > first))) list[atomicAdd(&s.count, 1u)] = e;
        __syncthreads();
      }
      m = static_cast<int>(s.count);
      if (kk == 0)
        bound = CUDART_INF_F;
      else if (c.thr)
        bound = key_score(c.thr);
      __syncthreads();
    }
  }
  return m;
}

// The cut of the kk largest (kk > 0) from the counts of `bins`: the bin that holds the kk-th, and among its
// keys, where they are few, the one with kk - 1 before it in order (a lower index is before an equal key).
// `at`: those taken before this CTA's part.  False if the bin holds too many.
__device__ __forceinline__ bool cut_of_bins(int m, uint32_t kk, int ranks, SelShared& s, const uint2* list, const Bins bins,
                                            Cut& cut, uint32_t& first, uint32_t& at_out) {
  const int tid = threadIdx.x, lane = tid & 31, rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  uint4 c = make_uint4(0, 0, 0, 0);      // thread q: bins 2047 - 4 q .. 2044 - 4 q
  if (ranks == 1) {
    c = reinterpret_cast<const uint4*>(s.hist)[kSelThreads - 1 - tid];
  } else {
    for (int r = 0; r < ranks; r += 2) {         // two loads under way
      const uint4 v = ld_cluster_v4(mapa_shared(s.hist + 4 * (kSelThreads - 1 - tid), r));
      const uint4 u = ld_cluster_v4(mapa_shared(s.hist + 4 * (kSelThreads - 1 - tid), r + 1));
      c.x += v.x + u.x, c.y += v.y + u.y, c.z += v.z + u.z, c.w += v.w + u.w;
    }
  }
  const uint32_t own = c.x + c.y + c.z + c.w;
  if (tid == 0) s.nears = 0, s.stat[2] = 0, s.stat[3] = 0;
  uint32_t before = block_prefix(own, s.wsum);
  if (before < kk && kk <= before + own) {       // exactly one thread
    uint32_t bin = kSelBins - 1 - 4 * tid, cnt = c.w;
    if (kk > before + cnt) before += cnt, --bin, cnt = c.z;
    if (kk > before + cnt) before += cnt, --bin, cnt = c.y;
    if (kk > before + cnt) before += cnt, --bin, cnt = c.x;
    s.found[0] = bin;
    s.found[1] = before;
    s.found[2] = cnt;
  }
  __syncthreads();
  const uint32_t bin = s.found[0], left = kk - s.found[1], cnt = s.found[2];
  if (cnt > kSelNear) return false;
  uint32_t above = 0;                            // forced, or of a bin above
  for (int i = tid; i < m; i += kSelThreads) {
    const uint2 e = list[i];
    const uint32_t b = e.x == kForcedKey ? static_cast<uint32_t>(kSelBins) : bins.of(key_score(e.x));
    if (b == bin) s.near[atomicAdd(&s.nears, 1u)] = e;
    above += b > bin ? 1u : 0u;
  }
  const uint2* all = s.near;
  uint32_t r = 0;        // the CTA that has entry tid
  if (ranks == 1) {
    __syncthreads();
  } else {
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    if (lane == 0) atomicAdd(&s.stat[3], above);
    cluster_sync();      // the others' keys are there, and they have read this CTA's counts
    all = reinterpret_cast<const uint2*>(s.hist);
    if (tid < kSelNear) {
      const uint32_t n = ld_ranks(&s.nears, ranks);
      uint32_t at = tid;
      bool past = true;                  // entry tid is past the CTAs' so far
      for (int i = 0; i < ranks; ++i) {
        const uint32_t here = __shfl_sync(0xFFFFFFFFu, n, i);
        if (past) r = i;
        past = past && at >= here;
        if (past) at -= here;
      }
      if (!past) reinterpret_cast<uint2*>(s.hist)[tid] = ld_cluster_v2(mapa_shared(s.near + at, r));
    }
    __syncthreads();
  }
  if (tid < static_cast<int>(cnt)) {
    const uint2 e = all[tid];
    uint32_t ahead = 0;
    for (uint32_t i = 0; i < cnt; ++i) {
      const uint2 o = all[i];
      ahead += o.x > e.x || (o.x == e.x && o.y < e.y) ? 1u : 0u;
    }
    if (ahead + 1 == left) s.found[0] = e.x, s.found[1] = e.y;
    if (ahead < left && r < static_cast<uint32_t>(rank)) atomicAdd(&s.stat[2], 1u);
  }
  __syncthreads();
  if (ranks > 1) at_out = s.stat[2] + __reduce_add_sync(0xFFFFFFFFu, lane < rank ? ld_ranks(&s.stat[3], ranks) : 0u);
  cut = Cut{s.found[0], 1u};
  first = ~s.found[1] - 1u;         // indices up to the cut's own
  return true;
}

// The bound of a row of n scores: the one of rank `rank` (1: the largest) in the sample, and the scale of the bins
// from there on (0: none, -1: no bound).  The sample is 512 groups of eight neighbours spread over the row (whole
// sectors: 1024 groups of four waited for twice as many requests, 4096 rows of 65536 took 288 us instead of
// 267), the same in every CTA of the cluster; its histogram divides the scores' range evenly.  Leaves hist
// empty.
__device__ __forceinline__ float2 sample_bound(const float* __restrict__ x, bool vec, int n, uint32_t rank, SelShared& s) {
  const int tid = threadIdx.x, lane = tid & 31;
  float f[8];
  float lo = CUDART_INF_F, hi = -CUDART_INF_F;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = sample_at(tid + j * kSelThreads, n);
    if (vec && i + 3 < n) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(x + i));
      f[4 * j] = w.x, f[4 * j + 1] = w.y, f[4 * j + 2] = w.z, f[4 * j + 3] = w.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * j + e] = i + e < n ? __ldg(x + i + e) : CUDART_NAN_F;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (fabsf(f[j]) < CUDART_INF_F) lo = fminf(lo, f[j]), hi = fmaxf(hi, f[j]);       // finite ones
  // order of floats as integers: the warps' extremes meet in shared memory
  const uint32_t wlo = __reduce_min_sync(0xFFFFFFFFu, score_key(lo)), whi = __reduce_max_sync(0xFFFFFFFFu, score_key(hi));
  if (tid == 0) s.stat[0] = 0xFFFFFFFFu, s.stat[1] = 0, s.stat[2] = 0;
  reinterpret_cast<uint4*>(s.hist)[tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (lane == 0) {
    atomicMin(&s.stat[0], wlo);
    atomicMax(&s.stat[1], whi);
  }
  __syncthreads();
  lo = key_score(s.stat[0]);
  hi = key_score(s.stat[1]);
  const float scale = 2047.f / (hi - lo);
  if (hi > lo && scale > 0.f && scale < CUDART_INF_F) {
    uint32_t inf = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (fabsf(f[j]) < CUDART_INF_F) atomicAdd(&s.hist[static_cast<int>((f[j] - lo) * scale)], 1u);
      inf += f[j] == CUDART_INF_F ? 1u : 0u;
    }
    if (inf) atomicAdd(&s.hist[kSelBins - 1], inf);
    __syncthreads();
    const uint4 c = reinterpret_cast<const uint4*>(s.hist)[kSelThreads - 1 - tid];      // bins 2047 - 4 tid .. 2044 - 4 tid
    const uint32_t own = c.x + c.y + c.z + c.w;
    uint32_t before = block_prefix(own, s.wsum);
    if (before < rank && rank <= before + own) {       // at most one thread
      uint32_t bin = kSelBins - 1 - 4 * tid;
      if (rank > before + c.w) before += c.w, --bin;
      if (bin == kSelBins - 2 - 4 * tid && rank > before + c.z) before += c.z, --bin;
      if (bin == kSelBins - 3 - 4 * tid && rank > before + c.y) --bin;
      s.found[0] = __float_as_uint(lo + static_cast<float>(bin) / scale);
      s.stat[2] = 1;
    }
    __syncthreads();
    reinterpret_cast<uint4*>(s.hist)[tid] = make_uint4(0, 0, 0, 0);
    if (s.stat[2]) {
      const float bound = __uint_as_float(s.found[0]);
      // room above the sample's largest: the row's tail may be as long again
      const float bins = (kSelBins / 2 - 1) / (hi - bound);
      return make_float2(bound, hi > bound && bins > 0.f && bins < CUDART_INF_F ? bins : 0.f);
    }
  }
  return make_float2(0.f, -1.f);
}

// Streams x[from .. to) and lists what the bound lets in (and the forced).  A warp takes 512 neighbouring scores
// at a time, 4 a lane and load; of a row that is let in whole 128, so that a short one is shared by the warps.
__device__ __forceinline__ void let_in(const float* __restrict__ x, bool vec, int from, int to, int f_lo, int f_hi, float bound,
                                    bool strict, uint32_t cap, SelShared& s, uint2* list) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (strict) {
    for (int i0 = from + warp * 128; i0 < to; i0 += kSelWarps * 128) {
      const int i = i0 + 4 * lane;
      float v[4];
      load_scores(x, vec, i, to, v);
      uint32_t take = forced_bits(i0, 1, to, f_lo, f_hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) take |= (v[j] > bound ? 1u : 0u) << j;
      const uint32_t mine = __popc(take);
      uint32_t inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += w;
      }
      uint32_t pos = 0;
      if (lane == 31) pos = atomicAdd(&s.count, inc);
      pos = __shfl_sync(0xFFFFFFFFu, pos, 31) + inc - mine;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (take >> j & 1u) {
          if (pos < cap) list[pos] = make_uint2(__float_as_uint(v[j]), static_cast<uint32_t>(i + j));
          ++pos;
        }
    }
  }
  for (int i0 = strict ? to : from + warp * 512; i0 < to; i0 += kSelWarps * 512) {
    float v[16];
    if (vec && i0 + 512 <= to) {
      const float4* x4 = reinterpret_cast<const float4*>(x + i0) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = __ldg(x4 + 32 * j);
        v[4 * j] = w.x, v[4 * j + 1] = w.y, v[4 * j + 2] = w.z, v[4 * j + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_scores(x, vec, i0 + 128 * j + 4 * lane, to, v + 4 * j);
    }
    uint32_t take = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) take |= (v[j] >= bound ? 1u : 0u) << j;
    if (i0 < f_lo || i0 + 512 > f_hi) take |= forced_bits(i0, 4, to, f_lo, f_hi);
    append(list, cap, &s.count, take, x, i0, false, f_lo, f_hi);
  }
}

// Rank in the sample of a bound that lets in the kk largest of n scores almost surely.
__device__ __forceinline__ float sample_rank(uint32_t kk, int n) {
  const float r = static_cast<float>(kk) * kSelSample / n;
  return r + 6.f * sqrtf(r) + 8.f;
}

// A part's list of what the bound of the sample's rank rho lets in, as keys, counted in `bins`.
struct List {
  int m;               // entries
  uint32_t total;      // of the row, with those that had no place
  bool good;           // all have a place, and they are at least topk or the row's all
  bool strict;         // no bound
  Bins bins;
  float bound;
};

__device__ __forceinline__ List list_of(const float* __restrict__ x, bool vec, int n, int from, int to, int f_lo, int f_hi, float rho,
                                        float tried, int ranks, uint32_t cap, int topk, SelShared& s, uint2* list) {
  const int tid = threadIdx.x;
  List l{0, 0, false, true, Bins{0.f, 0.f}, -CUDART_INF_F};
  float& bound = l.bound;
  if (tid == 0) s.count = 0;
  __syncthreads();
  if (n > static_cast<int>(cap)) {
    const float2 found = sample_bound(x, vec, n, static_cast<uint32_t>(fminf(fmaxf(rho, 1.f), kSelSample - 1.f)), s);
    if (found.y >= 0.f) bound = found.x, l.bins = Bins{found.x, found.y}, l.strict = false;
  }
  if (bound == tried) return l;
  let_in(x, vec, from, to, f_lo, f_hi, bound, l.strict, cap, s, list);
  __syncthreads();
  l.total = s.count;
  l.m = static_cast<int>(min(l.total, cap));
  bool fits = l.total <= cap;
  for (int i = tid; i < l.m; i += kSelThreads) {
    const uint2 e = list[i];
    const int at = static_cast<int>(e.y);
    const bool forced = at < f_lo || at >= f_hi;
    const float v = __uint_as_float(e.x);
    list[i].x = forced ? kForcedKey : score_key(v);
    if (l.bins.scale > 0.f && !forced) atomicAdd(&s.hist[l.bins.of(v)], 1u);
  }
  if (ranks == 1) {
    __syncthreads();
  } else {
    cluster_sync();
    const uint32_t c = ld_ranks(&s.count, ranks);
    l.total = __reduce_add_sync(0xFFFFFFFFu, c);
    fits = __all_sync(0xFFFFFFFFu, c <= cap);
  }
  l.good = fits && (l.strict || l.total >= static_cast<uint32_t>(topk));
  return l;
}

__device__ __forceinline__ bool select_row(const IndexSelectParams& p, int t, int rank, int ranks, int b, int64_t vis,
                                           uint32_t cap, SelShared& s, uint2* list) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* __restrict__ x = p.scores + t * p.s_stride;
  const int n = select_blocks_of(p, vis);
  const int f_lo = min(p.first, n), f_hi = max(f_lo, n - p.last);      // forced: below f_lo, from f_hi on
  const uint32_t kk = p.topk - (f_lo + n - f_hi);                // places of the others
  const int part = ((n + ranks - 1) / ranks + 3) & ~3;
  const int from = min(n, rank * part), to = min(n, from + part);
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  // ---- the bound: the score of the sample's rank that leaves room for its error
  const List l = list_of(x, vec, n, from, to, f_lo, f_hi, sample_rank(kk, n) * s.again, s.tried, ranks, cap, p.topk, s, list);
  int m = l.m;

  // ---- the cut, over the row
  Cut c{0, 0};
  uint32_t first = 0;
  uint32_t at = 0, all = p.topk;      // positions before this CTA's part, and of the row
  const bool binned = l.good && kk > 0 && l.bins.scale > 0.f && cut_of_bins(m, kk, ranks, s, list, l.bins, c, first, at);
  if (!binned) {
    const bool fresh = s.again == 1.f;         // read before the barrier: thread 0 writes it after
    if (ranks > 1) cluster_sync(); else __syncthreads();           // the counts have been read
    if (!l.good) {
      if (!l.strict && fresh) {                // once more, with a rank for the middle of the list's room
        if (tid == 0) {
          s.again = 0.5f * static_cast<float>(p.topk + cap) / static_cast<float>(l.total);
          s.tried = l.bound;
        }
        __syncthreads();
        return false;
      }
      m = ordered_list(x, vec, from, to, f_lo, f_hi, kk, cap, s, list);
      __syncthreads();
    }
    c = find_cut(m, kk, ranks, s, [&](int i) { return list[i].x == kForcedKey ? 0u : list[i].x; });
    if (c.ties) first = find_cut(m, c.ties, ranks, s, [&](int i) { return list[i].x == c.thr ? ~list[i].y : 0u; }).thr;
  }
  auto taken = [&](uint2 e) { return e.x > c.thr || (c.ties && e.x == c.thr && ~e.y > first); };
  int32_t* out = p.blocks + t * p.b_stride;
  int32_t* out_slots = p.slots ? p.slots + t * p.sl_stride : nullptr;
  if (ranks > 1 && !binned) {
    uint32_t mine = 0;
    for (int i = tid; i < m; i += kSelThreads) mine += taken(list[i]) ? 1u : 0u;
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    if (tid == 0) s.stat[3] = 0;
    __syncthreads();
    if (lane == 0) atomicAdd(&s.stat[3], mine);
    cluster_sync();
    const uint32_t v = ld_ranks(&s.stat[3], ranks);
    at = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? v : 0u);
    all = __reduce_add_sync(0xFFFFFFFFu, v);
  }
  // ---- the map, 65536 indices at a time, and its bits in order
  for (int w0 = from; w0 < to; w0 += 32 * kSelBins) {
    reinterpret_cast<uint4*>(s.hist)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint2 e = list[i];
      const uint32_t d = e.y - w0;
      if (d < static_cast<uint32_t>(min(to - w0, 32 * kSelBins)) && taken(e)) atomicOr(&s.hist[d >> 5], 1u << (d & 31));
    }
    __syncthreads();
    const uint4 w = reinterpret_cast<const uint4*>(s.hist)[tid];
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    const uint32_t own = __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
    uint32_t pos = at + block_prefix(own, s.wsum);
    if (tid == kSelThreads - 1) s.found[0] = pos + own;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      for (uint32_t bits = words[u]; bits; bits &= bits - 1)
        out[pos++] = w0 + 128 * tid + 32 * u + __ffs(bits) - 1;
    }
    __syncthreads();
    at = s.found[0];
    __syncthreads();
  }
  if (ranks == 1) all = at;
  // ---- -1 after the list
  for (int i = static_cast<int>(all) + rank * kSelThreads + tid; i < p.topk; i += ranks * kSelThreads) out[i] = -1;
  // the list is written, and no CTA leaves while another may read its count
  if (ranks > 1) cluster_sync(); else __syncthreads();
  if (!out_slots) return true;
  // ---- token slots of the taken blocks through the block table
  const int64_t slots = static_cast<int64_t>(p.topk) * p.block_tokens;
  for (int64_t i = rank * kSelThreads + tid; i < slots; i += ranks * kSelThreads) {
    const int64_t j = i / p.block_tokens;
    int32_t slot = -1;
    if (j < all) {
      const int64_t pos = static_cast<int64_t>(__ldcg(out + j)) * p.block_tokens + (i - j * p.block_tokens);
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
  return true;
}

__global__ void __launch_bounds__(kSelThreads, 3) mla_index_select_kernel(const IndexSelectParams p, int ranks, int cap) {
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelShared& s = *reinterpret_cast<SelShared*>(sel_smem);
  uint2* list = reinterpret_cast<uint2*>(sel_smem + kSelFixed);       // (score bits, then key; index)
  const int t = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  if (threadIdx.x < 32) {
    int64_t vis = 0;
    const int b = row_request(p.cu_q, p.seq_lens, p.B, t, &vis);
    if (threadIdx.x == 0) {
      s.row[0] = b;
      s.row[1] = vis;
      s.again = 1.f;
      s.tried = CUDART_NAN_F;
    }
  }
  __syncthreads();
  if (s.row[0] < 0) return;
  while (!select_row(p, t, rank, ranks, static_cast<int>(s.row[0]), s.row[1], cap, s, list)) {
  }
}

// ------------------------------------------------------------------------------------------
// Page lists.  One warp per row keeps the visible pages of its list in order and puts the partly
// visible one (the row's newest page, when its last tokens are hidden or unwritten) last, so that
// a length alone says which tokens the row attends: full pages x block_size + the part.
__global__ void __launch_bounds__(128) mla_page_list_kernel(const PageListParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  // launched as a programmatic dependent of the work before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x < 2 && p.sched[threadIdx.x]) *p.sched[threadIdx.x] = 0u;
  if (t >= p.T) return;
  const int c_first = lane < p.topk ? p.blocks[t * p.b_stride + lane] : -1;      // under way with the search below
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
    const int c = c0 == 0 ? c_first : c0 + lane < p.topk ? src[c0 + lane] : -1;
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

namespace {

template <int kVec>
cudaError_t insert_launch(int bf16, const IndexInsertParams& p, cudaStream_t stream) {
  const dim3 grid(p.T, (p.Hi + 8 * kVec - 1) / (8 * kVec));
  if (bf16)
    mla_index_insert_kernel<true, kVec><<<grid, 128, 0, stream>>>(p);
  else
    mla_index_insert_kernel<false, kVec><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

// (32 warps an SM, each with several steps; 24 and 40 within 3 %)
template <int kRows>
cudaError_t gather_launch(int bf16, const IndexGatherParams& p, int sms, cudaStream_t stream) {
  const int64_t all = (p.num_tokens + 4 * kRows - 1) / (4 * kRows), once = static_cast<int64_t>(sms) * 8;
  const unsigned grid = static_cast<unsigned>(all < once ? all : once);
  if (bf16)
    mla_index_gather_kernel<true, kRows><<<grid, 128, 0, stream>>>(p);
  else
    mla_index_gather_kernel<false, kRows><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Four vectors a half-warp for many, two for few (one wave of CTAs either way, the shorter ones end
// sooner): 8191 tokens of 64 heads 41.7 against 48.3 us, 512 4.3 against 4.6, 256 3.6 against 3.2, 32 2.9 against
// 2.4.  Eight held 80 registers a thread and took 49 us for 8191.
cudaError_t launch_index_insert(int bf16, const IndexInsertParams& p, cudaStream_t stream) {
  return static_cast<int64_t>(p.T) * p.Hi >= 32768 ? insert_launch<4>(bf16, p, stream) : insert_launch<2>(bf16, p, stream);
}

// 16 rows a warp for many, two for few: 512000 rows 35 against 78 us, 64000 5.4 against 10.4, 12000 3.5 against 3.6,
// 8192 3.1 against 3.0, 1021 3.0 against 2.4.  (8 rows: 512000 37 us, 32 rows 42.)
cudaError_t launch_index_gather(int bf16, const IndexGatherParams& p, int sms, cudaStream_t stream) {
  return p.num_tokens >= 10240 ? gather_launch<16>(bf16, p, sms, stream) : gather_launch<2>(bf16, p, sms, stream);
}

static_assert(kSelFixed + (kSelectMaxTopk + kSelChunk) * 8 <= 200 * 1024, "shared memory budget");

cudaError_t launch_index_select(const IndexSelectParams& p, int sms, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mla_index_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  // CTAs that share a row: while the batch leaves SMs idle and a part keeps 8192 scores
  int ranks = 1;
  while (ranks < 8 && static_cast<int64_t>(p.T) * ranks * 2 <= sms && p.width / (ranks * 2) >= 8192) ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T) * ranks);
  cfg.blockDim = dim3(kSelThreads);
  const int cap = select_capacity(p.topk, p.width > 1 ? p.width : 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSelFixed) + static_cast<size_t>(cap) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_index_select_kernel, p, ranks, cap);
}

cudaError_t launch_page_list(const PageListParams& p, cudaStream_t stream) {
  return launch_pdl(mla_page_list_kernel, dim3((p.T + 3) / 4), dim3(128), 0, stream, p);
}

}  // namespace mla
