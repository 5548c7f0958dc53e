// mla_index_scores.cu -- the cheap score that chooses what sparse attention reads: every visible
// cached index key against the index queries of a row,
//   s[t, j] = ks[j] * sum_h w[t, h] * relu(q[t, h, :] . k[j, :]),
// stored per token, or as the maximum over blocks of 16..128 tokens.
//
// Design.  The key tile (128 keys x 128 values, E4M3 or bf16) is the M operand and the query rows
// (up to 256 = 4 queries x 64 heads, 8 x 32, ...) the N operand of tcgen05.mma, so a TMEM lane
// is a key and a column a (query, head): one read of a key serves every row of the tile, the heads of a
// query are summed where the products are, and a warp's results are 32 neighbouring scores of one
// row.  relu and the weights run between the two, on CUDA cores, in fp32.
//
// Work is cut into units of one key tile x one query tile, enumerated over requests by a closed
// form (a causal row sees seq_len - rows + i + 1 keys), and every CTA takes an equal contiguous
// range of them: scores are independent, so nothing is merged and no counter is shared.
//
// Warps: 0 producer (TMA boxes of pages, lanes resolve page ids), 1 and 2 MMA issuers (1 owns TMEM),
// 4..19 four epilogue groups of four warps: two sets of two groups, each set with two of the four
// 128-column accumulator buffers and a warp of its own to issue for it.
//
// Measured (GB300).  A decode step over 64 contexts of 16384..131072 tokens (657 MB of keys, scores and
// queries): 119 us, 5.5 TB/s of the 6.8 TB/s a copy reaches.  4059 prefill rows against 20000..32768
// keys (1.97 TFLOP, E4M3): 1.02 ms, 1.92 PFLOP/s; with bf16 keys the products themselves bound it, 79 % of
// the measured bf16 rate.  With E4M3 the CUDA cores do: a product costs them a max at half rate and half an
// fma.f32x2, and without that arithmetic (the rest of the pipeline alone) the same kernel takes 70 % of
// the time.  What it took to get there, each against the form before it:
//   - weights in registers, 16 for 64 columns, by 16 x 256-bit accumulator loads (epilogue below);
//   - few instructions on the warps that issue: they run once a tile beside busy neighbours, and their
//     instructions are fetched again each time (two MMA warps, uniform operands, slow paths out of line;
//     237 -> 187 us on 608 rows x 32768 keys, bf16 71 -> 53 us on 608 x 8192);
//   - no division in the producer's loop (155 -> 130 us for 64 contexts of 65536).
// Tried and slower: 24 epilogue warps of 72 registers (spills; 187 -> 268 us), accumulator loads ahead of
// their use (187 -> 192 us), 104 registers for the epilogue by setmaxnreg (spills), one lane polling
// for its warp (187 -> 212 us), MMAs of N = 128 from one warp (198 -> 243 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "mla_index.h"
#include "mla_internal.h"
#include "mla_paged_tma.cuh"

namespace mla {
namespace {

constexpr int kIxCols = 256;                  // query rows (MMA N) of a tile
constexpr int kIxThreads = 32 * 20;
constexpr int kSegDepth = 4;

// A run of key tiles of one query tile.
struct Segment {
  int t0, nq;          // first row and rows of the query tile
  int j0, nt;          // first key tile and number of key tiles; nt = 0 ends the queue
  int vis0;            // keys that row t0 sees (row t0 + i: vis0 + i), may be <= 0
  int b, pad0, pad1;
};

// A stage fills one of four accumulator buffers of 128 columns: half of the columns of a key tile, a
// key tile of at most 128 columns, or two of at most 64.
constexpr int kStageCols = 128;
constexpr int kBufs = 4;
__device__ __forceinline__ int stage_tiles(int cols) { return cols <= 64 ? 2 : 1; }
__device__ __forceinline__ int tile_stages(int cols) { return cols > kStageCols ? 2 : 1; }

template <int F>
struct IndexCfg {
  static_assert(F == kBF16 || F == kFP8, "format");
  static constexpr int kHalves = F == kBF16 ? 2 : 1;            // 128-byte columns of a row
  static constexpr int kTileBytes = 128 * 128 * kHalves;
  static constexpr int kQBytes = kIxCols * 128 * kHalves;
  static constexpr int kS = F == kBF16 ? 4 : 8;                 // key tiles in flight
  static constexpr int kQB = F == kBF16 ? 1 : 2;                // query tiles in flight
  static constexpr int kSc = kS + 8;                            // scales in flight (see the producer)
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQB * kQBytes;
  static constexpr int kScale = kRing + kS * kTileBytes;
  static constexpr int kRed = kScale + kSc * 512;               // block maxima: 4 buffers x 2 groups x 4 warps x 8 queries
  static constexpr int kSeg = kRed + 2 * 16 * 8 * 4;
  static constexpr int kBad = kSeg + kSegDepth * 32;
  static constexpr int kBar = kBad + ((kSc * 4 + 7) & ~7);
  static constexpr int kNumBars = 2 * kS + 4 + 2 * kBufs + 2 * kSegDepth + 8 + 2;      // as carved in the kernel
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kAlloc = kMisc + 64 + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
};

// sum over y = 1..x of ceil(y / r) (0 for x <= 0)
__device__ __forceinline__ int64_t ceil_sum(int64_t x, int r) {
  if (x <= 0) return 0;
  const int64_t q = x / r, s = x - q * r;
  return r * (q * (q + 1) / 2) + s * (q + 1);
}

// Units of a request: query tiles of QT rows, tile i with ceil((a + i + 1) / r) key tiles, where
// a = ceil((L - n) / QT) and r = 128 / QT: ceil((L - n + (i + 1) QT) / 128).
struct Request {
  int64_t a;
  int row0, n, L, m;
  int64_t units;
};

template <int QT>
__device__ __forceinline__ Request load_request(const IndexScoresParams& p, int b) {
  Request q;
  if (p.cu_q) {
    q.row0 = min(max(p.cu_q[b], 0), p.T);
    q.n = max(min(p.cu_q[b + 1], p.T) - q.row0, 0);
  } else {
    q.row0 = b;
    q.n = b < p.T ? 1 : 0;
  }
  q.L = min(max(p.seq_lens[b], 0), 0x7FFFF000);      // positions of a tile's rows stay in 32 bits
  q.m = (q.n + QT - 1) / QT;
  const int d = q.L - q.n;
  q.a = d >= 0 ? (d + QT - 1) / QT : -((-d) / QT);
  q.units = ceil_sum(q.a + q.m, 128 / QT) - ceil_sum(q.a, 128 / QT);
  return q;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A position in a ring of N slots and the parity of its pass.
template <int N>
struct Cursor {
  int slot = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) slot = 0, par ^= 1u;
  }
};

// relu(d) * w summed into acc, for the C columns of one query: pairs of columns share an fma.f32x2
__device__ __forceinline__ void fma2(uint64_t& acc, float x0, float x1, uint64_t w) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(x0), "f"(x1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(x), "l"(w));
}
__device__ __forceinline__ float sum2(uint64_t a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
  return x + y;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}

// 16 lanes x 32 columns: lane 4 a + b gets, of every 8 columns c, v[4 c] and v[4 c + 1] = TMEM lane a,
// columns 2 b and 2 b + 1, and v[4 c + 2], v[4 c + 3] = TMEM lane a + 8.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// The rest of a bounded wait, out of line: the roles' loops stay short (a warp that runs a loop once
// a tile beside busy neighbours fetches all of its instructions again each time).
__device__ __noinline__ bool wait_rest(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return warp_wait(bar, parity, abort_flag);
}

// Bounded wait of a whole warp.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return wait_rest(bar, parity, abort_flag);
}

template <int F, int HP>
__global__ void __launch_bounds__(kIxThreads, 1)
    mla_index_scores_kernel(const __grid_constant__ IndexScoresParams p, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_q) {
  using C = IndexCfg<F>;
  constexpr int S = C::kS, SC = C::kSc, HV = C::kHalves, QB = C::kQB;
  constexpr int QT = kIxCols / HP;             // queries of a tile
  constexpr int QW = 64 / HP;                  // queries of an epilogue group
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, not through an integer: the compiler then still knows it is shared memory
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* qs = smem + C::kQ;
  uint8_t* ring = smem + C::kRing;
  float* scales = reinterpret_cast<float*>(smem + C::kScale);
  float* red = reinterpret_cast<float*>(smem + C::kRed);
  Segment* segs = reinterpret_cast<Segment*>(smem + C::kSeg);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::kBad);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* k_full = bars;                     // [S] key tile and its scales landed
  uint64_t* k_empty = k_full + S;              // [S] its MMAs are done
  uint64_t* q_full = k_empty + S;              // [2]
  uint64_t* q_empty = q_full + 2;              // [2]
  uint64_t* d_full = q_empty + 2;              // [4] accumulator ready
  uint64_t* d_empty = d_full + kBufs;          // [4] accumulator read
  uint64_t* seg_full = d_empty + kBufs;
  uint64_t* seg_empty = seg_full + kSegDepth;
  uint64_t* red_full = seg_empty + kSegDepth;  // [4 groups][2] block maxima of a group's warps written
  uint64_t* fin = red_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 8);
  int64_t* start = reinterpret_cast<int64_t*>(smem + C::kMisc + 16);      // [0] first unit's request, [1] its offset, [2] units
  int64_t* part = reinterpret_cast<int64_t*>(red);      // setup only: 20 warp totals

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 2);      // both MMA warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&d_full[i], 2);      // the MMAs, and the issuer's own arrival (see there)
      mbar_init(&d_empty[i], 8);
    }
    for (int i = 0; i < kSegDepth; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 18);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&red_full[i], 4);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    abort_flag[0] = 0;
    abort_flag[1] = 0;
    start[0] = p.B;
    start[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_q) : "memory");
  }
  // ---- this CTA's range of units, [W c / G, W (c + 1) / G), and the request it starts in: a prefix sum
  // over the requests' units, twice where one pass of the CTA does not hold them all
  int64_t lo = 0, hi = 0;
  const int chunks = (p.B + kIxThreads - 1) / kIxThreads;
  for (int pass = 0; pass < (chunks > 1 ? 2 : 1); ++pass) {
    int64_t before = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * kIxThreads + tid;
      const int64_t u = b < p.B ? load_request<QT>(p, b).units : 0;
      int64_t inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) part[warp] = inc;
      __syncthreads();
      int64_t base = before, all = 0;
#pragma unroll
      for (int w = 0; w < kIxThreads / 32; ++w) {
        const int64_t v = part[w];
        if (w < warp) base += v;
        all += v;
      }
      if (pass == 0 && c + 1 == chunks) {
        const uint64_t total = static_cast<uint64_t>(before + all), each = total / gridDim.x, rest = total % gridDim.x;
        lo = static_cast<int64_t>(each * blockIdx.x + (rest < blockIdx.x ? rest : blockIdx.x));
        hi = lo + static_cast<int64_t>(each + (blockIdx.x < rest ? 1 : 0));
      }
      if (chunks == 1 || pass == 1) {
        const int64_t first = base + inc - u;
        if (first <= lo && lo < first + u && lo < hi) {
          start[0] = b;
          start[1] = lo - first;
        }
      }
      before += all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    int b = static_cast<int>(start[0]);
    int64_t x = start[1], rem = hi - lo;
    const bool leader = elect_one();
    const int BR = p.BR, SP = 128 / BR;            // page slices of BR rows, SP of them a tile
    const int SB = p.block_size / BR;              // slices of a page
    const int TG = 32 / SP;                        // key tiles covered by one page lookup of the warp
    const uint32_t SM = (1u << SP) - 1;
    int tile = 0;                                  // key tiles issued
    Cursor<S> kc;
    Cursor<SC> sc;
    int nseg = 0;
    uint32_t errbits = 0;
    bool ok = true;
    while (ok && rem > 0 && b < p.B) {
      const Request rq = load_request<QT>(p, b);
      if (x >= rq.units) {
        ++b;
        x = 0;
        continue;
      }
      // the query tile that holds unit x
      constexpr int r = 128 / QT;
      const int64_t fa = ceil_sum(rq.a, r);
      int i0 = 0, i1 = rq.m - 1;
      while (i0 < i1) {
        const int mid = (i0 + i1 + 1) >> 1;
        if (ceil_sum(rq.a + mid, r) - fa <= x) i0 = mid; else i1 = mid - 1;
      }
      const int64_t y = x - (ceil_sum(rq.a + i0, r) - fa);
      const int64_t units_i = ceil_sum(rq.a + i0 + 1, r) - ceil_sum(rq.a + i0, r);
      const int64_t take = min(units_i - y, rem);
      x += take;
      rem -= take;
      Segment sg;
      sg.t0 = rq.row0 + i0 * QT;
      sg.nq = min(QT, rq.n - i0 * QT);
      sg.vis0 = rq.L - rq.n + i0 * QT + 1;
      sg.b = b;
      sg.pad0 = sg.pad1 = 0;
      // keys of the tile's last row, and those that have a column
      const int64_t seen = min(static_cast<int64_t>(sg.vis0) + sg.nq - 1, p.cap);
      const int64_t real = seen > 0 ? (seen + 127) / 128 : 0;
      sg.j0 = static_cast<int>(y);
      sg.nt = static_cast<int>(max(min(y + take, real) - y, static_cast<int64_t>(0)));
      if (sg.nt == 0) continue;
      const int k = nseg % kSegDepth;
      if (nseg >= kSegDepth && !warp_wait(&seg_empty[k], ((nseg / kSegDepth) - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      const int qb = nseg % QB;
      if (nseg >= QB && !warp_wait(&q_empty[qb], ((nseg / QB) - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        segs[k] = sg;
        mbar_arrive(&seg_full[k]);
        mbar_arrive_expect_tx(&q_full[qb], C::kQBytes);
#pragma unroll
        for (int h = 0; h < HV; ++h)
          tma_load_3d(qs + qb * C::kQBytes + h * kIxCols * 128, &tm_q, 128 * h, 0, sg.t0, &q_full[qb]);
      }
      ++nseg;
      // Pages of the slices j SP .. (j + TG) SP - 1, one per lane, looked up a group of TG tiles ahead.
      const int s_end = static_cast<int>((seen + BR - 1) / BR);          // slices with a visible key
      auto lookup = [&](int j, int& y) -> int {
        const int sl = j * SP + lane, col = SB == 1 ? sl : sl / SB;
        y = SB == 1 ? 0 : (sl - col * SB) * BR;
        if (j >= sg.j0 + sg.nt || sl >= s_end) return -2;                 // nothing to read
        const int id = col < p.bt_cols ? p.block_table[b * p.bt_stride + col] : -1;
        return (id < 0 || id >= p.num_blocks) ? -1 : id;
      };
      int cur, cy, nxt = 0, ny = 0;
      nxt = lookup(sg.j0, ny);
      uint32_t bad_m = 0, good_m = 0;
      int in = TG;      // tile of the lookup group
      for (int t = 0; t < sg.nt; ++t, ++tile) {
        if (in == TG) {
          in = 0;
          cur = nxt;
          cy = ny;
          bad_m = __ballot_sync(0xFFFFFFFFu, cur == -1);
          good_m = __ballot_sync(0xFFFFFFFFu, cur >= 0);
          if (bad_m) errbits |= 2u;
          nxt = lookup(sg.j0 + t + TG, ny);
        }
        const int slot = kc.slot, sslot = sc.slot;
        // Tile n - S's MMAs are done, so the accumulators of the stage four before its own had been
        // read: with at most 2 tiles a stage, the scales of tile n - S - 8 and before are free.
        if (tile >= S && !wait_all(&k_empty[slot], kc.par ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (leader) {
          bad[sslot] = (bad_m >> (in * SP)) & SM;
          mbar_arrive_expect_tx(&k_full[slot], C::kTileBytes + (F == kFP8 ? __popc((good_m >> (in * SP)) & SM) * BR * 4 : 0));
        }
#pragma unroll 1
        for (int q = 0; q < SP; ++q) {
          const int id = __shfl_sync(0xFFFFFFFFu, cur, in * SP + q), y = __shfl_sync(0xFFFFFFFFu, cy, in * SP + q);
          if (leader) {
#pragma unroll
            for (int h = 0; h < HV; ++h)
              tma_load_3d(ring + slot * C::kTileBytes + h * 128 * 128 + q * BR * 128, &tm_k, 128 * h, y, id >= 0 ? id : p.num_blocks, &k_full[slot]);
            if (F == kFP8 && id >= 0)
              bulk_g2s(scales + sslot * 128 + q * BR, p.key_scales + (id * p.ks_stride + y), BR * 4, &k_full[slot]);
          }
        }
        ++in;
        kc.step();
        sc.step();
      }
    }
    if (ok) {      // end of the queue
      const int k = nseg % kSegDepth;
      if (nseg < kSegDepth || warp_wait(&seg_empty[k], ((nseg / kSegDepth) - 1) & 1, abort_flag)) {
        if (lane == 0) {
          Segment e{};
          segs[k] = e;
          mbar_arrive(&seg_full[k]);
        }
      }
    }
    // never leave copies in flight behind us
    if (lane == 0) {
      volatile int no_abort[2] = {0, 0};
      for (int q = tile > S ? tile - S : 0; q < tile; ++q) mbar_wait(&k_full[q % S], (q / S) & 1, no_abort);
      for (int q = nseg > QB ? nseg - QB : 0; q < nseg; ++q) mbar_wait(&q_full[q % QB], (q / QB) & 1, no_abort);
    }
    __syncwarp();
    if (lane == 0 && errbits) set_device_error(p.err, errbits);
  } else if (warp <= 2) {
    // ------------------------------------------------------------------ MMA issuers
    // One for each set's stages: a single warp's loop (waits, 4 or 8 products, commits: some 700 cycles
    // a stage beside the epilogue's warps) set the kernel's pace.
    const uint32_t mine = warp - 1;
    // The whole warp walks the loop and one elected lane issues: addresses and descriptors then stay
    // warp-uniform (from a single-lane branch every operand of an MMA is moved to a uniform register
    // first, and this warp, which shares its scheduler with four busy ones, set the kernel's pace).
    const bool leader = elect_one();
    const uint32_t hi_desc = static_cast<uint32_t>(smem_desc(0, 16, 1024, kSwizzle128B) >> 32);
    const uint32_t dK0 = static_cast<uint32_t>(smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B));
    const uint32_t dQ0 = static_cast<uint32_t>(smem_desc(smem_u32(qs), 16, 1024, kSwizzle128B));
    auto desc = [&](uint32_t lo) -> uint64_t { return static_cast<uint64_t>(hi_desc) << 32 | lo; };
    Cursor<S> kc;
    uint32_t parity = 0;                       // of the stage count: this warp's stages are those of `mine`
    uint32_t x = 0, empty_par = 1;             // buffer mine + 2 x, free at first
    bool ok = true;
    for (uint32_t ns = 0; ok; ++ns) {
      const uint32_t k = ns % kSegDepth, qb = ns % QB;
      if (!wait_all(&seg_full[k], (ns / kSegDepth) & 1, abort_flag)) break;
      const int nt = __shfl_sync(0xFFFFFFFFu, segs[k].nt, 0), nq = __shfl_sync(0xFFFFFFFFu, segs[k].nq, 0);
      if (leader) mbar_arrive(&seg_empty[k]);
      if (nt == 0) break;
      if (!wait_all(&q_full[qb], (ns / QB) & 1, abort_flag)) break;
      const int n = (nq * HP + 15) & ~15;      // columns: a multiple of 16
      const int G = stage_tiles(n);
      const bool two = tile_stages(n) == 2;    // every tile has a stage of this warp, its first or second half
      const int half = two && parity != mine ? 1 : 0;
      const int cols = two ? (half ? n - kStageCols : kStageCols) : n;
      const uint32_t idesc = F == kBF16 ? idesc_f16(128, cols, 1, 1, 0, 0) : idesc_e4m3(128, cols, 0, 0);
      const uint32_t dQ = dQ0 + qb * (C::kQBytes >> 4) + half * (kStageCols * 128 >> 4);
      int in = 0;                              // tile of the stage
      // Every tile's barrier is waited for in order, the other warp's too: a phase is known to be over
      // before the next one of its slot is waited for.
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        if (!wait_all(&k_full[kc.slot], kc.par, abort_flag)) {
          ok = false;
          break;
        }
        const bool own = two || parity == mine, last = in + 1 == G || t + 1 == nt;
        if (own && in == 0 && !wait_all(&d_empty[mine + 2 * x], empty_par, abort_flag)) {
          ok = false;
          break;
        }
        if (leader) {
          if (own) {
            tc_fence_after();
            const uint32_t dK = dK0 + static_cast<uint32_t>(kc.slot) * (C::kTileBytes >> 4);
            const uint32_t d = tmem + (mine + 2 * x) * kStageCols + in * 64;
#pragma unroll
            for (int h = 0; h < HV; ++h)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint64_t a = desc(dK + ((h * 128 * 128 + kk * 32) >> 4));
                const uint64_t bq = desc(dQ + ((h * kIxCols * 128 + kk * 32) >> 4));
                if (F == kBF16)
                  mma_f16_ss(d, a, bq, idesc, h + kk > 0 ? 1u : 0u);
                else
                  mma_f8_ss(d, a, bq, idesc, h + kk > 0 ? 1u : 0u);
              }
            mma_commit(&k_empty[kc.slot]);
            if (last) {
              mma_commit(&d_full[mine + 2 * x]);
              // the scales and bad-page masks that came with the key tiles reach the epilogue by this
              // thread's release (it has seen k_full)
              mbar_arrive(&d_full[mine + 2 * x]);
            }
          } else {
            mbar_arrive(&k_empty[kc.slot]);
          }
        }
        __syncwarp();
        kc.step();
        ++in;
        if (last) {
          in = 0;
          if (own) {
            x ^= 1u;
            empty_par ^= x ^ 1u;
          }
          if (!two) parity ^= 1u;
        }
      }
      if (ok && leader) mma_commit(&q_empty[qb]);
    }
    if (leader) {      // no product is in flight when the accumulators are freed
      volatile int no_abort[2] = {0, 0};
      mma_commit(&fin[mine]);
      mbar_wait(&fin[mine], 0, no_abort);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    // Two sets of two groups: a set takes every second stage and has two of the four buffers, so that
    // the products of its next stage run while it reads this one; a group takes 64 columns.
    const int quad = warp & 3, group = (warp - 4) >> 2, set = group >> 1, sl = group & 1;
    // A thread's keys and columns: a 16 x 256-bit load gives lane 4 a + b the columns 2 b, 2 b + 1 of
    // every 8 for the keys a and a + 8, so its weights of 64 columns are 16 registers (a lane that had
    // one key and all columns would need them all, and reading them from shared memory for every
    // tile took twice the time of the products).  The four lanes of a key then exchange
    // their sums, and lane 4 a + b ends with key a + 8 b.
    const int la = lane >> 2, lb = lane & 3;
    const int key = 32 * quad + la + 8 * lb;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16) + sl * 64;
    float* red_g = red + (sl * 4 + quad) * 8;     // of buffer u: 64 u further
    const bool padded = p.Hi < HP;
    const bool early = !padded && p.block_tokens <= 32;       // nothing of the stage is needed after its columns
    const int bt = p.block_tokens, br_shift = 31 - __clz(p.BR), bt_shift = 31 - __clz(bt);
    const int cap = static_cast<int>(p.cap);
    uint32_t stage = 0;                           // stages before the segment
    int sbase = 0;                                // scale slot of the segment's first tile
    uint32_t uses = 0;                            // block maxima exchanged through red
    bool ok = true;
    for (uint32_t ns = 0; ok; ++ns) {
      const uint32_t k = ns % kSegDepth;
      if (!wait_all(&seg_full[k], (ns / kSegDepth) & 1, abort_flag)) break;
      const Segment sg = segs[k];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[k]);
      if (sg.nt == 0) break;
      // the segment's stages, the set's first one, and this group's tile and queries in it
      const int n = (sg.nq * HP + 15) & ~15, G = stage_tiles(n), NS = tile_stages(n);
      const int stages = NS == 2 ? 2 * sg.nt : (sg.nt + G - 1) / G;
      const int i0 = static_cast<int>(stage & 1) ^ set;
      const int g = G == 2 ? sl : 0;
      const int q0 = G == 2 ? 0 : (NS == 2 ? i0 * kStageCols + sl * 64 : sl * 64) / HP;
      const int nq = max(min(QW, sg.nq - q0), 0);
      int t = (NS == 2 ? 0 : i0 * G) + g;         // tile of the set's next stage
      const int dt = NS == 2 ? 1 : 2 * G;
      int slot = sbase + t;                       // and its scale slot
      if (slot >= SC) slot -= SC;
      const int first = sg.j0 * 128 + key;
      const int lim = min(sg.vis0 + q0, cap) - first;         // keys of the segment that the first query sees, less the thread's place
      const int edge = cap - first;
      float* row = p.scores + static_cast<int64_t>(sg.t0 + q0) * p.s_stride + (first >> bt_shift);
      const float* wsrc = p.weights + static_cast<int64_t>(sg.t0 + q0) * p.w_stride;
      auto weight = [&](int c) -> float {         // 0 for padded heads and queries
        const int q = c / HP, h = c % HP;
        return q < nq && h < p.Hi ? __ldg(wsrc + q * p.w_stride + h) : 0.f;
      };
      uint64_t w[8];                              // of the columns 8 c + 2 lb and the next
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = pack2(weight(8 * c + 2 * lb), weight(8 * c + 2 * lb + 1));
      for (int i = i0; i < stages; i += 2, t += dt) {
        const uint32_t at = stage + i, buf = at % kBufs;
        const bool has = nq > 0 && t < sg.nt;
        if (!wait_all(&d_full[buf], (at / kBufs) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const int s0 = slot;
        slot += dt;
        if (slot >= SC) slot -= SC;
        tc_fence_after();
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[buf]);
        };
        if (!has) {
          release();
          continue;
        }
        // the key's scale and bad pages, read before the release (their slots are reused after it)
        const uint32_t bm = bad[s0];
        const float ks = F == kFP8 ? scales[s0 * 128 + key] : 1.f;
        const uint32_t ta = tl + buf * kStageCols;
        // Load u: keys 16 (u / 2) .. + 15 of the warp's 32, columns 32 (u % 2) .. + 31.
        float v[QW];
        {
          float y[4][QW];                         // keys la + 8 i
          uint64_t acc[2][QW];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float d[16];
            tmem_ld_16x256(ta + 32 * (u & 1) + (static_cast<uint32_t>(16 * (u >> 1)) << 16), d);
            tmem_ld_wait();
            if (u == 3 && early) release();       // everything is in registers
#pragma unroll
            for (int c = 0; c < 4; ++c) {         // 8 columns
              const int q = (32 * (u & 1) + 8 * c) / HP;
              const bool start = (32 * (u & 1) + 8 * c) % HP == 0;
              const float* x = d + 4 * c;
              const uint64_t ww = w[4 * (u & 1) + c];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                if (start) acc[r][q] = 0;
                fma2(acc[r][q], max_nan(x[2 * r], 0.f), max_nan(x[2 * r + 1], 0.f), ww);
              }
            }
            if (u & 1)
#pragma unroll
              for (int q = 0; q < QW; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r) y[(u >> 1) * 2 + r][q] = sum2(acc[r][q]);
          }
          // the four lanes of a key: lane bit 1 keeps keys la, la + 8 or la + 16, la + 24, bit 0 one of them
#pragma unroll
          for (int q = 0; q < QW; ++q) {
            const bool h = lb & 2, o = lb & 1;
            const float k0 = h ? y[2][q] : y[0][q], k1 = h ? y[3][q] : y[1][q];
            const float g0 = h ? y[0][q] : y[2][q], g1 = h ? y[1][q] : y[3][q];
            const float z0 = k0 + __shfl_xor_sync(0xFFFFFFFFu, g0, 2), z1 = k1 + __shfl_xor_sync(0xFFFFFFFFu, g1, 2);
            v[q] = (o ? z1 : z0) + __shfl_xor_sync(0xFFFFFFFFu, o ? z0 : z1, 1);
          }
        }
        // a key with infinities or NaN meets the zeros of the padded heads: sum the heads alone
        if (padded) {
#pragma unroll
          for (int q = 0; q < QW; ++q) {
            if (!__any_sync(0xFFFFFFFFu, v[q] != v[q])) continue;
            float s = 0.f;
#pragma unroll 1
            for (int h = 0; h < p.Hi; ++h) {
              uint32_t e;
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(e) : "r"(ta + q * HP + h));
              tmem_ld_wait();
              s = fmaf(max_nan(__uint_as_float(e), 0.f), weight(q * HP + h), s);
            }
            // (in another order of the sum: only for the keys that need it, so that the others' bits do not depend on
            // what lies beside them, unwritten slots among it)
            s = __shfl_sync(0xFFFFFFFFu, s, la + 8 * lb);
            if (v[q] != v[q]) v[q] = s;
          }
        }
        const bool is_bad = bm && ((bm >> (key >> br_shift)) & 1u);
#pragma unroll
        for (int q = 0; q < QW; ++q) v[q] = is_bad ? -CUDART_INF_F : F == kFP8 ? v[q] * ks : v[q];
        const bool exchange = bt > 32;
        if (!exchange && !early) release();
        const int off = t * 128;
        float* r = row + (off >> bt_shift);
        if (bt == 1) {
#pragma unroll
          for (int q = 0; q < QW; ++q, r += p.s_stride)
            if ((QW == 1 || q < nq) && off < (QW == 1 ? lim : min(lim + q, edge))) *r = v[q];
          continue;
        }
#pragma unroll
        for (int q = 0; q < QW; ++q, r += p.s_stride) {
          if (q >= nq) break;
          const bool seen = off < min(lim + q, edge);
          float val = seen ? v[q] : -CUDART_INF_F;
          // over la and lb bit 0: 16 keys; over lb bit 1: 32
          val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 4));
          val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 8));
          val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 16));
          val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 1));
          if (bt > 16) val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 2));
          if (!exchange) {
            if ((key & (bt - 1)) == 0 && seen) *r = val;
          } else if (lane == 0) {
            red_g[64 * buf + q] = val;
          }
        }
        if (exchange) {       // blocks of 64 or 128 keys: two or four warps of the group
          uint64_t* rf = &red_full[group * 2 + (uses & 1)];
          if (lane == 0) mbar_arrive(rf);
          const uint32_t par = (uses++ >> 1) & 1u;
          const int wb = bt >> 5;                 // warps of a block; its first one joins them
          if ((quad & (wb - 1)) == 0) {
            if (!wait_all(rf, par, abort_flag)) {
              ok = false;
              break;
            }
            const int p0 = sg.j0 * 128 + off + 32 * quad;
            if (lane < nq && p0 < min(sg.vis0 + q0 + lane, cap)) {
              float mx = red_g[64 * buf + lane];
              for (int o = 1; o < wb; ++o) mx = max_nan(mx, red_g[64 * buf + 8 * o + lane]);
              p.scores[static_cast<int64_t>(sg.t0 + q0 + lane) * p.s_stride + (p0 >> bt_shift)] = mx;
            }
          }
          // red is free with the buffer: written again only for the stage that next uses it
          release();
        }
      }
      stage += stages;
      sbase = (sbase + sg.nt) % SC;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag == 2) set_device_error(p.err, 16u);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int F, int HP>
cudaError_t launch_hp(const IndexScoresParams& p, const void* tk, const void* tq, int grid, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mla_index_scores_kernel<F, HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             IndexCfg<F>::kAlloc);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  mla_index_scores_kernel<F, HP><<<grid, kIxThreads, IndexCfg<F>::kAlloc, stream>>>(
      p, *static_cast<const CUtensorMap*>(tk), *static_cast<const CUtensorMap*>(tq));
  return cudaGetLastError();
}

template <int F>
cudaError_t launch_f(int hp, const IndexScoresParams& p, const void* tk, const void* tq, int grid, cudaStream_t stream) {
  switch (hp) {
    case 8: return launch_hp<F, 8>(p, tk, tq, grid, stream);
    case 16: return launch_hp<F, 16>(p, tk, tq, grid, stream);
    case 32: return launch_hp<F, 32>(p, tk, tq, grid, stream);
    case 64: return launch_hp<F, 64>(p, tk, tq, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_index_scores(int bf16, int hp, const IndexScoresParams& p, const void* tk, const void* tq, int grid,
                                cudaStream_t stream) {
  return bf16 ? launch_f<kBF16>(hp, p, tk, tq, grid, stream) : launch_f<kFP8>(hp, p, tk, tq, grid, stream);
}

}  // namespace mla
