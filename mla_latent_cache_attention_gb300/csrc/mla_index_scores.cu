// mla_index_scores.cu -- the cheap score that chooses what sparse attention reads: every visible
// cached index key against the index queries of a row,
//   s[t, j] = ks[j] * sum_h w[t, h] * relu(q[t, h, :] . k[j, :]),
// stored per token, or as the maximum over blocks of 16..128 tokens.
//
// Design.  The key tile (128 keys x 128 values, E4M3 or bf16) is the M operand and the query rows
// (up to 256 = 4 queries x 64 heads, 8 x 32, ...) the N operand of tcgen05.mma, so a TMEM lane
// is a key and a column a (query, head): the sum over heads stays inside one thread, needs no
// exchange, and a warp's 32 results are 32 neighbouring scores of one row.  relu and the weights
// run between the two, on CUDA cores, in fp32; the weights of a thread's 64 columns stay in
// registers for all key tiles of a query tile.
//
// Work is cut into units of one key tile x one query tile, enumerated over requests by a closed
// form (a causal row sees seq_len - rows + i + 1 keys), and every CTA takes an equal contiguous
// range of them: scores are independent, so nothing is merged and no counter is shared.
//
// A stage is one accumulator buffer of 256 columns: one key tile, or two or four where the query
// tile has at most 128 or 64 columns (decode), so that the four epilogue groups always share it.
//
// Warps: 0 producer (TMA boxes of pages, lanes resolve page ids), 1 MMA issuer and TMEM owner, 
// 2..17 four epilogue groups of four warps.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "mla_index.h"
#include "mla_internal.h"
#include "mla_paged_tma.cuh"

namespace mla {
namespace {

constexpr int kIxCols = 256;                  // query rows (MMA N) of a tile
constexpr int kIxThreads = 32 * 18;
constexpr int kSegDepth = 4;

// A run of key tiles of one query tile.
struct Segment {
  int t0, nq;          // first row and rows of the query tile
  int j0, nt;          // first key tile and number of key tiles; nt = 0 ends the queue
  int vis0;            // keys that row t0 sees (row t0 + i: vis0 + i), may be <= 0
  int b, pad0, pad1;
};

// Key tiles of a stage (one accumulator buffer): query tiles of few columns share it.
__device__ __forceinline__ int stage_tiles(int cols) { return cols <= 64 ? 4 : cols <= 128 ? 2 : 1; }

template <int F>
struct IndexCfg {
  static_assert(F == kBF16 || F == kFP8, "format");
  static constexpr int kHalves = F == kBF16 ? 2 : 1;            // 128-byte columns of a row
  static constexpr int kTileBytes = 128 * 128 * kHalves;
  static constexpr int kQBytes = kIxCols * 128 * kHalves;
  static constexpr int kS = F == kBF16 ? 4 : 8;                 // key tiles in flight
  static constexpr int kQB = F == kBF16 ? 1 : 2;                // query tiles in flight
  static constexpr int kSc = kS + 12;                           // scales in flight (see the producer)
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQB * kQBytes;
  static constexpr int kScale = kRing + kS * kTileBytes;
  static constexpr int kRed = kScale + kSc * 512;               // block maxima: 2 buffers x 4 slices x 4 warps x 8 queries
  static constexpr int kSeg = kRed + 2 * 16 * 8 * 4;
  static constexpr int kBad = kSeg + kSegDepth * 32;
  static constexpr int kBar = kBad + ((kSc * 4 + 7) & ~7);
  static constexpr int kNumBars = 2 * kS + 8 + 2 * kSegDepth + 4 + 1;      // as carved in the kernel
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
  q.L = max(p.seq_lens[b], 0);
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

// Bounded wait of a whole warp: one look by every lane where the phase has completed already.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort_flag);
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
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
  uint64_t* d_full = q_empty + 2;              // [2] accumulator ready
  uint64_t* d_empty = d_full + 2;              // [2] accumulator read
  uint64_t* seg_full = d_empty + 2;
  uint64_t* seg_empty = seg_full + kSegDepth;
  uint64_t* red_full = seg_empty + kSegDepth;  // [4] block maxima of a group's warps written
  uint64_t* fin = red_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 8);
  int64_t* start = reinterpret_cast<int64_t*>(smem + C::kMisc + 16);      // [0] first unit's request, [1] its offset, [2] units
  int64_t* part = reinterpret_cast<int64_t*>(red);      // setup only: 18 warp totals

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&d_full[i], 2);      // the MMAs, and the issuer's own arrival (see there)
      mbar_init(&d_empty[i], 8);
    }
    for (int i = 0; i < kSegDepth; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 17);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&red_full[i], 4);
    mbar_init(fin, 1);
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
  // ---- this CTA's range of units: [W c / G, W (c + 1) / G), and the request it starts in
  int64_t total = 0, lo = 0, hi = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kIxThreads) {
      const int b = b0 + tid;
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
      for (int w = 0; w < kIxThreads / 32; ++w) {
        const int64_t v = part[w];
        if (w < warp) base += v;
        all += v;
      }
      if (pass == 1) {
        const int64_t first = base + inc - u;
        if (first <= lo && lo < first + u && lo < hi) {
          start[0] = b;
          start[1] = lo - first;
        }
      }
      before += all;
    }
    if (pass == 0) {
      total = before;
      lo = total / gridDim.x * blockIdx.x + min(total % gridDim.x, static_cast<int64_t>(blockIdx.x));
      hi = lo + total / gridDim.x + (blockIdx.x < total % gridDim.x ? 1 : 0);
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
      // Pages of the slices j SP .. (j + TG) SP - 1, one per lane, looked up a group of TG tiles ahead;
      // a lane then issues its own slice's copies when its tile comes.
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
        // Tile n - S's MMAs are done, so the accumulators of the stage two before its own had been
        // read: with at most 4 tiles a stage, the scales of tile n - S - 12 = n - SC are free.
        if (tile >= S && !wait_all(&k_empty[slot], kc.par ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          bad[sslot] = (bad_m >> (in * SP)) & SM;
          mbar_arrive_expect_tx(&k_full[slot], C::kTileBytes + (F == kFP8 ? __popc((good_m >> (in * SP)) & SM) * BR * 4 : 0));
        }
        __syncwarp();
        if (lane / SP == in) {
          const int row = (lane - in * SP) * BR, z = cur >= 0 ? cur : p.num_blocks;
#pragma unroll
          for (int h = 0; h < HV; ++h)
            tma_load_3d(ring + slot * C::kTileBytes + h * 128 * 128 + row * 128, &tm_k, 128 * h, cy, z, &k_full[slot]);
          if (F == kFP8 && cur >= 0)
            bulk_g2s(scales + sslot * 128 + row, p.key_scales + z * p.ks_stride + cy, BR * 4, &k_full[slot]);
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
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one elected lane issues: addresses and descriptors then stay
    // warp-uniform (from a single-lane branch every operand of an MMA is moved to a uniform register
    // first, and this warp, which shares its scheduler with four busy ones, set the kernel's pace).
    const bool leader = elect_one();
    const uint32_t hi_desc = static_cast<uint32_t>(smem_desc(0, 16, 1024, kSwizzle128B) >> 32);
    const uint32_t dK0 = static_cast<uint32_t>(smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B));
    const uint32_t dQ0 = static_cast<uint32_t>(smem_desc(smem_u32(qs), 16, 1024, kSwizzle128B));
    auto desc = [&](uint32_t lo) -> uint64_t { return static_cast<uint64_t>(hi_desc) << 32 | lo; };
    Cursor<S> kc;
    uint32_t stage = 0;
    bool ok = true;
    for (uint32_t ns = 0; ok; ++ns) {
      const uint32_t k = ns % kSegDepth, qb = ns % QB;
      if (!wait_all(&seg_full[k], (ns / kSegDepth) & 1, abort_flag)) break;
      const int nt = __shfl_sync(0xFFFFFFFFu, segs[k].nt, 0), nq = __shfl_sync(0xFFFFFFFFu, segs[k].nq, 0);
      if (leader) mbar_arrive(&seg_empty[k]);
      if (nt == 0) break;
      if (!wait_all(&q_full[qb], (ns / QB) & 1, abort_flag)) break;
      const int n = (nq * HP + 15) & ~15;      // columns: a multiple of 16
      const int G = stage_tiles(nq * HP), gcols = kIxCols / G;
      const uint32_t idesc = F == kBF16 ? idesc_f16(128, n, 1, 1, 0, 0) : idesc_e4m3(128, n, 0, 0);
      const uint32_t dQ = dQ0 + qb * (C::kQBytes >> 4);
      for (int t = 0; ok && t < nt; t += G, ++stage) {
        const uint32_t buf = stage & 1;
        const int g1 = min(G, nt - t);
        if (stage >= 2 && !wait_all(&d_empty[buf], ((stage >> 1) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        for (int g = 0; g < g1; ++g) {
          if (!wait_all(&k_full[kc.slot], kc.par, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dK = dK0 + static_cast<uint32_t>(kc.slot) * (C::kTileBytes >> 4);
          const uint32_t d = tmem + buf * kIxCols + g * gcols;
          if (leader) {
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
          }
          kc.step();
        }
        if (leader) {
          mma_commit(&d_full[buf]);
          // the scales and bad-page masks that came with the key tiles reach the epilogue by this
          // thread's release (it has seen k_full)
          mbar_arrive(&d_full[buf]);
          if (t + G >= nt) mma_commit(&q_empty[qb]);
        }
      }
    }
    if (leader) {      // no product is in flight when the accumulators are freed
      volatile int no_abort[2] = {0, 0};
      mma_commit(fin);
      mbar_wait(fin, 0, no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    // Two sets of two groups: a set takes every second stage (one accumulator buffer), so that one
    // set's waits hide behind the other's work; a group takes two 64-column slices of the buffer.
    const int quad = warp & 3, group = (warp - 2) >> 2, set = group >> 1;
    // A thread's keys and columns: a 16 x 256-bit load gives lane 4 a + b the columns 2 b, 2 b + 1 of
    // every 8 for the keys a and a + 8, so its weights of 64 columns are 16 registers (a lane that had
    // one key and all columns would need them all, and reading them from shared memory for every
    // tile took twice the time of the products).  The four lanes of a key then exchange
    // their sums, and lane 4 a + b ends with key a + 8 b.
    const int la = lane >> 2, lb = lane & 3;
    const int key = 32 * quad + la + 8 * lb;
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16) + set * kIxCols + (group & 1) * 128;
    float* red_g = red + (group * 2 * 4 + quad) * 8;          // slice j at + 32 j
    const bool padded = p.Hi < HP;
    const bool early = !padded && p.block_tokens <= 32;       // nothing of the stage is needed after its columns
    const int bt = p.block_tokens, br_shift = 31 - __clz(p.BR), bt_shift = 31 - __clz(bt);
    const int cap = static_cast<int>(min(p.cap, static_cast<int64_t>(0x7FFFFFFF)));
    uint32_t stage = 0;                           // stages before the segment
    int sbase = 0;                                // scale slot of the segment's first tile
    uint32_t full_par = 0;                        // parity of the set's next stage
    uint32_t uses = 0;                            // block maxima exchanged through red
    bool ok = true;
    for (uint32_t ns = 0; ok; ++ns) {
      const uint32_t k = ns % kSegDepth;
      if (!wait_all(&seg_full[k], (ns / kSegDepth) & 1, abort_flag)) break;
      const Segment sg = segs[k];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[k]);
      if (sg.nt == 0) break;
      // tile of a stage and queries of this group's two slices
      const int G = stage_tiles(sg.nq * HP), per = 4 / G;
      int g[2] = {}, q0[2] = {}, nq[2] = {};
      int lim[2] = {};                            // keys from the thread's first one that its first query sees
      float* row[2] = {};                         // where its first score goes
      auto weight = [&](int j, int c) -> float {  // 0 for padded heads and queries
        const int q = c / HP, h = c % HP;
        return q < nq[j] && h < p.Hi ? __ldg(p.weights + static_cast<int64_t>(sg.t0 + q0[j] + q) * p.w_stride + h) : 0.f;
      };
      uint64_t w[2][8];                           // of the slices' columns 8 c + 2 lb and the next
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int sl = (group & 1) * 2 + j;
        g[j] = sl / per;
        q0[j] = (sl % per) * QW;
        nq[j] = max(min(QW, sg.nq - q0[j]), 0);
        const int first = (sg.j0 + g[j]) * 128 + key;
        lim[j] = min(sg.vis0 + q0[j], cap) - first;
        row[j] = p.scores + static_cast<int64_t>(sg.t0 + q0[j]) * p.s_stride + (first >> bt_shift);
#pragma unroll
        for (int c = 0; c < 8; ++c) w[j][c] = pack2(weight(j, 8 * c + 2 * lb), weight(j, 8 * c + 2 * lb + 1));
      }
      const int first_own = (stage & 1) == static_cast<uint32_t>(set) ? 0 : G;
      int ss = sbase + first_own;                 // scale slot of the stage's first tile
      if (ss >= SC) ss -= SC;
      for (int t = first_own; t < sg.nt; t += 2 * G) {
        const bool has0 = nq[0] > 0 && t + g[0] < sg.nt, has1 = nq[1] > 0 && t + g[1] < sg.nt;      // has1 implies has0
        if (!wait_all(&d_full[set], full_par, abort_flag)) {
          ok = false;
          break;
        }
        full_par ^= 1u;
        const int s0 = ss;
        ss += 2 * G;
        if (ss >= SC) ss -= SC;
        tc_fence_after();
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[set]);
        };
        auto slot_of = [&](int j) -> int {
          const int s = s0 + g[j];
          return s >= SC ? s - SC : s;
        };
        if (!has0) {
          release();
          continue;
        }
        // the keys' scales and bad pages, read before the release (their slots are reused after it)
        const uint32_t bm[2] = {bad[slot_of(0)], has1 ? bad[slot_of(1)] : 0u};
        float ks[2];
        if (F == kFP8) {
          ks[0] = scales[slot_of(0) * 128 + key];
          ks[1] = has1 ? scales[slot_of(1) * 128 + key] : 0.f;
        }
        // Sums of the slices.  Load u of a slice: keys 16 (u / 2) .. + 15 of the warp's 32, columns
        // 32 (u % 2) .. + 31; the next load is under way meanwhile.
        float v[2][QW];
        auto load = [&](int j, int u, float (&x)[16]) {
          tmem_ld_16x256(tl + 64 * j + 32 * (u & 1) + (static_cast<uint32_t>(16 * (u >> 1)) << 16), x);
        };
        auto slice = [&](int j, bool more) {      // more: another slice follows
          float y[4][QW];                         // keys la + 8 i
          uint64_t acc[2][QW];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float d[16];
            load(j, u, d);
            tmem_ld_wait();
            if (u == 3 && !more && early) release();                          // everything is in registers
#pragma unroll
            for (int c = 0; c < 4; ++c) {         // 8 columns
              const int q = (32 * (u & 1) + 8 * c) / HP;
              const bool start = (32 * (u & 1) + 8 * c) % HP == 0;
              const float* x = d + 4 * c;
              const uint64_t ww = w[j][4 * (u & 1) + c];
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
            v[j][q] = (o ? z1 : z0) + __shfl_xor_sync(0xFFFFFFFFu, o ? z0 : z1, 1);
          }
        };
        slice(0, has1);
        if (has1) slice(1, false);
        const bool exchange = bt > 32;
        // a key with infinities or NaN meets the zeros of the padded heads: sum the heads alone
        if (padded) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j == 1 && !has1) break;
#pragma unroll
            for (int q = 0; q < QW; ++q) {
              if (!__any_sync(0xFFFFFFFFu, v[j][q] != v[j][q])) continue;
              float s = 0.f;
#pragma unroll 1
              for (int h = 0; h < p.Hi; ++h) {
                uint32_t e;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(e) : "r"(tl + 64 * j + q * HP + h));
                tmem_ld_wait();
                s = fmaf(max_nan(__uint_as_float(e), 0.f), weight(j, q * HP + h), s);
              }
              v[j][q] = __shfl_sync(0xFFFFFFFFu, s, la + 8 * lb);
            }
          }
        }
        if (F == kFP8) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < QW; ++q) v[j][q] *= ks[j];
        }
        if (bm[0] | bm[1]) {      // tokens of bad pages
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if ((bm[j] >> (key >> br_shift)) & 1u)
#pragma unroll
              for (int q = 0; q < QW; ++q) v[j][q] = -CUDART_INF_F;
        }
        if (!exchange && !early) release();
        const int off = t * 128;
        if (bt == 1) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j == 1 && !has1) break;
            if (QW == 1) {
              if (off < lim[j]) row[j][off] = v[j][0];
            } else {
              float* r = row[j] + off;
#pragma unroll
              for (int q = 0; q < QW; ++q, r += p.s_stride)
                if (q < nq[j] && off < min(lim[j] + q, cap - sg.j0 * 128 - g[j] * 128 - key)) *r = v[j][q];
            }
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j == 1 && !has1) break;
          float* r = row[j] + (off >> bt_shift);
          const int edge = cap - sg.j0 * 128 - g[j] * 128 - key;
#pragma unroll
          for (int q = 0; q < QW; ++q, r += p.s_stride) {
            if (q >= nq[j]) break;
            const bool seen = off < min(lim[j] + q, edge);
            float val = seen ? v[j][q] : -CUDART_INF_F;
            // over la and lb bit 0: 16 keys; over lb bit 1: 32
            val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 4));
            val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 8));
            val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 16));
            val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 1));
            if (bt > 16) val = max_nan(val, __shfl_xor_sync(0xFFFFFFFFu, val, 2));
            if (!exchange) {
              if ((key & (bt - 1)) == 0 && seen) *r = val;
            } else if (lane == 0) {
              red_g[32 * j + q] = val;
            }
          }
        }
        if (exchange) {       // blocks of 64 or 128 keys: two or four warps of the group
          if (lane == 0) mbar_arrive(&red_full[group]);
          const uint32_t par = uses++ & 1u;
          const int wb = bt >> 5;                 // warps of a block; its first one joins them
          if ((quad & (wb - 1)) == 0) {
            if (!wait_all(&red_full[group], par, abort_flag)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (j == 1 && !has1) break;
              const int p0 = (sg.j0 + t + g[j]) * 128 + 32 * quad;
              if (lane < nq[j] && p0 < min(sg.vis0 + q0[j] + lane, cap)) {
                float mx = red_g[32 * j + lane];
                for (int o = 1; o < wb; ++o) mx = max_nan(mx, red_g[32 * j + 8 * o + lane]);
                p.scores[static_cast<int64_t>(sg.t0 + q0[j] + lane) * p.s_stride + (p0 >> bt_shift)] = mx;
              }
            }
          }
          // red is free with the buffer: written again only for the stage that next uses it
          release();
        }
      }
      stage += (sg.nt + G - 1) / G;
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
  static bool configured[64] = {};
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
