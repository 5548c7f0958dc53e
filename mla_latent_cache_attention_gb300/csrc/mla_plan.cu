// mla_plan.cu -- the blocks and slots of a step, from the requests' lengths.
//
// With L_b the cached tokens of request b (0 where it is finished), n_b its new ones and s the block size, request b
// needs ceil((L_b + n_b) / s) - ceil(L_b / s) new blocks.  Exclusive sums over the requests say which blocks of the
// stack of free ones are whose and which rows of the step are whose; then every row's slot is a lookup.
//
// Latency counts: a decode step has a few hundred rows.  One CTA makes the sums, 1024 requests at a time, and does the
// rest as well where there is little of it; where many blocks may come back or many rows are written, the eight CTAs of
// a cluster make the same sums each and share the copies (256 requests, 32 of them finished with 1000 blocks each:
// 43 us with one CTA, whose warps copied a request's blocks one load at a time).
#include "mla_ptx.cuh"
#include "mla_step.h"

namespace mla {
namespace {

constexpr int kPlanThreads = kPlanKept, kPlanCtas = 8;
constexpr uint32_t kErrFree = 32u;      // MLA_DEVERR_FREE

struct Pair {
  int64_t a, b;
};

// Exclusive sums of two values over the CTA; the totals in `total`.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* ws, Pair& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t a = __shfl_up_sync(0xFFFFFFFFu, x.a, o), b = __shfl_up_sync(0xFFFFFFFFu, x.b, o);
    if (lane >= o) x.a += a, x.b += b;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Pair s = ws[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t a = __shfl_up_sync(0xFFFFFFFFu, s.a, o), b = __shfl_up_sync(0xFFFFFFFFu, s.b, o);
      if (lane >= o) s.a += a, s.b += b;
    }
    ws[lane] = s;
  }
  __syncthreads();
  total = ws[31];
  const Pair before = warp ? ws[warp - 1] : Pair{0, 0};
  __syncthreads();      // ws may be written again
  return Pair{before.a + x.a - v.a, before.b + x.b - v.b};
}

__device__ __forceinline__ int64_t blocks_of(int64_t tokens, int block_size) {
  return static_cast<int64_t>(static_cast<uint64_t>(tokens + block_size - 1) / static_cast<uint32_t>(block_size));
}

// The sums of up to 1024 requests, kept for the rows (more requests are looked up in the outputs).
struct Kept {
  int32_t cu[kPlanThreads + 1], len[kPlanThreads];
  uint8_t served[kPlanThreads];
};

// Positions and slots of rows r0, r0 + step, ...
template <bool kKept>
__device__ __forceinline__ void write_rows(const PlanParams& p, const Kept& kept, int r0, int step) {
  const int32_t* cu = kKept ? kept.cu : p.cu;
  const int total = cu[p.B];
  for (int r = r0; r < p.T; r += step) {
    int64_t pos = 0, slot = -1;
    if (r < total) {
      int lo = 0, hi = p.B - 1;      // the last request b with cu[b] <= r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= r)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int c0 = cu[lo], len = kKept ? kept.len[lo] : p.seq_out[lo];
      if (kKept ? kept.served[lo] : p.served[lo]) {
        pos = static_cast<int64_t>(len) - (cu[lo + 1] - c0) + (r - c0);
        const uint32_t col = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.block_size);
        const int id = p.table[static_cast<int64_t>(lo) * p.t_stride + col];
        if (id >= 0) slot = static_cast<int64_t>(id) * p.block_size + (pos - static_cast<int64_t>(col) * p.block_size);
      } else {
        pos = static_cast<int64_t>(len) + (r - c0);
      }
    }
    p.positions[r] = pos;
    p.slots[r] = slot;
  }
}

// kCtas CTAs (a cluster), each with the same sums.  Every CTA reads the lengths and the count of free blocks before the
// first one writes them (they may be the same memory).
template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ Pair ws[32];
  __shared__ int64_t base[kPlanThreads];      // first place on the stack of a finished request's blocks
  __shared__ Kept kept;
  __shared__ unsigned long long taken;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = kCtas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  auto meet = [&]() {
    __syncwarp();
    if (kCtas > 1)
      cluster_sync();      // (releases and acquires the CTAs' writes to global memory)
    else
      __syncthreads();
  };
  if (tid == 0) taken = 0;
  int64_t free = min(max(static_cast<int64_t>(*p.num_free), int64_t(0)), p.capacity);
  uint32_t err = 0;
  // the blocks of finished requests go on top of the stack, in the order of the requests and of their tables: copied
  // as one run of entries, four loads of a thread on their way at once
  if (p.finished) {
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int64_t back = 0;
      if (b < p.B && p.finished[b]) back = min(blocks_of(max(p.seq_lens[b], 0), p.block_size), static_cast<int64_t>(p.cols));
      Pair total;
      base[tid] = block_scan(Pair{back, 0}, ws, total).a;
      __syncthreads();
      const int64_t n = min(total.a, p.capacity - free);
      if (n < total.a) err |= kErrFree;
      const int last = min(kPlanThreads, p.B - b0) - 1;
      for (int64_t e0 = static_cast<int64_t>(rank) * kPlanThreads + tid; e0 < n; e0 += 4 * kCtas * kPlanThreads) {
        int32_t id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t e = e0 + static_cast<int64_t>(u) * kCtas * kPlanThreads;
          if (e >= n) continue;
          int lo = 0, hi = last;      // the last request whose run begins at or before e (those with none share its start)
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (base[mid] <= e)
              lo = mid;
            else
              hi = mid - 1;
          }
          id[u] = p.table[static_cast<int64_t>(b0 + lo) * p.t_stride + (e - base[lo])];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t e = e0 + static_cast<int64_t>(u) * kCtas * kPlanThreads;
          if (e < n) p.free_blocks[free + e] = id[u];
        }
      }
      __syncthreads();      // base may be written again
      free += n;
    }
    meet();      // written to the stack, and read from the finished rows, before blocks are taken
  }
  // every request takes what it needs from the top: in order, until the blocks or the rows run out
  int64_t rows = 0, wanted = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int64_t L = 0, n = 0, have = 0, need = 0;
    bool fits = true;
    if (b < p.B) {
      n = max(p.new_lens[b], 0);
      if (!(p.finished && p.finished[b])) L = max(p.seq_lens[b], 0);
      have = blocks_of(L, p.block_size);
      need = blocks_of(L + n, p.block_size) - have;
      fits = have + need <= p.cols && L + n <= 0x7FFFFFFF;
      if (!fits) need = 0;
    }
    Pair total;
    const Pair x = block_scan(Pair{n, need}, ws, total);
    const int64_t r0 = rows + x.a, off = wanted + x.b;
    const bool served = fits && (need == 0 || off + need <= free) && r0 + n <= p.T;
    // the chunk's lengths have been read by every CTA (by this one: the barriers of the scan; by the others: the next
    // chunk's are other requests')
    if (kCtas > 1) cluster_sync();
    if (b < p.B) {
      const int32_t at = static_cast<int32_t>(min(r0, static_cast<int64_t>(p.T))), end = static_cast<int32_t>(min(r0 + n, static_cast<int64_t>(p.T)));
      const int32_t len = static_cast<int32_t>(served ? L + n : L);
      kept.cu[tid] = at;      // of use where all requests fit one chunk
      kept.len[tid] = len;
      kept.served[tid] = served;
      if (b == p.B - 1) kept.cu[tid + 1] = end;
      if (rank == 0) {
        p.cu[b] = at;
        if (b == p.B - 1) p.cu[p.B] = end;
        p.seq_out[b] = len;
        if (p.served) p.served[b] = served;
        if (!served) err |= kErrFree;
      }
    }
    // new table entries: a warp has the requests of its lanes, one after the other, every CTA its share of them
    const int64_t take = served ? need : 0;
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, take > 0); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int64_t k = __shfl_sync(0xFFFFFFFFu, take, src), first = free - 1 - __shfl_sync(0xFFFFFFFFu, off, src);
      int32_t* row = p.table + static_cast<int64_t>(b - lane + src) * p.t_stride + __shfl_sync(0xFFFFFFFFu, have, src);
      if (src % kCtas != rank) continue;
      for (int64_t i = lane; i < k; i += 32) row[i] = p.free_blocks[first - i];
    }
    if (take > 0) atomicMax(&taken, static_cast<unsigned long long>(off + take));
    rows += total.a;
    wanted += total.b;
  }
  meet();      // table entries and outputs are written
  if (rank == 0 && tid == 0) *p.num_free_out = static_cast<int32_t>(free - static_cast<int64_t>(taken));
  err = __reduce_or_sync(0xFFFFFFFFu, err);
  if (lane == 0 && err) set_device_error(p.err, err);
  if (p.B <= kPlanThreads)
    write_rows<true>(p, kept, rank * kPlanThreads + tid, kCtas * kPlanThreads);
  else
    write_rows<false>(p, kept, rank * kPlanThreads + tid, kCtas * kPlanThreads);
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  // The cluster costs a small step 2 us.  How many blocks come back is known to the GPU alone: what the table can hold counts.
  const bool small = p.T <= 2 * kPlanThreads && (!p.finished || static_cast<int64_t>(p.B) * p.cols <= 8 * kPlanThreads);
  if (small) {
    plan_kernel<1><<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel<kPlanCtas>, p);
}

}  // namespace mla
