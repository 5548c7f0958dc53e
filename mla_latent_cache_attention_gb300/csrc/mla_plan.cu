// mla_plan.cu -- the blocks and slots of a step, from the requests' lengths.
//
// With L_b the cached tokens of request b (0 where it is finished), n_b its new ones and s the block size, request b
// needs ceil((L_b + n_b) / s) - ceil(L_b / s) new blocks.  Exclusive sums over the requests say which blocks of the
// stack of free ones are whose and which rows of the step are whose; then every row's slot is a lookup.
//
// Latency counts: a decode step has a few hundred rows.  The sums, the stack and the new table entries are the work of
// one CTA, which takes its requests 1024 at a time; it also writes the rows of a small step.  The rows of a larger
// one are written by a second kernel, launched as a programmatic dependent.
#include "mla_internal.h"
#include "mla_ptx.cuh"
#include "mla_step.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024, kOneCtaRows = 4096;
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

// Positions and slots of rows r0, r0 + step, ... from cu, seq_out, served and the table.
__device__ __forceinline__ void write_rows(const PlanParams& p, int r0, int step) {
  const int total = p.cu[p.B];
  for (int r = r0; r < p.T; r += step) {
    int64_t pos = 0, slot = -1;
    if (r < total) {
      int lo = 0, hi = p.B - 1;      // the last request b with cu[b] <= r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= r)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int c0 = p.cu[lo], len = p.seq_out[lo];
      if (p.served[lo]) {
        pos = static_cast<int64_t>(len) - (p.cu[lo + 1] - c0) + (r - c0);
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

template <bool kRows>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ Pair ws[32];
  __shared__ unsigned long long taken;
  const int tid = threadIdx.x, lane = tid & 31;
  if (!kRows && tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) taken = 0;
  int64_t free = min(max(static_cast<int64_t>(*p.num_free), int64_t(0)), p.capacity);
  uint32_t err = 0;
  // the blocks of finished requests go on top of the stack, in the order of the requests and of their tables
  if (p.finished) {
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int64_t back = 0;
      if (b < p.B && p.finished[b]) back = min(blocks_of(max(p.seq_lens[b], 0), p.block_size), static_cast<int64_t>(p.cols));
      Pair total;
      const int64_t base = free + block_scan(Pair{back, 0}, ws, total).a;
      for (uint32_t m = __ballot_sync(0xFFFFFFFFu, back > 0); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int64_t n = __shfl_sync(0xFFFFFFFFu, back, src), at = __shfl_sync(0xFFFFFFFFu, base, src);
        const int32_t* row = p.table + static_cast<int64_t>(b - lane + src) * p.t_stride;
        for (int64_t i = lane; i < n; i += 32) {
          if (at + i < p.capacity)
            p.free_blocks[at + i] = row[i];
          else
            err |= kErrFree;
        }
      }
      free = min(free + total.a, p.capacity);
    }
    __syncthreads();      // written to the stack, and read from the finished rows, before blocks are taken
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
    if (b < p.B) {
      p.cu[b] = static_cast<int32_t>(min(r0, static_cast<int64_t>(p.T)));
      if (b == p.B - 1) p.cu[p.B] = static_cast<int32_t>(min(r0 + n, static_cast<int64_t>(p.T)));
      p.seq_out[b] = static_cast<int32_t>(served ? L + n : L);
      p.served[b] = served;
      if (!served) err |= kErrFree;
    }
    const int64_t take = served ? need : 0;
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, take > 0); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int64_t k = __shfl_sync(0xFFFFFFFFu, take, src), first = free - 1 - __shfl_sync(0xFFFFFFFFu, off, src);
      int32_t* row = p.table + static_cast<int64_t>(b - lane + src) * p.t_stride + __shfl_sync(0xFFFFFFFFu, have, src);
      for (int64_t i = lane; i < k; i += 32) row[i] = p.free_blocks[first - i];
    }
    if (take > 0) atomicMax(&taken, static_cast<unsigned long long>(off + take));
    rows += total.a;
    wanted += total.b;
  }
  __syncthreads();
  if (tid == 0) *p.num_free_out = static_cast<int32_t>(free - static_cast<int64_t>(taken));
  err = __reduce_or_sync(0xFFFFFFFFu, err);
  if (lane == 0 && err) set_device_error(p.err, err);
  if (kRows) write_rows(p, tid, kPlanThreads);
}

__global__ void __launch_bounds__(256) plan_rows_kernel(const __grid_constant__ PlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  write_rows(p, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  if (p.T <= kOneCtaRows) {
    plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(plan_rows_kernel, dim3(static_cast<unsigned>((p.T + 255) / 256)), dim3(256), 0, stream, p);
}

}  // namespace mla
