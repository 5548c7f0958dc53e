// Decode kernel instantiations for the mxfp4 cache.
#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

// The joined results of requests that several runs share: out = sum_i e^{lse_i - lse} O_i over the request's parts, and zeros
// for requests without keys.  Grid (rows * H, 4): a CTA has 128 of a row and head's 512 values.
struct Fp4MergeParams {
  const float* part_o;
  const float* part_lse;
  const int64_t* first;
  const int32_t* seq_lens;
  int B, q_len, H, W;
  uint8_t* out;
  int64_t o_s0b, o_s1b;
  float* lse;
};

__global__ void __launch_bounds__(128) mla_fp4_merge_kernel(const __grid_constant__ Fp4MergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t rh = blockIdx.x;
  const int row = static_cast<int>(rh / p.H), h = static_cast<int>(rh % p.H), b = row / p.q_len;
  const int tid = threadIdx.x, d = blockIdx.y * 128 + tid;
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out + row * p.o_s0b + h * p.o_s1b) + d;
  const int L = p.seq_lens[b];
  if (L <= 0) {
    *dst = __float2bfloat16_rn(0.f);
    if (p.lse && d == 0) p.lse[rh] = -CUDART_INF_F;
    return;
  }
  const int64_t run = p.first[p.B], t0 = p.first[b], t1 = t0 + (static_cast<int64_t>(L) + kTile - 1) / kTile;
  const int w0 = static_cast<int>(t0 / run), n = static_cast<int>((t1 - 1) / run) - w0 + 1;
  if (n == 1) return;      // written by the run that has all of it
  // part i is slot 2 (w0 + i), the first one 2 w0 + 1
  __shared__ float wt[128];
  __shared__ float red[4];
  const int cols = p.q_len * p.H, c = (row % p.q_len) * p.H + h;
  auto at = [&](int i) -> int64_t { return (2 * static_cast<int64_t>(w0 + i) + (i == 0 ? 1 : 0)) * cols + c; };
  const int lane = tid & 31, warp = tid >> 5;
  float m = -CUDART_INF_F;
  for (int i = tid; i < n; i += 128) m = fmaxf(m, p.part_lse[at(i)]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float mu = m == -CUDART_INF_F ? 0.f : m;
  float acc = 0.f, sum = 0.f;
  for (int i0 = 0; i0 < n; i0 += 128) {
    __syncthreads();
    wt[tid] = i0 + tid < n ? expf(p.part_lse[at(i0 + tid)] - mu) : 0.f;      // (a part's NaN goes on)
    __syncthreads();
    const int k = min(n - i0, 128);
    for (int i = 0; i < k; i += 8) {
      float o[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = i + y < k ? p.part_o[at(i0 + i + y) * kLora + d] : 0.f;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        if (i + y >= k) break;
        const float x = wt[i + y];
        sum += x;
        if (x != 0.f) acc = fmaf(x, o[y], acc);
      }
    }
  }
  *dst = __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
  if (p.lse && d == 0) p.lse[rh] = sum == 0.f ? -CUDART_INF_F : mu + logf(sum);
}

template <int NQ>
cudaError_t launch_nq(const Fp4Params& p, int grid, cudaStream_t stream) {
  using C = Fp4Cfg<NQ>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mla_fp4_kernel<NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_pdl(mla_fp4_kernel<NQ>, dim3(grid), dim3(C::kThreads), C::kAlloc, stream, p);
}

}  // namespace

cudaError_t launch_fp4_paged(int nq, const Fp4Params& p, cudaStream_t stream) {
  return nq == 16 ? launch_nq<16>(p, p.W * p.G, stream) : launch_nq<32>(p, p.W * p.G, stream);
}

cudaError_t launch_fp4_merge(const Fp4Params& p, cudaStream_t stream) {
  const Fp4MergeParams m{p.part_o, p.part_lse, p.first, p.seq_lens, p.B, p.q_len, p.H, p.W, p.out, p.o_s0b, p.o_s1b, p.lse};
  const int64_t n = static_cast<int64_t>(p.B) * p.cols;
  return launch_pdl(mla_fp4_merge_kernel, dim3(static_cast<unsigned>(n), 4), dim3(128), 0, stream, m);
}

}  // namespace mla

#ifdef MLA_TIMELINE
extern "C" __attribute__((visibility("default"))) int mla_debug_timeline_fp4(void* events, void* counts) {
  cudaMemcpyFromSymbol(events, mla::g_tl, sizeof(mla::g_tl));
  cudaMemcpyFromSymbol(counts, mla::g_tl_n, sizeof(mla::g_tl_n));
  const int zero[mla::kTlCtas][mla::kTlRoles] = {};
  return cudaMemcpyToSymbol(mla::g_tl_n, zero, sizeof(zero)) == cudaSuccess ? 0 : -3;
}
#endif
