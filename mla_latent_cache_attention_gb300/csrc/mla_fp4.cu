// Decode kernel instantiations for the mxfp4 cache.
#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

// The joined results of requests that several runs share: out = sum_i e^{lse_i - lse} O_i over the request's parts.  Grid
// (query columns, min(B, W)): CTA (c, y) joins column c of the y-th such request, if there are as many.
// kJoin: loads of a thread on their way at once, by fours as there are parts.  32 where the runs are many to a request, 8 else
// (registers, and so CTAs an SM): one request of 131072 keys 35.7 against 53.2 us with its decode, 128 of 8k to 32k keys of
// 96 heads 963 against 940 (with two terms a weight).
template <int kJoin>
__global__ void __launch_bounds__(256) mla_fp4_merge_kernel(const __grid_constant__ Fp4Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int found[8], mine[3];
  int w0 = -1, n = 0, left = blockIdx.y;      // requests before this one
  int64_t b = -1;
  for (int i0 = 0; i0 < p.W; i0 += 256) {
    const int2 span = i0 + tid < p.W ? p.span[i0 + tid] : make_int2(-1, 0);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, span.x >= 0);
    if (lane == 0) found[warp] = __popc(some);
    __syncthreads();
    int before = __popc(some & ((1u << lane) - 1u)), all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < warp) before += found[i];
      all += found[i];
    }
    if (span.x >= 0 && before == left) mine[0] = i0 + tid, mine[1] = span.x, mine[2] = span.y;
    __syncthreads();
    if (left < all) {
      w0 = mine[0], b = mine[1], n = mine[2];
      break;
    }
    left -= all;
  }
  if (w0 < 0) return;
  // part i is slot 2 (w0 + i), the first one 2 w0 + 1
  auto at = [&](int i) -> int64_t { return (2 * static_cast<int64_t>(w0 + i) + (i == 0 ? 1 : 0)) * p.cols + c; };
  __shared__ float wt[256];
  __shared__ float red[8];
  float2 o[kJoin];
  auto load = [&](int i, int k) {
#pragma unroll
    for (int y = 0; y < kJoin; ++y) {
      if (y % 4 == 0 && i + y >= k) break;
      o[y] = i + y < k ? reinterpret_cast<const float2*>(p.part_o + at(i + y) * kLora)[tid] : make_float2(0.f, 0.f);
    }
  };
  load(0, n);      // on their way before the weights are known
  float m = -CUDART_INF_F;
  for (int i = tid; i < n; i += 256) m = fmaxf(m, p.part_lse[at(i)]);
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
  if (lane == 0) red[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  const float mu = m == -CUDART_INF_F ? 0.f : m;
  float2 acc = make_float2(0.f, 0.f);
  float sum = 0.f;
  for (int i0 = 0; i0 < n; i0 += 256) {
    __syncthreads();
    wt[tid] = i0 + tid < n ? expf(p.part_lse[at(i0 + tid)] - mu) : 0.f;      // (a part's NaN goes on)
    __syncthreads();
    const int k = min(n - i0, 256);
    for (int i = 0; i < k; i += kJoin) {
      if (i0 + i > 0) load(i0 + i, n);
#pragma unroll
      for (int y = 0; y < kJoin; ++y) {
        if (y % 4 == 0 && i + y >= k) break;
        const float x = i + y < k ? wt[i + y] : 0.f;
        sum += x;
        if (x != 0.f) {
          acc.x = fmaf(x, o[y].x, acc.x);
          acc.y = fmaf(x, o[y].y, acc.y);
        }
      }
    }
  }
  const int64_t row = b * p.q_len + c / p.H;
  const int h = c % p.H;
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out + row * p.o_s0b + h * p.o_s1b) + 2 * tid;
  dst[0] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc.x / sum);
  dst[1] = __float2bfloat16_rn(sum == 0.f ? 0.f : acc.y / sum);
  if (p.lse && tid == 0) p.lse[row * p.H + h] = sum == 0.f ? -CUDART_INF_F : mu + logf(sum);
}

template <int NQ>
cudaError_t launch_nq(const Fp4Params& p, cudaStream_t stream) {
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
  return launch_pdl(mla_fp4_kernel<NQ>, dim3(p.G, p.W), dim3(C::kThreads), C::kAlloc, stream, p);
}

}  // namespace

cudaError_t launch_fp4_paged(int nq, const Fp4Params& p, cudaStream_t stream) {
  return nq == 16 ? launch_nq<16>(p, stream) : nq == 32 ? launch_nq<32>(p, stream) : nq == 48 ? launch_nq<48>(p, stream) : launch_nq<64>(p, stream);
}

cudaError_t launch_fp4_merge(const Fp4Params& p, cudaStream_t stream) {
  return launch_pdl(p.W / 8 >= p.B ? mla_fp4_merge_kernel<32> : mla_fp4_merge_kernel<8>, dim3(p.cols, p.B < p.W ? p.B : p.W), dim3(256), 0, stream, p);
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
