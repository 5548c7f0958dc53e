// Decode kernel instantiations for the mxfp4 cache.
#include "mla_fp4.cuh"
#include "mla_internal.h"

namespace mla {
namespace {

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

cudaError_t launch_fp4_paged(int nq, const Fp4Params& p, int grid, cudaStream_t stream) {
  return nq == 16 ? launch_nq<16>(p, grid, stream) : launch_nq<32>(p, grid, stream);
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
