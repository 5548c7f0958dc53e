// mla_rope.cu -- rotary positions of queries and keys in one launch, and the table of cosines and sines.
//
// Pair (a, b) of a head at position p turns by the angle of its frequency: a' = a c - b s, b' = b c + a s, with c and s
// from the fp32 table and fp32 arithmetic (one product rounded before the fused multiply-add, as in the fused
// epilogues), rounded once to the tensor's type.  The inverse takes -s: the transposed rotation, which is the rotation's
// gradient.
//
// Bound by memory: every value is read and written once.  A CTA takes a token; a thread keeps one place in the head (a
// 16-byte piece, in the half layout one of either half) for all the heads it serves, so that its cosines and
// sines are loaded once and stay in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_ptx.cuh"
#include "mla_step.h"

namespace mla {
namespace {

template <int kType>
struct Elem;
template <>
struct Elem<0> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<1> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<2> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fmaf_rn(x, c, -__fmul_rn(y, s));
  b = __fmaf_rn(y, c, __fmul_rn(x, s));
}

// The units of a head: first the rotated ones, then the copied ones (none in place).  W values (16 bytes) a piece;
// interleaved: R / W pieces of W / 2 pairs; half: R / (2 W) units of a piece of either half; copied: (D - R) / W pieces.
template <int kType, bool kHalf, bool kCopy>
__device__ __forceinline__ void rope_tensor(const RopeTensor& x, const RopeParams& p, int64_t t, const float* cs) {
  using E = Elem<kType>;
  using T = typename E::T;
  constexpr int S = sizeof(T), W = 16 / S, kPairs = kHalf ? W : W / 2;
  struct alignas(16) Piece {
    T v[W];
  };
  const int heads = blockDim.x / x.units;                    // at once
  const int h0 = threadIdx.x / x.units, u = threadIdx.x % x.units;
  if (h0 >= heads) return;
  const int R = p.R, turned = kHalf ? R / (2 * W) : R / W;
  const uint8_t* in = x.in + t * x.i_s0;
  uint8_t* out = x.out + t * x.o_s0;
  if (kCopy && u >= turned) {
    const int c = (u - turned) * W, d = (c < x.at ? c : c + R) * S;
#pragma unroll 4
    for (int h = h0; h < x.H; h += heads)
      *reinterpret_cast<Piece*>(out + h * x.o_s1 + d) = *reinterpret_cast<const Piece*>(in + h * x.i_s1 + d);
    return;
  }
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    c[i] = __ldg(cs + u * kPairs + i);
    s[i] = __ldg(cs + R / 2 + u * kPairs + i);
    if (p.inverse) s[i] = -s[i];
  }
  const int d = (x.at + u * W) * S, e = d + R / 2 * S;
#pragma unroll 4
  for (int h = h0; h < x.H; h += heads) {
    Piece a = *reinterpret_cast<const Piece*>(in + h * x.i_s1 + d);
    if constexpr (kHalf) {
      Piece b = *reinterpret_cast<const Piece*>(in + h * x.i_s1 + e);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float y0 = E::get(a.v[i]), y1 = E::get(b.v[i]);
        turn(y0, y1, c[i], s[i]);
        a.v[i] = E::put(y0);
        b.v[i] = E::put(y1);
      }
      *reinterpret_cast<Piece*>(out + h * x.o_s1 + e) = b;
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        float y0 = E::get(a.v[2 * i]), y1 = E::get(a.v[2 * i + 1]);
        turn(y0, y1, c[i], s[i]);
        a.v[2 * i] = E::put(y0);
        a.v[2 * i + 1] = E::put(y1);
      }
    }
    *reinterpret_cast<Piece*>(out + h * x.o_s1 + d) = a;
  }
}

// Rows, widths or offsets that are not whole pieces: a pair or a copied value a thread.
template <int kType, bool kHalf, bool kCopy>
__device__ __forceinline__ void rope_scalar(const RopeTensor& x, const RopeParams& p, int64_t t, const float* cs) {
  using E = Elem<kType>;
  using T = typename E::T;
  const int R = p.R, half = R / 2, units = half + (kCopy ? x.D - R : 0);
  for (int i = threadIdx.x; i < x.H * units; i += blockDim.x) {
    const int h = i / units, u = i - h * units;
    const T* in = reinterpret_cast<const T*>(x.in + t * x.i_s0 + h * x.i_s1);
    T* out = reinterpret_cast<T*>(x.out + t * x.o_s0 + h * x.o_s1);
    if (u >= half) {
      const int c = u - half, d = c < x.at ? c : c + R;
      out[d] = in[d];
      continue;
    }
    const int d = x.at + (kHalf ? u : 2 * u), e = d + (kHalf ? half : 1);
    float y0 = E::get(in[d]), y1 = E::get(in[e]);
    const float sn = __ldg(cs + half + u);
    turn(y0, y1, __ldg(cs + u), p.inverse ? -sn : sn);
    out[d] = E::put(y0);
    out[e] = E::put(y1);
  }
}

template <int kType, bool kHalf, bool kVec, bool kCopy>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeParams p) {
  const int64_t t = blockIdx.x;
  int64_t pos = p.positions[t];
  if (pos < 0 || pos >= p.max_position) {
    if (threadIdx.x == 0) set_device_error(p.err, 8u);
    pos = pos < 0 ? 0 : p.max_position - 1;
  }
  const float* cs = p.cos_sin + pos * p.R;
  for (int i = 0; i < 2; ++i) {
    if (p.x[i].H == 0) continue;
    if constexpr (kVec)
      rope_tensor<kType, kHalf, kCopy>(p.x[i], p, t, cs);
    else
      rope_scalar<kType, kHalf, kCopy>(p.x[i], p, t, cs);
  }
}

// Angles in 64 bits: at position 2^20 an fp32 angle is off by up to 0.06.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  const int half = p.R / 2;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.n * half) return;
  const int64_t pos = i / half;
  const int k = static_cast<int>(i - pos * half);
  double s, c;
  sincos(static_cast<double>(pos) * p.freq[k], &s, &c);
  p.out[pos * p.R + k] = static_cast<float>(c * p.scale);
  p.out[pos * p.R + half + k] = static_cast<float>(s * p.scale);
}

template <int kType, bool kHalf>
cudaError_t launch_t(bool vec, bool copy, RopeParams& p, cudaStream_t stream) {
  const int W = vec ? (kType == 2 ? 4 : 8) : 1;
  int most = 0, threads = 64;
  for (RopeTensor& x : p.x) {
    if (x.H == 0) continue;
    x.units = (vec && !kHalf ? p.R / W : p.R / (2 * W)) + (copy ? (x.D - p.R) / W : 0);
    most = x.H * x.units > most ? x.H * x.units : most;
    while (vec && threads < x.units) threads *= 2;      // at most 256: D <= 1024
  }
  while (threads < 256 && threads < most) threads *= 2;
  const dim3 grid(static_cast<unsigned>(p.T));
  if (vec && copy)
    rope_kernel<kType, kHalf, true, true><<<grid, threads, 0, stream>>>(p);
  else if (vec)
    rope_kernel<kType, kHalf, true, false><<<grid, threads, 0, stream>>>(p);
  else if (copy)
    rope_kernel<kType, kHalf, false, true><<<grid, threads, 0, stream>>>(p);
  else
    rope_kernel<kType, kHalf, false, false><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int type, bool half, bool vec, bool copy, RopeParams p, cudaStream_t stream) {
  if (type == 0) return half ? launch_t<0, true>(vec, copy, p, stream) : launch_t<0, false>(vec, copy, p, stream);
  if (type == 1) return half ? launch_t<1, true>(vec, copy, p, stream) : launch_t<1, false>(vec, copy, p, stream);
  return half ? launch_t<2, true>(vec, copy, p, stream) : launch_t<2, false>(vec, copy, p, stream);
}

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream) {
  const int64_t n = p.n * (p.R / 2);
  rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
