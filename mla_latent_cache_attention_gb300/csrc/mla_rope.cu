// mla_rope.cu -- rotary positions of queries and keys in one launch, and the table of cosines and sines.
//
// Pair (a, b) of a head at position p turns by the angle of its frequency: a' = a c - b s, b' = b c + a s, with c and s
// from the fp32 table and fp32 arithmetic (one product rounded before the fused multiply-add, as in the fused
// epilogues), rounded once to the tensor's type.  The inverse takes -s: the transposed rotation, which is the rotation's
// gradient.
//
// Bound by memory: every value is read and written once.  A CTA takes a token, or its queries or keys where their heads differ
// in shape; a thread keeps one place in the head (a 16-byte piece, in the half layout one of either half) for all the
// heads it serves, so that its cosines and sines are loaded once, behind its values.
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

// Row of the table for token t.
__device__ __forceinline__ int64_t row(const RopeParams& p, int64_t t) {
  const int64_t pos = p.positions[t];
  return pos < 0 ? 0 : pos >= p.max_position ? p.max_position - 1 : pos;
}

// The units of a head: first the rotated ones, then the copied ones (none in place).  W values (16 bytes) a piece;
// interleaved: R / W pieces of W / 2 pairs; half: R / (2 W) units of a piece of either half; copied: (D - R) / W pieces.
template <int kType, bool kHalf, bool kCopy, bool kStream>
__device__ __forceinline__ void rope_tensor(const RopeTensor& x, const RopeTensor& more, const RopeParams& p, int64_t t) {
  using E = Elem<kType>;
  using T = typename E::T;
  constexpr int S = sizeof(T), W = 16 / S, kPairs = kHalf ? W : W / 2;
  struct alignas(16) Piece {
    T v[W];
  };
  const int heads = blockDim.x / x.units;                    // at once
  const int h0 = threadIdx.x / x.units, u = threadIdx.x % x.units, all = x.H + more.H;
  if (h0 >= heads) return;
  const int R = p.R, turned = kHalf ? R / (2 * W) : R / W;
  auto in = [&](int h) -> const uint8_t* { return h < x.H ? x.in + t * x.i_s0 + h * x.i_s1 : more.in + t * more.i_s0 + (h - x.H) * more.i_s1; };
  auto out = [&](int h) -> uint8_t* { return h < x.H ? x.out + t * x.o_s0 + h * x.o_s1 : more.out + t * more.o_s0 + (h - x.H) * more.o_s1; };
  // A head at a time: two or three on their way cost the registers of more CTAs (8191 tokens of 72 heads of 128: 78 and
  // 94 us against 71).  Streams of more than the L2 pass it by both ways: 53 us, by the stores alone 66.
  auto load = [&](const uint8_t* at) -> Piece {
    const float4* from = reinterpret_cast<const float4*>(at);
    const float4 v = kStream ? __ldcs(from) : *from;
    return *reinterpret_cast<const Piece*>(&v);
  };
  auto store = [&](uint8_t* at, const Piece& v) {
    float4* to = reinterpret_cast<float4*>(at);
    if constexpr (kStream)
      __stcs(to, *reinterpret_cast<const float4*>(&v));
    else
      *to = *reinterpret_cast<const float4*>(&v);
  };
  if (kCopy && u >= turned) {
    const int c = (u - turned) * W, d = (c < x.at ? c : c + R) * S;
    for (int h = h0; h < all; h += heads) store(out(h) + d, load(in(h) + d));
    return;
  }
  float c[kPairs], s[kPairs];
  bool have = false;                    // the table's values are loaded: after the first head's loads are on their way
  const int d = (x.at + u * W) * S, e = d + R / 2 * S;
  for (int h = h0; h < all; h += heads) {
    Piece a = load(in(h) + d), b;
    if constexpr (kHalf) b = load(in(h) + e);
    if (!have) {
      const float* cs = p.cos_sin + row(p, t) * R;
#pragma unroll
      for (int i = 0; i < kPairs; i += kPairs < 4 ? 2 : 4) {      // (the table's rows are aligned to 16 bytes where kVec is)
        if constexpr (kPairs >= 4) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + u * kPairs + i)), s4 = __ldg(reinterpret_cast<const float4*>(cs + R / 2 + u * kPairs + i));
          c[i] = c4.x, c[i + 1] = c4.y, c[i + 2] = c4.z, c[i + 3] = c4.w;
          s[i] = s4.x, s[i + 1] = s4.y, s[i + 2] = s4.z, s[i + 3] = s4.w;
        } else {
          const float2 c2 = __ldg(reinterpret_cast<const float2*>(cs + u * kPairs + i)), s2 = __ldg(reinterpret_cast<const float2*>(cs + R / 2 + u * kPairs + i));
          c[i] = c2.x, c[i + 1] = c2.y;
          s[i] = s2.x, s[i + 1] = s2.y;
        }
      }
      if (p.inverse) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s[i] = -s[i];
      }
      have = true;
    }
    if constexpr (kHalf) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float y0 = E::get(a.v[j]), y1 = E::get(b.v[j]);
        turn(y0, y1, c[j], s[j]);
        a.v[j] = E::put(y0);
        b.v[j] = E::put(y1);
      }
      store(out(h) + e, b);
    } else {
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        float y0 = E::get(a.v[2 * j]), y1 = E::get(a.v[2 * j + 1]);
        turn(y0, y1, c[j], s[j]);
        a.v[2 * j] = E::put(y0);
        a.v[2 * j + 1] = E::put(y1);
      }
    }
    store(out(h) + d, a);
  }
}

// Rows, widths or offsets that are not whole pieces: a pair or a copied value a thread.
template <int kType, bool kHalf, bool kCopy>
__device__ __forceinline__ void rope_scalar(const RopeTensor& x, const RopeParams& p, int64_t t) {
  using E = Elem<kType>;
  using T = typename E::T;
  const float* cs = p.cos_sin + row(p, t) * p.R;
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

// (40 registers a thread: with the 64 of two CTAs of 512 the prefill above takes 60 us, with 32 they spill: 99 us)
template <int kType, bool kHalf, bool kVec, bool kCopy, bool kStream>
__global__ void __launch_bounds__(512, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  const int64_t t = blockIdx.x;
  if constexpr (kVec) {
    const RopeTensor none{};
    if (p.joint)
      rope_tensor<kType, kHalf, kCopy, kStream>(p.x[0], p.x[1], p, t);
    else
      rope_tensor<kType, kHalf, kCopy, kStream>(p.x[blockIdx.y], none, p, t);
  } else {
    rope_scalar<kType, kHalf, kCopy>(p.x[blockIdx.y], p, t);
  }
  if (blockIdx.y > 0) return;
  if (threadIdx.x == 0) {
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_position) set_device_error(p.err, 8u);
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
  for (RopeTensor& x : p.x) x.units = (vec && !kHalf ? p.R / W : p.R / (2 * W)) + (copy ? (x.D - p.R) / W : 0);
  const bool two = p.x[1].H > 0;
  // heads of the same shape are one run of heads; else the keys are CTAs of their own
  p.joint = vec && two && p.x[0].D == p.x[1].D && p.x[0].at == p.x[1].at;
  // Tensors larger than the L2 (129 MB) keep nothing there for who comes next.
  int64_t bytes = 0;
  for (const RopeTensor& x : p.x) bytes += static_cast<int64_t>(p.T) * x.H * (copy ? x.D : p.R) * (kType == 2 ? 4 : 2);
  const bool stream_by = bytes > (64ll << 20);
  int threads = 64;
  for (int i = 0; i < (two && !p.joint ? 2 : 1); ++i) {
    const int units = p.x[i].units, heads = p.x[i].H + (p.joint ? p.x[1].H : 0);
    // vec: two heads a thread where up to 512 threads can (a head has at most 256 units: D <= 1024); else a unit a thread
    const int at_once = vec ? (heads + 1) / 2 * units <= 512 ? (heads + 1) / 2 : 512 / units : heads;
    const int want = at_once * units < 256 || vec ? at_once * units : 256;
    if (want > threads) threads = want;
  }
  threads = (threads + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(p.T), two && !p.joint ? 2 : 1);
  if (vec && copy && stream_by)
    rope_kernel<kType, kHalf, true, true, true><<<grid, threads, 0, stream>>>(p);
  else if (vec && copy)
    rope_kernel<kType, kHalf, true, true, false><<<grid, threads, 0, stream>>>(p);
  else if (vec && stream_by)
    rope_kernel<kType, kHalf, true, false, true><<<grid, threads, 0, stream>>>(p);
  else if (vec)
    rope_kernel<kType, kHalf, true, false, false><<<grid, threads, 0, stream>>>(p);
  else if (copy)
    rope_kernel<kType, kHalf, false, true, false><<<grid, threads, 0, stream>>>(p);
  else
    rope_kernel<kType, kHalf, false, false, false><<<grid, threads, 0, stream>>>(p);
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
