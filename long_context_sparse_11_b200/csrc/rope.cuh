// Rotary positions (dsa_rope) and the angle arithmetic that the cache append shares.
//
// Pair i of the rotated dims turns by a = pos * inv_freq[i]; both are held in double and the angle is
// reduced to [-pi, pi] before its sine and cosine, so positions of 10^6 and more lose nothing (an fp32
// angle of 10^6 radians is off by 0.03).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace dsa {
namespace rope {

constexpr int MAX_PAIRS = 128;
constexpr int THREADS = 256;

struct Freqs {
  double f[MAX_PAIRS];
};

// Sine and cosine of pos * freq.  The reduction subtracts k * 2 pi in two parts (the double nearest to
// 2 pi and the rest), each in one fused step.
__device__ __forceinline__ void sin_cos(int32_t pos, double freq, double& s, double& c) {
  const double a = static_cast<double>(pos) * freq;
  const double k = rint(a * 0.15915494309189533577);
  double r = fma(-k, 6.283185307179586232, a);
  r = fma(-k, 2.4492935982947064e-16, r);
  sincos(r, &s, &c);
}

struct Params {
  const uint8_t* x;
  uint8_t* out;
  const int32_t* pos;
  int64_t x_tok, x_head, out_tok, out_head;  // strides in elements
  int32_t n_tokens, n_heads, dim, offset, rot;
  int32_t tok_per_cta, head_per_cta, head_groups;
  int32_t half;       // 1: pairs (i, i + rot / 2), 0: pairs (2i, 2i + 1)
  int32_t copy_rest;  // 1: the dims outside the rotated ones are copied (out is another tensor than x)
  double sin_sign;    // -1 turns the other way (the gradient)
  double mscale;
};

template <typename T>
struct Vec {
  static constexpr int N = 16 / static_cast<int>(sizeof(T));
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
union Pack {
  uint4 u;
  T t[Vec<T>::N];
};

// One CTA: tok_per_cta tokens x head_per_cta heads.  The tokens' sines and cosines are formed once, in shared
// memory; then one 16-byte vector (half layout: one of each half) per thread and step.  Bound by the tensor's
// bytes; each value is rounded once.
template <typename T>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ Params p,
                                                       const __grid_constant__ Freqs fr) {
  grid_dependency_sync();
  extern __shared__ float2 cs[];  // [tok_per_cta][rot / 2] (cos, sin), scaled
  constexpr int V = Vec<T>::N;
  const int32_t tg = static_cast<int32_t>(blockIdx.x / p.head_groups);
  const int32_t t0 = tg * p.tok_per_cta;
  const int32_t h0 = static_cast<int32_t>(blockIdx.x % p.head_groups) * p.head_per_cta;
  const int32_t nt = min(p.tok_per_cta, p.n_tokens - t0), nh = min(p.head_per_cta, p.n_heads - h0);
  const int32_t pairs = p.rot / 2;
  for (int32_t i = threadIdx.x; i < nt * pairs; i += THREADS) {
    double s, c;
    sin_cos(p.pos[t0 + i / pairs], fr.f[i % pairs], s, c);
    cs[i] = make_float2(static_cast<float>(c * p.mscale), static_cast<float>(s * p.mscale * p.sin_sign));
  }
  __syncthreads();
  const int32_t turn_units = p.half ? pairs / V : p.rot / V;
  const int32_t units = turn_units + (p.copy_rest ? (p.dim - p.rot) / V : 0);
  const int32_t n = nt * nh * units;
  for (int32_t i = threadIdx.x; i < n; i += THREADS) {
    const int32_t u = i % units, th = i / units;
    const int32_t t = th / nh, h = th % nh;
    const T* src = reinterpret_cast<const T*>(p.x) + (t0 + t) * p.x_tok + (h0 + h) * p.x_head;
    T* dst = reinterpret_cast<T*>(p.out) + (t0 + t) * p.out_tok + (h0 + h) * p.out_head;
    if (u >= turn_units) {
      int32_t d = (u - turn_units) * V;
      if (d >= p.offset) d += p.rot;
      *reinterpret_cast<uint4*>(dst + d) = *reinterpret_cast<const uint4*>(src + d);
      continue;
    }
    const float2* ct = cs + t * pairs;
    if (p.half) {
      const int32_t d = p.offset + u * V;
      Pack<T> a, b;
      a.u = *reinterpret_cast<const uint4*>(src + d);
      b.u = *reinterpret_cast<const uint4*>(src + d + pairs);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 w = ct[u * V + j];
        const float xa = to_f32(a.t[j]), xb = to_f32(b.t[j]);
        a.t[j] = from_f32<T>(xa * w.x - xb * w.y);
        b.t[j] = from_f32<T>(xa * w.y + xb * w.x);
      }
      *reinterpret_cast<uint4*>(dst + d) = a.u;
      *reinterpret_cast<uint4*>(dst + d + pairs) = b.u;
    } else {
      const int32_t d = p.offset + u * V;
      Pack<T> a;
      a.u = *reinterpret_cast<const uint4*>(src + d);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 w = ct[(u * V + j) / 2];
        const float xa = to_f32(a.t[j]), xb = to_f32(a.t[j + 1]);
        a.t[j] = from_f32<T>(xa * w.x - xb * w.y);
        a.t[j + 1] = from_f32<T>(xa * w.y + xb * w.x);
      }
      *reinterpret_cast<uint4*>(dst + d) = a.u;
    }
  }
}

}  // namespace rope
}  // namespace dsa
