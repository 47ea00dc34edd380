// Rotary positions (dsa_rope) and the angle arithmetic that the cache append shares.
//
// Pair i of the rotated dims turns by a = pos * inv_freq[i]; both are held in double and the angle is
// reduced to [-pi/4, pi/4] before its sine and cosine, so positions of 10^6 and more lose nothing (an fp32
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

// Sine and cosine of pos * freq in double, both to about 2^-52.  The reduction to [-pi/4, pi/4] subtracts k * pi/2 in two
// parts (the double nearest to pi/2 and the rest), each in one fused step; the rest is the Taylor series, whose first term
// left out is r^17 / 17! <= 5e-17.  About 25 operations: double ones are the scarce kind here.
__device__ __forceinline__ void sin_cos(int32_t pos, double freq, double& s, double& c) {
  const double a = static_cast<double>(pos) * freq;
  const double k = rint(a * 0.63661977236758134308);
  double r = fma(-k, 1.570796326794896558, a);
  r = fma(-k, 6.123233995736766036e-17, r);
  const double q = r * r;
  double u = -1.0 / 1307674368000.0;  // -1/15!
  u = fma(u, q, 1.0 / 6227020800.0);
  u = fma(u, q, -1.0 / 39916800.0);
  u = fma(u, q, 1.0 / 362880.0);
  u = fma(u, q, -1.0 / 5040.0);
  u = fma(u, q, 1.0 / 120.0);
  u = fma(u, q, -1.0 / 6.0);
  u = fma(u * q, r, r);
  double v = 1.0 / 20922789888000.0;  // 1/16!
  v = fma(v, q, -1.0 / 87178291200.0);
  v = fma(v, q, 1.0 / 479001600.0);
  v = fma(v, q, -1.0 / 3628800.0);
  v = fma(v, q, 1.0 / 40320.0);
  v = fma(v, q, -1.0 / 720.0);
  v = fma(v, q, 1.0 / 24.0);
  v = fma(v, q, -0.5);
  v = fma(v, q, 1.0);
  const int n = static_cast<int>(static_cast<long long>(k)) & 3;  // quarter turns
  s = n & 1 ? v : u;
  c = n & 1 ? u : v;
  if (n & 2) s = -s;
  if ((n + 1) & 2) c = -c;
}

// Division of numbers below 2^31 by a fixed one, with a multiplication: n / d = (n * mul) >> (32 + shift).
struct Div {
  uint32_t d, mul, shift;
};
inline Div make_div(uint32_t d) {
  Div r{d, 0, 0};
  while ((1ull << (r.shift + 1)) <= d) ++r.shift;  // floor(log2 d)
  // ceil(2^(32 + shift) / d) for d not a power of two (fits 32 bits); powers of two shift only
  r.mul = (d & (d - 1)) ? static_cast<uint32_t>(((1ull << (32 + r.shift)) + d - 1) / d) : 0u;
  return r;
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Div& v) {
  return v.mul ? __umulhi(n, v.mul) >> v.shift : n >> v.shift;
}

struct Params {
  const uint8_t* x;
  uint8_t* out;
  const int32_t* pos;
  int64_t x_tok, x_head, out_tok, out_head;  // strides in elements
  int32_t n_tokens, n_heads, dim, offset, rot;
  int32_t tok_per_cta, head_per_cta, head_groups;
  Div by_groups, by_pairs, by_units, by_heads;  // head_groups, rot / 2, 16-byte steps of a head, head_per_cta
  int32_t half;       // 1: pairs (i, i + rot / 2), 0: pairs (2i, 2i + 1)
  int32_t copy_rest;  // 1: the dims outside the rotated ones are copied (out is another tensor than x)
  double sin_sign;    // -1 turns the other way (the gradient)
  double mscale;
};

template <typename T>
struct Vec {
  static constexpr int N = 16 / static_cast<int>(sizeof(T));
};

// A pair's cosine and sine, scaled.  16-bit types turn in fp32: three roundings of 2^-24 of |a| + |b| before the one to T,
// which is 2^13 times as coarse and more.  fp32 turns in double, so that its one rounding is the result's.
template <typename T>
struct Turn {
  using Real = float;
  using Pair = float2;
};
template <>
struct Turn<float> {
  using Real = double;
  using Pair = double2;
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

template <typename T>
constexpr int MIN_BLOCKS = sizeof(T) == 2 ? 0 : 4;  // per SM; 0: as many as the registers leave

// One CTA: tok_per_cta tokens x head_per_cta heads.  The tokens' sines and cosines are formed once, in shared memory; then
// each thread takes 16-byte steps (half layout: one in each half), UNROLL at a time with their loads first (4 take 97
// registers in bf16, and a prefill chunk's queries 41 instead of 26 us).  Bound by the tensor's bytes: 8,192 tokens x 64
// heads x 64 dims in bf16 25.7 us, 5.2 TB/s; a decode step's 32 tokens 4 us alone, a launch.  fp32 is held to 4 blocks per SM:
// 4,097 tokens x 8 heads of 128 dims, 64 turned, 8.3 us (11.1 at 72 registers and 3 blocks; 8.0 with fp32 arithmetic).
template <typename T>
__global__ void __launch_bounds__(THREADS, MIN_BLOCKS<T>) rope_kernel(const __grid_constant__ Params p,
                                                       const __grid_constant__ Freqs fr) {
  grid_dependency_sync();
  using Real = typename Turn<T>::Real;
  using Pair = typename Turn<T>::Pair;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  Pair* cs = reinterpret_cast<Pair*>(rope_smem);  // [tok_per_cta][rot / 2]
  constexpr int V = Vec<T>::N, UNROLL = 2;
  const int32_t tg = static_cast<int32_t>(quotient(blockIdx.x, p.by_groups));
  const int32_t t0 = tg * p.tok_per_cta;
  const int32_t h0 = (static_cast<int32_t>(blockIdx.x) - tg * p.head_groups) * p.head_per_cta;
  const int32_t nt = min(p.tok_per_cta, p.n_tokens - t0), nh = min(p.head_per_cta, p.n_heads - h0);
  const int32_t pairs = p.rot / 2;
  for (int32_t i = threadIdx.x; i < nt * pairs; i += THREADS) {
    const int32_t t = static_cast<int32_t>(quotient(i, p.by_pairs));
    double s, c;
    sin_cos(p.pos[t0 + t], fr.f[i - t * pairs], s, c);
    cs[i] = Pair{static_cast<Real>(c * p.mscale), static_cast<Real>(s * p.mscale * p.sin_sign)};
  }
  __syncthreads();
  const int32_t turn_units = p.half ? pairs / V : p.rot / V, units = static_cast<int32_t>(p.by_units.d);
  const int32_t n = nt * p.head_per_cta * units;  // heads past the last are skipped
  for (int32_t i0 = threadIdx.x; i0 < n; i0 += THREADS * UNROLL) {
    Pack<T> a[UNROLL], b[UNROLL];
    T* dst[UNROLL];
    int32_t step[UNROLL], tok[UNROLL];  // step < 0: nothing to do
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int32_t i = i0 + k * THREADS;
      const int32_t th = static_cast<int32_t>(quotient(i, p.by_units)), u = i - th * units;
      const int32_t t = static_cast<int32_t>(quotient(th, p.by_heads)), h = th - t * p.head_per_cta;
      step[k] = i < n && h < nh ? u : -1;
      tok[k] = t;
      if (step[k] < 0) continue;
      const T* src = reinterpret_cast<const T*>(p.x) + (t0 + t) * p.x_tok + (h0 + h) * p.x_head;
      dst[k] = reinterpret_cast<T*>(p.out) + (t0 + t) * p.out_tok + (h0 + h) * p.out_head;
      int32_t d = p.offset + u * V;
      if (u >= turn_units) {
        d = (u - turn_units) * V;
        if (d >= p.offset) d += p.rot;
      } else if (p.half) {
        b[k].u = *reinterpret_cast<const uint4*>(src + d + pairs);
      }
      a[k].u = *reinterpret_cast<const uint4*>(src + d);
      dst[k] += d;
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (step[k] < 0) continue;
      if (step[k] < turn_units) {
        const Pair* ct = cs + tok[k] * pairs;
        if (p.half) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const Pair w = ct[step[k] * V + j];
            const Real xa = to_f32(a[k].t[j]), xb = to_f32(b[k].t[j]);
            a[k].t[j] = from_f32<T>(static_cast<float>(xa * w.x - xb * w.y));
            b[k].t[j] = from_f32<T>(static_cast<float>(xa * w.y + xb * w.x));
          }
          *reinterpret_cast<uint4*>(dst[k] + pairs) = b[k].u;
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const Pair w = ct[(step[k] * V + j) / 2];
            const Real xa = to_f32(a[k].t[j]), xb = to_f32(a[k].t[j + 1]);
            a[k].t[j] = from_f32<T>(static_cast<float>(xa * w.x - xb * w.y));
            a[k].t[j + 1] = from_f32<T>(static_cast<float>(xa * w.y + xb * w.x));
          }
        }
      }
      *reinterpret_cast<uint4*>(dst[k]) = a[k].u;
    }
  }
}

}  // namespace rope
}  // namespace dsa
