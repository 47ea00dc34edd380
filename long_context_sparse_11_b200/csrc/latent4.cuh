// Latent cache rows in 4 bits: the row format, the append that normalises, rotates and quantises on the way into
// a paged cache (4-bit or e4m3), and the read of cached rows.
//
// A 4-bit row is 320 bytes: 576 values as 18 blocks of 32, a value = c * 2^e with c an e2m1 code
// (+-{0, .5, 1, 1.5, 2, 3, 4, 6}) and e the block's exponent, in [-13, 13].
//   bytes 0..287    72 little-endian words of 8 values: bits 4i..4i+2 of a word = magnitude code of value i,
//                   bit 8i + 7 = sign of value i (i < 4), bit 8i + 3 = sign of value 4 + i
//   bytes 288..305  exponent of block b plus 127, bytes 306..319 zero
// A block with a NaN is stored as 32 codes 7 with the exponent 14, where code 7 is e5m2's NaN: reading it needs no
// case of its own.
// The signs sit where a byte permutation that looks up four magnitudes at once leaves room for them: four values
// decode with one lookup and one logical operation.  Exponents stay within [-13, 13] so that every value is a
// normal e5m2 number, which the tensor cores take as it is.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "ptx.cuh"
#include "rope.cuh"

namespace dsa {
namespace lat {

constexpr int DIM = 576, NOPE = 512, ROT = 64;
constexpr int ROW4 = 320, EXP_OFF = 288;
constexpr int EXP_MIN = -13, EXP_MAX = 13, EXP_NAN = 14 + 127;

// Physical slot of position t of sequence b, or -1.
__device__ __forceinline__ int64_t slot_of(int32_t b, int32_t t, const int32_t* block_table, int32_t batch,
                                           int32_t max_pages, int32_t n_pages) {
  if (b < 0 || b >= batch || t < 0 || (t >> 6) >= max_pages) return -1;
  const int32_t page = block_table[static_cast<int64_t>(b) * max_pages + (t >> 6)];
  if (page < 0 || page >= n_pages) return -1;
  return static_cast<int64_t>(page) * 64 + (t & 63);
}

// ------------------------------------------------------------------------------------- quantisation

// Exponent of a block from its largest magnitude: the least e with amax <= 6 * 2^e, within [-13, 13].
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 129 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return min(max(e, EXP_MIN), EXP_MAX);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two values to e2m1 codes (round to nearest even, saturating), the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r & 255u;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight codes, value i in nibble i, to a word of the row format (the signs move).
__device__ __forceinline__ uint32_t arrange(uint32_t x) {
  const uint32_t s = x & 0x88888888u;
  uint32_t lo = s & 0xFFFFu, hi = s >> 16;
  lo = (lo | (lo << 8)) & 0x00FF00FFu;
  lo = (lo | (lo << 4)) & 0x0F0F0F0Fu;
  hi = (hi | (hi << 8)) & 0x00FF00FFu;
  hi = (hi | (hi << 4)) & 0x0F0F0F0Fu;
  return (x & 0x77777777u) | (lo << 4) | hi;
}

// ------------------------------------------------------------------------------------- decoding

// e5m2 bytes of the magnitudes c * 2^e, codes 0..3 in x and 4..7 in y, for an exponent byte of a row: those of
// exponent 0 with 4 e added to each byte but the zero's.  Two multiply-adds, which leave the ALU to the permutations.
__device__ __forceinline__ uint2 mag_table(uint32_t exp_byte) {
  return make_uint2(exp_byte * 0x04040400u + (0x3E3C3800u - 127u * 0x04040400u),
                    exp_byte * 0x04040404u + (0x46444240u - 127u * 0x04040404u));
}
// The eight values of a word as e5m2 bytes: values 0..3 in x, 4..7 in y.
__device__ __forceinline__ uint2 word_to_e5m2(uint32_t w, uint2 tab) {
  const uint32_t m = w & 0x77777777u;
  uint2 r;
  r.x = __byte_perm(tab.x, tab.y, m) | (w & 0x80808080u);
  r.y = __byte_perm(tab.x, tab.y, __umulhi(m, 65536u)) | ((w * 16u) & 0x80808080u);
  return r;
}

// ------------------------------------------------------------------------------------- append

struct AppendParams {
  const uint8_t* x;  // rows of 576 bf16 or fp32 values
  int64_t x_stride;  // elements
  const float* gamma;
  double eps;
  const int32_t* seq;
  const int32_t* pos;
  const int32_t* block_table;
  uint8_t* pool;
  float* scale;  // e4m3 pools
  int* status;
  int32_t n_rows, batch, max_pages, n_pages;
  int32_t rotate, half;
  double mscale;
};
struct RotFreqs {
  double f[ROT / 2];
};

__device__ __forceinline__ float load1(const uint8_t* row, int d, bool f32) {
  return f32 ? reinterpret_cast<const float*>(row)[d]
             : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[d]) << 16);
}

// One warp per row.  Lane l holds values 8l..8l+7 and 256 + 8l.. of the latent dims and pair l of the RoPE dims.
// The norm and the rotation are formed to 48 bits and more (the sum of squares and the rotation in double, the products in
// pairs of fp32 numbers, which cost the double unit nothing) and rounded to fp32 once, so that which side of a 4-bit border
// a value falls on does not depend on the order of a sum; the quantisation is fp32 arithmetic without rounding (power-of-two
// steps), or the e4m3 rule of dsa_quant_e4m3.
// Bound by the latency of that chain (position, page; sum, root; maxima) at 32 rows per SM, which its 62 registers allow: 8,192
// bf16 rows 11.8 us alone and from cold caches, 32 rows 5.4 us.  Fewer registers (48: 14.2 us for 13.6 with the read back, 40:
// 15.5) spill.
template <bool F32, bool MX>
__global__ void __launch_bounds__(256) latent_append_kernel(const __grid_constant__ AppendParams p,
                                                            const __grid_constant__ RotFreqs fr) {
  grid_dependency_sync();
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (r >= p.n_rows) return;
  const int32_t t = p.pos[r];
  const int32_t b = p.seq ? p.seq[r] : static_cast<int32_t>(r);
  // the row and gamma are on their way before the page is known
  const uint8_t* row = p.x + r * p.x_stride * (F32 ? 4 : 2);
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int d = 256 * i + 8 * lane;
    if (F32) {
      const float4 a = *reinterpret_cast<const float4*>(row + d * 4);
      const float4 b = *reinterpret_cast<const float4*>(row + d * 4 + 16);
      v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
      v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + d * 2);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i][2 * j] = __uint_as_float(w[j] << 16);
        v[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
  const int da = p.half ? NOPE + lane : NOPE + 2 * lane, db = p.half ? NOPE + 32 + lane : NOPE + 2 * lane + 1;
  float ra = load1(row, da, F32), rb = load1(row, db, F32);
  __align__(16) float g[2][8];
  if (p.gamma) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(&g[i >> 1][4 * (i & 1)]) =
          __ldg(reinterpret_cast<const float4*>(p.gamma + 256 * (i >> 1) + 8 * lane + 4 * (i & 1)));
  }
  const int64_t slot = slot_of(b, t, p.block_table, p.batch, p.max_pages, p.n_pages);
  if (slot < 0) {
    if (lane == 0) atomicOr(p.status, DEVERR_BOUNDS);
    return;
  }
  if (p.gamma) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma(static_cast<double>(v[i][j]), static_cast<double>(v[i][j]), ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double inv = 1.0 / sqrt(ss * (1.0 / NOPE) + p.eps);
    const float ih = static_cast<float>(inv), il = static_cast<float>(inv - static_cast<double>(ih));
    float probe = 0.f;  // NaN once a result is not finite
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[i][j];
        const float gh = ih * g[i][j], gl = fmaf(il, g[i][j], fmaf(ih, g[i][j], -gh));  // inv * gamma as gh + gl
        const float y = x * gh;
        v[i][j] = y + fmaf(x, gl, fmaf(x, gh, -y));
        probe = fmaf(v[i][j], 0.f, probe);
      }
    // Where the pairs leave fp32's range (a result or 1 / rms above it, a subnormal 1 / rms): the products in double
    if (probe != 0.f || ih < 1e-25f) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = static_cast<float>(static_cast<double>(load1(row, 256 * i + 8 * lane + j, F32)) * inv *
                                       static_cast<double>(g[i][j]));
    }
  }
  if (p.rotate) {
    double s, c;
    rope::sin_cos(t, fr.f[lane], s, c);
    s *= p.mscale;
    c *= p.mscale;
    const double a = ra, b = rb;
    ra = static_cast<float>(a * c - b * s);
    rb = static_cast<float>(a * s + b * c);
  }
  if (MX) {
    uint8_t* dst = p.pool + slot * ROW4;
    uint32_t ex[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[i][j]));
      // the integer order of non-negative floats puts NaN above infinity
      uint32_t u = __float_as_uint(amax);
      u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
      u = max(u, __shfl_xor_sync(0xffffffffu, u, 2));
      const bool bad = u > 0x7F800000u;
      const int e = bad ? 0 : block_exp(__uint_as_float(u));
      ex[i] = bad ? EXP_NAN : static_cast<uint32_t>(e + 127);
      const float inv = exp2_int(-e);
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= e2m1_pair(v[i][2 * j] * inv, v[i][2 * j + 1] * inv) << (8 * j);
      if (bad) w = 0x77777777u;
      *reinterpret_cast<uint32_t*>(dst + (32 * i + lane) * 4) = arrange(w);
    }
    // RoPE dims: interleaved pairs put blocks 16 and 17 on lanes 0-15 and 16-31; halves put block 16 on ra, 17 on rb
    uint32_t ua = __float_as_uint(fabsf(ra)), ub = __float_as_uint(fabsf(rb));
    if (!p.half) ua = ub = max(ua, ub);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      if (o == 16 && !p.half) break;
      ua = max(ua, __shfl_xor_sync(0xffffffffu, ua, o));
      ub = max(ub, __shfl_xor_sync(0xffffffffu, ub, o));
    }
    const bool bad_a = ua > 0x7F800000u, bad_b = ub > 0x7F800000u;
    const int ea = bad_a ? 0 : block_exp(__uint_as_float(ua)), eb = bad_b ? 0 : block_exp(__uint_as_float(ub));
    uint32_t code = e2m1_pair(ra * exp2_int(-ea), rb * exp2_int(-eb));
    if (bad_a) code = (code & 0xF0u) | 7u;
    if (bad_b) code = (code & 0x0Fu) | 0x70u;
    if (!p.half) {
      uint32_t w = code << (8 * (lane & 3));
      w |= __shfl_xor_sync(0xffffffffu, w, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(dst + 256 + lane) = arrange(w);
    } else {
      uint32_t wa = (code & 15u) << (4 * (lane & 7)), wb = (code >> 4) << (4 * (lane & 7));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        wa |= __shfl_xor_sync(0xffffffffu, wa, o);
        wb |= __shfl_xor_sync(0xffffffffu, wb, o);
      }
      if ((lane & 7) == 0) {
        *reinterpret_cast<uint32_t*>(dst + 256 + lane / 2) = arrange(wa);
        *reinterpret_cast<uint32_t*>(dst + 272 + lane / 2) = arrange(wb);
      }
    }
    // exponent bytes: words 0..3 = blocks 0..15 (block b of half i sits on lanes 4(b % 8)..), word 4 = blocks 16, 17
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e0 = __shfl_sync(0xffffffffu, ex[0], 16 * (lane & 1) + 4 * j);
      const uint32_t e1 = __shfl_sync(0xffffffffu, ex[1], 16 * (lane & 1) + 4 * j);
      word |= (lane < 2 ? e0 : e1) << (8 * j);
    }
    const uint32_t xa = bad_a ? EXP_NAN : static_cast<uint32_t>(ea + 127);
    const uint32_t xb = bad_b ? EXP_NAN : static_cast<uint32_t>(eb + 127);
    const uint32_t x16 = __shfl_sync(0xffffffffu, xa, 0), x17 = __shfl_sync(0xffffffffu, xb, 16);
    if (lane == 4) word = x16 | (x17 << 8);
    if (lane > 4) word = 0;
    if (lane < 8) *reinterpret_cast<uint32_t*>(dst + EXP_OFF + 4 * lane) = word;
  } else {
    float amax = fmaxf(fabsf(ra), fabsf(rb));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    uint8_t* dst = p.pool + slot * DIM;
    auto pair = [&](float a, float b) {
      return static_cast<uint32_t>(
          __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s)), __NV_SATFINITE, __NV_E4M3));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint2 w;
      w.x = pair(v[i][0], v[i][1]) | (pair(v[i][2], v[i][3]) << 16);
      w.y = pair(v[i][4], v[i][5]) | (pair(v[i][6], v[i][7]) << 16);
      *reinterpret_cast<uint2*>(dst + 256 * i + 8 * lane) = w;
    }
    const uint32_t c = pair(ra, rb);
    dst[da] = static_cast<uint8_t>(c & 255u);
    dst[db] = static_cast<uint8_t>(c >> 8);
    if (lane == 0) p.scale[slot] = s;
  }
}

// ------------------------------------------------------------------------------------- read

struct ReadParams {
  const uint8_t* pool;
  const float* scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* seq;
  const int32_t* pos;
  uint16_t* out;  // [n_rows, out_stride] bf16
  int64_t out_stride;
  int* status;
  int32_t n_rows, batch, max_pages, n_pages;
};

// 12 threads per row, thread w with words w, w + 12, .. of 8 values (4 or 8 bytes of codes in, 16 bytes of bf16 out): the
// loads of a row are in flight together behind its chain of position and page, and neighbouring threads store neighbouring
// bytes.  4-bit values are exact in bf16; an e4m3 code times its fp32 scale is rounded once.  Bound by that chain and the
// stores: 32,768 4-bit rows in 11.0 us, 4.4 TB/s of codes and values (a thread per word, four rows each, spent 73% of the
// issue slots mostly on addresses and took 12.9).
constexpr int READ_LANES = 12, READ_WORDS = 6, READ_THREADS = 288;
constexpr int READ_ROWS = READ_THREADS / READ_LANES;
template <bool MX>
__global__ void __launch_bounds__(READ_THREADS, 7) latent_read_kernel(const __grid_constant__ ReadParams p) {
  grid_dependency_sync();
  const int32_t g = threadIdx.x / READ_LANES, w = threadIdx.x - g * READ_LANES;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * READ_ROWS + g;
  if (r >= p.n_rows) return;
  const int32_t b = p.seq ? p.seq[r] : static_cast<int32_t>(r), t = p.pos[r];
  const int64_t slot = slot_of(b, t, p.block_table, p.batch, p.max_pages, p.n_pages);
  if (slot < 0 || t >= p.seq_lens[b]) {
    if (w == 0) atomicOr(p.status, DEVERR_BOUNDS);
    return;
  }
  const uint8_t* row = p.pool + slot * (MX ? ROW4 : DIM);
  uint2 codes[READ_WORDS];
  uint32_t ex[READ_WORDS];
  float scale = 1.f;
#pragma unroll
  for (int u = 0; u < READ_WORDS; ++u) {
    if (MX) {
      codes[u].x = __ldg(reinterpret_cast<const uint32_t*>(row + 4 * w + 4 * READ_LANES * u));
      ex[u] = __ldg(row + EXP_OFF + w / 4 + READ_LANES / 4 * u);
    } else {
      codes[u] = __ldg(reinterpret_cast<const uint2*>(row + 8 * w + 8 * READ_LANES * u));
    }
  }
  if (!MX) scale = __ldg(p.scale + slot);
  uint16_t* out = p.out + r * p.out_stride + 8 * w;
#pragma unroll
  for (int u = 0; u < READ_WORDS; ++u) {
    uint32_t o[4];
    if (MX) {
      const uint2 m = word_to_e5m2(codes[u].x, mag_table(ex[u]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // an e5m2 byte is the high byte of the f16 of the same value
        const uint32_t h2 = __byte_perm(0u, i < 2 ? m.x : m.y, i & 1 ? 0x7060 : 0x5040);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c2 = ((i < 2 ? codes[u].x : codes[u].y) >> (16 * (i & 1))) & 0xFFFFu;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2), __NV_E4M3);
        const __nv_bfloat162 v = __floats2bfloat162_rn(__half2float(__ushort_as_half(h.x)) * scale,
                                                       __half2float(__ushort_as_half(h.y)) * scale);
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *reinterpret_cast<uint4*>(out + 8 * READ_LANES * u) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace lat
}  // namespace dsa
