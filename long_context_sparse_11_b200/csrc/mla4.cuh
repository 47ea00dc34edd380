// Sparse MLA attention over a paged latent cache held in 4 bits (row format: latent4.cuh).
//   z[h, j] = scale * q[h, :] . kv[idx_j, :576],  p = softmax_j(z),  out[h] = sum_j p kv[idx_j, :512]
//
// Both products run on the 8-bit tensor path with nothing lost in the cache and next to nothing in q and p:
//   * a cache value c * 2^e (e2m1 times a power of two in [2^-13, 2^13]) is an e5m2 number, exactly.  Four of them
//     decode with one byte permutation (a table of the block's eight magnitudes) and one logical operation;
//   * q is scaled per head by a power of two to a largest magnitude in [128, 256) and split into the nearest e4m3
//     number and 16 times the rest, also e4m3: 8 significant bits, all that bf16 has.  The two parts are 128 columns
//     of one product, summed with the factor 1/16 in the softmax;
//   * p is split into the nearest e4m3 number and the nearest e5m2 number of the rest (7 to 8 bits, as bf16, and a
//     floor of 2^-20 of the row's largest probability), two products into the same accumulator.
// In the form of the FP8 kernel (mla.cuh), every MMA has M = 128:
//   S^T[key, q part] = KV[key, 0:576] . Q[part, 0:576]   N = 128, K = 32: 18 steps of 64 clocks
//   O^T[dim, head]  += V^T[dim, key] . P^T[key, head]    N = 64, 4 blocks of 128 dims, 2 parts: 32 steps of 48 clocks
// so a tile of 128 keys takes the tensor core about 2,700 clocks (operand reads at 128 B a clock set both rates).
// The decoded tile is 72 KB, half of an f16 one, so nearly two tiles fit in shared memory (eight 128-dim sub-tiles in
// a ring, one RoPE sub-tile): S^T of tile j + 1 runs while the softmax of tile j does, and PV of tile j while tile
// j + 2 is decoded into the sub-tiles it frees.
//
// Warps 0..7: softmax and output (warp w: TMEM lane quadrant w % 4, 32 heads from 32 (w / 4)); 8 decode warps: the
// query rows, and tile g + 1's 320-byte rows loaded into registers while tile g is decoded; last warp: MMA issuer.
// CTAs are persistent over equal contiguous ranges of the (row, key tile) sequence; rows that a range boundary cuts
// leave fp32 partials for combine4_kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include "latent4.cuh"
#include "mla.cuh"
#include "ptx.cuh"

namespace dsa {
namespace mla4 {

constexpr int TILE = 128;
constexpr int SUB = 128 * 128;  // one sub-tile: 128 keys (or q parts) x 128 dims, 1 byte each
constexpr int RSUB = 128 * 64;  // the RoPE dims of 128 keys (or q parts)
constexpr int SLOTS = 8;
constexpr int OFF_Q = 0;
constexpr int OFF_QR = 4 * SUB;
constexpr int OFF_KV = OFF_QR + RSUB;
constexpr int OFF_KR = OFF_KV + SLOTS * SUB;
constexpr int OFF_P = OFF_KR + RSUB;  // [2 parts][128 keys][64 heads]
constexpr int OFF_MISC = OFF_P + 2 * RSUB;
constexpr int N_BARS = 6 + SLOTS * 2 + 1;
constexpr int M_TMEM = 192, M_ABORT = 196;
constexpr int M_NEED = 200;  // int [4 tiles]: "a head's maximum moved"
constexpr int M_MASK = 216;  // uint16 [4 tiles][8 warps]: keys that count
constexpr int M_ZS = 288;    // float [4 items][64]: logit scale of a head
constexpr int M_MRUN = M_ZS + 1024;
constexpr int M_ALPHA = M_MRUN + 256;  // after an item's last tile: the inverse row sums
constexpr int M_RED = M_ALPHA + 256;   // float [4 quadrants][64]
constexpr int SMEM_BYTES = OFF_MISC + M_RED + 1024;
static_assert(N_BARS * 8 <= M_TMEM && SMEM_BYTES <= 232448, "shared memory");

constexpr int SM_WARPS = 8, DEC_WARPS = 8, HPW = 32;
constexpr int SM_THREADS = SM_WARPS * 32;
constexpr int MMA_WARP = SM_WARPS + DEC_WARPS;
constexpr int THREADS = (MMA_WARP + 1) * 32;
constexpr uint32_t TM_S = 256;  // S^T buffers at columns 256 and 384; O^T at 0..255

constexpr int B_QFULL = 0, B_SFULL = 1 /* and 2 */, B_PFULL = 3, B_PVDONE = 4, B_RFULL = 5, B_FULL = 6,
              B_EMPTY = B_FULL + SLOTS;

// p is held as 2^(z - m + BIAS): at most 2^(BIAS + GROW) <= 256 (e4m3 ends at 448) while the running maximum m
// trails the true one by up to GROW, and with e5m2's smallest step of 2^-16 exact to 2^-20 of the largest.
constexpr float BIAS = 4.f, GROW = 4.f;

struct Params {
  const uint16_t* q;  // [n_q, 64, 576] bf16
  const uint8_t* kv;  // [n_pages, 64, 320]
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* idx;  // [n_q / rows_per_idx, k]
  uint16_t* out;       // [n_q, 64, 512] bf16
  float* lse;          // [n_q, 64] or null
  // A CTA's range holds at most two cut rows: one begun before it (fragment 0), one that ends after it (fragment 1).
  float* part_o;       // [grid, 2, 64, 512] fp32
  float* part_ml;      // [grid, 2, 2, 64] (m in log2 units, l)
  int32_t n_q, rows_per_idx, k, batch, max_pages, n_pages;
  int32_t tiles, tiles_per_row;  // tiles = n_q * tiles_per_row
  float scale_log2;
  int* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ uint64_t make_sdesc64(uint32_t saddr) {  // 64-byte swizzle, 8-row groups of 512 bytes
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(512 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)4 << 61;
  return d;
}
// Byte offset of 16-byte chunk c (0..3) of row r inside a 64-byte-swizzled region.
__device__ __forceinline__ uint32_t sw64_off(uint32_t r, uint32_t c) { return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4); }

// First global tile of CTA c.
__host__ __device__ __forceinline__ int32_t range_begin(int64_t c, int64_t tiles, int64_t grid) {
  return static_cast<int32_t>(c * tiles / grid);
}

// One block of 32 values (16 bytes) to its e5m2 bytes.
__device__ __forceinline__ void decode32(const uint4& raw, uint32_t exp_byte, uint4& o0, uint4& o1) {
  const uint2 tab = lat::mag_table(exp_byte);
  const uint2 a = lat::word_to_e5m2(raw.x, tab), b = lat::word_to_e5m2(raw.y, tab);
  const uint2 c = lat::word_to_e5m2(raw.z, tab), d = lat::word_to_e5m2(raw.w, tab);
  o0 = make_uint4(a.x, a.y, b.x, b.y);
  o1 = make_uint4(c.x, c.y, d.x, d.y);
}

// One query head's 8 bf16 values to 8 e4m3 bytes of the scaled value and 8 of 16 times the rest.
__device__ __forceinline__ void split_q(const uint4& raw, float mul, bool nan, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16) * mul, b = __uint_as_float(w[i] & 0xFFFF0000u) * mul;
    const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(p, __NV_E4M3);
    const float ra = (a - __half2float(__ushort_as_half(r.x))) * 16.f, rb = (b - __half2float(__ushort_as_half(r.y))) * 16.f;
    h[i] = nan ? 0x7F7Fu : p;
    l[i] = nan ? 0u : __nv_cvt_float2_to_fp8x2(make_float2(ra, rb), __NV_SATFINITE, __NV_E4M3);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// Two probabilities to e4m3 bytes (low half of the result) and e5m2 bytes of the rest (high half).
__device__ __forceinline__ uint32_t split_p(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  const __half2_raw hr = h;
  const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(hr, __NV_SATFINITE, __NV_E4M3);
  const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3);
  const __half2_raw rest = __hsub2(h, __half2(back));
  const uint32_t lo = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E5M2);
  return hi | (lo << 16);
}

__global__ void __launch_bounds__(THREADS, 1) sparse_mla4_kernel(const __grid_constant__ Params p) {
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  uint8_t* misc = smem + OFF_MISC;
  const uint32_t bar0 = base + OFF_MISC;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + M_ABORT);
  volatile int* need_flags = reinterpret_cast<volatile int*>(misc + M_NEED);
  volatile uint16_t* masks = reinterpret_cast<volatile uint16_t*>(misc + M_MASK);
  float* zs = reinterpret_cast<float*>(misc + M_ZS);
  float* m_run = reinterpret_cast<float*>(misc + M_MRUN);
  float* alpha = reinterpret_cast<float*>(misc + M_ALPHA);
  float* red = reinterpret_cast<float*>(misc + M_RED);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (base & 1023u) {  // the swizzled layouts need it; the driver places dynamic shared memory so
    if (threadIdx.x == 0) atomicOr(p.status, DEVERR_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(B_QFULL), DEC_WARPS);
    mbar_init(bar(B_SFULL), 2);
    mbar_init(bar(B_SFULL + 1), 2);
    mbar_init(bar(B_PFULL), SM_WARPS);
    mbar_init(bar(B_PVDONE), 1);
    mbar_init(bar(B_RFULL), DEC_WARPS);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(bar(B_FULL + i), DEC_WARPS);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) need_flags[i] = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_holder), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int32_t tpr = p.tiles_per_row;
  const int32_t g_begin = range_begin(blockIdx.x, p.tiles, gridDim.x);
  const int32_t g_end = range_begin(blockIdx.x + 1, p.tiles, gridDim.x);
  const int32_t n = g_end - g_begin;  // this CTA's tiles; below, tile i is global tile g_begin + i

  if (warp >= SM_WARPS && warp < MMA_WARP) {
    // ================================================================= decode warps
    // Warp dw holds keys 16 dw .. 16 dw + 15 of every tile.  Latent sub-tile d: lane l decodes blocks 4 d + l % 4 of
    // keys l / 4 and l / 4 + 8 (64 consecutive bytes of a row per four lanes); RoPE: block 16 + l % 2 of key l / 2.
    const int dw = warp - SM_WARPS;
    const int c4 = lane & 3, r4 = lane >> 2;
    auto wait = [&](int b, uint32_t par) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), par, abort_flag, p.status, p.wait_ns));
    };
    auto publish = [&](int b) {  // this warp's stores are visible to the tensor core, then one arrival
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    // selected position of key 16 dw + lane of tile i (lanes 0..15), -1 past the end
    auto load_idx = [&](int32_t i) -> int32_t {
      if (i >= n || lane >= 16) return -1;
      const int32_t row = (g_begin + i) / tpr, j = (g_begin + i) % tpr;
      const int32_t at = j * TILE + 16 * dw + lane;
      return at < p.k ? p.idx[static_cast<int64_t>(row / p.rows_per_idx) * p.k + at] : -1;
    };
    auto resolve = [&](int32_t i, int32_t t) -> int32_t {
      if (t < 0) return -1;
      const int32_t irow = (g_begin + i) / tpr / p.rows_per_idx;
      int64_t s = -1;
      if (t < p.seq_lens[irow]) s = lat::slot_of(irow, t, p.block_table, p.batch, p.max_pages, p.n_pages);
      if (s < 0) atomicOr(p.status, DEVERR_BOUNDS);
      return static_cast<int32_t>(s);
    };
    uint4 raw[8], raw_r, ex_a, ex_b;
    uint32_t ex_r;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto row_ptr = [&](int32_t slot, int src) -> const uint8_t* {
      const int32_t s = __shfl_sync(0xffffffffu, slot, src);
      return s < 0 ? nullptr : p.kv + static_cast<int64_t>(s) * lat::ROW4;
    };
    auto ld16 = [&](const uint8_t* r, int off) { return r ? __ldg(reinterpret_cast<const uint4*>(r + off)) : zero; };

    // Query row of item `it`: copied as bf16 into the rows that its two parts will fill, then split in place, one
    // head per step of its warp.
    auto q_copy = [&](int32_t row) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q) + static_cast<int64_t>(row) * 64 * 1152;
      for (int i = 0; i < 8; ++i) {
        const int h = dw * 8 + i;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const int c = lane + 32 * u;
          if (c < 64) cp_async16(base + OFF_Q + (c >> 4) * SUB + sw128_off(h + 64 * ((c >> 3) & 1), c & 7), src + h * 1152 + c * 16, 16);
          else if (c < 72) cp_async16(base + OFF_QR + sw64_off(h + 64 * ((c >> 2) & 1), c & 3), src + h * 1152 + c * 16, 16);
        }
      }
    };
    auto q_split = [&](int32_t item) {
      cp_async_wait_all();
      __syncwarp();
      for (int i = 0; i < 8; ++i) {
        const int h = dw * 8 + i;
        uint4 v[3];
        uint32_t amax = 0;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const int c = lane + 32 * u;
          v[u] = zero;
          if (c < 64) v[u] = *reinterpret_cast<const uint4*>(smem + OFF_Q + (c >> 4) * SUB + sw128_off(h + 64 * ((c >> 3) & 1), c & 7));
          else if (c < 72) v[u] = *reinterpret_cast<const uint4*>(smem + OFF_QR + sw64_off(h + 64 * ((c >> 2) & 1), c & 3));
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) amax = max(amax, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const bool nan = amax >= 0x7F800000u;  // a head that is not finite becomes NaN throughout
        int sh = amax == 0u || nan ? 0 : 134 - static_cast<int>(amax >> 23);
        sh = min(max(sh, -120), 126);
        const float mul = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          const int c = lane + 32 * u;
          uint2 hi, lo;
          split_q(v[u], mul, nan, hi, lo);
          if (c < 64) {
            uint8_t* d = smem + OFF_Q + (c >> 4) * SUB + (c & 1) * 8;
            *reinterpret_cast<uint2*>(d + sw128_off(h, (c & 15) >> 1)) = hi;
            *reinterpret_cast<uint2*>(d + sw128_off(64 + h, (c & 15) >> 1)) = lo;
          } else if (c < 72) {
            uint8_t* d = smem + OFF_QR + (c & 1) * 8;
            *reinterpret_cast<uint2*>(d + sw64_off(h, (c & 7) >> 1)) = hi;
            *reinterpret_cast<uint2*>(d + sw64_off(64 + h, (c & 7) >> 1)) = lo;
          }
        }
        if (lane == 0) zs[(item & 3) * 64 + h] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
      }
      publish(B_QFULL);
    };

    bool ok = true;
    if (n > 0) q_copy(g_begin / tpr);
    int32_t slot = resolve(0, load_idx(0));
    {
      const uint8_t *a = row_ptr(slot, r4), *b = row_ptr(slot, r4 + 8), *c = row_ptr(slot, lane >> 1);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        raw[2 * d] = ld16(a, d * 64 + c4 * 16);
        raw[2 * d + 1] = ld16(b, d * 64 + c4 * 16);
      }
      ex_a = ld16(a, lat::EXP_OFF), ex_b = ld16(b, lat::EXP_OFF);
      raw_r = ld16(c, 256 + (lane & 1) * 16);
      ex_r = c ? __ldg(c + lat::EXP_OFF + 16 + (lane & 1)) : 0u;
    }
    int32_t slot_next = resolve(1, load_idx(1));
    int32_t idx_next2 = load_idx(2);
    int32_t item = 0;
    if (n > 0) q_split(0);
    for (int32_t i = 0; i < n && ok; ++i) {
      const uint8_t *na = row_ptr(slot_next, r4), *nb = row_ptr(slot_next, r4 + 8), *nc = row_ptr(slot_next, lane >> 1);
      const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0) & 0xFFFFu;
      const uint32_t xa[4] = {ex_a.x, ex_a.y, ex_a.z, ex_a.w}, xb[4] = {ex_b.x, ex_b.y, ex_b.z, ex_b.w};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int s = 4 * (i & 1) + d;
        if (ok && i >= 2) ok = wait(B_EMPTY + s, ((i >> 1) & 1) ^ 1);
        if (ok) {
          if (d == 0 && lane == 0) masks[(i & 3) * 8 + dw] = static_cast<uint16_t>(live);
          uint4 o0, o1;
          uint8_t* dst = smem + OFF_KV + s * SUB;
          decode32(raw[2 * d], (xa[d] >> (8 * c4)) & 255u, o0, o1);
          *reinterpret_cast<uint4*>(dst + sw128_off(16 * dw + r4, 2 * c4)) = o0;
          *reinterpret_cast<uint4*>(dst + sw128_off(16 * dw + r4, 2 * c4 + 1)) = o1;
          decode32(raw[2 * d + 1], (xb[d] >> (8 * c4)) & 255u, o0, o1);
          *reinterpret_cast<uint4*>(dst + sw128_off(16 * dw + r4 + 8, 2 * c4)) = o0;
          *reinterpret_cast<uint4*>(dst + sw128_off(16 * dw + r4 + 8, 2 * c4 + 1)) = o1;
          raw[2 * d] = ld16(na, d * 64 + c4 * 16);
          raw[2 * d + 1] = ld16(nb, d * 64 + c4 * 16);
          publish(B_FULL + s);
        }
      }
      ex_a = ld16(na, lat::EXP_OFF), ex_b = ld16(nb, lat::EXP_OFF);
      // S^T of the tile before has read its RoPE sub-tile (and its query row)
      if (ok && i >= 1) ok = wait(B_SFULL + ((i - 1) & 1), ((i - 1) >> 1) & 1);
      if (ok && i >= 1 && (g_begin + i) % tpr == 0) {
        q_copy((g_begin + i) / tpr);
        q_split(++item);
      }
      if (ok) {
        uint4 o0, o1;
        decode32(raw_r, ex_r, o0, o1);
        uint8_t* dst = smem + OFF_KR;
        const int r = 16 * dw + (lane >> 1), b = lane & 1;
        *reinterpret_cast<uint4*>(dst + sw64_off(r, 2 * b)) = o0;
        *reinterpret_cast<uint4*>(dst + sw64_off(r, 2 * b + 1)) = o1;
        raw_r = ld16(nc, 256 + b * 16);
        ex_r = nc ? __ldg(nc + lat::EXP_OFF + 16 + b) : 0u;
        publish(B_RFULL);
      }
      slot = slot_next;
      slot_next = resolve(i + 2, idx_next2);
      idx_next2 = load_idx(i + 3);
    }
  } else if (warp == MMA_WARP) {
    // ================================================================= MMA issuer
    if (lane == 0) {
      constexpr uint32_t ID_S = make_idesc(1, 0, 0, 0, 128, 128);    // e5m2 keys, e4m3 q parts
      constexpr uint32_t ID_PV[2] = {make_idesc(1, 0, 1, 1, 128, 64),  // e5m2 values, e4m3 p
                                     make_idesc(1, 1, 1, 1, 128, 64)};  // and the e5m2 rest of p
      auto wait = [&](int b, uint32_t par) {
        if (!mbar_wait(bar(b), par, abort_flag, p.status, p.wait_ns)) return false;
        tc_fence_after();
        return true;
      };
      int32_t item = 0;
      bool ok = true;
      for (int32_t i = 0; i <= n && ok; ++i) {
        if (i < n) {
          if (i == 0 || (g_begin + i) % tpr == 0) {
            ok = wait(B_QFULL, item & 1);
            ++item;
          }
          const uint32_t ds = tmem + TM_S + 128u * (i & 1);
          for (int d = 0; d < 4 && ok; ++d) {
            const int s = 4 * (i & 1) + d;
            if (!(ok = wait(B_FULL + s, (i >> 1) & 1))) break;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8(ds, make_sdesc(base + OFF_KV + s * SUB + kk * 32, 16, 1024),
                     make_sdesc(base + OFF_Q + d * SUB + kk * 32, 16, 1024), ID_S, (d | kk) != 0);
          }
          if (ok) ok = wait(B_RFULL, i & 1);
          if (!ok) break;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            mma_f8(ds, make_sdesc64(base + OFF_KR + kk * 32), make_sdesc64(base + OFF_QR + kk * 32), ID_S, 1);
          mma_commit(bar(B_SFULL + (i & 1)));
          mbar_arrive(bar(B_SFULL + (i & 1)));  // and what the decode warps left in shared memory (masks, scales)
        }
        if (i >= 1) {
          const int32_t t = i - 1;
          const bool first = t == 0 || (g_begin + t) % tpr == 0;
          if (!(ok = wait(B_PFULL, t & 1))) break;
          for (int mb = 0; mb < 4; ++mb) {
            const int s = 4 * (t & 1) + mb;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t a = make_sdesc(base + OFF_KV + s * SUB + kk * 4096, SUB, 1024);
#pragma unroll
              for (int u = 0; u < 2; ++u)
                mma_f8(tmem + 64u * mb, a, make_sdesc64(base + OFF_P + u * RSUB + kk * 2048), ID_PV[u], !first || kk + u > 0);
            }
            mma_commit(bar(B_EMPTY + s));
          }
          mma_commit(bar(B_PVDONE));
        }
      }
    }
  } else {
    // ================================================================= softmax / output warps
    const int quad = warp & 3, hh = warp >> 2;
    const int key = quad * 32 + lane;  // TMEM lane: key of S^T, dim of an O^T block
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int hcol = HPW * hh;
    int32_t item = 0;
    bool ok = true;
    float lsum[HPW];
    // As in mla.cuh: a failed wait is recorded and acted on at the next named_bar_or, where all softmax threads leave
    // together; before a warp-collective TMEM access the lanes of a warp agree on it.
    bool fail = false;
    for (int32_t i = 0; i < n; ++i) {
      const int32_t row = (g_begin + i) / tpr, j = (g_begin + i) % tpr;
      const bool first = i == 0 || j == 0, last = i == n - 1 || j == tpr - 1;
      if (first) {
        if (quad == 0) m_run[hcol + lane] = -INFINITY;
        named_bar(1, SM_THREADS);
#pragma unroll
        for (int h = 0; h < HPW; ++h) lsum[h] = 0.f;
      }
      {
        const bool got = mbar_wait(bar(B_SFULL + (i & 1)), (i >> 1) & 1, abort_flag, p.status, p.wait_ns);
        fail = __any_sync(0xffffffffu, fail || !got);
      }
      tc_fence_after();
      const bool valid = (masks[(i & 3) * 8 + (key >> 4)] >> (key & 15)) & 1;
      float z[HPW];
      bool exceed = false;
      if (!fail) {
        const float* zi = zs + (item & 3) * 64 + hcol;
        const uint32_t ts = tmem + TM_S + 128u * (i & 1) + hcol + lane_off;
#pragma unroll
        for (int c = 0; c < HPW / 16; ++c) {
          uint32_t a[16], b[16];
          DSA_TMEM_LD_X16(ts + 16u * c, a);
          DSA_TMEM_LD_X16(ts + 64u + 16u * c, b);
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            const float s = fmaf(__uint_as_float(b[h]), 0.0625f, __uint_as_float(a[h]));
            z[16 * c + h] = valid ? s * zi[16 * c + h] : -INFINITY;
            exceed |= z[16 * c + h] > m_run[hcol + 16 * c + h] + GROW;
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < HPW; ++h) z[h] = -INFINITY;
      }
      volatile int* need = need_flags + (i & 3);
      if (__any_sync(0xffffffffu, exceed) && lane == 0) *need = 1;
      if (named_bar_or(1, SM_THREADS, fail)) {
        ok = false;
        break;
      }
      // a later tile's flag: its last readers have passed this barrier, its next writers wait for the next one
      if (threadIdx.x == 0) need_flags[(i + 2) & 3] = 0;
      const bool resc = *need != 0;
      if (resc) {
        const float wmax = mla::warp_reduce32<true>(z, lane);
        red[quad * 64 + hcol + lane] = wmax;
        named_bar(1, SM_THREADS);
        if (quad == 0) {
          const int h = hcol + lane;
          const float tmax = fmaxf(fmaxf(red[h], red[64 + h]), fmaxf(red[128 + h], red[192 + h]));
          const float mo = m_run[h];
          float a = 1.f;
          if (tmax > -INFINITY && (mo == -INFINITY || tmax > mo + GROW)) {
            a = mo == -INFINITY ? 0.f : ex2_approx(mo - tmax);
            m_run[h] = tmax;
          }
          alpha[h] = a;
        }
        named_bar(1, SM_THREADS);
#pragma unroll
        for (int h = 0; h < HPW; ++h) lsum[h] *= alpha[hcol + h];
      }
      uint32_t ph[HPW / 4], pl[HPW / 4];
#pragma unroll
      for (int h = 0; h < HPW; h += 4) {
        float e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float m = m_run[hcol + h + u];
          e[u] = ex2_approx(z[h + u] - (m == -INFINITY ? 0.f : m) + BIAS);  // 0 for a masked key
          lsum[h + u] += e[u];
        }
        const uint32_t s0 = split_p(e[0], e[1]), s1 = split_p(e[2], e[3]);
        ph[h / 4] = __byte_perm(s0, s1, 0x5410);
        pl[h / 4] = __byte_perm(s0, s1, 0x7632);
      }
      // PV of the tile before has read P^T, and O^T holds its sum
      if (i > 0) {
        const bool got = mbar_wait(bar(B_PVDONE), (i - 1) & 1, abort_flag, p.status, p.wait_ns);
        fail = __any_sync(0xffffffffu, fail || !got);
        tc_fence_after();
      }
      if (resc && !first) {
#pragma unroll 1
        for (int mb = 0; mb < 4 && !fail; ++mb) {
          const uint32_t ta = tmem + 64u * mb + hcol + lane_off;
          uint32_t x[HPW];
          DSA_TMEM_LD_X32(ta, x);
#pragma unroll
          for (int c = 0; c < HPW; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * alpha[hcol + c]);
          DSA_TMEM_ST_X32(ta, x);
        }
      }
#pragma unroll
      for (int c = 0; c < HPW / 16; ++c) {
        const uint32_t off = sw64_off(key, (hcol >> 4) + c);
        *reinterpret_cast<uint4*>(smem + OFF_P + off) = make_uint4(ph[4 * c], ph[4 * c + 1], ph[4 * c + 2], ph[4 * c + 3]);
        *reinterpret_cast<uint4*>(smem + OFF_P + RSUB + off) = make_uint4(pl[4 * c], pl[4 * c + 1], pl[4 * c + 2], pl[4 * c + 3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PFULL));
      if (!last) continue;
      // ---- end of item: wait for its last PV, reduce the row sums, write the output
      ++item;
      {
        const bool got = mbar_wait(bar(B_PVDONE), i & 1, abort_flag, p.status, p.wait_ns);
        fail = __any_sync(0xffffffffu, fail || !got);
        tc_fence_after();
      }
      red[quad * 64 + hcol + lane] = mla::warp_reduce32<false>(lsum, lane);
      if (named_bar_or(1, SM_THREADS, fail)) {
        ok = false;
        break;
      }
      float l = 0.f;  // row sum of head hcol + lane (quadrant 0)
      if (quad == 0) {
        const int h = hcol + lane;
        l = red[h] + red[64 + h] + red[128 + h] + red[192 + h];
        alpha[h] = l == 0.f ? 0.f : 1.f / l;
      }
      named_bar(1, SM_THREADS);
      const int32_t row0 = row * tpr;  // this row's first global tile
      if (row0 >= g_begin && row0 + tpr <= g_end) {
        uint16_t* orow = p.out + static_cast<int64_t>(row) * 64 * 512;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t x[HPW];
          DSA_TMEM_LD_X32(tmem + 64u * mb + hcol + lane_off, x);
#pragma unroll
          for (int c = 0; c < HPW; ++c) {
            const __nv_bfloat16 o = __float2bfloat16_rn(__uint_as_float(x[c]) * alpha[hcol + c]);
            orow[(hcol + c) * 512 + mb * 128 + key] = *reinterpret_cast<const uint16_t*>(&o);
          }
        }
        if (p.lse && quad == 0)
          p.lse[static_cast<int64_t>(row) * 64 + hcol + lane] =
              l == 0.f ? -INFINITY : (m_run[hcol + lane] - BIAS + log2f(l)) * 0.69314718055994531f;
      } else {
        const int64_t pr = static_cast<int64_t>(blockIdx.x) * 2 + (row0 >= g_begin ? 1 : 0);
        float* po = p.part_o + pr * 64 * 512;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t x[HPW];
          DSA_TMEM_LD_X32(tmem + 64u * mb + hcol + lane_off, x);
#pragma unroll
          for (int c = 0; c < HPW; ++c) po[(hcol + c) * 512 + mb * 128 + key] = __uint_as_float(x[c]);
        }
        if (quad == 0) {
          p.part_ml[pr * 128 + hcol + lane] = l == 0.f ? -INFINITY : m_run[hcol + lane] - BIAS;
          p.part_ml[pr * 128 + 64 + hcol + lane] = l;
        }
      }
      tc_fence_before();
      named_bar(1, SM_THREADS);  // m_run, alpha and red are the next item's
    }
    (void)ok;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// Rows cut over several CTAs: out = sum_s w_s O_s / sum_s w_s l_s, w_s = 2^(m_s - max m).  One CTA per (range
// boundary, 4 heads), 4 dims per thread; the first boundary inside a row does the row.  A row has at most 16 fragments
// (k <= 2,048); batches of 8 are loaded before any weight is known, so a row costs one or two memory latencies.
constexpr int COMBINE_THREADS = 512;
__global__ void __launch_bounds__(COMBINE_THREADS) combine4_kernel(const float* __restrict__ part_o,
                                                                   const float* __restrict__ part_ml, int32_t tpr,
                                                                   int32_t tiles, int32_t grid,
                                                                   uint16_t* __restrict__ out, float* __restrict__ lse) {
  grid_dependency_sync();
  const int32_t c = blockIdx.x + 1, h = blockIdx.y * 4 + threadIdx.x / 128, t = threadIdx.x % 128;
  const int32_t b = range_begin(c, tiles, grid), row = b / tpr;
  if (b % tpr == 0 || range_begin(c - 1, tiles, grid) > row * tpr) return;
  int32_t n = 2;  // fragments: CTA c - 1 (its fragment 1), then CTAs c, c + 1, ... (their fragment 0)
  while (c + n - 1 < grid && range_begin(c + n - 1, tiles, grid) < (row + 1) * tpr) ++n;
  auto at = [&](int s) { return static_cast<int64_t>(c - 1 + s) * 2 + (s == 0 ? 1 : 0); };
  constexpr int EARLY = 8;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  for (int s0 = 0; s0 < n; s0 += EARLY) {
    float4 o[EARLY];
    float m[EARLY], l[EARLY];
#pragma unroll
    for (int u = 0; u < EARLY; ++u) {
      const bool in = s0 + u < n;
      const int64_t f = at(s0 + u);
      o[u] = in ? *reinterpret_cast<const float4*>(part_o + (f * 64 + h) * 512 + 4 * t) : make_float4(0.f, 0.f, 0.f, 0.f);
      m[u] = in ? part_ml[f * 128 + h] : -INFINITY;
      l[u] = in ? part_ml[f * 128 + 64 + h] : 0.f;
    }
    float mn = M;
#pragma unroll
    for (int u = 0; u < EARLY; ++u) mn = fmaxf(mn, m[u]);
    const float a = M == -INFINITY ? 0.f : exp2f(M - mn);
    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a, L *= a;
#pragma unroll
    for (int u = 0; u < EARLY; ++u) {
      if (l[u] == 0.f) continue;  // a fragment without a key
      const float w = exp2f(m[u] - (mn == -INFINITY ? 0.f : mn));
      acc.x = fmaf(w, o[u].x, acc.x);
      acc.y = fmaf(w, o[u].y, acc.y);
      acc.z = fmaf(w, o[u].z, acc.z);
      acc.w = fmaf(w, o[u].w, acc.w);
      L = fmaf(w, l[u], L);
    }
    M = mn;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&x);
  pk.y = *reinterpret_cast<const uint32_t*>(&y);
  *reinterpret_cast<uint2*>(out + (static_cast<int64_t>(row) * 64 + h) * 512 + 4 * t) = pk;
  if (lse && t == 0) lse[static_cast<int64_t>(row) * 64 + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace mla4
}  // namespace dsa
