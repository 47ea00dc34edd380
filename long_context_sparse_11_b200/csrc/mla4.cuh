// Sparse MLA attention over a paged latent cache held in 4 bits (row format: latent4.cuh).
//   z[h, j] = scale * q[h, :] . kv[idx_j, :576],  p = softmax_j(z),  out[h] = sum_j p kv[idx_j, :512]
// One CTA per (query row, 8 heads): 32 keys at a time are decoded to fp32 in shared memory, their logits formed by
// one thread per (head, key), and the softmax runs over them with a running maximum and sum in fp32.
#pragma once
#include <cuda_bf16.h>
#include "latent4.cuh"
#include "ptx.cuh"

namespace dsa {
namespace mla4 {

constexpr int HPC = 8, KEYS = 32, THREADS = 256;
constexpr int LD = 577;  // odd row stride: the 32 keys of a warp's logits fall into 32 banks
constexpr int SMEM_BYTES = (KEYS * LD + HPC * 576 + HPC * KEYS) * 4;

struct Params {
  const uint16_t* q;  // [n_q, 64, 576] bf16
  const uint8_t* kv;  // [n_pages, 64, 320]
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* idx;  // [n_q / rows_per_idx, k]
  uint16_t* out;       // [n_q, 64, 512] bf16
  float* lse;          // [n_q, 64] or null
  int32_t n_q, rows_per_idx, k, batch, max_pages, n_pages;
  float scale_log2;
  int* status;
};

__global__ void __launch_bounds__(THREADS) sparse_mla4_kernel(const __grid_constant__ Params p) {
  grid_dependency_sync();
  extern __shared__ float sm[];
  float* kv = sm;                   // [32][577]
  float* qs = sm + KEYS * LD;       // [8][576]
  float* ps = qs + HPC * 576;       // [8][32]
  __shared__ int64_t slots[KEYS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t row = blockIdx.x, h0 = blockIdx.y * HPC, irow = row / p.rows_per_idx;
  for (int i = tid; i < HPC * 576; i += THREADS)
    qs[i] = __uint_as_float(static_cast<uint32_t>(p.q[(static_cast<int64_t>(row) * 64 + h0) * 576 + i]) << 16);
  const int32_t len = p.seq_lens[irow];
  float m = -INFINITY, l = 0.f;     // of head `warp`, the same in all lanes
  float acc[HPC][2] = {};           // dims 2 tid, 2 tid + 1
  for (int32_t j0 = 0; j0 < p.k; j0 += KEYS) {
    __syncthreads();
    if (tid < KEYS) {
      const int32_t t = j0 + tid < p.k ? p.idx[static_cast<int64_t>(irow) * p.k + j0 + tid] : -1;
      int64_t s = -1;
      if (t >= 0) {
        if (t < len) s = lat::slot_of(irow, t, p.block_table, p.batch, p.max_pages, p.n_pages);
        if (s < 0) atomicOr(p.status, DEVERR_BOUNDS);
      }
      slots[tid] = s;
    }
    __syncthreads();
    for (int i = tid; i < KEYS * 72; i += THREADS) {
      const int key = i / 72, w = i % 72;
      uint2 b = make_uint2(0u, 0u);
      if (slots[key] >= 0) {
        const uint8_t* r = p.kv + slots[key] * lat::ROW4;
        b = lat::word_to_e5m2(*reinterpret_cast<const uint32_t*>(r + 4 * w), lat::mag_table(r[lat::EXP_OFF + w / 4]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t by = ((e < 4 ? b.x : b.y) >> (8 * (e & 3))) & 255u;
        kv[key * LD + 8 * w + e] = __half2float(__ushort_as_half(static_cast<unsigned short>(by << 8)));
      }
    }
    __syncthreads();
    float z = -INFINITY;
    if (slots[lane] >= 0) {
      float a = 0.f;
      for (int d = 0; d < 576; ++d) a = fmaf(qs[warp * 576 + d], kv[lane * LD + d], a);
      z = a * p.scale_log2;
    }
    float mx = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float pr = slots[lane] >= 0 ? exp2f(z - mn) : 0.f;
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    float sum = pr;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * alpha + sum;
    m = mn;
    ps[warp * KEYS + lane] = pr;
    __shared__ float alphas[HPC];
    if (lane == 0) alphas[warp] = alpha;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < HPC; ++h) {
      float a0 = acc[h][0] * alphas[h], a1 = acc[h][1] * alphas[h];
      for (int j = 0; j < KEYS; ++j) {
        const float w = ps[h * KEYS + j];
        if (w != 0.f || w != w) {
          a0 = fmaf(w, kv[j * LD + 2 * tid], a0);
          a1 = fmaf(w, kv[j * LD + 2 * tid + 1], a1);
        }
      }
      acc[h][0] = a0, acc[h][1] = a1;
    }
  }
  __shared__ float ls[HPC];
  if (lane == 0) {
    ls[warp] = l;
    if (p.lse) p.lse[static_cast<int64_t>(row) * 64 + h0 + warp] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HPC; ++h) {
    const float inv = ls[h] == 0.f ? 0.f : 1.f / ls[h];
    const __nv_bfloat162 o = __floats2bfloat162_rn(acc[h][0] * inv, acc[h][1] * inv);
    *reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(row) * 64 + h0 + h) * 512 + 2 * tid) =
        *reinterpret_cast<const uint32_t*>(&o);
  }
}

}  // namespace mla4
}  // namespace dsa
