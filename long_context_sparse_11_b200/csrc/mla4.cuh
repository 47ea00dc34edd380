// Sparse MLA attention over a paged latent cache held in 4 bits (row format: latent4.cuh).
//   z[h, j] = scale * q[h, :] . kv[idx_j, :576],  p = softmax_j(z),  out[h] = sum_j p kv[idx_j, :512]
//
// Both products run on the 8-bit tensor path with nothing lost in the cache and next to nothing in q and p:
//   * a cache value c * 2^e (e2m1 times a power of two in [2^-13, 2^13]) is an e5m2 number, exactly.  Four of them
//     decode with one byte permutation (a table of the block's eight magnitudes) and one logical operation;
//   * q is scaled per head by a power of two to a largest magnitude in [128, 256) and split into the nearest e4m3
//     number and 16 times the rest, also e4m3: 8 significant bits, all that bf16 has, down to 2^-13 of the head's largest
//     value (smaller ones are off by up to 2^-21 of it).  The two parts are 128 rows of one product, summed with the
//     factor 1/16 in the softmax;
//   * p is rounded to f16 and split into the nearest e4m3 number and the nearest e5m2 number of the rest: off by less than
//     2^-8 of it, the most that bf16 is, and by up to 2^-18 of the row's largest probability where p is below 2^-10 of that.
//     Two products into the same accumulator; the sum of p is of the unsplit fp32 values.
//   S[q part, key]  = Q[part, 0:576] . KV[key, 0:576]    M = 128, N = 128, K = 32: 18 steps of 64 clocks
//   O^T[dim, head] += V^T[dim, key] . P[head, key]       M = 128 dims x 4, N = 64, K = 32, 2 parts: 32 steps of 48 clocks
// so a tile of 128 keys takes the tensor core about 2,700 clocks, the second product at the rate of shared memory (6 KB per
// step).  A tile in fact takes about 4,000 (with the merge, 32 x 5 rows of 2,048 keys 66 us; 512 rows of one sequence 173 to 175
// us, 840 TFLOP/s of the products as they are defined): its 72 KB of decoded values, written beside the 272 KB that the products read, and the
// instructions of decode and softmax share the SM with it (512 rows: issue slots 56% busy, the L1 data pipe 59%).
//
// The chain of one tile (rows, decode, S, softmax, PV) is several times that long, so three tiles are in flight: a decoded tile
// is 64 KB (plus 8 KB of RoPE dims, one buffer), and the query row, which would take that much again, stays in tensor memory as
// the A operand of S.  It passes through a tile's slot of the ring on its way there.  Tensor memory: O^T in columns 0..255, S in
// 256..383, Q (512 dims) in 384..511; Q's RoPE dims in shared memory.
//
// Warps 0..15: query rows, softmax and output (warp w: heads 16 (w % 4) .. + 15, keys 32 (w / 4) .. + 31; a lane holds 16
// keys of one head); 8 decode warps: the next tile's 320-byte rows loaded into registers while one is decoded; 2 warps
// issue the MMAs.  CTAs are persistent over whole rows and, last, an equal part of a row that several CTAs share, which leaves
// fp32 partials for combine4_kernel.  A change of rows costs about 12,000 clocks (the next query's two parts, the output).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include "latent4.cuh"
#include "ptx.cuh"

namespace dsa {
namespace mla4 {

constexpr int TILE = 128;
constexpr int SUB = 128 * 128;  // one sub-tile: 128 keys (or q parts) x 128 dims, 1 byte each
constexpr int RSUB = 128 * 64;  // the RoPE dims of 128 keys (or q parts)
constexpr int SLOTS = 3;        // of 4 sub-tiles
constexpr int OFF_QR = 0;       // RoPE dims of the 128 q parts
constexpr int OFF_KV = OFF_QR + RSUB;
constexpr int OFF_KR = OFF_KV + SLOTS * 4 * SUB;
constexpr int OFF_P = OFF_KR + RSUB;  // [2 parts][64 heads][128 keys]
constexpr int OFF_MISC = OFF_P + SUB;
constexpr int N_BARS = 6 + 2 * SLOTS;
constexpr int M_TMEM = 208, M_ABORT = 212;
constexpr int M_MASK = 224;  // uint16 [4 tiles][8 warps]: keys that count
constexpr int M_ZS = 288;    // float [4 items][64]: logit scale of a head
constexpr int M_ALPHA = M_ZS + 1024;  // float [64]: factor on a head's sums; after its last tile: inverse row sum
constexpr int M_RED = M_ALPHA + 256;  // float [4 key groups][64]
constexpr int SMEM_BYTES = OFF_MISC + M_RED + 1024;
static_assert(N_BARS * 8 <= M_TMEM && SMEM_BYTES <= 232448, "shared memory");

constexpr int SM_WARPS = 16, DEC_WARPS = 8, HPW = 16;
constexpr int SM_THREADS = SM_WARPS * 32;
constexpr int MMA_WARP = SM_WARPS + DEC_WARPS;
constexpr int THREADS = (MMA_WARP + 4) * 32;  // seven whole warpgroups (three warps of the last one idle)
// Registers per thread: 72 at launch for 896 threads; the issuers' warpgroup gives some of its own to the decode.
// Spills would go to L2, since shared memory leaves the L1 cache next to nothing.
constexpr int REGS_LAUNCH = 72, REGS_SM = 72, REGS_DEC = 88, REGS_MMA = 40;
static_assert(SM_THREADS * REGS_SM + DEC_WARPS * 32 * REGS_DEC + 128 * REGS_MMA <= THREADS * REGS_LAUNCH, "register split");
constexpr uint32_t TM_S = 256, TM_Q = 384;

// S complete, its RoPE operand free, S read, P written, PV complete, query staged; then the slots
constexpr int B_SFULL = 0, B_RFREE = 1, B_SREAD = 2, B_PFULL = 3, B_PVDONE = 4, B_QFULL = 5, B_FULL = 6,
              B_EMPTY = B_FULL + SLOTS;

// p is 2^(z - m + 4), held as e = p / 256 = 2^(z + nn), nn = BIAS - m: p is at most 2^8 (e4m3 ends at 448) while the running
// maximum m trails the true one by up to GROW.  Below p = 2^-6 the e4m3 part is subnormal and the rest up to 2^-10, whose e5m2
// number is off by up to 2^-14: 2^-18 of a largest p of 2^4 or more.  A smaller GROW would keep more of small p and move the
// maximum more often: 2 gives 2^-20, and 512 rows 193 us for 175; 3 gives 2^-19 and 181.
constexpr float BIAS = -4.f, GROW = 4.f;
static_assert(BIAS + GROW == 0.f, "e <= 1");

struct Params {
  const uint16_t* q;  // [n_q, 64, 576] bf16
  const uint8_t* kv;  // [n_pages, 64, 320]
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* idx;  // [n_q / rows_per_idx, k]
  uint16_t* out;       // [n_q, 64, 512] bf16
  float* lse;          // [n_q, 64] or null
  float* part_o;       // [parts of rows, 16, 512, 4] fp32 (16 quads of heads, 512 dims, 4 heads)
  float* part_ml;      // [parts of rows, 2, 64] (m in log2 units, l)
  int32_t n_q, rows_per_idx, k, batch, max_pages, n_pages;
  // CTA c has the whole rows whole_rows * c ..; the rows behind those of all CTAs are cut into `parts` equal parts (1: not
  // cut), and CTA c < n_parts has part c of them.
  int32_t tiles_per_row, whole_rows, parts, n_parts;
  float scale_log2;
  int* status;
  uint64_t wait_ns;
};

// Shared-memory matrix descriptors whose low word is the address / 16 (plus 1 << 16, a leading offset that none of
// these layouts reads): 128-byte swizzle with 8-row groups of 1,024 bytes, 64-byte swizzle with groups of 512.
__device__ __forceinline__ uint64_t desc128(uint32_t lo) {
  return (static_cast<uint64_t>((1024u >> 4) | (1u << 14) | (2u << 29)) << 32) | lo;
}
__device__ __forceinline__ uint64_t desc64(uint32_t lo) {
  return (static_cast<uint64_t>((512u >> 4) | (1u << 14) | (4u << 29)) << 32) | lo;
}
// Byte offset of 16-byte chunk c (0..3) of row r inside a 64-byte-swizzled region.
__device__ __forceinline__ uint32_t sw64_off(uint32_t r, uint32_t c) { return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4); }

// Row k of a CTA in its order: its whole rows, then its part of a cut row (which ends with the CTA's tiles).  Worked out anew
// at each row's end: more of it kept in registers, and the softmax warps spill.
struct Row {
  int32_t row, first;  // first: its first tile
};
__device__ __forceinline__ Row row_of(const Params& p, int32_t k) {
  const int32_t c = blockIdx.x;
  if (k < p.whole_rows) return Row{p.whole_rows * c + k, 0};
  const int32_t r = c / p.parts, s = c - r * p.parts;
  return Row{p.whole_rows * static_cast<int32_t>(gridDim.x) + r, s * p.tiles_per_row / p.parts};
}

// Keeps the arithmetic on loaded registers behind this point (moved up, it would wait for loads just issued).
__device__ __forceinline__ void pin(uint4& v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }

// One block of 32 values (16 bytes) to its e5m2 bytes.
__device__ __forceinline__ void decode32(const uint4& raw, uint32_t exp_byte, uint4& o0, uint4& o1) {
  const uint2 tab = lat::mag_table(exp_byte);
  const uint2 a = lat::word_to_e5m2(raw.x, tab), b = lat::word_to_e5m2(raw.y, tab);
  const uint2 c = lat::word_to_e5m2(raw.z, tab), d = lat::word_to_e5m2(raw.w, tab);
  o0 = make_uint4(a.x, a.y, b.x, b.y);
  o1 = make_uint4(c.x, c.y, d.x, d.y);
}

// 8 bf16 values of one query head, scaled by `mul` (a power of two), to 8 e4m3 bytes and 8 of 16 times the rest.
__device__ __forceinline__ void split_q(const uint4& raw, float mul, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[4], l[4];
  const __half2 sixteen = __float2half2_rn(16.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // exact in f16: 8 significant bits, at most 256 (f16's smallest step is 2^-31 of the head's largest)
    const __half2 v = __floats2half2_rn(__uint_as_float(w[i] << 16) * mul, __uint_as_float(w[i] & 0xFFFF0000u) * mul);
    const __half2_raw vr = v;
    h[i] = __nv_cvt_halfraw2_to_fp8x2(vr, __NV_SATFINITE, __NV_E4M3);
    const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h[i]), __NV_E4M3);
    const __half2_raw rest = __hmul2(__hsub2(v, __half2(back)), sixteen);
    l[i] = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// Two fp32 values side by side in a register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four values e = p / 256 to the e4m3 bytes and, of the rest, the e5m2 bytes of p.  At this scale the f16 of e has the
// exponent field of p's e4m3 (bias 15 against 7 + 8), normal or not: rounding it to three mantissa bits and taking its
// bits 14..7 is the conversion.  An e5m2 number is the high byte of an f16.  Both round to nearest (ties away from zero) by
// adding half a last place; two ALU operations a pair instead of five conversions and permutations.
__device__ __forceinline__ void split_p(float a, float b, float c, float d, uint32_t one, uint32_t& hi, uint32_t& lo) {
  const __half2 u = __floats2half2_rn(a, b), v = __floats2half2_rn(c, d);
  // multiply-adds by an opaque 1 (the FMA pipe; the ALU is the busier one)
  const uint32_t ru = *reinterpret_cast<const uint32_t*>(&u) * one + 0x00400040u;
  const uint32_t rv = *reinterpret_cast<const uint32_t*>(&v) * one + 0x00400040u;
  hi = __byte_perm(ru * 2u, rv * 2u, 0x7531);
  const uint32_t tu = ru & 0xFF80FF80u, tv = rv & 0xFF80FF80u;
  const __half2 scale = __float2half2_rn(256.f);
  const __half2 su = __hmul2(__hsub2(u, *reinterpret_cast<const __half2*>(&tu)), scale);
  const __half2 sv = __hmul2(__hsub2(v, *reinterpret_cast<const __half2*>(&tv)), scale);
  lo = __byte_perm(*reinterpret_cast<const uint32_t*>(&su) * one + 0x00800080u,
                   *reinterpret_cast<const uint32_t*>(&sv) * one + 0x00800080u, 0x7531);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// *ptr where `cond` holds, else -1 (and no access).  Nothing waits for the load before its result is used, as it would
// at the join of a branch.
__device__ __forceinline__ int32_t load_if(bool cond, const int32_t* ptr) {
  int32_t r;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tmov.b32 %0, -1;\n\t@p ld.global.nc.b32 %0, [%2];\n\t}"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(cond)), "l"(ptr));
  return r;
}

// A whole warp waits for a phase.  Each try sleeps until the phase completes or 20 us have passed (a loop of short tries
// would take issue slots from the warps that work).  A wait that runs out sets the abort flag and the status word; from then
// on every wait of the CTA gives up after one try.  Nothing leaves its loop early: all roles run through their steps (on
// whatever the buffers hold) and end together, so none is left waiting for one that has gone.
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                           uint64_t limit_ns) {
  auto attempt = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
  };
  if (!attempt()) {
    const uint64_t t0 = globaltimer_ns();
    while (!*abort && !attempt()) {
      if (globaltimer_ns() - t0 > limit_ns) {
        *abort = 1;
        atomicOr(status, DEVERR_TIMEOUT);
      }
    }
  }
  __syncwarp();
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// D += A B^T with A (K-major, 4 bytes per column) in tensor memory.
__device__ __forceinline__ void mma_f8_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 128 rows x 32 bytes of shared memory to 8 columns of tensor memory.
__device__ __forceinline__ void tmem_copy(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What keys that do not count read instead of a cache row: codes 0 are zeros whatever the exponents.
__device__ __align__(16) const uint8_t zero_row[lat::ROW4] = {};

__global__ void __launch_bounds__(THREADS, 1) sparse_mla4_kernel(const __grid_constant__ Params p) {
  grid_dependency_sync();
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  uint8_t* misc = smem + OFF_MISC;
  const uint32_t bar0 = base + OFF_MISC;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + M_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + M_ABORT);
  volatile uint16_t* masks = reinterpret_cast<volatile uint16_t*>(misc + M_MASK);
  float* zs = reinterpret_cast<float*>(misc + M_ZS);
  float* alpha = reinterpret_cast<float*>(misc + M_ALPHA);
  float* red = reinterpret_cast<float*>(misc + M_RED);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: a uniform value
  if (base & 1023u) {  // the swizzled layouts need it; the driver places dynamic shared memory so
    if (threadIdx.x == 0) atomicOr(p.status, DEVERR_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(B_SFULL), 2);
    mbar_init(bar(B_RFREE), 1);
    mbar_init(bar(B_SREAD), SM_WARPS);
    mbar_init(bar(B_PFULL), SM_WARPS);
    mbar_init(bar(B_PVDONE), 1);
    mbar_init(bar(B_QFULL), SM_WARPS);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(bar(B_FULL + i), DEC_WARPS);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_holder), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int32_t tpr = p.tiles_per_row;
  auto wait = [&](int b, uint32_t par) { wait_phase(bar(b), par, abort_flag, p.status, p.wait_ns); };
  int32_t n = p.whole_rows * tpr;  // this CTA's tiles
  if (blockIdx.x < p.n_parts) {
    const int32_t s = blockIdx.x % p.parts;
    n += (s + 1) * tpr / p.parts - s * tpr / p.parts;
  }
  const Row row0 = row_of(p, 0);

  // The ring's slots in the order of their use: a row's query, then its tiles.  On a fresh barrier the wait for the phase
  // before the first passes.
  struct Ring {
    int32_t slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
      if (++slot == SLOTS) slot = 0, phase ^= 1;
    }
  };
  // Row of S of a head's first part; its second is 16 rows further, in the same lane quadrant of tensor memory.
  auto q_row = [](int h) { return 32 * (h >> 4) + (h & 15); };
  // Four heads of a query row, eight lanes each (lane l % 8 of a head holds 16-byte chunks l % 8 + 8 u; the last are the RoPE
  // dims), split into the rows of a slot.  The RoPE parts are returned: their one buffer is free only after the last S of
  // the row before.
  auto q_stage = [&](int32_t row, int32_t item, int32_t slot, int h4, uint2& rope_hi, uint2& rope_lo) {
    const int h = h4 + (lane >> 3), l8 = lane & 7, r = q_row(h);
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(row) * 64 + h) * 576) + l8;
    uint4 v[9];
#pragma unroll
    for (int u = 0; u < 9; ++u) v[u] = __ldg(src + 8 * u);
    uint32_t am = 0;
#pragma unroll
    for (int u = 0; u < 9; ++u) {
      am = max_u16x2(max_u16x2(am, v[u].x & 0x7FFF7FFFu), v[u].y & 0x7FFF7FFFu);
      am = max_u16x2(max_u16x2(am, v[u].z & 0x7FFF7FFFu), v[u].w & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) am = max_u16x2(am, __shfl_xor_sync(0xffffffffu, am, o));
    am = max(am & 0xFFFFu, am >> 16);  // bf16 bits of the head's largest magnitude
    const bool nan = am >= 0x7F80u;    // a head that is not finite becomes NaN throughout
    int sh = am == 0u || nan ? 0 : 134 - static_cast<int>(am >> 7);
    sh = min(max(sh, -120), 126);
    const float mul = nan ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
#pragma unroll
    for (int u = 0; u < 8; ++u) {  // chunk l8 + 8 u: 8 bytes of either part
      uint2 hi, lo;
      split_q(v[u], mul, hi, lo);
      uint8_t* d = smem + OFF_KV + (4 * slot + (u >> 1)) * SUB + (l8 & 1) * 8;
      const uint32_t c = 4 * (u & 1) + (l8 >> 1);
      *reinterpret_cast<uint2*>(d + sw128_off(r, c)) = hi;
      *reinterpret_cast<uint2*>(d + sw128_off(r + 16, c)) = lo;
    }
    split_q(v[8], mul, rope_hi, rope_lo);
    if (l8 == 0) zs[(item & 3) * 64 + h] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
  };
  auto q_stage_rope = [&](int h4, const uint2& hi, const uint2& lo) {
    const int r = q_row(h4 + (lane >> 3)), l8 = lane & 7;
    uint8_t* d = smem + OFF_QR + (l8 & 1) * 8;
    *reinterpret_cast<uint2*>(d + sw64_off(r, l8 >> 1)) = hi;
    *reinterpret_cast<uint2*>(d + sw64_off(r + 16, l8 >> 1)) = lo;
  };

  if (warp >= SM_WARPS && warp < MMA_WARP) {
    // ================================================================= decode warps
    regs_inc<REGS_DEC>();
    // Warp dw holds keys 16 dw .. 16 dw + 15 of every tile.  Latent dims: lane l decodes block `blk` of keys 2 k + `odd`, k = 0..7
    // (256 consecutive bytes of two rows in a load: what these loads cost is the lines they touch); RoPE: block 16 + l % 2 of
    // key l / 2.  Eight neighbouring lanes store to 128 different bytes modulo 128: four chunks of an even row, four of an odd.
    const int dw = warp - SM_WARPS;
    const int blk = (lane & 3) | ((lane >> 3) << 2), odd = (lane >> 2) & 1;
    auto publish = [&](int b) {  // this warp's stores are visible to the tensor core, then one arrival
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    // The cache slot of key 16 dw + lane (lanes 0..15) of a tile, in three steps a tile apart, so that no step waits for
    // the load of the one before: the selected position (-1: none), its page number, the slot.  `ahead` walks the tiles.
    // A position or page out of range is reported and skipped.
    struct Pos {
      int32_t t, len, irow;
    };
    struct Page {
      int32_t t, page;
    };
    struct {
      int32_t left, at, item, irow;
    } ahead;
    ahead.left = n;
    ahead.item = 0;
    ahead.irow = row0.row / p.rows_per_idx;
    ahead.at = row0.first * TILE + 16 * dw + lane;
    auto position = [&]() -> Pos {
      const bool in = ahead.left > 0;
      const Pos q{load_if(in && lane < 16 && ahead.at < p.k, p.idx + static_cast<int64_t>(ahead.irow) * p.k + ahead.at),
                  load_if(in, p.seq_lens + ahead.irow), ahead.irow};
      --ahead.left;
      ahead.at += TILE;
      if (ahead.at >= tpr * TILE) {
        const Row next = row_of(p, ++ahead.item);
        ahead.irow = next.row / p.rows_per_idx;
        ahead.at = next.first * TILE + 16 * dw + lane;
      }
      return q;
    };
    auto find_page = [&](const Pos& q) -> Page {
      return Page{q.t, load_if(q.t >= 0 && q.t < q.len && (q.t >> 6) < p.max_pages,
                               p.block_table + static_cast<int64_t>(q.irow) * p.max_pages + (q.t >> 6))};
    };
    auto find_slot = [&](const Page& g) -> int32_t {
      if (g.t < 0) return -1;
      if (g.page < 0 || g.page >= p.n_pages) {
        atomicOr(p.status, DEVERR_BOUNDS);
        return -1;
      }
      return g.page * 64 + (g.t & 63);
    };
    uint4 raw[8], raw_r;
    uint32_t ex[8], ex_r;
    auto row_ptr = [&](int32_t slot, int src) -> const uint8_t* {  // a key that does not count reads a row of zeros
      const int32_t s = __shfl_sync(0xffffffffu, slot, src);
      return s < 0 ? zero_row : p.kv + static_cast<int64_t>(s) * lat::ROW4;
    };
    auto ld16 = [&](const uint8_t* r, int off) { return __ldg(reinterpret_cast<const uint4*>(r + off)); };

    const uint8_t* rr;  // row of this lane's RoPE block
    auto load_latent = [&](int32_t slots, int k) {
      const uint8_t* r = row_ptr(slots, 2 * k + odd);
      raw[k] = ld16(r, 16 * blk);
      ex[k] = __ldg(r + lat::EXP_OFF + blk);
    };
    auto load_rope = [&] {
      raw_r = ld16(rr, 256 + (lane & 1) * 16);
      ex_r = __ldg(rr + lat::EXP_OFF + 16 + (lane & 1));
    };

    auto q_prefetch = [&](int32_t row) {  // 72 lines of this warp's heads
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q) + static_cast<int64_t>(row) * 64 * 1152 + dw * 8 * 1152;
      for (int l = lane; l < 72; l += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + l * 128));
    };
    Ring ring;
    const Pos t0 = position(), t1 = position(), t2 = position();
    Pos t3 = position();  // in the loop: of tile i + 3
    const Page g0 = find_page(t0), g1 = find_page(t1);
    Page g2 = find_page(t2);  // of tile i + 2
    int32_t slot = find_slot(g0), slot_next;
#pragma unroll
    for (int k = 0; k < 8; ++k) load_latent(slot, k);
    rr = row_ptr(slot, lane >> 1);
    load_rope();
    slot_next = find_slot(g1);
    int32_t item = 0, row_left = tpr - row0.first;
    // A row's query is the softmax warps' work: here its use of a slot only keeps the barriers' phases in step.  The wait
    // belongs to that: a slot's release is one bit of its phase, and a warp that left one out would, with rows of one tile,
    // take the tile's slot while PV of the tile two uses before still reads it.
    auto skip_query = [&] {
      wait(B_EMPTY + ring.slot, ring.phase ^ 1);
      if (lane == 0) mbar_arrive(bar(B_FULL + ring.slot));
      ring.next();
    };
    if (n > 0) skip_query();
    // where block blk of key 16 dw + odd goes in the 128-byte swizzle; of keys further on: 256 k bytes further, chunks ^ 2 k
    const uint32_t at0 = (blk >> 2) * SUB + sw128_off(16 * dw + odd, 2 * (blk & 3));
    for (int32_t i = 0; i < n; ++i) {
      const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0) & 0xFFFFu;
      rr = row_ptr(slot_next, lane >> 1);
      wait(B_EMPTY + ring.slot, ring.phase ^ 1);
      if (lane == 0) masks[(i & 3) * 8 + dw] = static_cast<uint16_t>(live);
      uint8_t* const dst = smem + OFF_KV + 4 * ring.slot * SUB;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint4 o0, o1;
        pin(raw[k]);
        decode32(raw[k], ex[k], o0, o1);
        const uint32_t at = (at0 ^ (32 * (k & 3))) + 256 * k;
        *reinterpret_cast<uint4*>(dst + at) = o0;
        *reinterpret_cast<uint4*>(dst + (at ^ 16u)) = o1;
        load_latent(slot_next, k);  // of the next tile
      }
      if (i >= 1) wait(B_RFREE, (i - 1) & 1);  // the one RoPE sub-tile
      {
        uint4 o0, o1;
        pin(raw_r);
        decode32(raw_r, ex_r, o0, o1);
        const uint32_t o = sw64_off(16 * dw + (lane >> 1), 2 * (lane & 1));
        *reinterpret_cast<uint4*>(smem + OFF_KR + o) = o0;
        *reinterpret_cast<uint4*>(smem + OFF_KR + (o ^ 16u)) = o1;
      }
      load_rope();
      publish(B_FULL + ring.slot);
      ring.next();
      slot = slot_next;
      slot_next = find_slot(g2);
      g2 = find_page(t3);
      t3 = position();
      if (row_left == 3 && i + 3 < n) q_prefetch(row_of(p, item + 1).row);
      if (--row_left == 0) {
        row_left = tpr;  // (a part's tiles end with n)
        ++item;
        if (i + 1 < n) skip_query();
      }
    }
  } else if (warp >= MMA_WARP) {
    // ================================================================= MMA issuer
    regs_dec<REGS_MMA>();
    // Two warps, so that neither product waits behind the other's inputs: S of a tile once it is decoded, PV as its
    // probabilities arrive (S runs a tile ahead).  A whole warp runs each loop and one elected lane issues:
    // every address stays in uniform registers, and an MMA costs one instruction.  (Issued by one lane of a divergent branch
    // they took 75 to 120 clocks each; one warp that polled for both streams left the tensor core idle between steps.)
    const uint32_t lo0 = (base >> 4) | (1u << 16);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    Ring ring;
    int32_t row_left = 0, item = 0;
    if (warp == MMA_WARP) {
      constexpr uint32_t ID_S = make_idesc(0, 1, 0, 0, 128, 128);  // e4m3 q parts, e5m2 keys
      for (int32_t i = 0; i < n; ++i) {
        if (row_left == 0) {  // the row's query to tensor memory, behind the last S that reads the one before
          wait(B_FULL + ring.slot, ring.phase);
          wait(B_QFULL, item++ & 1);
          if (i > 0) wait(B_SFULL, (i - 1) & 1);
          tc_fence_after();
          const uint64_t a = desc128(lo0 + (OFF_KV + 4 * ring.slot * SUB) / 16);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 16; ++c) tmem_copy(tm + TM_Q + 8 * c, a + (c >> 2) * (SUB / 16) + 2 * (c & 3));
            mma_commit(bar(B_EMPTY + ring.slot));
          }
          __syncwarp();
          ring.next();
          row_left = i == 0 ? tpr - row0.first : tpr;
        }
        --row_left;
        if (i > 0) wait(B_SREAD, (i - 1) & 1);
        wait(B_FULL + ring.slot, ring.phase);
        tc_fence_after();
        const uint64_t b = desc128(lo0 + (OFF_KV + 4 * ring.slot * SUB) / 16);
        const uint64_t ar = desc64(lo0 + OFF_QR / 16), br = desc64(lo0 + OFF_KR / 16);
        if (elect_one()) {
          // the RoPE dims first: their one buffer is then free for the next tile while the rest runs
          mma_f8(tm + TM_S, ar, br, ID_S, 0);
          mma_f8(tm + TM_S, ar + 2, br + 2, ID_S, 1);
          mma_commit(bar(B_RFREE));
#pragma unroll
          for (int kk = 0; kk < 16; ++kk)
            mma_f8_ta(tm + TM_S, tm + TM_Q + 8 * kk, b + (kk >> 2) * (SUB / 16) + 2 * (kk & 3), ID_S, 1);
          mma_commit(bar(B_SFULL));
          mbar_arrive(bar(B_SFULL));  // and what the decode warps left in shared memory (masks)
        }
        __syncwarp();
        ring.next();
      }
    } else if (warp == MMA_WARP + 1) {
      constexpr uint32_t ID_PV = make_idesc(1, 0, 1, 0, 128, 64);   // e5m2 values, e4m3 p
      constexpr uint32_t ID_PVR = make_idesc(1, 1, 1, 0, 128, 64);  // and the e5m2 rest of p
      for (int32_t i = 0; i < n; ++i) {
        const uint32_t keep = row_left == 0 ? 0u : 1u;  // a row's first tile starts its sum
        if (row_left == 0) {
          row_left = i == 0 ? tpr - row0.first : tpr;
          ring.next();  // past the row's query
        }
        --row_left;
        wait(B_PFULL, i & 1);
        tc_fence_after();
        const uint64_t a = desc128(lo0 + (OFF_KV + 4 * ring.slot * SUB) / 16), b = desc128(lo0 + OFF_P / 16);
        if (elect_one()) {
#pragma unroll
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // 32 keys: 4 groups of 8 rows of V, 32 bytes of a row of P
              mma_f8(tm + 64u * mb, a + mb * (SUB / 16) + 256 * kk, b + 2 * kk, ID_PV, kk > 0 ? 1u : keep);
              mma_f8(tm + 64u * mb, a + mb * (SUB / 16) + 256 * kk, b + RSUB / 16 + 2 * kk, ID_PVR, 1);
            }
          }
          mma_commit(bar(B_EMPTY + ring.slot));
          mma_commit(bar(B_PVDONE));
        }
        __syncwarp();
        ring.next();
      }
    }
  } else {
    // ================================================================= softmax / output warps
    static_assert(REGS_SM == REGS_LAUNCH, "no change");
    Ring ring;
    if (n > 0) {
      uint2 hi, lo;
      q_stage(row0.row, 0, 0, 4 * warp, hi, lo);
      q_stage_rope(4 * warp, hi, lo);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_QFULL));
      ring.next();
    }
    // Lanes l and l + 16 of a warp hold one head's keys 0..15 and 16..31 of the warp's 32: its scale, maximum and sum are one
    // register each, and a lane's probabilities are 16 consecutive bytes of P.
    const int quad = warp & 3, grp = warp >> 2;
    const int head = 16 * quad + (lane & 15), upper = lane >> 4;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int dim = quad * 32 + lane, hcol = HPW * grp;  // of the O^T fragment this lane scales and writes: 16 heads of a dim
    uint32_t one;
    asm volatile("mov.b32 %0, 1;" : "=r"(one));
    int32_t item = 0;
    float z = 0.f, nn = BIAS;  // logit scale, BIAS minus the running maximum
    uint64_t lsum = 0ull;     // two partial row sums
    bool seen = false;        // the item has had a key that counts (its maxima are set)
    int32_t left = min(tpr - row0.first, n);  // left: tiles of the row still to come
    for (int32_t i = 0; i < n; ++i) {
      wait(B_SFULL, i & 1);
      tc_fence_after();
      if (!seen) z = zs[(item & 3) * 64 + head];
      const uint32_t mine = *reinterpret_cast<const uint32_t*>(misc + M_MASK + (i & 3) * 16 + grp * 4);
      uint64_t t[8];  // log2 of p / 256 of keys 2 u, 2 u + 1
      {
        const uint32_t ts = tmem + TM_S + 32u * grp + lane_off;
        uint32_t a[16], b[16];
        DSA_TMEM_LD_16X32X2_X16(ts, a);
        DSA_TMEM_LD_16X32X2_X16(ts + (16u << 16), b);
        DSA_TMEM_WAIT_LD_X16(a, b);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SREAD));
        const uint64_t part = pack2(0.0625f, 0.0625f), zz = pack2(z, z), mm = pack2(nn, nn);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint64_t sum = fma2(pack2(__uint_as_float(b[2 * u]), __uint_as_float(b[2 * u + 1])), part,
                                    pack2(__uint_as_float(a[2 * u]), __uint_as_float(a[2 * u + 1])));
          t[u] = fma2(sum, zz, mm);
        }
      }
      if (mine != 0xFFFFFFFFu) {  // the same in the whole warp
        const uint32_t m = mine >> (16 * upper);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float2 v = unpack2(t[u]);
          t[u] = pack2((m >> (2 * u)) & 1u ? v.x : -INFINITY, (m >> (2 * u + 1)) & 1u ? v.y : -INFINITY);
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float2 v = unpack2(t[u]);
        top = max3(top, v.x, v.y);
      }
      bool rescale_o = false;
      // The running maxima stay unless a head has outgrown its own
      if (named_bar_or(1, SM_THREADS, top > BIAS + GROW || !seen)) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        if (upper == 0) red[grp * 64 + head] = top;
        named_bar(1, SM_THREADS);
        const float m = fmaxf(fmaxf(red[head], red[64 + head]), fmaxf(red[128 + head], red[192 + head]));
        // the change of nn: a head's maximum becomes BIAS where it is the first or has grown past the margin
        const float d = m > -INFINITY && (!seen || m > BIAS + GROW) ? BIAS - m : 0.f;
        rescale_o = seen;
        if (seen) {
          const float f = ex2_approx(d);
          lsum = mul2(lsum, pack2(f, f));
          if (grp == 0 && upper == 0) alpha[head] = f;
          named_bar(1, SM_THREADS);
        } else {
          const uint4 live = *reinterpret_cast<const uint4*>(misc + M_MASK + (i & 3) * 16);
          seen = (live.x | live.y | live.z | live.w) != 0u;
        }
        nn += d;
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = add2(t[u], pack2(d, d));
      }
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 v = unpack2(t[2 * u]), w = unpack2(t[2 * u + 1]);
        const float e0 = ex2_approx(v.x), e1 = ex2_approx(v.y), e2 = ex2_approx(w.x), e3 = ex2_approx(w.y);
        lsum = add2(lsum, add2(pack2(e0, e1), pack2(e2, e3)));
        split_p(e0, e1, e2, e3, one, ph[u], pl[u]);
      }
      // PV of the tile before has read P, and O^T holds its sum
      if (i > 0) wait(B_PVDONE, (i - 1) & 1);
      tc_fence_after();
      if (rescale_o) {
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          const uint32_t ta = tmem + 64u * mb + hcol + lane_off;
          uint32_t x[HPW];
          DSA_TMEM_LD_X16(ta, x);
#pragma unroll
          for (int c = 0; c < HPW; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * alpha[hcol + c]);
          DSA_TMEM_ST_X16(ta, x);
        }
      }
      uint8_t* const at = smem + OFF_P + sw128_off(head, 2 * grp + upper);
      *reinterpret_cast<uint4*>(at) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
      *reinterpret_cast<uint4*>(at + RSUB) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_PFULL));
      ring.next();
      if (--left > 0) continue;
      if (i + 1 < n) {  // the next row's query, while the last PV runs (S has read the present one)
        wait(B_EMPTY + ring.slot, ring.phase ^ 1);
        uint2 hi, lo;
        q_stage(row_of(p, item + 1).row, item + 1, ring.slot, 4 * warp, hi, lo);
        q_stage_rope(4 * warp, hi, lo);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_QFULL));
        ring.next();
      }
      // ---- end of item: wait for its last PV, reduce the row sums, write the output
      const int32_t row = row_of(p, item++).row;
      float l = unpack2(lsum).x + unpack2(lsum).y;
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      wait(B_PVDONE, i & 1);  // every warp has written P, so none still reads its tile's maxima in red
      tc_fence_after();
      if (upper == 0) red[grp * 64 + head] = l;
      named_bar(1, SM_THREADS);
      const bool whole = p.parts == 1 || row < p.whole_rows * static_cast<int32_t>(gridDim.x);
      const int64_t pr = blockIdx.x;
      if (grp == 0 && upper == 0) {
        l = 256.f * (red[head] + red[64 + head] + red[128 + head] + red[192 + head]);  // sum of p
        alpha[head] = l == 0.f ? 0.f : 1.f / l;
        if (!whole) {
          p.part_ml[pr * 128 + head] = l == 0.f ? -INFINITY : -nn - 8.f;
          p.part_ml[pr * 128 + 64 + head] = l;
        } else if (p.lse) {
          p.lse[static_cast<int64_t>(row) * 64 + head] = l == 0.f ? -INFINITY : (log2f(l) - nn - 8.f) * 0.69314718055994531f;
        }
      }
      if (whole) {
        named_bar(1, SM_THREADS);  // alpha
        uint16_t* orow = p.out + static_cast<int64_t>(row) * 64 * 512;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t x[HPW];
          DSA_TMEM_LD_X16(tmem + 64u * mb + hcol + lane_off, x);
#pragma unroll
          for (int c = 0; c < HPW; c += 4) {  // 4 heads of one dim per lane -> 4 dims of one head per lane
            const float4 a = *reinterpret_cast<const float4*>(alpha + hcol + c);
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(__uint_as_float(x[c]) * a.x, __uint_as_float(x[c + 1]) * a.y);
            const __nv_bfloat162 b1 = __floats2bfloat162_rn(__uint_as_float(x[c + 2]) * a.z, __uint_as_float(x[c + 3]) * a.w);
            uint32_t u = *reinterpret_cast<const uint32_t*>(&b0), v = *reinterpret_cast<const uint32_t*>(&b1);
            const uint32_t un = __shfl_xor_sync(0xffffffffu, u, 1), vn = __shfl_xor_sync(0xffffffffu, v, 1);
            u = lane & 1 ? __byte_perm(un, u, 0x7632) : __byte_perm(u, un, 0x5410);  // two dims of head c + lane % 2
            v = lane & 1 ? __byte_perm(vn, v, 0x7632) : __byte_perm(v, vn, 0x5410);  // and of head c + 2 + lane % 2
            const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 2 ? u : v, 2);
            const uint2 w = lane & 2 ? make_uint2(got, v) : make_uint2(u, got);
            *reinterpret_cast<uint2*>(orow + (hcol + c + (lane & 3)) * 512 + mb * 128 + (dim & ~3)) = w;
          }
        }
      } else {
        float4* po = reinterpret_cast<float4*>(p.part_o + pr * 64 * 512);  // [16 head quads][512 dims] of 4 heads
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t x[HPW];
          DSA_TMEM_LD_X16(tmem + 64u * mb + hcol + lane_off, x);
#pragma unroll
          for (int c = 0; c < HPW; c += 4)
            po[((hcol + c) >> 2) * 512 + mb * 128 + dim] =
                make_float4(__uint_as_float(x[c]), __uint_as_float(x[c + 1]), __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]));
        }
      }
      left = min(tpr, n - 1 - i);
      nn = BIAS;
      lsum = 0ull;
      seen = false;
      tc_fence_before();
      named_bar(1, SM_THREADS);  // alpha and red are the next item's
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// Cut rows: out = sum_s w_s O_s / sum_s w_s l_s, w_s = 2^(m_s - max m).  One block of 128 threads per 4 heads of a cut row
// (DIMS = 4: 4 dims of 4 heads per thread), or per 4 heads and 128 dims (DIMS = 1) when the rows are few and cut into many
// parts (at most 16: k <= 2,048).  One warp forms the weights while the first EARLY parts are on their way to everyone.
// Bound by the latency of its loads: 7.1 us alone and from cold caches for 6 rows of 16 parts (12.6 MB).
constexpr int COMBINE_THREADS = 128;
template <int DIMS, int EARLY>
__global__ void __launch_bounds__(COMBINE_THREADS) combine4_kernel(const float* __restrict__ part_o,
                                                                   const float* __restrict__ part_ml, int32_t n,
                                                                   int32_t base, uint16_t* __restrict__ out,
                                                                   float* __restrict__ lse) {
  grid_dependency_sync();
  __shared__ __align__(16) float wgt[16][4];  // a fragment's weights are read at once
  __shared__ float inv[4];
  const int32_t hq = blockIdx.y, dim = (DIMS == 1 ? blockIdx.z * COMBINE_THREADS : 0) + threadIdx.x;
  const int32_t row = base + blockIdx.x;  // the cut rows' parts, n each, follow one another
  auto frag = [&](int s) { return static_cast<int32_t>(blockIdx.x) * n + s; };
  float4 o[EARLY][DIMS];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int u = 0; u < EARLY; ++u)
#pragma unroll
      for (int d = 0; d < DIMS; ++d)
        o[u][d] = s0 + u < n ? reinterpret_cast<const float4*>(part_o)[(static_cast<int64_t>(frag(s0 + u)) * 16 + hq) * 512 +
                                                                      dim + d * COMBINE_THREADS]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  fetch(0);
  if (threadIdx.x < 32) {  // lane = (fragment, head) of fragments 0..7, and the same of 8..15
    const int s = threadIdx.x >> 2, e = threadIdx.x & 3;
    float m[2], l[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool in = s + 8 * u < n;
      m[u] = in ? part_ml[frag(s + 8 * u) * 128 + hq * 4 + e] : -INFINITY;
      l[u] = in ? part_ml[frag(s + 8 * u) * 128 + 64 + hq * 4 + e] : 0.f;
    }
    float M = fmaxf(m[0], m[1]);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float L = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float w = l[u] == 0.f ? 0.f : exp2f(m[u] - (M == -INFINITY ? 0.f : M));  // 0: a fragment without a key
      wgt[s + 8 * u][e] = w;
      L = fmaf(w, l[u], L);
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    if (s == 0) {
      inv[e] = L == 0.f ? 0.f : 1.f / L;
      if (lse && (DIMS == 4 || blockIdx.z == 0))
        lse[static_cast<int64_t>(row) * 64 + hq * 4 + e] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  float4 acc[DIMS];
#pragma unroll
  for (int d = 0; d < DIMS; ++d) acc[d] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += EARLY) {
    if (s0 > 0) fetch(s0);
#pragma unroll
    for (int u = 0; u < EARLY; ++u) {
      if (s0 + u >= n) break;
      const float4 w = *reinterpret_cast<const float4*>(wgt[s0 + u]);
#pragma unroll
      for (int d = 0; d < DIMS; ++d) {
        acc[d].x = fmaf(w.x, o[u][d].x, acc[d].x);
        acc[d].y = fmaf(w.y, o[u][d].y, acc[d].y);
        acc[d].z = fmaf(w.z, o[u][d].z, acc[d].z);
        acc[d].w = fmaf(w.w, o[u][d].w, acc[d].w);
      }
    }
  }
#pragma unroll
  for (int d = 0; d < DIMS; ++d) {
    const float a[4] = {acc[d].x, acc[d].y, acc[d].z, acc[d].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat16 v = __float2bfloat16_rn(a[e] * inv[e]);
      out[(static_cast<int64_t>(row) * 64 + hq * 4 + e) * 512 + dim + d * COMBINE_THREADS] = *reinterpret_cast<const uint16_t*>(&v);
    }
  }
}

}  // namespace mla4
}  // namespace dsa
