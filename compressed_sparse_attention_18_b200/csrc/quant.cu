// FP8 quantisation in blocks of 128 channels: E4M3 codes with one fp32 scale for 128 channels of one row
// (activations) or for a block of 128 rows x 128 channels (weights), the operands of csa_gemm_fp8.
//
//   scale = fp32(amax / 448), code = E4M3_rne_satfinite(fp32(x / scale)), -0 -> +0; amax == 0 -> scale 0,
//   codes 0 (the rule of the FP8 window rows, with 128 channels to a block).  A NaN has no part in amax and
//   becomes the NaN code; an infinity makes the scale infinite, itself NaN and the block's other codes 0.
//
// Bound by HBM: 2 bytes read and 1 written an element (4096 x 4096 in rows: 10.0 us, 5.1 TB/s), with the instructions of
// the quotients close behind (11.8 an element, 60 % of the issue slots).  A block is kept in registers between its
// maximum and its codes, so the source is read once.
#include "csa_common.cuh"

namespace csa {

constexpr int Q8_BLOCK = 128;

// The divisor of a block and how to divide by it.  fp32(x / s) for many x and one s: with r the correctly rounded
// 1 / s and q = x r, q + r (x - q s) with two fused multiply-adds is the correctly rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990) as long as nothing leaves the
// normal range.  s in [2^-60, 2^60] keeps 1 / s, q and the residual in it, except where x / s is so small that its code
// is 0 whatever the residual; other scales take the plain division.
struct Q8Div {
  float s, r;
  bool fast;
};
__device__ __forceinline__ Q8Div q8_div(float sc) {
  Q8Div d;
  d.s = sc > 0.0f ? sc : 1.0f;                     // a block of zeros (and NaN)
  d.fast = sc >= 0x1p-60f && sc <= 0x1p60f;
  d.r = d.fast ? __frcp_rn(sc) : 0.0f;
  return d;
}

// Four E4M3 bytes, -0 as +0.
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  const uint32_t w = (uint32_t)lo | ((uint32_t)hi << 16);
  // a byte keeps its sign bit only if its magnitude is not 0
  const uint32_t m = w & 0x7F7F7F7Fu;
  return w & (m | (m + 0x7F7F7F7Fu));
}

// E4M3 bytes of fp32(x_e / s), 8 elements to a uint2.
__device__ __forceinline__ uint2 q8_codes8(const float* x, const Q8Div& d) {
  float q[8];
  if (d.fast) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = x[e] * d.r;
      q[e] = __fmaf_rn(d.r, __fmaf_rn(-y, d.s, x[e]), y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(x[e], d.s);
  }
  return make_uint2(q8_pack4(q[0], q[1], q[2], q[3]), q8_pack4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ void q8_unpack(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = bf16_bits_to_f(w[e] & 0xFFFFu);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float q8_amax8(const float* x) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(x[e]));
  return a;
}

// Rows: 8 lanes take one block of one row, two vectors of 8 elements (16 bytes) each.  EVEN (K a multiple of 128): the
// blocks of all rows follow one another, block u at element 128 u.  Two blocks a lane
// in flight take a tenth longer, four half as long again (fewer warps fit), 16 lanes a block a quarter (the scale's two
// divisions are paid by each lane).
template <bool EVEN>
__global__ void __launch_bounds__(256) quant_rows_kernel(const uint16_t* __restrict__ src, long long total, int K, int KB,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int sub = threadIdx.x & 7;
  pdl_trigger();
  pdl_wait();
  // every lane of a warp takes part in the reduction, the ones behind the last block with zeros
  const long long u = (long long)blockIdx.x * 32 + (threadIdx.x >> 3);
  long long at = -1;                               // the lane's first element of the block, -1 where there is none
  int left = Q8_BLOCK;                             // elements of the row from there on
  if (EVEN) {
    if (u < total) at = u * Q8_BLOCK + 8 * sub;
  } else {
    const long long row = u / KB;
    const int k0 = (int)(u - row * KB) * Q8_BLOCK + 8 * sub;
    left = K - k0;
    if (u < total && left > 0) at = row * K + k0;
  }
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (at >= 0) v0 = *reinterpret_cast<const uint4*>(src + at);
  if (at >= 0 && left > 64) v1 = *reinterpret_cast<const uint4*>(src + at + 64);
  float x[16];
  q8_unpack(v0, x);
  q8_unpack(v1, x + 8);
  float amax = fmaxf(q8_amax8(x), q8_amax8(x + 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float sc = __fdiv_rn(amax, 448.0f);
  const Q8Div d = q8_div(sc);
  if (at >= 0) *reinterpret_cast<uint2*>(codes + at) = q8_codes8(x, d);
  if (at >= 0 && left > 64)
    *reinterpret_cast<uint2*>(codes + at + 64) = q8_codes8(x + 8, d);
  if (sub == 0 && u < total) scales[u] = sc;
}

// Weights: one CTA takes one block of 128 rows x 128 channels, VEC vectors of 8 elements a thread.
template <int VEC>
__global__ void __launch_bounds__(Q8_BLOCK * Q8_BLOCK / 8 / VEC) quant_blocks_kernel(const uint16_t* __restrict__ src, long long rows, int K,
                                                                            uint8_t* __restrict__ codes,
                                                                            float* __restrict__ scales) {
  constexpr int THREADS = Q8_BLOCK * Q8_BLOCK / 8 / VEC, STEP = THREADS / 16;   // STEP: rows the CTA covers at once
  __shared__ float red[THREADS / 32];
  const int KB = (K + Q8_BLOCK - 1) / Q8_BLOCK;
  const int kb = (int)(blockIdx.x % KB);
  const long long r0 = (long long)(blockIdx.x / KB) * Q8_BLOCK + (threadIdx.x >> 4);
  const int k0 = kb * Q8_BLOCK + 8 * (threadIdx.x & 15);
  pdl_trigger();
  pdl_wait();
  uint4 v[VEC];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (r0 + STEP * i < rows && k0 < K) v[i] = *reinterpret_cast<const uint4*>(src + (r0 + STEP * i) * K + k0);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    float x[8];
    q8_unpack(v[i], x);
    amax = fmaxf(amax, q8_amax8(x));
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) amax = fmaxf(amax, red[i]);
  const float sc = __fdiv_rn(amax, 448.0f);
  const Q8Div d = q8_div(sc);
  if (threadIdx.x == 0) scales[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if (r0 + STEP * i >= rows || k0 >= K) continue;
    float x[8];
    q8_unpack(v[i], x);
    *reinterpret_cast<uint2*>(codes + (r0 + STEP * i) * K + k0) = q8_codes8(x, d);
  }
}

template <bool EVEN>
static csa_status launch_quant_rows(const csa_quant_fp8_args* a, cudaStream_t st) {
  const int KB = (a->K + Q8_BLOCK - 1) / Q8_BLOCK;
  const long long total = (long long)a->rows * KB, blocks = (total + 31) / 32;
  CSA_SUPPORTED(blocks <= 0x7fffffffLL);
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)quant_rows_kernel<EVEN>, 0, attr_done);
  return launch_pdl(quant_rows_kernel<EVEN>, dim3((unsigned)blocks), dim3(256), 0, st, (const uint16_t*)a->src, total,
                    a->K, KB, a->codes, a->scales);
}

template <int VEC>
static csa_status launch_quant_blocks(const csa_quant_fp8_args* a, unsigned blocks, cudaStream_t st) {
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)quant_blocks_kernel<VEC>, 0, attr_done);
  return launch_pdl(quant_blocks_kernel<VEC>, dim3(blocks), dim3(Q8_BLOCK * Q8_BLOCK / 8 / VEC), 0, st,
                    (const uint16_t*)a->src, (long long)a->rows, a->K, a->codes, a->scales);
}

}  // namespace csa

using namespace csa;

extern "C" csa_status csa_quant_fp8(const csa_quant_fp8_args* a, void* stream) {
  CSA_REQUIRE(a != nullptr && a->struct_size == sizeof(csa_quant_fp8_args));
  CSA_REQUIRE(a->rows >= 0 && a->K >= 1);
  CSA_REQUIRE(a->block_rows == 1 || a->block_rows == Q8_BLOCK);
  CSA_SUPPORTED(a->K % 16 == 0);
  if (a->rows == 0) return CSA_OK;
  CSA_REQUIRE(a->src && a->codes && a->scales);
  CSA_SUPPORTED(((uintptr_t)a->src & 15) == 0 && ((uintptr_t)a->codes & 15) == 0 && ((uintptr_t)a->scales & 3) == 0);
  if (a->block_rows == 1)
    return a->K % Q8_BLOCK == 0 ? launch_quant_rows<true>(a, (cudaStream_t)stream) : launch_quant_rows<false>(a, (cudaStream_t)stream);
  const long long KB = (a->K + Q8_BLOCK - 1) / Q8_BLOCK;
  const long long blocks = ((long long)a->rows + Q8_BLOCK - 1) / Q8_BLOCK * KB;
  CSA_SUPPORTED(blocks <= 0x7fffffffLL);
  // 1024 threads a block while one wave takes them all (the shortest chain: 1000 x 2064 in 2.6 us, 3.8 with 512), 512
  // beyond (4096 x 4096 in 15.3 us, 3.3 TB/s; 23.4 with 1024, 17.8 with 256)
  return blocks <= 2 * 148 ? launch_quant_blocks<2>(a, (unsigned)blocks, (cudaStream_t)stream)
                           : launch_quant_blocks<4>(a, (unsigned)blocks, (cudaStream_t)stream);
}
