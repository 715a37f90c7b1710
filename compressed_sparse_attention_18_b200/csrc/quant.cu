// FP8 quantisation in blocks of 128 channels: E4M3 codes with one fp32 scale for 128 channels of one row
// (activations) or for a block of 128 rows x 128 channels (weights), the operands of csa_gemm_fp8.
//
//   scale = fp32(amax / 448), code = E4M3_rne_satfinite(fp32(x / scale)), -0 -> +0; amax == 0 -> scale 0,
//   codes 0 (the rule of the FP8 window rows, with 128 channels to a block).  A NaN has no part in amax and
//   becomes the NaN code; an infinity makes the scale infinite, itself NaN and the block's other codes 0.
//
// Bound by HBM: 2 bytes read and 1 written an element.  A block is kept in registers between its maximum and
// its codes, so the source is read once.
#include "csa_common.cuh"

namespace csa {

constexpr int Q8_BLOCK = 128;

// Four E4M3 bytes of fp32(x_e / sc), -0 as +0.
__device__ __forceinline__ uint32_t q8_codes4(const float* x, float sc) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t c = f32_to_e4m3(__fdiv_rn(x[e], sc));
    w |= ((c & 0x7Fu) ? c : 0u) << (8 * e);
  }
  return w;
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

// Rows: 16 lanes take one block of one row, 8 elements (16 bytes) each.
__global__ void __launch_bounds__(256) quant_rows_kernel(const uint16_t* __restrict__ src, long long rows, int K,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int KB = (K + Q8_BLOCK - 1) / Q8_BLOCK;
  const int sub = threadIdx.x & 15;
  const long long total = rows * KB;
  pdl_trigger();
  pdl_wait();
  // every lane of a warp takes part in the reduction, the ones behind the last block with zeros
  for (long long u0 = (long long)blockIdx.x * 16; u0 < total; u0 += (long long)gridDim.x * 16) {
    const long long u = u0 + (threadIdx.x >> 4);
    const long long row = u / KB;
    const int kb = (int)(u % KB);
    const int k0 = kb * Q8_BLOCK + 8 * sub;
    const bool in = u < total && k0 < K;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = *reinterpret_cast<const uint4*>(src + row * K + k0);
    float x[8];
    q8_unpack(v, x);
    float amax = q8_amax8(x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float sc = __fdiv_rn(amax, 448.0f);
    const float den = sc > 0.0f ? sc : 1.0f;          // a block of zeros (and NaN)
    const uint2 c = make_uint2(q8_codes4(x, den), q8_codes4(x + 4, den));
    if (in) *reinterpret_cast<uint2*>(codes + row * K + k0) = c;
    if (u < total && sub == 0) scales[u] = sc;
  }
}

// Weights: one CTA takes one block of 128 rows x 128 channels, 8 vectors of 8 elements a thread.
__global__ void __launch_bounds__(256) quant_blocks_kernel(const uint16_t* __restrict__ src, long long rows, int K,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float red[8];
  const int KB = (K + Q8_BLOCK - 1) / Q8_BLOCK;
  const int kb = (int)(blockIdx.x % KB);
  const long long r0 = (long long)(blockIdx.x / KB) * Q8_BLOCK;
  const int k0 = kb * Q8_BLOCK + 8 * (threadIdx.x & 15);
  pdl_trigger();
  pdl_wait();
  uint4 v[8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long row = r0 + 16 * i + (threadIdx.x >> 4);
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && k0 < K) v[i] = *reinterpret_cast<const uint4*>(src + row * K + k0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x[8];
    q8_unpack(v[i], x);
    amax = fmaxf(amax, q8_amax8(x));
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, red[i]);
  const float sc = __fdiv_rn(amax, 448.0f);
  const float den = sc > 0.0f ? sc : 1.0f;
  if (threadIdx.x == 0) scales[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long row = r0 + 16 * i + (threadIdx.x >> 4);
    if (row >= rows || k0 >= K) continue;
    float x[8];
    q8_unpack(v[i], x);
    const uint2 c = make_uint2(q8_codes4(x, den), q8_codes4(x + 4, den));
    *reinterpret_cast<uint2*>(codes + row * K + k0) = c;
  }
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
  const long long KB = (a->K + Q8_BLOCK - 1) / Q8_BLOCK;
  if (a->block_rows == 1) {
    static std::atomic<unsigned> attr_done{0};
    set_smem_once((const void*)quant_rows_kernel, 0, attr_done);
    long long blocks = (a->rows * KB + 15) / 16;
    if (blocks > 148 * 16) blocks = 148 * 16;
    return launch_pdl(quant_rows_kernel, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream,
                      (const uint16_t*)a->src, (long long)a->rows, a->K, a->codes, a->scales);
  }
  const long long blocks = ((long long)a->rows + Q8_BLOCK - 1) / Q8_BLOCK * KB;
  CSA_SUPPORTED(blocks <= 0x7fffffffLL);
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)quant_blocks_kernel, 0, attr_done);
  return launch_pdl(quant_blocks_kernel, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream,
                    (const uint16_t*)a->src, (long long)a->rows, a->K, a->codes, a->scales);
}
