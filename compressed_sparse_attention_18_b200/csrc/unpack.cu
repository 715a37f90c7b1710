// Reading the caches back: entries of an FP4 cache and rows of an FP8 window as bf16 rows, a range of rows
// or a list of ids per sequence.
//
//   FP4:  x = bf16(fp32(e2m1 * e4m3 * g))   (e2m1 * e4m3 has at most 6 significant bits: exact; one fp32 rounding
//         by g, none when g is a power of two, and the bf16 rounding, which is exact then too)
//   FP8:  x = bf16(fp32(e4m3 * scale))
//   the RoPE channels are copied.
//
// Bound by HBM: 366 bytes read and 1024 written an FP4 entry of 512 channels, 604 and 1024 an FP8 row.
#include "csa_common.cuh"

namespace csa {

struct UnpackParams {
  long long total;        // B * n output rows
  int n, d_n, d_r, n_max; // n_max: rows a sequence holds (window: Wn)
  float g;
  const uint8_t* codes;
  const uint8_t* scales8;  // FP4: E4M3 bytes
  const float* scales32;   // FP8
  const uint16_t* rope;
  const int32_t* row0;
  const int32_t* idx;
  uint16_t* out;
  csa_page_map pm;
};

// One warp per output row; a lane writes 8 channels (16 bytes) at a time.
template <bool FP8>
__global__ void __launch_bounds__(256) unpack_kernel(const UnpackParams P) {
  const int lane = threadIdx.x & 31;
  const int d = P.d_n + P.d_r;
  const int nb = P.d_n / (FP8 ? 64 : 32), nb_pad = (nb + 3) & ~3;
  pdl_trigger();
  pdl_wait();
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < P.total; r += (long long)gridDim.x * 8) {
    const int b = (int)(r / P.n);
    const long long j = r % P.n;
    const long long i = P.idx ? (long long)P.idx[r] : (long long)(P.row0 ? P.row0[b] : 0) + j;
    long long row = -1;                            // absent: a zero row
    if (i >= 0 && i < P.n_max) row = FP8 ? (long long)b * P.n_max + i : page_row(P.pm, b, P.n_max, i);
    uint4* o = reinterpret_cast<uint4*>(P.out + r * d);
    for (int c = lane; c < (d >> 3); c += 32) {
      const int e = 8 * c;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row >= 0 && e >= P.d_n) {
        v = *reinterpret_cast<const uint4*>(P.rope + row * P.d_r + (e - P.d_n));
      } else if (row >= 0 && FP8) {
        const uint2 w = *reinterpret_cast<const uint2*>(P.codes + row * P.d_n + e);
        const float s = P.scales32[row * nb_pad + (e >> 6)];
        const uint32_t w2[2] = {w.x, w.y};
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t two = w2[k >> 1] >> (16 * (k & 1));
          y[k] = pack_bf16x2(__fmul_rn(e4m3_to_f32(two), s), __fmul_rn(e4m3_to_f32(two >> 8), s));
        }
        v = make_uint4(y[0], y[1], y[2], y[3]);
      } else if (row >= 0) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(P.codes + row * (P.d_n >> 1) + (e >> 1));
        const float s = e4m3_to_f32(P.scales8[row * nb_pad + (e >> 5)]);
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t h2 = e2m1x2_to_h2(w >> (8 * k));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          y[k] = pack_bf16x2(__fmul_rn(f.x * s, P.g), __fmul_rn(f.y * s, P.g));
        }
        v = make_uint4(y[0], y[1], y[2], y[3]);
      }
      o[c] = v;
    }
  }
}

template <bool FP8>
static csa_status launch_unpack(const UnpackParams& P, cudaStream_t st) {
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)unpack_kernel<FP8>, 0, attr_done);
  long long blocks = (P.total + 7) / 8;
  if (blocks > 148 * 16) blocks = 148 * 16;
  return launch_pdl(unpack_kernel<FP8>, dim3((unsigned)blocks), dim3(256), 0, st, P);
}

}  // namespace csa

using namespace csa;

extern "C" csa_status csa_unpack_fp4(const csa_unpack_args* a, void* stream) {
  CSA_REQUIRE(a != nullptr && a->struct_size == sizeof(csa_unpack_args));
  CSA_REQUIRE(a->B >= 0 && a->n >= 0 && a->d > 0 && a->d_rope >= 0 && a->d_rope <= a->d && a->n_max >= 0);
  CSA_SUPPORTED((a->d - a->d_rope) % 32 == 0 && a->d_rope % 8 == 0);
  {
    const csa_status pv = check_page_map(a->pages, a->n_max);
    if (pv != CSA_OK) return pv;
  }
  if ((long long)a->B * a->n == 0) return CSA_OK;
  CSA_REQUIRE(a->out && !(a->idx && a->row0));
  CSA_REQUIRE(a->n_max == 0 || a->d == a->d_rope || (a->codes && a->scales));
  CSA_REQUIRE(a->n_max == 0 || a->d_rope == 0 || a->rope);
  CSA_REQUIRE(a->global_scale > 0.0f);
  CSA_SUPPORTED((((uintptr_t)a->out | (uintptr_t)a->codes | (uintptr_t)a->rope) & 15) == 0 &&
                ((uintptr_t)a->scales & 3) == 0);
  UnpackParams P{};
  P.total = (long long)a->B * a->n;
  P.n = a->n; P.d_n = a->d - a->d_rope; P.d_r = a->d_rope; P.n_max = a->n_max; P.g = a->global_scale;
  P.codes = a->codes; P.scales8 = (const uint8_t*)a->scales; P.rope = (const uint16_t*)a->rope;
  P.row0 = a->row0; P.idx = a->idx; P.out = (uint16_t*)a->out; P.pm = a->pages;
  return launch_unpack<false>(P, (cudaStream_t)stream);
}

extern "C" csa_status csa_unpack_fp8_window(const csa_unpack_args* a, void* stream) {
  CSA_REQUIRE(a != nullptr && a->struct_size == sizeof(csa_unpack_args));
  CSA_REQUIRE(a->B >= 0 && a->n >= 0 && a->d > 0 && a->d_rope >= 0 && a->d_rope <= a->d && a->n_max >= 0);
  CSA_SUPPORTED((a->d - a->d_rope) % 64 == 0 && a->d_rope % 8 == 0);
  CSA_SUPPORTED(a->pages.table == nullptr);       // windows are not paged
  if ((long long)a->B * a->n == 0) return CSA_OK;
  CSA_REQUIRE(a->out && !(a->idx && a->row0));
  CSA_REQUIRE(a->n_max == 0 || a->d == a->d_rope || (a->codes && a->scales));
  CSA_REQUIRE(a->n_max == 0 || a->d_rope == 0 || a->rope);
  CSA_SUPPORTED((((uintptr_t)a->out | (uintptr_t)a->codes | (uintptr_t)a->rope | (uintptr_t)a->scales) & 15) == 0);
  UnpackParams P{};
  P.total = (long long)a->B * a->n;
  P.n = a->n; P.d_n = a->d - a->d_rope; P.d_r = a->d_rope; P.n_max = a->n_max; P.g = 1.0f;
  P.codes = a->codes; P.scales32 = (const float*)a->scales; P.rope = (const uint16_t*)a->rope;
  P.row0 = a->row0; P.idx = a->idx; P.out = (uint16_t*)a->out;
  return launch_unpack<true>(P, (cudaStream_t)stream);
}
