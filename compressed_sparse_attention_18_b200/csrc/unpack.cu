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
  uint32_t total, n;      // output rows, and of one sequence
  int cpr;                // 16-byte chunks of an output row (d / 8)
  int d_n, d_r, n_max;    // n_max: rows a sequence holds (window: Wn)
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

// One warp writes one row, a lane two chunks of 8 channels (16 bytes) at a time, both loaded before either is used; the
// many small warps keep more reads in flight than several rows a warp (32768 FP4 entries: 11.8 us, 3.9 TB/s; two rows
// 12.9, four 17.4).
template <bool FP8>
__global__ void __launch_bounds__(256) unpack_kernel(const UnpackParams P) {
  const int nb_pad = (P.d_n / (FP8 ? 64 : 32) + 3) & ~3;
  const uint32_t r = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  if (r >= P.total) return;
  const int b = (int)(r / P.n);
  const long long i = P.idx ? (long long)__ldg(P.idx + r) : (long long)(P.row0 ? __ldg(P.row0 + b) : 0) + (r - b * P.n);
  long long row = -1;                              // absent: a zero row
  if (i >= 0 && i < P.n_max) row = FP8 ? (long long)b * P.n_max + i : page_row(P.pm, b, P.n_max, i);
  for (int c0 = threadIdx.x & 31; c0 < P.cpr; c0 += 64) {
    uint4 raw[2];                                  // RoPE slice: the chunk; else its codes in x (FP8: x, y), FP4 scale in y
    float s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 8 * (c0 + 32 * u);
      raw[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.f;
      if (row < 0 || c0 + 32 * u >= P.cpr) continue;
      if (e >= P.d_n) {
        raw[u] = __ldg(reinterpret_cast<const uint4*>(P.rope + row * P.d_r + (e - P.d_n)));
      } else if (FP8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(P.codes + row * P.d_n + e));
        raw[u].x = w.x;
        raw[u].y = w.y;
        s[u] = __ldg(P.scales32 + row * nb_pad + (e >> 6));
      } else {
        raw[u].x = __ldg(reinterpret_cast<const uint32_t*>(P.codes + row * (P.d_n >> 1) + (e >> 1)));
        raw[u].y = __ldg(P.scales8 + row * nb_pad + (e >> 5));
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (c0 + 32 * u >= P.cpr) continue;
      uint4 v = raw[u];
      if (8 * (c0 + 32 * u) < P.d_n) {
        uint32_t y[4];
        const float sc = FP8 ? s[u] : e4m3_to_f32(raw[u].y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t h2;
          if (FP8) {
            const uint16_t two = (uint16_t)((k < 2 ? raw[u].x : raw[u].y) >> (16 * (k & 1)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
          } else {
            h2 = e2m1x2_to_h2(raw[u].x >> (8 * k));
          }
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          y[k] = FP8 ? pack_bf16x2(__fmul_rn(f.x, sc), __fmul_rn(f.y, sc))
                     : pack_bf16x2(__fmul_rn(f.x * sc, P.g), __fmul_rn(f.y * sc, P.g));
        }
        v = make_uint4(y[0], y[1], y[2], y[3]);
      }
      reinterpret_cast<uint4*>(P.out)[(unsigned long long)r * P.cpr + c0 + 32 * u] = v;
    }
  }
}

template <bool FP8>
static csa_status launch_unpack(const csa_unpack_args* a, UnpackParams P, cudaStream_t st) {
  const long long total = (long long)a->B * a->n;
  CSA_SUPPORTED(total <= 0x7fffffffLL);
  P.total = (uint32_t)total;
  P.n = (uint32_t)a->n;
  P.cpr = a->d / 8;
  P.d_n = a->d - a->d_rope;
  P.d_r = a->d_rope;
  P.n_max = a->n_max;
  P.codes = a->codes;
  P.rope = (const uint16_t*)a->rope;
  P.row0 = a->row0;
  P.idx = a->idx;
  P.out = (uint16_t*)a->out;
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)unpack_kernel<FP8>, 0, attr_done);
  return launch_pdl(unpack_kernel<FP8>, dim3((unsigned)((total + 7) / 8)), dim3(256), 0, st, P);
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
  P.g = a->global_scale;
  P.scales8 = (const uint8_t*)a->scales;
  P.pm = a->pages;
  return launch_unpack<false>(a, P, (cudaStream_t)stream);
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
  P.scales32 = (const float*)a->scales;
  return launch_unpack<true>(a, P, (cudaStream_t)stream);
}
