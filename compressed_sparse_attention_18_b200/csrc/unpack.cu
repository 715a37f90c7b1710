// Reading the caches back: entries of an FP4 cache and rows of an FP8 window as bf16 rows, a range of rows
// or a list of ids per sequence.
//
//   FP4:  x = bf16(fp32(e2m1 * e4m3 * g))   (e2m1 * e4m3 has at most 6 significant bits: exact; one fp32 rounding
//         by g, none when g is a power of two, and the bf16 rounding, which is exact then too)
//   FP8:  x = bf16(fp32(e4m3 * scale))
//   the RoPE channels are copied.
//
// 366 bytes are read and 1024 written an FP4 entry of 512 channels, 604 and 1024 an FP8 row.  FP4 is bound by the
// conversions' instructions (17 an element, 82 % of the issue slots): 32768 entries take 10.7 us, 8.0 with the bytes
// stored as they are; filling as much memory with zeros takes 9.4.  FP8 is bound by HBM, and there by the writes: 65536
// rows take 22.2 us, 21.4 with the bytes as they are, a fill 17.7 (3.8 TB/s).
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

// Eight channels as bf16: of an FP4 entry (4 code bytes, scale byte, global scale), of an FP8 row (8 codes, scale).
__device__ __forceinline__ uint4 fp4x8_to_bf16(uint32_t codes, uint32_t scale, float g) {
  const float sc = e4m3_to_f32(scale);
  uint32_t y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t h2 = e2m1x2_to_h2(codes >> (8 * k));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    y[k] = pack_bf16x2(__fmul_rn(f.x * sc, g), __fmul_rn(f.y * sc, g));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ uint4 fp8x8_to_bf16(uint32_t c0, uint32_t c1, float sc) {
  uint32_t y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h2;
    const uint16_t two = (uint16_t)((k < 2 ? c0 : c1) >> (16 * (k & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    y[k] = pack_bf16x2(__fmul_rn(f.x, sc), __fmul_rn(f.y, sc));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// One warp writes one row, a lane two chunks of 8 channels (16 bytes) at a time, both loaded before either is used; the
// many small warps keep more reads in flight than several rows a warp (32768 FP4 entries: 10.8 us; two rows a warp 12.9,
// four 17.4).
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
      if (8 * (c0 + 32 * u) < P.d_n) v = FP8 ? fp8x8_to_bf16(raw[u].x, raw[u].y, s[u]) : fp4x8_to_bf16(raw[u].x, raw[u].y, P.g);
      reinterpret_cast<uint4*>(P.out)[(unsigned long long)r * P.cpr + c0 + 32 * u] = v;
    }
  }
}

// A sequence's own keys for the shared-prefix attention, bf16 rows of 512: cache entries first .. n_max - 1 (zero from
// n_c on: the cache holds anything there), then the window buffer.  A row with a NaN or an infinity becomes zero and is
// marked, since the attention multiplies rows with weights of queries that do not see them.  One warp per row as above.
struct OwnRowsParams {
  uint32_t total, per;     // rows, and of one sequence: E entries, then the window's
  int first, E, n_max, Wn;
  float g;
  const int32_t* n_c;
  const uint8_t* codes;
  const uint8_t* scales;
  const uint16_t* rope;
  const uint16_t* win;     // bf16 window, or null:
  const uint8_t* wcodes;
  const float* wscales;
  const uint16_t* wrope;
  uint16_t* out;
  uint8_t* bad;            // [B][stride]: 1 for a row that is not finite
  uint32_t stride;
  csa_page_map pm;
};

__global__ void __launch_bounds__(256) own_rows_kernel(const OwnRowsParams P) {
  const uint32_t r = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // in this order: the attention behind this kernel reads inputs of earlier work as soon as it starts
  pdl_wait();
  pdl_trigger();
  if (r >= P.total) return;
  const int b = (int)(r / P.per), u = (int)(r % P.per);
  uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (u < P.E) {
    const int i = P.first + u;
    const long long row = i < min(__ldg(P.n_c + b), P.n_max) ? page_row(P.pm, b, P.n_max, i) : -1;
    if (row >= 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = lane + 32 * k;
        if (c >= 56)
          v[k] = __ldg(reinterpret_cast<const uint4*>(P.rope + row * 64) + (c - 56));
        else
          v[k] = fp4x8_to_bf16(__ldg(reinterpret_cast<const uint32_t*>(P.codes + row * 224) + c), __ldg(P.scales + row * 16 + (c >> 2)), P.g);
      }
    }
  } else {
    const long long row = (long long)b * P.Wn + (u - P.E);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = lane + 32 * k;
      if (P.win) {
        v[k] = __ldg(reinterpret_cast<const uint4*>(P.win + row * 512) + c);
      } else if (c >= 56) {
        v[k] = __ldg(reinterpret_cast<const uint4*>(P.wrope + row * 64) + (c - 56));
      } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(P.wcodes + row * 448) + c);
        v[k] = fp8x8_to_bf16(w.x, w.y, __ldg(P.wscales + row * 8 + (c >> 3)));
      }
    }
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (x[i] & 0x7F800000u) == 0x7F800000u || (x[i] & 0x7F80u) == 0x7F80u;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad) v[0] = v[1] = make_uint4(0, 0, 0, 0);
  if (lane == 0) P.bad[(size_t)b * P.stride + u] = bad;
  uint4* o = reinterpret_cast<uint4*>(P.out + (size_t)r * 512);
  o[lane] = v[0];
  o[lane + 32] = v[1];
}

// Writes [B][n_max - first + Wn][512] and, behind it, the marks, one byte a row and 256-byte multiples a sequence; the caller checked shapes and alignment (d = 512, d_rope = 64).
csa_status launch_own_rows(const csa_attn_args* a, int first, void* out, cudaStream_t st) {
  OwnRowsParams P{};
  const bool has_win = attn_has_window(a);
  P.first = first; P.E = a->n_max - first; P.n_max = a->n_max; P.Wn = has_win ? a->Wn : 0;
  const long long per = (long long)P.E + P.Wn, total = per * a->B;
  CSA_SUPPORTED(total <= 0x7fffffffLL);
  P.per = (uint32_t)per; P.total = (uint32_t)total;
  P.g = a->g_kv; P.n_c = a->n_c; P.codes = a->kv_codes; P.scales = a->kv_scales; P.rope = (const uint16_t*)a->kv_rope;
  if (a->win_format == CSA_WIN_FP8) {
    P.wcodes = a->win_codes; P.wscales = a->win_scales; P.wrope = (const uint16_t*)a->win_rope;
  } else {
    P.win = (const uint16_t*)a->win_kv;
  }
  P.out = (uint16_t*)out; P.pm = a->kv_pages;
  P.bad = (uint8_t*)out + (size_t)total * 1024; P.stride = (uint32_t)((per + 255) / 256 * 256);
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)own_rows_kernel, 0, attr_done);
  return launch_pdl(own_rows_kernel, dim3((unsigned)((total + 7) / 8)), dim3(256), 0, st, P);
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
