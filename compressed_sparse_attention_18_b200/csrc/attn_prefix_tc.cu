// HCA attention over a prefix of compressed entries that every sequence of the batch shares, on the 5th-generation
// tensor cores: the partial softmax attention of all query rows (each a head of a query) over the prefix's bf16 rows.
// Since the prefix is the same for all and there is one shared KV head, the rows of the whole batch form one matrix,
// and a CTA attends with 96 of them at a time over tiles of 128 entries:
//
//   S^T[key][row] = K[key][:] . Q[row][:]          M = 128 keys, N = 96 rows, K = 512 (32 MMAs, K-major)
//   P^T = exp2(S^T * scale*log2e - m_row)          m: a running reference per row, see below
//   O^T[dim][row] += sum_key K[key][dim] P^T[key][row]   M = 4 x 128 dims, N = 96, K = 128 (32 MMAs, both MN-major)
//
// The per-query kernels dequantise every entry again for every query and reach an N of 64; here entries arrive as
// bf16 by TMA and N = 96 costs no more than 64: an M = 128 bf16 MMA takes 59 cycles at N = 64 and at N = 96 (64 at 128,
// measured), so 96 rows run at 6650 of the 8190 flop a cycle and SM.  O^T takes 4 x 96 columns of tensor memory, S^T 96.
//
// Shared memory: Q (96 KB) stays; the 8 chunks (128 keys x 64 dims, 16 KB) of a tile pass through a ring of 6.  S needs
// chunks 0..7, then O takes 2 3 | 4 5 | 6 7, which are still there, and 0 1, which come a second time: 10 loads a tile.
// Softmax: the reference m of a row moves only when a tile's scores exceed it by more than 2^8 (or in a part's first
// tile), which the threads of a column group agree on with one barrier; the sum stays in registers, one partial sum
// per thread and row, until the part ends.
// Parts: the tiles of all blocks of 96 rows form one line that is cut evenly over the CTAs, so a CTA works on the
// end of one block and the start of the next, and each leaves a partial (O / l in bf16, lse) that the split merge adds.
// Sources: "DeepSeek-V4: エージェントが実際に使える100万トークンのコンテキスト", §ハイブリッド注意, Fig. 4 (the 128x layer
// attends densely over all visible entries).
#include "csa_common.cuh"
#include "sm100.cuh"

namespace csa {

using namespace sm100;

constexpr int PX_COLS = 96;                 // query rows of a block
constexpr int PX_KEYS = 128;
constexpr int PX_WORKERS = 384;             // warps 0-11: 4 lane quadrants (keys, dims) x 3 groups of 32 rows
constexpr int PX_THREADS = PX_WORKERS + 64; // warp 12: TMA, warp 13: tensor memory and MMA
constexpr int PX_SLOTS = 6, PX_CHUNK = PX_KEYS * 128, PX_LOADS = 10;
constexpr uint32_t PX_COL_S = 0, PX_COL_O = 96;
constexpr float PX_SLACK = 8.0f;            // log2 units: probabilities stay <= 2^8
constexpr float PX_LOG2E = 1.4426950408889634f, PX_LN2 = 0.6931471805599453f;

struct PxSmem {
  alignas(1024) uint8_t Q[8][PX_COLS * 128];     // [dim block][row][128 B], 128-byte swizzle
  alignas(1024) uint8_t K[PX_SLOTS][PX_CHUNK];   // [key][128 B], 128-byte swizzle
  alignas(1024) uint8_t P[3][PX_KEYS * 64];      // [group][key][32 rows bf16], 64-byte swizzle
  alignas(16) float m[PX_COLS];                  // reference (log2 units); 0 for a row that sees no key
  alignas(16) float inv[PX_COLS];                // 1 / l at a part's end
  float red[4][PX_COLS];
  alignas(8) uint64_t full[PX_SLOTS], rel[PX_SLOTS];
  uint64_t bar_q, bar_qfree, bar_s, bar_p, bar_o;
  uint32_t tmem_base;
  uint32_t err;
};

struct PxParams {
  long long R;            // query rows: B * Nq * H
  long long T;            // tiles of all blocks
  int tiles;              // tiles of one block: ceil(n_p / 128)
  int Nq, H, ratio, n_p, n_max;
  int slot0, slots;       // partial slots of a query: this kernel's first, and all
  int pslots;             // this kernel's
  float scale_log2;
  const int64_t* q_pos;
  const int32_t* n_c;
  uint16_t* part_o;       // [query][slots][H][512] bf16
  float* part_lse;        // [query][slots][H]
};

// The CTA that tile g of the line belongs to when it is cut into G even parts [i T / G, (i + 1) T / G).
__host__ __device__ __forceinline__ long long px_cta_of(long long g, long long G, long long T) { return ((g + 1) * G - 1) / T; }

__device__ __forceinline__ float px_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void px_group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
// Barrier of a column group that returns whether any of its threads passed true.
__device__ __forceinline__ bool px_group_any(int g, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %2, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r) : "r"(1 + g), "r"((uint32_t)v) : "memory");
  return r != 0;
}
// 32 values per lane reduced over the warp's lanes, transposed: lane l returns the reduction of value l.
template <bool kMax>
__device__ __forceinline__ float px_transpose_reduce(float (&v)[32], int lane) {
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, s);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}
__device__ __forceinline__ void px_tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  tmem_st_x16(taddr, r);
  tmem_st_x16(taddr + 16, r + 16);
}

__global__ void __launch_bounds__(PX_THREADS, 1)
    attn_prefix_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const PxParams P) {
  extern __shared__ uint8_t smem_raw[];
  PxSmem& S = *reinterpret_cast<PxSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long G = gridDim.x, g_begin = blockIdx.x * P.T / G, g_end = (blockIdx.x + 1) * P.T / G;
  if (tid == 0) {
    S.err = 0;
    for (int i = 0; i < PX_SLOTS; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.rel[i], 1); }
    mbar_init(&S.bar_q, 1);
    mbar_init(&S.bar_qfree, 1);
    mbar_init(&S.bar_s, 1);
    mbar_init(&S.bar_p, PX_WORKERS / 32);
    mbar_init(&S.bar_o, 1);
    fence_mbar_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
  }
  if (warp == 13) { tmem_alloc(&S.tmem_base, 512); tmem_relinquish(); }
  pdl_trigger();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = S.tmem_base;
  bool ok = true;
  pdl_wait();

  if (warp == 12) {
    // ------------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t n = 0, part = 0;
      for (long long g = g_begin; g < g_end && ok; ++part) {
        const long long blk = g / P.tiles, blk_end = (blk + 1) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
        // the previous part's S MMAs have read Q
        if (part > 0 && !mbar_wait(&S.bar_qfree, (part - 1) & 1)) { ok = false; break; }
        mbar_arrive_expect_tx(&S.bar_q, 8 * PX_COLS * 128);
        for (int j = 0; j < 8; ++j) tma_load_2d(S.Q[j], &qmap, j * 64, (int)(blk * PX_COLS), &S.bar_q);
        for (; g < e && ok; ++g) {
          const int key0 = (int)(g - blk * P.tiles) * PX_KEYS;
          for (int k = 0; k < PX_LOADS; ++k, ++n) {
            const uint32_t s = n % PX_SLOTS, f = n / PX_SLOTS;
            if (f > 0 && !mbar_wait(&S.rel[s], (f - 1) & 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&S.full[s], PX_CHUNK);
            tma_load_2d(S.K[s], &kmap, (k & 7) * 64, key0, &S.full[s]);
          }
        }
      }
      if (!ok) {
        atomicOr(&S.err, 1u);
        // drain: the copies this thread issued complete before the CTA may leave
        for (uint32_t i = n > PX_SLOTS ? n - PX_SLOTS : 0; i < n; ++i)
          mbar_wait(&S.full[i % PX_SLOTS], (i / PX_SLOTS) & 1, 1u << 16);
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t ids = idesc_bf16(128, PX_COLS, 0, 0), ido = idesc_bf16(128, PX_COLS, 1, 1);
      const uint64_t kdesc = smem_desc(smem_addr(S.K[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t qdesc = smem_desc(smem_addr(S.Q[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t vdesc = smem_desc(smem_addr(S.K[0]), PX_CHUNK, 1024, LAYOUT_SW128);
      const uint64_t pdesc = smem_desc(smem_addr(S.P[0]), PX_KEYS * 64, 512, LAYOUT_SW64);
      uint32_t n0 = 0, f = 0, part = 0;
      auto chunk_ready = [&](uint32_t n) {
        uint64_t* bar = &S.full[n % PX_SLOTS];
        const uint32_t ph = (n / PX_SLOTS) & 1;
        if (!mbar_test(bar, ph)) ok = ok && mbar_wait(bar, ph);
      };
      for (long long g = g_begin; g < g_end && ok; ++part) {
        const long long blk_end = (g / P.tiles + 1) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
        ok = mbar_wait(&S.bar_q, part & 1);
        for (long long t = g; t < e && ok; ++t, ++f, n0 += PX_LOADS) {
          // S^T = K Q^T, chunk by chunk as they land
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            chunk_ready(n0 + j);
            if (!ok) continue;
            tc_fence_after();
            const uint32_t s = (n0 + j) % PX_SLOTS;
#pragma unroll
            for (int s2 = 0; s2 < 4; ++s2)
              mma_bf16_ss(tb + PX_COL_S, kdesc + (uint64_t)((s * PX_CHUNK + s2 * 32) >> 4),
                          qdesc + (uint64_t)((j * PX_COLS * 128 + s2 * 32) >> 4), ids, (j | s2) != 0);
            if (j < 2) mma_commit(&S.rel[s]);        // chunks 0 and 1 come again for O
          }
          mma_commit(&S.bar_s);
          if (t + 1 == e) mma_commit(&S.bar_qfree);
          ok = ok && mbar_wait(&S.bar_p, f & 1);
          if (ok) tc_fence_after();
          // O^T += V^T P^T: dims 128.., 256.., 384.. from the chunks that stayed, then 0..
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int mt = (i + 1) & 3;
            const uint32_t n = n0 + (mt ? 2 * mt : 8), s = n % PX_SLOTS;
            if (mt == 0) { chunk_ready(n); chunk_ready(n + 1); }
            if (!ok) continue;
            tc_fence_after();
#pragma unroll
            for (int s2 = 0; s2 < 8; ++s2)
              mma_bf16_ss(tb + PX_COL_O + PX_COLS * mt, vdesc + (uint64_t)((s * PX_CHUNK + s2 * 2048) >> 4),
                          pdesc + (uint64_t)((s2 * 1024) >> 4), ido, t > g || s2 > 0);
            mma_commit(&S.rel[s]);
            mma_commit(&S.rel[s + 1]);
          }
          if (t + 1 == e) mma_commit(&S.bar_o);
        }
        g = e;
      }
      if (!ok) atomicOr(&S.err, 1u);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------ softmax and epilogue
    const int quad = warp & 3, grp = warp >> 2;
    const int kr = 32 * quad + lane;             // the thread's key of a tile, and its dim of 128 in the epilogue
    const uint32_t lane_base = tb + ((uint32_t)(32 * quad) << 16) + 32 * grp;
    uint8_t* prow = &S.P[grp][kr * 64];
    const float4* m4 = reinterpret_cast<const float4*>(&S.m[32 * grp]);
    uint32_t f = 0, part = 0;
    for (long long g = g_begin; g < g_end; ++part) {
      const long long blk = g / P.tiles, blk_end = (blk + 1) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
      // lane l of every warp speaks for row l of its group: how many entries it sees (rows behind the last
      // query row see all of them: their Q is zero and nothing is stored), its reference, its partial's place
      const long long col = blk * PX_COLS + 32 * grp + lane;
      const bool real = col < P.R;
      int nv = P.n_p;
      long long prt = 0;                         // row of the partial arrays, without the slot
      if (real) {
        const long long bq = col / P.H;
        const int b = (int)(bq / P.Nq);
        const long long see = (P.q_pos[bq] + 1) / P.ratio;
        nv = (int)max(0LL, min((long long)min(P.n_p, min(P.n_c[b], P.n_max)), see));
        prt = bq * P.slots * P.H + (col - bq * P.H);
      }
      int nv_min = nv;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) nv_min = min(nv_min, __shfl_xor_sync(0xffffffffu, nv_min, o));
      float m_l = -INFINITY;
      float l[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) l[j] = 0.f;
      for (long long t = g; t < e; ++t, ++f) {
        const bool first = t == g;
        const int key0 = (int)(t - blk * P.tiles) * PX_KEYS;
        ok = ok && mbar_wait(&S.bar_s, f & 1);
        tc_fence_after();
        float z[32];
        {
          uint32_t v[32];
          tmem_ld_x32(lane_base + PX_COL_S, v);
          tmem_wait_ld_x32(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(v[j]);
        }
        if (key0 + PX_KEYS > nv_min) {           // some row of the group does not see the whole tile
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (key0 + kr >= __shfl_sync(0xffffffffu, nv, j)) z[j] = -INFINITY;
        }
        bool move = first;
        if (!first) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 mm = m4[j >> 2];
            top = fmaxf(top, fmaxf(fmaxf(fmaf(z[j], P.scale_log2, -mm.x), fmaf(z[j + 1], P.scale_log2, -mm.y)),
                                   fmaxf(fmaf(z[j + 2], P.scale_log2, -mm.z), fmaf(z[j + 3], P.scale_log2, -mm.w))));
          }
          move = px_group_any(grp, top > PX_SLACK);
        }
        if (move) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = z[j] * P.scale_log2;
          S.red[quad][32 * grp + lane] = px_transpose_reduce<true>(v, lane);
          px_group_sync(grp);
          const int c = 32 * grp + lane;
          const float mt = fmaxf(fmaxf(S.red[0][c], S.red[1][c]), fmaxf(S.red[2][c], S.red[3][c]));
          const float mn = first || mt > m_l + PX_SLACK ? fmaxf(m_l, mt) : m_l;
          const float fc = first || mn == m_l ? 1.f : exp2f(m_l - mn);
          m_l = mn;
          if (quad == 0) S.m[c] = mn == -INFINITY ? 0.f : mn;
          px_group_sync(grp);
          if (!first && __any_sync(0xffffffffu, fc != 1.f)) {
            // the sums and O^T of the rows whose reference moved (the O MMAs so far completed before S did)
#pragma unroll
            for (int j = 0; j < 32; ++j) l[j] *= __shfl_sync(0xffffffffu, fc, j);
#pragma unroll 1
            for (int mt4 = 0; mt4 < 4; ++mt4) {
              uint32_t o[32];
              const uint32_t at = lane_base + PX_COL_O + PX_COLS * mt4;
              tmem_ld_x32(at, o);
              tmem_wait_ld_x32(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * __shfl_sync(0xffffffffu, fc, j));
              px_tmem_st_x32(at, o);
            }
            tmem_wait_st();
          }
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          const float4 ma = m4[j >> 2], mb = m4[(j >> 2) + 1];
          const float mm[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] = px_exp2(fmaf(z[j + i], P.scale_log2, -mm[i]));
            l[j + i] += p[i];
          }
          // P is rounded to bf16 for the MMA (2^-8 of a probability); l adds the unrounded values
          *reinterpret_cast<uint4*>(prow + ((((j >> 3) ^ (kr >> 1)) & 3) << 4)) =
              make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.bar_p);
      }
      // ---- the part's partial: O^T / l, lane = dim, columns = rows
      const long long first_cta = px_cta_of(blk * P.tiles, G, P.T);
      const int slot = P.slot0 + (int)(blockIdx.x - first_cta);
      S.red[quad][32 * grp + lane] = px_transpose_reduce<false>(l, lane);
      px_group_sync(grp);
      {
        const int c = 32 * grp + lane;
        const float lt = (S.red[0][c] + S.red[1][c]) + (S.red[2][c] + S.red[3][c]);
        if (quad == 0) {
          S.inv[c] = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);       // (a NaN stays one)
          if (real) {
            P.part_lse[prt + (long long)slot * P.H] = lt == 0.f ? -INFINITY : (m_l + log2f(lt)) * PX_LN2;
            // slots of this block that no CTA fills
            if (e == blk_end)
              for (int s = slot + 1; s < P.slot0 + P.pslots; ++s) P.part_lse[prt + (long long)s * P.H] = -INFINITY;
          }
        }
      }
      px_group_sync(grp);
      ok = ok && mbar_wait(&S.bar_o, part & 1);
      tc_fence_after();
      const float4* i4 = reinterpret_cast<const float4*>(&S.inv[32 * grp]);
      const int n_real = (int)min(32LL, P.R - (blk * PX_COLS + 32 * grp));
      const long long row = prt + (long long)slot * P.H;
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t o[32];
        tmem_ld_x32(lane_base + PX_COL_O + PX_COLS * mt, o);
        tmem_wait_ld_x32(o);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 iv = i4[j >> 2];
          const float f4[4] = {iv.x, iv.y, iv.z, iv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long r = __shfl_sync(0xffffffffu, row, j + i);
            if (j + i < n_real)
              P.part_o[r * 512 + 128 * mt + kr] = (uint16_t)f_to_bf16_bits(__uint_as_float(o[j + i]) * f4[i]);
          }
        }
      }
      tc_fence_before();
      // the group's red and inv are rewritten only after all of its warps have read them
      px_group_sync(grp);
      g = e;
    }
    if (!ok && lane == 0) atomicOr(&S.err, 1u);
  }
  __syncthreads();
  if (warp == 13) {
    if (S.err && lane == 0) atomicOr(&g_csa_device_error, 1u);
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// The prefix kernel's plan for R query rows over n_p entries: CTAs, and partial slots a query needs (at most `most`).
void attn_prefix_plan(long long R, int n_p, int most, int* ctas, int* slots) {
  const long long blocks = (R + PX_COLS - 1) / PX_COLS, tiles = ((long long)n_p + PX_KEYS - 1) / PX_KEYS, T = blocks * tiles;
  long long G = T < 148 ? T : 148;
  if (G > blocks * (most - 1)) G = blocks * (most - 1);    // a block is cut into at most ceil(G / blocks) + 1 parts
  long long worst = 1;
  // (with no fewer blocks than CTAs every part is at least a block's worth: two CTAs a block at most)
  if (blocks >= G) {
    worst = blocks == G ? 1 : 2;
  } else {
    for (long long b = 0; b < blocks; ++b) {
      const long long n = px_cta_of((b + 1) * tiles - 1, G, T) - px_cta_of(b * tiles, G, T) + 1;
      if (n > worst) worst = n;
    }
  }
  *ctas = (int)G;
  *slots = (int)worst;
}

csa_status launch_attn_prefix(const csa_attn_args* a, const void* prefix, int n_p, int ctas, int slot0, int pslots, int slots,
                              uint16_t* part_o, float* part_lse, cudaStream_t st) {
  const long long R = (long long)a->B * a->Nq * a->H;
  CUtensorMap qm, km;
  auto encode = [](CUtensorMap* map, const void* base, long long rows, int box) {
    const cuuint64_t gdim[2] = {512, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {1024};
    const cuuint32_t bx[2] = {64, (cuuint32_t)box};
    const cuuint32_t estr[2] = {1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, bx, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!encode(&qm, a->q, R, PX_COLS) || !encode(&km, prefix, n_p, PX_KEYS)) return CSA_ERR_CUDA;
  PxParams P{};
  P.R = R;
  P.tiles = (n_p + PX_KEYS - 1) / PX_KEYS;
  P.T = (R + PX_COLS - 1) / PX_COLS * P.tiles;
  P.Nq = a->Nq; P.H = a->H; P.ratio = a->ratio; P.n_p = n_p; P.n_max = a->n_max;
  P.slot0 = slot0; P.slots = slots; P.pslots = pslots;
  P.scale_log2 = (a->softmax_scale != 0.0f ? a->softmax_scale : 1.0f / sqrtf(512.0f)) * PX_LOG2E;
  P.q_pos = a->q_pos; P.n_c = a->n_c; P.part_o = part_o; P.part_lse = part_lse;
  const int smem = (int)sizeof(PxSmem) + 1024;
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)attn_prefix_tc_kernel, smem, attr_done);
  return launch_pdl(attn_prefix_tc_kernel, dim3((unsigned)ctas), dim3(PX_THREADS), (size_t)smem, st, qm, km, P);
}

}  // namespace csa
