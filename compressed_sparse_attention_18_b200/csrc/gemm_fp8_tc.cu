// Block-scaled FP8 matrix product on the 5th-generation tensor cores, for the compressor's projections with
// FP8 weights: for each of one or two weights
//
//   out[m][n] = bf16( sum_kb sx[m][kb] sw[n / 128][kb] sum_{k in block kb} x[m][k] W[n][k] )
//
// x [M][K] and W [N][K] are E4M3 codes, sx holds one fp32 scale per row and 128 channels, sw one per 128 x 128 block.
// The scales are not powers of two, so they cannot ride in the MMA: each 128-wide block of K is one accumulator in
// tensor memory (4 MMAs of K = 32, first one overwriting), which the epilogue warps read, multiply by the block's
// scale and add in fp32 registers while the MMAs of the next block fill the other buffer.
//
// Tile: 128 rows of one operand (MMA M) x BN of the other (MMA N) x 128 of K per pipeline stage, both by TMA with
// the 128-byte swizzle (a row of a stage is exactly one 128-byte line).  Three arrangements:
//   SWAP = false  the 128 rows are tokens, BN = 128 channels: a thread holds one token, its scale is one register;
//   SWAP = true   the 128 rows are channels, BN = 16 .. 64 tokens: few tokens do not pay for 128, and a CTA's
//                 channels share one weight scale;
//   pairs         (below) two CTAs on 256 tokens x 256 channels.
// A cluster of ks CTAs can share a tile, each taking a part of K; the partial sums meet in distributed shared
// memory and are added in rank order (the same result at every run).
// Bounds, measured on B200 (replayed graphs, SM clock 1.7 GHz under the power cap): 4096 tokens into two weights of
// 512 x 4096 23.6 us = 1450 TFLOP/s, 8192 x 4096 x 4096 1690 TFLOP/s.  The same pair kernel without reading the
// accumulators until the end reaches 1630 / 2000, without the loads as well 1970 / 2300.  So at 4096 tokens the hand-over
// of two accumulators (all of tensor memory) costs 11 %, operands from L2 17 %; the larger rest against the rate of the
// MMAs is that each pair has one tile there, with nothing beside its first loads and its stores, and 10 of 74 have none.
// Few tokens are bound by latency:
// 32 tokens into the two weights take 4.5 us, 4 MB of weights at the copy rate 0.65 us.
// Warp roles (384 threads): warps 0-7 scale and accumulate (4 lane quadrants x 2 column halves), warp 8 TMA, warps
// 9 and 10 MMA, warp 11 tensor memory.  Every wait is bounded; a wait that gives up records device error 1 and the kernel leaves.
#include "csa_common.cuh"
#include "sm100.cuh"

namespace csa {

using namespace sm100;

constexpr int GF_ROWS = 128, GF_BK = 128;
constexpr int GF_EPI = 256, GF_THREADS = GF_EPI + 128;
constexpr int GF_MAX_CLUSTER = 8;
constexpr int GF_SC_CHUNK = 16;            // K blocks whose token scales are staged at once (SWAP)

template <int BN>
struct GfCfg {
  static constexpr int NB = 4;                              // accumulator buffers
  static constexpr uint32_t TMEM_COLS = NB * BN;
  static constexpr int A_BYTES = GF_ROWS * GF_BK;           // 16 KB
  static constexpr int B_BYTES = BN * GF_BK;
  static constexpr int STAGES = BN == 128 ? 6 : 8;
  static constexpr int STAGE_LD = BN + 4;                   // floats per staged row: no bank conflicts
};

template <int BN>
struct GfSmem {
  alignas(1024) uint8_t a[GfCfg<BN>::STAGES][GfCfg<BN>::A_BYTES];
  alignas(1024) uint8_t b[GfCfg<BN>::STAGES][GfCfg<BN>::B_BYTES];
  alignas(16) float sc[2][GF_SC_CHUNK][BN];  // SWAP: token scales x weight scale
  alignas(8) uint64_t full[GfCfg<BN>::STAGES];
  uint64_t mma[GfCfg<BN>::STAGES];           // the stage's MMAs have completed: it is free, its accumulator is full
  uint64_t acc_empty[GfCfg<BN>::NB];
  uint64_t done;
  uint32_t tmem_base;
  uint32_t err;
};

struct GfParams {
  const float* sx;          // [M][KB]
  const float* sw[2];       // [ceil(N / 128)][KB]
  uint16_t* out[2];         // [M][N]
  int M, N, KB;
  int tiles_a, tiles_b;     // pairs: tiles of the tokens and of the channels, for one weight
  int tiles;                // pairs: all
  int ks;                   // CTAs that share a tile (a cluster): 1, 2, 4 or 8
};

// kind::f8f6f4 instruction descriptor: E4M3 A and B (K-major), fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}

// CW columns of an accumulator: acc += f * column (f one factor, or SWAP: one per column from shared memory).
template <int CW, bool SWAP>
__device__ __forceinline__ void gf_accumulate(uint32_t taddr, float f, const float* fcol, float (&acc)[CW]) {
  if constexpr (CW >= 32) {
#pragma unroll
    for (int c = 0; c < CW; c += 32) {
      uint32_t v[32];
      tmem_ld_x32(taddr + c, v);
      tmem_wait_ld_x32(v);
      if constexpr (SWAP) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 s = *reinterpret_cast<const float4*>(fcol + c + j);
          acc[c + j] = fmaf(s.x, __uint_as_float(v[j]), acc[c + j]);
          acc[c + j + 1] = fmaf(s.y, __uint_as_float(v[j + 1]), acc[c + j + 1]);
          acc[c + j + 2] = fmaf(s.z, __uint_as_float(v[j + 2]), acc[c + j + 2]);
          acc[c + j + 3] = fmaf(s.w, __uint_as_float(v[j + 3]), acc[c + j + 3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(f, __uint_as_float(v[j]), acc[c + j]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < CW; c += 8) {
      float v[8];
      tmem_ld_x8(taddr + c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[c + j] = fmaf(SWAP ? fcol[c + j] : f, v[j], acc[c + j]);
    }
  }
}

template <int BN, bool SWAP>
__global__ void __launch_bounds__(GF_THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap w0map,
                    const __grid_constant__ CUtensorMap w1map, const GfParams P) {
  using Cfg = GfCfg<BN>;
  constexpr int ST = Cfg::STAGES, NB = Cfg::NB, CW = BN / 2;
  extern __shared__ uint8_t smem_raw[];
  GfSmem<BN>& S = *reinterpret_cast<GfSmem<BN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A cluster has one tile: its place among the 128-row operand's, the other one's, and the weight.  (No division:
  // with the tile's place from one running number the smallest call took 3.6 us instead of 3.0.)
  const int rank = (int)blockIdx.x & (P.ks - 1), lg = __popc(P.ks - 1);
  const int kb0 = P.KB * rank >> lg, kb1 = P.KB * (rank + 1) >> lg;
  const int ta = (int)blockIdx.x >> lg, tb = (int)blockIdx.y, w = (int)blockIdx.z;
  if (threadIdx.x == 0) {
    S.err = 0;
    for (int s = 0; s < ST; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.mma[s], 1); }
    for (int a = 0; a < NB; ++a) mbar_init(&S.acc_empty[a], GF_EPI / 32);
    mbar_init(&S.done, 2);
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&w0map);
    prefetch_tensormap(&w1map);
  }
  if (warp == 11) { tmem_alloc(&S.tmem_base, Cfg::TMEM_COLS); tmem_relinquish(); }
  pdl_trigger();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = S.tmem_base;
  bool ok = true;
  pdl_wait();                                // operands may be written by the previous kernel
  if (warp == 8) {
    // ------------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int issued = 0;
      const CUtensorMap* wm = w ? &w1map : &w0map;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        const int s = issued % ST, f = issued / ST;
        if (f > 0 && !mbar_wait(&S.mma[s], (f - 1) & 1)) { ok = false; break; }
        mbar_arrive_expect_tx(&S.full[s], Cfg::A_BYTES + Cfg::B_BYTES);
        tma_load_2d(S.a[s], SWAP ? wm : &xmap, kb * GF_BK, ta * GF_ROWS, &S.full[s]);
        tma_load_2d(S.b[s], SWAP ? &xmap : wm, kb * GF_BK, tb * BN, &S.full[s]);
      }
      if (!ok) atomicOr(&S.err, 1u);
      // drain: the copies this thread issued complete before the CTA may leave
      for (int i = max(0, issued - ST); i < issued; ++i) mbar_wait(&S.full[i % ST], (i / ST) & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == 9 || warp == 10) {
    // ------------------------------------------------------------------------ MMA issuers
    // Two threads take the K blocks in turn: a thread's waits and its commit cost about 400 cycles a block, and
    // few MMAs queue behind the running one, so a single issuer left the tensor pipe idle for half of the time.
    if (lane == 0) {
      const uint32_t idesc = idesc_e4m3(GF_ROWS, BN);
      const uint64_t ad0 = smem_desc(smem_addr(S.a[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t bd0 = smem_desc(smem_addr(S.b[0]), 16, 1024, LAYOUT_SW128);
      const int n = kb1 - kb0;
      for (int it = warp - 9; it < n; it += 2) {
        const int s = it % ST, a = it % NB;
        if (it >= NB && !mbar_wait(&S.acc_empty[a], (uint32_t)(it / NB - 1) & 1)) { ok = false; break; }
        if (!mbar_wait(&S.full[s], (uint32_t)(it / ST) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint64_t ad = ad0 + (uint64_t)(s * (Cfg::A_BYTES >> 4)), bd = bd0 + (uint64_t)(s * (Cfg::B_BYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < GF_BK / 32; ++kk)
          mma_f8_ss(tbase + (uint32_t)(a * BN), ad + kk * 2, bd + kk * 2, idesc, kk != 0);
        mma_commit(&S.mma[s]);
      }
      mma_commit(&S.done);
      if (!ok) atomicOr(&S.err, 1u);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------------ scale and accumulate
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const int arow = 32 * quad + lane;           // row of the tile (token, or channel when SWAP)
    const float* swr = w ? P.sw[1] : P.sw[0];
    const float* sxr = nullptr;
    if (!SWAP) {
      // this thread's token (rows behind the last read the last one's scale; they are not stored) and the
      // 128-channel block of its column half
      sxr = P.sx + (long long)min(ta * GF_ROWS + arow, P.M - 1) * P.KB;
      swr += (long long)min((tb * BN + half * CW) / 128, (P.N - 1) / 128) * P.KB;
    } else {
      swr += (long long)ta * P.KB;             // a tile's 128 channels are one scale block
    }
    float acc[CW];
#pragma unroll
    for (int j = 0; j < CW; ++j) acc[j] = 0.f;
    // scales, read four K blocks ahead of their use
    float sx4[4], sw4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sx4[i] = !SWAP && kb0 + i < kb1 ? __ldg(sxr + kb0 + i) : 0.f;
      sw4[i] = !SWAP && kb0 + i < kb1 ? __ldg(swr + kb0 + i) : 0.f;
    }
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      const int it = kb - kb0, a = it % NB;
      float f = 0.f;
      const float* fcol = nullptr;
      if constexpr (SWAP) {
        if (it % GF_SC_CHUNK == 0) {
          // the factors of the next K blocks, [K block][token]: two buffers, so the one being read by a
          // slower warp (at most one chunk behind) is not the one written
          float* dst = &S.sc[(it / GF_SC_CHUNK) & 1][0][0];
          const int n = min(GF_SC_CHUNK, kb1 - kb);
          for (int i = threadIdx.x; i < BN * GF_SC_CHUNK; i += GF_EPI) {
            const int c = i / GF_SC_CHUNK, k = i % GF_SC_CHUNK;
            const int m = tb * BN + c;
            dst[k * BN + c] = k < n && m < P.M ? P.sx[(long long)m * P.KB + kb + k] * swr[kb + k] : 0.f;
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        fcol = &S.sc[(it / GF_SC_CHUNK) & 1][it % GF_SC_CHUNK][half * CW];
      } else {
        f = sx4[0] * sw4[0];
#pragma unroll
        for (int i = 0; i < 3; ++i) { sx4[i] = sx4[i + 1]; sw4[i] = sw4[i + 1]; }
        if (kb + 4 < kb1) { sx4[3] = __ldg(sxr + kb + 4); sw4[3] = __ldg(swr + kb + 4); }
      }
      ok = ok && mbar_wait(&S.mma[it % ST], (it / ST) & 1);
      tc_fence_after();
      gf_accumulate<CW, SWAP>(tbase + lane_off + (uint32_t)(a * BN + half * CW), f, fcol, acc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&S.acc_empty[a]);
    }
    uint16_t* out = w ? P.out[1] : P.out[0];
    if (!SWAP && P.ks == 1) {
      // a token's CW columns straight from the registers, 16 bytes at a time (N % 8 == 0)
      const int m = ta * GF_ROWS + arow, n0 = tb * BN + half * CW;
      if (m < P.M) {
        uint16_t* dst = out + (long long)m * P.N + n0;
#pragma unroll
        for (int j = 0; j < CW; j += 8)
          if (n0 + j < P.N)
            *reinterpret_cast<uint4*>(dst + j) =
                make_uint4(pack_bf16x2(acc[j], acc[j + 1]), pack_bf16x2(acc[j + 2], acc[j + 3]),
                           pack_bf16x2(acc[j + 4], acc[j + 5]), pack_bf16x2(acc[j + 6], acc[j + 7]));
      }
    } else {
      // staged in fp32 over the operand ring (every MMA has read it: this tile is the CTA's only one and
      // its last accumulator has arrived), token-major: [token][channel]
      float* stage = reinterpret_cast<float*>(&S.a[0][0]);
      if (SWAP) {
#pragma unroll
        for (int j = 0; j < CW; ++j) stage[(half * CW + j) * GF_ROWS + arow] = acc[j];
      } else {
#pragma unroll
        for (int j = 0; j < CW; j += 4)
          *reinterpret_cast<float4*>(&stage[arow * Cfg::STAGE_LD + half * CW + j]) =
              make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      }
    }
    if (!ok && lane == 0) atomicOr(&S.err, 1u);
  }
  if (SWAP || P.ks > 1) {
    // ---- the cluster's partial sums: every CTA adds and stores its share of the tile's tokens
    __syncwarp();
    if (P.ks > 1) cluster_sync_all(); else __syncthreads();
    constexpr int TOK = SWAP ? BN : GF_ROWS, CH = SWAP ? GF_ROWS : BN, LD = SWAP ? GF_ROWS : Cfg::STAGE_LD;
    const int m0 = SWAP ? tb * BN : ta * GF_ROWS, n0 = SWAP ? ta * GF_ROWS : tb * BN;
    const int tok0 = TOK * rank >> lg, tok1 = TOK * (rank + 1) >> lg;
    const float* stage = reinterpret_cast<const float*>(&S.a[0][0]);
    uint32_t base[GF_MAX_CLUSTER];
#pragma unroll
    for (int r = 0; r < GF_MAX_CLUSTER; ++r) base[r] = P.ks > 1 && r < P.ks ? peer_addr(stage, r) : 0u;
    for (int i = threadIdx.x; i < (tok1 - tok0) * (CH / 4); i += GF_THREADS) {
      const int tok = tok0 + i / (CH / 4), ch = 4 * (i % (CH / 4));
      if (m0 + tok >= P.M || n0 + ch >= P.N) continue;
      float4 v[GF_MAX_CLUSTER];
      if (P.ks == 1) {
        v[0] = *reinterpret_cast<const float4*>(&stage[tok * LD + ch]);
      } else {
#pragma unroll
        for (int r = 0; r < GF_MAX_CLUSTER; ++r)
          if (r < P.ks) v[r] = ld_peer_v4(base[r] + (uint32_t)((tok * LD + ch) * 4));
      }
      float4 s = v[0];
#pragma unroll
      for (int r = 1; r < GF_MAX_CLUSTER; ++r)
        if (r < P.ks) { s.x += v[r].x; s.y += v[r].y; s.z += v[r].z; s.w += v[r].w; }
      *reinterpret_cast<uint2*>((w ? P.out[1] : P.out[0]) + (long long)(m0 + tok) * P.N + n0 + ch) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
    if (P.ks > 1) cluster_sync_all();            // the peers have read this CTA's shared memory
  }
  __syncthreads();
  if (warp == 11) {
    // every MMA this CTA issued has completed before its tensor memory is released
    mbar_wait(&S.done, 0, 1u << 20);
    tc_fence_after();
    tmem_dealloc(tbase, Cfg::TMEM_COLS);
  }
  if (S.err && threadIdx.x == 0) atomicOr(&g_csa_device_error, 1u);
}

// ---------------------------------------------------------------------------------------------- CTA pairs
// The same product with two CTAs to a tile of 256 tokens x BN channels (cta_group::2): each CTA loads its own 128
// tokens and half of the channels and keeps the accumulators of its own tokens, so a K block brings 128 + BN/2 rows
// into an SM instead of 128 + BN, and the MMA reads as many.  The even CTA issues the MMAs for both.
struct GpCfg {
  static constexpr int BN = 256;
  static constexpr int NB = 512 / BN;                       // accumulator buffers: all of tensor memory
  static constexpr int A_BYTES = GF_ROWS * GF_BK;
  static constexpr int B_BYTES = BN / 2 * GF_BK;
  static constexpr int STAGES = 6;
};

struct GpSmem {
  alignas(1024) uint8_t a[GpCfg::STAGES][GpCfg::A_BYTES];
  alignas(1024) uint8_t b[GpCfg::STAGES][GpCfg::B_BYTES];
  alignas(8) uint64_t full[GpCfg::STAGES];   // even CTA: both CTAs' operands of the stage have landed
  uint64_t mma[GpCfg::STAGES];               // both: the stage's MMAs have completed
  uint64_t acc_empty[GpCfg::NB];             // even CTA: both CTAs' warps have read the accumulator
  uint64_t done;                                 // both: all MMAs have completed
  uint32_t tmem_base;
  uint32_t err;
};

__device__ __forceinline__ void mma_f8_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}

__global__ void __launch_bounds__(GF_THREADS, 1) __cluster_dims__(2, 1, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap w0map,
                         const __grid_constant__ CUtensorMap w1map, const GfParams P) {
  using Cfg = GpCfg;
  constexpr int BN = Cfg::BN, ST = Cfg::STAGES, NB = Cfg::NB, CW = BN / 2;
  extern __shared__ uint8_t smem_raw[];
  GpSmem& S = *reinterpret_cast<GpSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)blockIdx.x & 1;
  const int t0 = (int)blockIdx.x >> 1, tstep = (int)gridDim.x >> 1;
  const int KB = P.KB;
  if (threadIdx.x == 0) {
    S.err = 0;
    for (int s = 0; s < ST; ++s) { mbar_init(&S.full[s], 1); mbar_init(&S.mma[s], 1); }
    for (int a = 0; a < NB; ++a) mbar_init(&S.acc_empty[a], 2 * (GF_EPI / 32));
    mbar_init(&S.done, 2);
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&w0map);
    prefetch_tensormap(&w1map);
  }
  if (warp == 11) { tmem_alloc_pair(&S.tmem_base, 512); tmem_relinquish_pair(); }
  pdl_trigger();
  __syncthreads();
  cluster_sync_all();                        // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tbase = S.tmem_base;
  bool ok = true;
  pdl_wait();

  if (warp == 8) {
    // ------------------------------------------------------------------------ TMA producer (one per CTA)
    // 128 sums a thread need more than an even share of the registers: 8 x 232 + 4 x 40 = 12 x 168 warps' worth
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (lane == 0) {
      int it = 0;
      for (int t = t0; t < P.tiles && ok; t += tstep) {
        const int tb = t % P.tiles_b, ta = t / P.tiles_b % P.tiles_a, w = t / P.tiles_b / P.tiles_a;
        const CUtensorMap* wm = w ? &w1map : &w0map;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int s = it % ST, f = it / ST;
          if (f > 0 && !mbar_wait(&S.mma[s], (f - 1) & 1)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2 * (Cfg::A_BYTES + Cfg::B_BYTES));
          const uint32_t bar = peer_addr(&S.full[s], 0);
          tma_load_2d_pair(S.a[s], &xmap, kb * GF_BK, (2 * ta + rank) * GF_ROWS, bar);
          tma_load_2d_pair(S.b[s], wm, kb * GF_BK, tb * BN + rank * (BN / 2), bar);
        }
      }
      if (!ok) atomicOr(&S.err, 1u);
      // drain: the pair's copies complete before it may leave
      if (rank == 0)
        for (int i = max(0, it - ST); i < it; ++i) mbar_wait(&S.full[i % ST], (i / ST) & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == 9 || warp == 10) {
    // ------------------------------------------------------------------------ MMA issuers (even CTA)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (rank == 0) {
      const uint32_t idesc = idesc_e4m3(2 * GF_ROWS, BN);
      const uint64_t ad0 = smem_desc(smem_addr(S.a[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t bd0 = smem_desc(smem_addr(S.b[0]), 16, 1024, LAYOUT_SW128);
      const int ntile = t0 < P.tiles ? (P.tiles - 1 - t0) / tstep + 1 : 0;
      const long long n = (long long)ntile * KB;
      uint32_t s = warp - 9, sph = 0;            // stage and its round
      uint32_t aph = 0;                          // round of this thread's accumulator (NB = 2: one each)
      for (long long it = warp - 9; it < n && ok; it += 2) {
        const int a = warp - 9;
        if (aph > 0 && !mbar_test(&S.acc_empty[a], (aph - 1) & 1)) ok = mbar_wait(&S.acc_empty[a], (aph - 1) & 1);
        if (!mbar_test(&S.full[s], sph)) ok = ok && mbar_wait(&S.full[s], sph);
        tc_fence_after();
        const uint64_t ad = ad0 + (uint64_t)(s * (Cfg::A_BYTES >> 4)), bd = bd0 + (uint64_t)(s * (Cfg::B_BYTES >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < GF_BK / 32; ++kk)
            mma_f8_ss_pair(tbase + (uint32_t)(a * BN), ad + kk * 2, bd + kk * 2, idesc, kk != 0);
          mma_commit_pair(&S.mma[s]);
        }
        __syncwarp();
        ++aph;
        s += 2;
        if (s >= ST) { s -= ST; sph ^= 1; }
      }
      if (elect_one()) mma_commit_pair(&S.done);
      __syncwarp();
      if (!ok && lane == 0) atomicOr(&S.err, 1u);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------------ scale and accumulate
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t taddr = tbase + ((uint32_t)(32 * quad) << 16) + (uint32_t)(half * CW);
    const int arow = 32 * quad + lane;
    const uint32_t empty0 = peer_addr(&S.acc_empty[0], 0);
    int it = 0;
    for (int t = t0; t < P.tiles; t += tstep) {
      const int tb = t % P.tiles_b, ta = t / P.tiles_b % P.tiles_a, w = t / P.tiles_b / P.tiles_a;
      const int m = (2 * ta + rank) * GF_ROWS + arow, n0 = tb * BN + half * CW;
      const float* sxr = P.sx + (long long)min(m, P.M - 1) * KB;
      const float* swr = (w ? P.sw[1] : P.sw[0]) + (long long)min(n0 / 128, (P.N - 1) / 128) * KB;
      float acc[CW];
#pragma unroll
      for (int j = 0; j < CW; ++j) acc[j] = 0.f;
      // scales, read four K blocks ahead of their use
      float sx4[4], sw4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sx4[i] = i < KB ? __ldg(sxr + i) : 0.f;
        sw4[i] = i < KB ? __ldg(swr + i) : 0.f;
      }
#pragma unroll 1
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int a = it % NB;
        const float f = sx4[0] * sw4[0];
#pragma unroll
        for (int i = 0; i < 3; ++i) { sx4[i] = sx4[i + 1]; sw4[i] = sw4[i + 1]; }
        if (kb + 4 < KB) { sx4[3] = __ldg(sxr + kb + 4); sw4[3] = __ldg(swr + kb + 4); }
        ok = ok && mbar_wait(&S.mma[it % ST], (it / ST) & 1);
        tc_fence_after();
        gf_accumulate<CW, false>(taddr + (uint32_t)(a * BN), f, nullptr, acc);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_cluster(empty0 + 8 * a);
      }
      if (m < P.M) {
        uint16_t* dst = (w ? P.out[1] : P.out[0]) + (long long)m * P.N + n0;
#pragma unroll
        for (int j = 0; j < CW; j += 8)
          if (n0 + j < P.N)
            *reinterpret_cast<uint4*>(dst + j) =
                make_uint4(pack_bf16x2(acc[j], acc[j + 1]), pack_bf16x2(acc[j + 2], acc[j + 3]),
                           pack_bf16x2(acc[j + 4], acc[j + 5]), pack_bf16x2(acc[j + 6], acc[j + 7]));
      }
    }
    if (!ok && lane == 0) atomicOr(&S.err, 1u);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
  }
  // every MMA of the pair has completed (they read both CTAs' operands and write both tensor memories), and no
  // arrival is on its way to a CTA that has left
  __syncthreads();
  if (warp == 11 && !mbar_wait(&S.done, 0, 1u << 20) && lane == 0) atomicOr(&S.err, 1u);
  __syncthreads();
  if (S.err && threadIdx.x == 0) atomicOr(&g_csa_device_error, 1u);
  cluster_sync_all();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

static bool encode_2d_u8(CUtensorMap* map, const void* base, uint64_t K, uint64_t rows, uint32_t box_rows) {
  const cuuint64_t gdim[2] = {K, rows};
  const cuuint64_t gstride[1] = {K};
  const cuuint32_t box[2] = {GF_BK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool SWAP>
static csa_status launch_gemm_fp8(const csa_gemm_fp8_args* a, int ks, cudaStream_t st) {
  const int nw = a->W[1] ? 2 : 1;
  CUtensorMap xm, wm[2];
  if (!encode_2d_u8(&xm, a->x, a->K, a->M, SWAP ? BN : GF_ROWS)) return CSA_ERR_CUDA;
  for (int w = 0; w < 2; ++w)
    if (!encode_2d_u8(&wm[w], a->W[w < nw ? w : 0], a->K, a->N, SWAP ? GF_ROWS : BN)) return CSA_ERR_CUDA;
  GfParams P{};
  P.sx = a->x_scales;
  for (int w = 0; w < nw; ++w) { P.sw[w] = a->W_scales[w]; P.out[w] = (uint16_t*)a->out[w]; }
  P.M = a->M; P.N = a->N; P.KB = (a->K + GF_BK - 1) / GF_BK;
  const long long ra = SWAP ? a->N : a->M, rb = SWAP ? a->M : a->N;
  const long long ta = (ra + GF_ROWS - 1) / GF_ROWS, tb = (rb + BN - 1) / BN;
  P.ks = ks;
  const int smem = (int)sizeof(GfSmem<BN>) + 1024;
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)gemm_fp8_kernel<BN, SWAP>, smem, attr_done);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)(ta * ks), (unsigned)tb, (unsigned)nw), dim3(GF_THREADS), smem, st, attr);
  if (ks > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<BN, SWAP>, xm, wm[0], wm[1], P);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return CSA_ERR_CUDA;
  }
  return launch_status();
}

static csa_status launch_gemm_fp8_pair(const csa_gemm_fp8_args* a, cudaStream_t st) {
  constexpr int BN = GpCfg::BN;
  const int nw = a->W[1] ? 2 : 1;
  CUtensorMap xm, wm[2];
  if (!encode_2d_u8(&xm, a->x, a->K, a->M, GF_ROWS)) return CSA_ERR_CUDA;
  for (int w = 0; w < 2; ++w)
    if (!encode_2d_u8(&wm[w], a->W[w < nw ? w : 0], a->K, a->N, BN / 2)) return CSA_ERR_CUDA;
  GfParams P{};
  P.sx = a->x_scales;
  for (int w = 0; w < nw; ++w) { P.sw[w] = a->W_scales[w]; P.out[w] = (uint16_t*)a->out[w]; }
  P.M = a->M; P.N = a->N; P.KB = (a->K + GF_BK - 1) / GF_BK; P.ks = 1;
  const long long ta = ((long long)a->M + 2 * GF_ROWS - 1) / (2 * GF_ROWS), tb = ((long long)a->N + BN - 1) / BN;
  const long long tiles = ta * tb * nw;
  if (tiles > 0x7fffffffLL / 2) return CSA_ERR_UNSUPPORTED;
  P.tiles_a = (int)ta; P.tiles_b = (int)tb; P.tiles = (int)tiles;
  int sms = 148;
  {
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  }
  const int smem = (int)sizeof(GpSmem) + 1024;
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)gemm_fp8_pair_kernel, smem, attr_done);
  const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch_pdl(gemm_fp8_pair_kernel, dim3((unsigned)(2 * pairs)), dim3(GF_THREADS), smem, st, xm, wm[0], wm[1], P);
}

}  // namespace csa

using namespace csa;

extern "C" csa_status csa_gemm_fp8(const csa_gemm_fp8_args* a, void* stream) {
  CSA_REQUIRE(a != nullptr && a->struct_size == sizeof(csa_gemm_fp8_args));
  CSA_REQUIRE(a->M >= 0 && a->N >= 1 && a->K >= 1);
  CSA_SUPPORTED(a->K % 16 == 0 && a->N % 8 == 0);
  if (a->M == 0) return CSA_OK;
  CSA_REQUIRE(a->x && a->x_scales && a->W[0] && a->W_scales[0] && a->out[0]);
  CSA_REQUIRE(a->W[1] ? (a->W_scales[1] && a->out[1] && a->out[1] != a->out[0]) : (!a->W_scales[1] && !a->out[1]));
  CSA_SUPPORTED((((uintptr_t)a->x | (uintptr_t)a->W[0] | (uintptr_t)a->W[1] | (uintptr_t)a->out[0] |
                  (uintptr_t)a->out[1]) & 15) == 0);
  CSA_SUPPORTED(tensor_map_encoder() != nullptr);
  cudaStream_t st = (cudaStream_t)stream;
  const int KB = (a->K + GF_BK - 1) / GF_BK, nw = a->W[1] ? 2 : 1;
  // Parts of K: doubled while the CTAs still fit one wave, each has a K block, and the clusters find room (GPCs hold
  // one or two of 8 CTAs; 16 such clusters ran in two waves).  Measured, two weights of 512 x 4096: 32 tokens
  // 10.2 / 7.5 / 5.8 / 5.2 us in 1 / 2 / 4 / 8 parts, 256 tokens 12.5 / 9.9 / 8.0 / 15.2, 1024 tokens 12.9 / 10.9.
  auto parts = [&](long long tiles, int most) {
    int ks = 1;
    while (ks < most && 2 * ks <= KB && tiles * ks * 2 <= 148) ks *= 2;
    return ks == 8 && tiles > 14 ? 4 : ks;
  };
  // Up to 64 tokens the channels are the MMA's 128 rows.  Measured, two weights of 512 x 4096, channels / tokens there:
  // 1 token 4.6 / 6.0 us, 32 5.1 / 6.9, 64 6.5 / 7.0, 96 8.2 / 7.3, 128 9.0 / 7.7 (all 0.4 more than now).
  if (a->M <= 64) {
    const long long tiles = ((long long)a->N + 127) / 128 * nw;
    const int ks = parts(tiles, GF_MAX_CLUSTER);
    if (a->M <= 16) return launch_gemm_fp8<16, true>(a, ks, st);
    if (a->M <= 32) return launch_gemm_fp8<32, true>(a, ks, st);
    return launch_gemm_fp8<64, true>(a, ks, st);
  }
  // Tiles of 128 x 128 while they fill one wave at most, pairs of CTAs on 256 x 256 beyond: 2304 / 2560 / 4096 tokens
  // into two weights of 512 x 4096 take 14.9 / 25.1 / 28.4 us with the former and 20.0 / 20.5 / 23.6 us with the latter.
  const long long tiles128 = ((long long)a->M + 127) / 128 * (((long long)a->N + 127) / 128) * nw;
  if (tiles128 < 148) return launch_gemm_fp8<128, false>(a, parts(tiles128, 4), st);
  return launch_gemm_fp8_pair(a, st);
}
