// HCA attention over a prefix of compressed entries that every sequence of the batch shares, on the 5th-generation
// tensor cores: the partial softmax attention of all query rows (each a head of a query) over the prefix's bf16 rows.
// Since the prefix is the same for all and there is one shared KV head, the rows of the whole batch form one matrix;
// a pair of CTAs attends with 128 of them at a time over tiles of 256 entries (K = V, 512 wide):
//
//   S[row][key] = Q[row][:] . K[key][:]              M = 128 rows, N = 256 keys, K = 512 (32 MMAs)
//   P = exp2(S * scale*log2e - m_row)                m: a running reference per row, see below
//   O[row][dim] += sum_key P[row][key] K[key][dim]   M = 128, N = 2 x 256 dims, K = 256 (32 MMAs)
//
// What bounds it is shared memory: an SM reads 128 bytes a cycle, and 16-deep MMAs that keep both operands there need
// 7 KB for 128 x 96 (one CTA, entries as the 128 rows: 8560 cycles a tile of 128 keys x 96 rows were measured, 2940
// flop a cycle) but 6 KB for 64 x 256 an SM here: with cta_group::2 each CTA holds 64 rows of A and half of B, and M = 128
// over a pair runs at the full rate from N = 256 on (64 cycles, measured).  O takes 256 columns of tensor memory, S 128:
// a CTA's lanes 0-63 hold its 64 rows over the first half of N, lanes 64-127 the same rows over the second half.
//
// Operands: S wants from CTA c the tile's keys 128 c .. 128 c + 127 over all dims (8 chunks of 128 keys x 64 dims,
// 16 KB), O wants all 256 keys over the dims 128 c .. and 256 + 128 c ..  Half of the chunks serve both; the others
// are replaced in place once S has read them (12 loads a tile instead of 16):
//   slot        0    1    2    3    4    5    6    7
//   S  (c)    dims 64 j .. of keys 128 c ..
//   O  (0)    kept kept new  new  kept kept new  new     (keys 0 .. in slots 0 1 4 5, keys 128 .. in 2 3 6 7;
//   O  (1)    new  new  kept kept new  new  kept kept     dims 128 c + 64 (j & 1) .. in 0-3, 256 more in 4-7)
// Softmax: a row's reference m moves only when a tile's scores exceed it by more than 2^8 (or in a part's first tile);
// the probabilities are written with the old one and the CTA's threads agree afterwards, with one barrier, whether that
// did; a thread sums its own columns until the part ends.
// A block's last tiles can be the own keys of the sequences it touches (bf16 rows from own_rows_kernel), masked to the rows
// of their sequence and to what each sees.  An own row that is not finite would reach every row of the block through
// 0 x NaN: own_rows_kernel writes it as zero and marks it, and the rows that see it get NaN.
// Parts: the tiles of all blocks of 128 rows form one line that is cut evenly over the pairs, so a pair works on the end
// of one block and the start of the next, and each leaves a partial (O / l in scaled fp16, lse) that the
// merge adds.
// Measured (replayed graphs, 1.85 GHz under the power cap): 64 sequences of 64 heads over 8192 shared entries take about
// 70 us here, 6700 cycles a tile (128 rows x 256 keys a pair) of which the MMAs need 4096: S 2700 (its operands arrive
// at the L2's rate), the wake-up of the softmax warps 300, softmax 2000, O 1750.  One pair has no room for a second
// S (O's accumulator and the operands fill tensor and shared memory), so softmax and MMAs take turns.
// Every wait is bounded; a wait that gives up records device error 1 and the kernel leaves.
// Sources: "DeepSeek-V4: エージェントが実際に使える100万トークンのコンテキスト", §ハイブリッド注意, Fig. 4 (the 128x layer
// attends densely over all visible entries).
#include "csa_common.cuh"
#include "sm100.cuh"

namespace csa {

using namespace sm100;

constexpr int PX_ROWS = 128;                // query rows of a block: 64 a CTA
constexpr int PX_KEYS = 256;                // entries of a tile
constexpr int PX_WORKERS = 512;             // warps 0-15: 4 lane quadrants x 4 quarters of a lane's columns
constexpr int PX_THREADS = PX_WORKERS + 64; // warp 16: TMA, warp 17: tensor memory, MMA (rank 0)
constexpr int PX_CHUNK = 128 * 128;         // 128 keys x 64 dims bf16
constexpr uint32_t PX_COL_S = 0, PX_COL_O = 128;
constexpr float PX_SLACK = 8.0f;            // log2 units: probabilities stay <= 2^8
constexpr float PX_LOG2E = 1.4426950408889634f, PX_LN2 = 0.6931471805599453f;

struct PxSmem {
  alignas(1024) uint8_t Q[8][64 * 128];     // [dim block][row][128 B], 128-byte swizzle
  alignas(1024) uint8_t K[8][PX_CHUNK];     // [slot][key][128 B], 128-byte swizzle
  alignas(1024) uint8_t P[4][64 * 128];     // [64 keys][row][128 B], 128-byte swizzle
  alignas(8) uint64_t full[8];              // rank 0: a slot's operands have landed in both CTAs (twice a tile: S, O)
  uint64_t rel[8];                          // both: a slot has been read (twice a tile: by S, by O)
  uint64_t bar_q[8];                        // rank 0: a dim block of Q has landed in both
  uint64_t bar_qfree, bar_s, bar_o;         // both: Q read; S complete; O complete
  uint64_t bar_p;                           // rank 0: P written (and S read) in both
  uint32_t tmem_base;
  uint32_t err;
};

struct PxParams {
  long long R;            // query rows: B * Nq * H
  long long T;            // tiles of all blocks (< 2^31), its quotient and remainder by the pairs
  int T_quot, T_rem;
  int tiles;              // tiles of one block: of the prefix, then nseq * otiles of own keys
  int ptiles;             // tiles of the prefix: ceil(n_p / 256)
  int nseq, otiles;       // own keys: sequences a block can touch, tiles of one sequence (0: attended elsewhere)
  int B, Nq, H, ratio, n_p, n_max;
  int E, Wn, window;      // own rows of a sequence: entries n_p .. n_p + E - 1, then Wn window rows
  const uint8_t* bad;     // [B][256 otiles] 1: an own row that holds NaN or infinities (and reads as zero)
  int early;              // the kernel before this one is own_rows_kernel: only own tiles wait for it
  const int64_t* win_pos0;
  int slot0, slots;       // partial slots of a query: this kernel's first, and all
  int pslots;             // this kernel's
  float scale_log2;
  const int64_t* q_pos;
  const int32_t* n_c;
  uint16_t* part_o;       // [query][slots][H][512] fp16, times
  float* part_scale;      // [query][slots][H][8]: a power of two for 64 dims
  float* part_lse;        // [query][slots][H]
};

// The pair that tile g of the line belongs to when it is cut into G even parts [i T / G, (i + 1) T / G).
__host__ __device__ __forceinline__ long long px_pair_of(long long g, long long G, long long T) { return ((g + 1) * G - 1) / T; }

// Tile i of a block: prefix rows from row0 on (b = -1), or own rows of sequence b, its keys key0 on.
struct PxTile {
  int b, key0, row0;
};
__device__ __forceinline__ PxTile px_tile(const PxParams& P, long long blk, int i) {
  PxTile t;
  if (i < P.ptiles) {
    t.b = -1;
    t.key0 = t.row0 = i * PX_KEYS;
  } else {
    const int o = i - P.ptiles, s = o / P.otiles;
    t.b = (int)((uint32_t)(blk * PX_ROWS) / (uint32_t)(P.Nq * P.H)) + s;
    t.key0 = (o - s * P.otiles) * PX_KEYS;
    // (a sequence behind the last: some rows that no query row is matched with)
    t.row0 = min(t.b, P.B - 1) * (P.E + P.Wn) + t.key0;
  }
  return t;
}

// The lowest n bits (n may be anything).
__device__ __forceinline__ uint32_t px_low(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

__device__ __forceinline__ float px_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void px_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
// Barrier of the softmax warps that returns whether any of their threads passed true.
__device__ __forceinline__ bool px_any(bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, 1, 512, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r) : "r"((uint32_t)v) : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(PX_THREADS, 1) __cluster_dims__(2, 1, 1)
    attn_prefix_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap omap, const PxParams P) {
  extern __shared__ uint8_t smem_raw[];
  PxSmem& S = *reinterpret_cast<PxSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x & 1;
  const long long pair = blockIdx.x >> 1, G = gridDim.x >> 1;
  // floor(pair T / G) and the next pair's, from T's quotient and remainder by G
  auto cut = [&](int i) { return i * P.T_quot + (int)((uint32_t)(i * P.T_rem) / (uint32_t)G); };
  const long long g_begin = cut((int)pair), g_end = cut((int)pair + 1);
  if (tid == 0) {
    S.err = 0;
    for (int i = 0; i < 8; ++i) { mbar_init(&S.full[i], 1); mbar_init(&S.rel[i], 1); mbar_init(&S.bar_q[i], 1); }
    mbar_init(&S.bar_qfree, 1);
    mbar_init(&S.bar_s, 1);
    mbar_init(&S.bar_o, 1);
    mbar_init(&S.bar_p, 2 * PX_WORKERS / 32);
    fence_mbar_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    if (P.otiles > 0) prefetch_tensormap(&omap);
  }
  if (warp == 17) { tmem_alloc_pair(&S.tmem_base, 512); tmem_relinquish_pair(); }
  pdl_trigger();
  __syncthreads();
  cluster_sync_all();                        // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tb = S.tmem_base;
  bool ok = true;
  // own_rows_kernel lets this grid start only after all work before it has completed, and writes nothing but own rows
  if (!P.early) pdl_wait();

  if (warp == 16) {
    // ------------------------------------------------------------------------ TMA producer (one per CTA)
    if (lane == 0) {
      uint32_t tile = 0, part = 0;
      for (long long g = g_begin; g < g_end && ok; ++part) {
        const long long blk = (uint32_t)g / (uint32_t)P.tiles, blk_end = (blk + 1) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
        // the previous part's S MMAs have read Q
        if (part > 0 && !mbar_wait(&S.bar_qfree, (part - 1) & 1)) { ok = false; break; }
        bool q_due = true;                       // Q's dim blocks go with the first tile's chunks
        for (; g < e && ok; ++g, ++tile) {
          const PxTile w = px_tile(P, blk, (int)(g - blk * P.tiles));
          const CUtensorMap* map = w.b < 0 ? &kmap : &omap;
          if (w.b >= 0) pdl_wait();              // (again and again: a no-op after the first)
          for (int j = 0; j < 8 && ok; ++j) {
            if (tile > 0 && !mbar_wait(&S.rel[j], 1)) { ok = false; break; }      // read by the previous tile's O
            if (q_due) {
              if (rank == 0) mbar_arrive_expect_tx(&S.bar_q[j], 2 * 64 * 128);
              tma_load_2d_pair(S.Q[j], &qmap, j * 64, (int)(blk * PX_ROWS) + 64 * rank, peer_addr(&S.bar_q[j], 0));
            }
            if (rank == 0) mbar_arrive_expect_tx(&S.full[j], 2 * PX_CHUNK);
            tma_load_2d_pair(S.K[j], map, j * 64, w.row0 + 128 * rank, peer_addr(&S.full[j], 0));
          }
          q_due = false;
          for (int j = 0; j < 8 && ok; ++j) {
            if (!mbar_wait(&S.rel[j], 0)) { ok = false; break; }                  // read by S
            const int owner = (j & 2) ? 0 : 1;                                    // whose chunk is not the one O wants
            if (rank == 0) mbar_arrive_expect_tx(&S.full[j], PX_CHUNK);
            if (rank == owner)
              tma_load_2d_pair(S.K[j], map, ((j & 4) ? 256 : 0) + 128 * rank + 64 * (j & 1), w.row0 + ((j & 2) ? 128 : 0),
                               peer_addr(&S.full[j], 0));
          }
        }
      }
      if (!ok) {
        atomicOr(&S.err, 1u);
        for (int i = 0; i < 1000; ++i) __nanosleep(200);       // copies in flight land before the CTA may leave
      }
    }
    __syncwarp();
  } else if (warp == 17) {
    // ------------------------------------------------------------------------ MMA issuer
    // (the whole warp of rank 0 walks, one lane issues: see elect_one)
    if (rank == 0) {
      const uint32_t ids = idesc_bf16(128, 256, 0, 0), ido = idesc_bf16(128, 256, 0, 1);
      const uint64_t qdesc = smem_desc(smem_addr(S.Q[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t kdesc = smem_desc(smem_addr(S.K[0]), 16, 1024, LAYOUT_SW128);
      const uint64_t vdesc = smem_desc(smem_addr(S.K[0]), PX_CHUNK, 1024, LAYOUT_SW128);
      const uint64_t pdesc = smem_desc(smem_addr(S.P[0]), 16, 1024, LAYOUT_SW128);
      auto landed = [&](uint64_t* bar, uint32_t ph) {
        if (!mbar_test(bar, ph)) ok = ok && mbar_wait(bar, ph);
      };
      uint32_t f = 0, part = 0;
      for (long long g = g_begin; g < g_end && ok; ++part) {
        const long long blk_end = ((uint32_t)g / (uint32_t)P.tiles + 1LL) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
        const int n = (int)(e - g);
#pragma unroll 1
        for (int t = 0; t < n && ok; ++t, ++f) {
          // (the loops are kept short: a part's first pass fetches this code from L2)
#pragma unroll 1
          for (int j = 0; j < 8; ++j) {
            if (t == 0) landed(&S.bar_q[j], part & 1);
            landed(&S.full[j], 0);
            tc_fence_after();
            const uint64_t qd = qdesc + (uint64_t)(j * (64 * 128 >> 4)), kd = kdesc + (uint64_t)(j * (PX_CHUNK >> 4));
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < 4; ++s) mma_bf16_ss_pair(tb + PX_COL_S, qd + 2 * s, kd + 2 * s, ids, (j | s) != 0);
              mma_commit_pair(&S.rel[j]);
              if (j == 7) {
                mma_commit_pair(&S.bar_s);
                if (t + 1 == n) mma_commit_pair(&S.bar_qfree);
              }
            }
            __syncwarp();
          }
          ok = ok && mbar_wait(&S.bar_p, f & 1);
          tc_fence_after();
          // slots 2 i, 2 i + 1: keys 128 (i & 1) .., dims 256 (i >> 1) ..
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            landed(&S.full[2 * i], 1);
            landed(&S.full[2 * i + 1], 1);
            tc_fence_after();
            const uint64_t pd = pdesc + (uint64_t)((i & 1) * (2 * 64 * 128 >> 4)), vd = vdesc + (uint64_t)(i * (2 * PX_CHUNK >> 4));
            const uint32_t d = tb + PX_COL_O + 128 * (i >> 1);
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < 8; ++s)
                mma_bf16_ss_pair(d, pd + (uint64_t)(((s >> 2) * 64 * 128 + (s & 3) * 32) >> 4), vd + 128 * s, ido,
                                 t > 0 || (i & 1) || s > 0);
              mma_commit_pair(&S.rel[2 * i]);
              mma_commit_pair(&S.rel[2 * i + 1]);
              if (i == 3 && t + 1 == n) mma_commit_pair(&S.bar_o);
            }
            __syncwarp();
          }
        }
        g = e;
      }
      if (!ok && lane == 0) atomicOr(&S.err, 1u);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------ softmax and epilogue
    // warp: lane quadrant `quad`, quarter `ch` of its lanes' columns.  A thread has one row, and of a tile the 32 keys
    // of eighth kq.  (16 warps of 32 keys: 8 warps of 64 spilled and hid less latency.)
    const int quad = warp & 3, ch = warp >> 2;
    const int row = 32 * (quad & 1) + lane, kq = 4 * (quad >> 1) + ch;
    const uint32_t lane_base = tb + ((uint32_t)(32 * quad) << 16);
    uint8_t* prow = &S.P[kq >> 1][row * 128];
    float (*red)[64] = reinterpret_cast<float (*)[64]>(S.P[0]);   // [key eighth][row], while P holds nothing of use
    const int pc = 4 * (kq & 1);                 // the thread's 16-byte chunks of that row: pc .. pc + 3
    const uint32_t bar_p = peer_addr(&S.bar_p, 0);
    uint32_t f = 0, part = 0;
    for (long long g = g_begin; g < g_end; ++part) {
      const long long blk = (uint32_t)g / (uint32_t)P.tiles, blk_end = (blk + 1) * P.tiles, e = blk_end < g_end ? blk_end : g_end;
      // how many entries the row sees (rows behind the last query row: all of them, their Q is zero and nothing is
      // stored), and its place in the partials without the slot
      const long long qr = blk * PX_ROWS + 64 * rank + row;
      const bool real = qr < P.R;
      // (own keys 0 .. ve - 1 are visible entries, wl .. wh - 1 the window)
      int nv = P.n_p, b = -2, ve = 0, wl = 0, wh = 0;
      long long prt = 0;
      if (real) {
        const long long bq = (uint32_t)qr / (uint32_t)P.H, tq = P.q_pos[bq];
        b = (int)bq / P.Nq;
        const int see = (int)max(0LL, min((long long)min(P.n_c[b], P.n_max), (tq + 1) / P.ratio));
        nv = min(P.n_p, see);
        ve = max(0, see - P.n_p);
        if (P.otiles > 0 && P.Wn > 0) {
          const long long p0 = P.win_pos0[b], lo = max(max(0LL, tq - P.window + 1), p0), hi = min(tq, p0 + P.Wn - 1);
          if (hi >= lo) { wl = P.E + (int)(lo - p0); wh = P.E + (int)(hi - p0) + 1; }
        }
        prt = bq * P.slots * P.H + (qr - bq * P.H);
      }
      float m = -INFINITY;                       // the row's reference (log2 units); its four threads agree
      float l = 0.f;                             // this thread's part of the row's sum
      for (long long t = g; t < e; ++t, ++f) {
        const bool first = t == g;
        const PxTile w = px_tile(P, blk, (int)(t - blk * P.tiles));
        const int k0 = w.key0 + 32 * kq;         // this thread's first key
        uint32_t see = 0;                        // which of its 32 keys the row sees
        bool bad = false;                        // one of them has no finite row: the row's result is NaN
        if (w.b < 0) {
          see = px_low(nv - k0);
        } else if (w.b == b) {
          see = px_low(ve - k0) | (px_low(wh - k0) & ~px_low(wl - k0));
          if (see) {
            pdl_wait();
            const uint4* at = reinterpret_cast<const uint4*>(P.bad + (size_t)b * P.otiles * PX_KEYS + k0);
            const uint4 x = at[0], y = at[1];
            if (x.x | x.y | x.z | x.w | y.x | y.y | y.z | y.w) {
              const uint8_t* s = reinterpret_cast<const uint8_t*>(at);
              for (int j = 0; j < 32; ++j) bad |= ((see >> j) & 1) && s[j] != 0;
            }
          }
        }
        const bool all = see == 0xffffffffu;
        ok = ok && mbar_wait(&S.bar_s, f & 1);
        tc_fence_after();
        // The tile is done with the reference as it is; where that turns out too low for some row (every thread of the CTA
        // learns of it at once), or in a part's first tile, once more with moved references.  The columns come 16 at a
        // time and the loops stay rolled: unrolled over all columns the kernel outgrows the instruction caches, and a
        // tile took a tenth longer.
        auto scores = [&](int c, float (&z)[16]) -> float {             // columns 16 c ..; returns their maximum
          uint32_t v[16];
          tmem_ld_x16(lane_base + PX_COL_S + 32 * ch + 16 * c, v);
          tmem_wait_ld_x16(v);
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = __uint_as_float(v[j]);
          if (!all) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!((see >> (16 * c + j)) & 1)) z[j] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) top = fmaxf(top, z[j]);
          return top;
        };
        float lt;                                // this thread's part of the tile's sum
        for (bool again = first;; again = true) {
          if (again) {
            float z[16], top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) top = fmaxf(top, scores(c, z));
            red[kq][row] = top * P.scale_log2;   // (the scale is positive)
            px_sync();
            float mt = red[0][row];
#pragma unroll
            for (int i = 1; i < 8; ++i) mt = fmaxf(mt, red[i][row]);
            const float mn = first || mt > m + PX_SLACK ? fmaxf(m, mt) : m;
            const float fc = first || mn == m ? 1.f : exp2f(m - mn);
            m = mn;
            l *= fc;
            if (!first && __any_sync(0xffffffffu, fc != 1.f)) {
              // O of the rows whose reference moved (the O MMAs so far completed before S did); this thread's
              // quarter of its lane's 256 columns
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t o[16];
                const uint32_t at = lane_base + PX_COL_O + 64 * ch + 16 * c;
                tmem_ld_x16(at, o);
                tmem_wait_ld_x16(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fc);
                tmem_st_x16(at, o);
              }
              tmem_wait_st();
            }
            px_sync();                           // red has been read
          }
          const float mm = m == -INFINITY ? 0.f : m;   // (a row that sees no key: every z is -inf)
          float top = -INFINITY;
          lt = 0.f;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float z[16];
            top = fmaxf(top, scores(c, z));
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
              float p[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                p[i] = px_exp2(fmaf(z[j + i], P.scale_log2, -mm));
                lt += p[i];
              }
              // P is rounded to bf16 for the MMA (2^-8 of a probability); the sum takes the unrounded values
              *reinterpret_cast<uint4*>(prow + ((((pc + 2 * c + (j >> 3)) ^ row) & 7) << 4)) =
                  make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]));
            }
          }
          if (again || !px_any(top * P.scale_log2 > m + PX_SLACK)) break;
        }
        l += bad ? __int_as_float(0x7fffffff) : lt;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(bar_p);
      }
      // ---- the part's partial: O / l
      const int slot = P.slot0 + (int)(pair - px_pair_of(blk * P.tiles, G, P.T));
      const long long out = prt + (long long)slot * P.H;
      ok = ok && mbar_wait(&S.bar_o, part & 1);
      tc_fence_after();
      red[kq][row] = l;
      px_sync();
      float ls = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ls += red[i][row];
      px_sync();                                 // red is free again
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      if (real && kq == 0) {
        P.part_lse[out] = ls == 0.f ? -INFINITY : (m + log2f(ls)) * PX_LN2;
        // slots of this block that no pair fills
        if (e == blk_end)
          for (int s = slot + 1; s < P.slot0 + P.pslots; ++s) P.part_lse[prt + (long long)s * P.H] = -INFINITY;
      }
      // This thread's columns 64 ch .. are the dims 64 blk64 .. of its row: fp16 values times a power of two for the 64
      // (from their largest), 2^-11 off at most where bf16 would be 2^-8, at no more bytes.
      const int blk64 = 4 * (ch >> 1) + 2 * (quad >> 1) + (ch & 1);
      float big = 0.f;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[16];
        tmem_ld_x16(lane_base + PX_COL_O + 64 * ch + 16 * c, o);
        tmem_wait_ld_x16(o);
#pragma unroll
        for (int j = 0; j < 16; ++j) big = fmaxf(big, fabsf(__uint_as_float(o[j])));
      }
      const uint32_t ex = min(max(__float_as_uint(big * inv) >> 23, 1u), 253u);
      const bool finite = big * inv < INFINITY;
      const float fac = finite ? inv * __uint_as_float((254u - ex) << 23) : inv;
      if (real) P.part_scale[out * 8 + blk64] = finite ? __uint_as_float(ex << 23) : 1.f;
      // 32 columns at a time through this warp's 2 KB of the P buffer (the O MMAs have read it) so that 4 lanes store 64
      // bytes of a row (16 bytes a row and store took 6000 cycles)
      uint8_t* stage = S.P[0] + 2048 * warp;
      uint16_t* dst = P.part_o + 64 * blk64 + 8 * (lane & 3);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t o[32];
        tmem_ld_x32(lane_base + PX_COL_O + 64 * ch + 32 * c, o);
        tmem_wait_ld_x32(o);
        __syncwarp();                            // the rows of the round before have been read
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(__uint_as_float(o[8 * k + 2 * i]) * fac, __uint_as_float(o[8 * k + 2 * i + 1]) * fac);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(stage + lane * 64 + (((k ^ (lane >> 1)) & 3) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 8 * k + (lane >> 2);
          const long long ro = __shfl_sync(0xffffffffu, real ? out : -1LL, r);
          const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 + ((((lane & 3) ^ (r >> 1)) & 3) << 4));
          if (ro >= 0) *reinterpret_cast<uint4*>(dst + ro * 512 + 32 * c) = w;
        }
      }
      tc_fence_before();
      px_sync();                                 // the next part's first tile writes red, which is warp 0's stage
      g = e;
    }
    if (!ok && lane == 0) atomicOr(&S.err, 1u);
  }
  // every MMA has completed (the last part's O was waited for in both CTAs) and no arrival is on its way to a CTA
  // that has left
  __syncthreads();
  if (S.err && tid == 0) atomicOr(&g_csa_device_error, 1u);
  if (P.early && tid == 0) pdl_wait();           // the grid completes only after its predecessor
  cluster_sync_all();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc_pair(tb, 512);
  }
}

// Tiles of own keys that a block of rows has when the prefix kernel takes them too: the sequences it can touch, and the
// tiles of one.
static void px_own(const csa_attn_args* a, int n_p, int* nseq, int* otiles) {
  const long long rs = (long long)a->Nq * a->H;             // rows of a sequence
  const long long n = PX_ROWS % rs == 0 ? PX_ROWS / rs : rs % PX_ROWS == 0 ? 1 : (PX_ROWS + rs - 2) / rs + 1;
  *nseq = (int)(n < a->B ? n : a->B);
  *otiles = (int)(((long long)a->n_max - n_p + (attn_has_window(a) ? a->Wn : 0) + PX_KEYS - 1) / PX_KEYS);
}

// Whether the prefix kernel takes the own keys too (as bf16 rows written by own_rows_kernel), or the per-query attention
// does: by their times.  A tile takes a pair 4.0 us, rows are written at about 4.2 TB/s; the per-query kernels take about
// 10 us and 7.9 us a wave of tiles of 128 keys.  Here every row of the window buffer counts, there the `window` rows of
// it that a query can see at most.  Measured, here / there: 16 sequences of 64 heads with 64 own entries
// after 8192 shared ones 32.7 / 44.6 us, 40 of 16 heads with 3000 after 200 94.6 / 111.4; 64 of 64 with 64 after 8192 and
// 1024 window rows 127 / 86, 1 of 64 heads and 4096 queries with 64 after 8192 and 4223 window rows 5974 / 4303.  Over 21
// shapes of 1 to 4096 queries and windows of up to 32 times their length the rule's choice costs 1.3 % on average,
// 13 % at most (128 of 16 heads with 500 after 512: 69.9 / 61.7, the wrong one).
bool attn_prefix_takes_own(const csa_attn_args* a, int n_p) {
  int nseq, otiles;
  px_own(a, n_p, &nseq, &otiles);
  const double rows = (double)a->B * a->Nq, R = rows * a->H;
  const double ent = (double)a->n_max - n_p;
  const double own = ent + (attn_has_window(a) ? a->Wn : 0);
  const double seen = ent + (attn_has_window(a) ? (a->Wn < a->window ? a->Wn : a->window) : 0);
  if (own * a->B > 2147483647.0) return false;
  const double blocks = (double)((long long)(R + PX_ROWS - 1) / PX_ROWS);
  const double t_here = 4.0 * blocks * nseq * otiles / 74 + a->B * own * 1024 / 4.2e6;
  const double waves = (double)(long long)((rows * (double)(long long)((seen + 127) / 128) + 147) / 148);
  return t_here < 10.0 + 7.9 * waves;
}

// The prefix kernel's plan: pairs of CTAs, and partial slots a query needs (at most `most`); 0 pairs: too many tiles.
void attn_prefix_plan(const csa_attn_args* a, int n_p, bool own, int most, int* pairs, int* slots) {
  const long long R = (long long)a->B * a->Nq * a->H;
  int nseq = 0, otiles = 0;
  if (own) px_own(a, n_p, &nseq, &otiles);
  const long long blocks = (R + PX_ROWS - 1) / PX_ROWS;
  const long long tiles = ((long long)n_p + PX_KEYS - 1) / PX_KEYS + (long long)nseq * otiles, T = blocks * tiles;
  *pairs = *slots = 0;
  if (T > 0x7fffffffLL) return;                            // (the kernel counts tiles in 32 bits)
  // Every part costs about as much as 1.2 tiles on top (its first operands from L2, its epilogue).  Cut evenly over all
  // pairs a pair often has two parts; cut at the blocks' ends (a whole number of pairs a block) it has one, of ever so
  // many more tiles: 16 sequences of 64 heads over 8192 entries, 8 blocks of 34 tiles, 35.8 us with 74 pairs, 32.8 with
  // 72; 24 over 4096 36.6 and 28.4; 64 over 1024 38.2 and 31.4.
  long long G = T < 74 ? T : 74;
  if (T > 74 && blocks <= 74) {
    const long long k = 74 / blocks < tiles ? 74 / blocks : tiles;
    if ((double)((tiles + k - 1) / k) + 1.2 < (double)T / 74 + 2.4) G = blocks * k;
  }
  if (G > blocks * (most - 1)) G = blocks * (most - 1);    // a block is cut into at most ceil(G / blocks) + 1 parts
  long long worst = 1;
  if (blocks >= G) {
    worst = blocks == G ? 1 : 2;                           // every part is at least a block's worth
  } else {
    for (long long b = 0; b < blocks; ++b) {
      const long long n = px_pair_of((b + 1) * tiles - 1, G, T) - px_pair_of(b * tiles, G, T) + 1;
      if (n > worst) worst = n;
    }
  }
  *pairs = (int)G;
  *slots = (int)worst;
}

// own_rows: own_rows_kernel's output, or null (the own keys are attended elsewhere).
csa_status launch_attn_prefix(const csa_attn_args* a, const void* prefix, int n_p, const void* own_rows, int pairs, int slot0,
                              int pslots, int slots, uint16_t* part_o, float* part_scale, float* part_lse,
                              cudaStream_t st) {
  const long long R = (long long)a->B * a->Nq * a->H;
  CUtensorMap qm, km, om;
  auto encode = [](CUtensorMap* map, const void* base, long long rows, int box) {
    const cuuint64_t gdim[2] = {512, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {1024};
    const cuuint32_t bx[2] = {64, (cuuint32_t)box};
    const cuuint32_t estr[2] = {1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, bx, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  PxParams P{};
  P.E = a->n_max - n_p;
  P.Wn = attn_has_window(a) ? a->Wn : 0;
  if (!encode(&qm, a->q, R, 64) || !encode(&km, prefix, n_p, 128)) return CSA_ERR_CUDA;
  if (own_rows == nullptr)
    om = km;                                   // never read
  else if (!encode(&om, own_rows, (long long)a->B * (P.E + P.Wn), 128))
    return CSA_ERR_CUDA;
  P.R = R;
  P.ptiles = (n_p + PX_KEYS - 1) / PX_KEYS;
  if (own_rows) px_own(a, n_p, &P.nseq, &P.otiles);
  P.tiles = P.ptiles + P.nseq * P.otiles;
  P.early = own_rows != nullptr;
  P.bad = (const uint8_t*)own_rows + (size_t)a->B * (P.E + P.Wn) * 1024;
  P.B = a->B; P.window = a->window; P.win_pos0 = a->win_pos0;
  P.T = (R + PX_ROWS - 1) / PX_ROWS * P.tiles;
  P.T_quot = (int)(P.T / pairs); P.T_rem = (int)(P.T % pairs);
  P.Nq = a->Nq; P.H = a->H; P.ratio = a->ratio; P.n_p = n_p; P.n_max = a->n_max;
  P.slot0 = slot0; P.slots = slots; P.pslots = pslots;
  P.scale_log2 = (a->softmax_scale != 0.0f ? a->softmax_scale : 1.0f / sqrtf(512.0f)) * PX_LOG2E;
  P.q_pos = a->q_pos; P.n_c = a->n_c; P.part_o = part_o; P.part_scale = part_scale; P.part_lse = part_lse;
  const int smem = (int)sizeof(PxSmem) + 1024;
  static_assert(sizeof(PxSmem) + 1024 <= 232448, "shared memory of a CTA");
  static std::atomic<unsigned> attr_done{0};
  set_smem_once((const void*)attn_prefix_tc_kernel, smem, attr_done);
  return launch_pdl(attn_prefix_tc_kernel, dim3((unsigned)(2 * pairs)), dim3(PX_THREADS), (size_t)smem, st, qm, km, om, P);
}

}  // namespace csa
