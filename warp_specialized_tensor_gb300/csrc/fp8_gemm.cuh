// fp8_gemm.cuh -- persistent, warp-specialized product of 8-bit floating-point
// matrices with an fp32 scale for each block of 128 along K, dense and grouped,
// on CTA pairs.
//
//   C[t][n] = sum_kb sA[kb][t] sB[kb][n] sum_{k in block kb} A[t][k] B[g][n][k]
//
// sA: one scale per token row and K block.  sB: one per feature row and K block
// (1 x 128), or one per 128 features (128 x 128).
//
// The tensor core computes the transposed tile D[n][t] (features on the 256-row
// MMA side, tokens on the N side in multiples of 16 up to 256, as in the bf16
// grouped GEMM: a ragged group wastes at most 15 token columns).  A K block of
// 128 is one 128-byte swizzled row per operand and four MMAs; its unscaled
// product goes to one of two tensor-memory accumulators, from where the epilogue
// warps add it, scaled, to fp32 sums in registers while the tensor core fills
// the other one.  Per K block a pair tile of 256 x 256 costs the tensor core
// about 512 cycles, and each of the four sub-cores of an SM 256 tensor-memory
// columns, 256 fused multiply-adds and 64 shared
// loads of the token scales.
//
// Roles per CTA (persistent, one CTA per SM, pairs in clusters of 2):
//   warp 0     TMA producer: this CTA's 128 rows of B[g] and its half of the
//              token tile, 128 bytes of K each; both CTAs' copies complete on
//              the leader's full[s].
//   warp 1     MMA issuer (leader CTA only), kind::f8f6f4, M = 256.
//   warp 2     tensor-memory allocation, offset check.
//   warp 3     scales of each K block to shared memory: those of the tokens
//              (4-byte loads: a group may start at any row), with 128 x 128
//              weight scales already times the CTA's one weight scale.
//   warps 4-11 epilogue: two warps per 32 features, each half of the tokens.
//
// Few tiles (short token tiles of a decoding step): when the tiles fill less
// than half of the pairs, each tile's K blocks are split over several pairs;
// every pair stores its fp32 sums to the workspace, and the last one to arrive
// (a counter per tile and CTA, which it sets back to 0) adds them in the order
// of the splits, so the result does not depend on which one is last.
#pragma once

#include "wst_common.cuh"

namespace wst {

constexpr int kF8Tile = 256;      // features per pair, tokens per tile
constexpr int kF8BK = 128;        // K per block, one scale each
constexpr int kF8Stages = 5;
constexpr int kF8EpiWarps = 8;
constexpr int kF8Parts = kF8EpiWarps / 4;       // warps that share 32 features
constexpr int kF8PartCols = kF8Tile / kF8Parts;  // their token columns
constexpr int kF8Threads = 128 + 32 * kF8EpiWarps;
constexpr int kF8WBytes = 128 * kF8BK;
constexpr int kF8XBytes = 128 * kF8BK;
constexpr int kF8StageBytes = kF8WBytes + kF8XBytes;
constexpr int kF8ThinRows = 16;   // token rows per TMA box of a tile of at most 128 tokens
constexpr int kF8ScaleStages = 8;
constexpr int kF8StgBytes = 2048;  // 32 features x 32 tokens (bf16) or 16 tokens (fp32)
constexpr int kF8TabMax = 256;
constexpr int kF8WalkBytes = 128;  // an epilogue warp's place in the walk over the tiles
constexpr size_t kF8SmemBytes = (size_t)kF8Stages * kF8StageBytes + kF8ScaleStages * kF8Tile * 4 +
                                kF8EpiWarps * kF8StgBytes + 512 + kF8TabMax * 4 + kF8EpiWarps * kF8WalkBytes + 1024;
static_assert(kF8SmemBytes <= 232448, "shared memory per CTA");
// Workspace: header (its padding holds one counter per split tile, 0 between
// calls, one half of it for each CTA of the pair) | one slot of fp32 sums per
// split unit and CTA.  Two splits at least, so at most half as many tiles as
// units.
constexpr int kF8MaxUnits = 120;
static_assert(kF8MaxUnits / 2 <= 60, "counters fit the header's padding");
constexpr size_t kF8SlotFloats = 128 * kF8Tile;
constexpr size_t kF8WorkspaceBytes = kWsHeaderBytes + (size_t)kF8MaxUnits * 2 * kF8SlotFloats * 4;

struct F8Args {
  int G, M_total, N, K;
  int n_tiles, k_blocks;
  const int* offsets;  // device int32[G+1]; NULL: one group of M_total rows
  const float* sa;     // sa[kb * ldsa + t]
  long long ldsa;
  const float* sb;     // rows: sb[g * strideSB + kb * ldsb + n]; blocks: sb[g * strideSB + (n / 128) * ldsb + kb]
  long long ldsb, strideSB;
  uint32_t idesc;      // without N
  const __nv_bfloat16* bias;
  long long bias_stride;
  int epi;
  void* C;
  long long ldc;
  int w_shared;
  int pairs;           // CTA pairs that can be resident at once
  int max_units;       // split units the workspace holds (0: never split)
  WsHeader* ws;
  unsigned long long timeout_ns;
};

// Splits of each tile's K loop: as many as keep every unit on a pair of its own.
__host__ __device__ inline int f8_splits(long long tiles, int pairs, int k_blocks, int max_units) {
  const int room = pairs < max_units ? pairs : max_units;
  if (tiles <= 0 || tiles > room) return 1;
  int s = room / (int)tiles;
  if (s > k_blocks / 4) s = k_blocks / 4;  // at least four K blocks each
  return s < 2 ? 1 : s;
}

struct F8Tile {
  int g, t0, nt, nmma, n0;
};

// Walks the groups in order; offsets are clamped into [0, M_total].
struct F8Walker {
  int g;
  long long base, count;
  int r0, r1, tt;
  const int* tab;

  __device__ __forceinline__ int off(const F8Args& p, int i) const {
    if (!p.offsets) return i ? p.M_total : 0;
    return tab ? tab[i] : __ldg(p.offsets + i);
  }
  __device__ __forceinline__ void load(const F8Args& p) {
    if (g >= p.G) { count = 0; return; }
    r0 = min(max(off(p, g), 0), p.M_total);
    r1 = min(max(off(p, g + 1), r0), p.M_total);
    tt = (r1 - r0 + kF8Tile - 1) / kF8Tile;
    count = (long long)tt * p.n_tiles;
  }
  __device__ __forceinline__ void init(const F8Args& p, const int* table) {
    tab = table;
    g = 0;
    base = 0;
    load(p);
  }
  __device__ __forceinline__ bool seek(const F8Args& p, long long t) {
    while (g < p.G && t >= base + count) {
      base += count;
      ++g;
      load(p);
    }
    return g < p.G;
  }
  __device__ __forceinline__ F8Tile tile(const F8Args& p, long long t) const {
    const int r = (int)(t - base);
    const int tok = r / p.n_tiles;
    F8Tile x;
    x.g = g;
    x.t0 = r0 + tok * kF8Tile;
    x.nt = min(kF8Tile, r1 - x.t0);
    x.nmma = (x.nt + 15) & ~15;
    x.n0 = (r - tok * p.n_tiles) * kF8Tile;
    return x;
  }
};

// Tiles of the problem, counted by a whole warp with the walker's clamping.
__device__ __forceinline__ long long f8_total_tiles(const F8Args& p) {
  if (!p.offsets) return (long long)((p.M_total + kF8Tile - 1) / kF8Tile) * p.n_tiles;
  long long cnt = 0;
  for (int g = (int)(threadIdx.x & 31); g < p.G; g += 32) {
    const int a = min(max(__ldg(p.offsets + g), 0), p.M_total);
    const int b = min(max(__ldg(p.offsets + g + 1), a), p.M_total);
    cnt += (b - a + kF8Tile - 1) / kF8Tile;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  return cnt * p.n_tiles;
}

// Non-decreasing from 0; rows behind the last group belong to none.
__device__ __forceinline__ void f8_check_offsets(const int* offsets, int G, int M_total, WsHeader* ws) {
  bool bad = __ldg(offsets) != 0;
  int prev = 0;
  for (int g = 0; g <= G && !bad; ++g) {
    const int v = __ldg(offsets + g);
    bad = v < prev || v > M_total;
    prev = v;
  }
  if (bad) latch_error(ws, kErrBadOffsets, 2);
}

// One unit of work: K blocks [k0, k1) of a tile; split < 0: the whole tile.
struct F8Unit {
  F8Tile tile;
  long long index;
  int split, k0, k1;
};

struct F8Units {
  F8Walker w;
  long long tiles;
  int splits;

  __device__ __forceinline__ void init(const F8Args& p, const int* table, long long total, int s) {
    w.init(p, table);
    tiles = total;
    splits = s;
  }
  __device__ __forceinline__ bool get(const F8Args& p, long long u, F8Unit& x) {
    x.index = splits > 1 ? (int)u / splits : u;  // (few units where they are split)
    if (x.index >= tiles || !w.seek(p, x.index)) return false;
    x.tile = w.tile(p, x.index);
    if (splits > 1) {
      x.split = (int)(u - x.index * splits);
      x.k0 = p.k_blocks * x.split / splits;
      x.k1 = p.k_blocks * (x.split + 1) / splits;
    } else {
      x.split = -1;
      x.k0 = 0;
      x.k1 = p.k_blocks;
    }
    return true;
  }
};

// An epilogue warp keeps its place in the walk in shared memory: its registers
// hold 64 sums per lane, and the walk moves once per tile.
struct F8Place {
  F8Units units;
  F8Unit unit;
  int more;
};
static_assert(sizeof(F8Place) <= kF8WalkBytes, "walk bytes");

// Sixteen fp32 columns of this thread's TMEM lane, valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_load16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor-memory loads; naming the registers keeps
// their uses behind the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// wait_phase without a call.  The epilogue waits with most of its registers
// live, and a call would save them to local memory each time it has to wait;
// and a kernel with calls gets one register budget for all its roles.
template <bool CLUSTER>
__device__ __forceinline__ bool f8_wait(const Guard& g, uint32_t bar, uint32_t parity, uint32_t info) {
  if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (uint32_t it = 1; it < (1u << 28); ++it) {
    if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0u && (*g.abort || globaltimer_ns() - t0 > g.limit_ns)) break;
  }
  if (!*g.abort) {
    *g.abort = 1u;
    latch_error(g.ws, kErrTimeout, info);
  }
  return false;
}

__device__ __forceinline__ float f8_act(int epi, float v) {
  if (epi == 2) {
    float t;
    asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(0.5f * v));
    return v * fmaf(0.5f, t, 0.5f);
  }
  if (epi == 3) return v * normcdff(v);
  return v;
}

// SB_ROWS: B has one scale per feature and K block (else one per 128 features).
template <bool OUT_F32, bool SB_ROWS, bool EPI>
__global__ void __launch_bounds__(kF8Threads, 1)
    k_gemm_fp8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmXt, const __grid_constant__ CUtensorMap tmC, const F8Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smW = smem;
  uint8_t* smX = smW + kF8Stages * kF8WBytes;
  float* smS = reinterpret_cast<float*>(smX + kF8Stages * kF8XBytes);
  uint8_t* smStg = reinterpret_cast<uint8_t*>(smS + kF8ScaleStages * kF8Tile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smStg + kF8EpiWarps * kF8StgBytes);
  // bars: full[S] | empty[S] | acc_full[2] | acc_empty[2] | scale_full[SS] | scale_empty[SS]
  constexpr int kNumBars = 2 * kF8Stages + 4 + 2 * kF8ScaleStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* last_flag = tmem_slot + 2;
  static_assert(kNumBars * 8 + 16 <= 512, "barrier area");
  int* off_tab = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
  const int* tab = p.offsets && p.G < kF8TabMax ? off_tab : nullptr;

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t bar_base = smem_addr(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kF8Stages + s); };
  auto accf_bar = [&](int a) { return bar_base + 8u * (2 * kF8Stages + a); };
  auto acce_bar = [&](int a) { return bar_base + 8u * (2 * kF8Stages + 2 + a); };
  auto scf_bar = [&](int s) { return bar_base + 8u * (2 * kF8Stages + 4 + s); };
  auto sce_bar = [&](int s) { return bar_base + 8u * (2 * kF8Stages + 4 + kF8ScaleStages + s); };
  const uint32_t rank = cluster_ctarank();
  const long long pair_id = blockIdx.x / 2;
  const int num_pairs = (int)(gridDim.x / 2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kF8Stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf_bar(a), 1);
      mbar_init(acce_bar(a), 2 * kF8EpiWarps);
    }
    for (int s = 0; s < kF8ScaleStages; ++s) {
      mbar_init(scf_bar(s), 1);
      mbar_init(sce_bar(s), kF8EpiWarps);
    }
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmXt);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 2) {
    tmem_alloc<2>(smem_addr(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  if (warp == 3 && tab) {
    for (int i = (int)lane; i <= p.G; i += 32) off_tab[i] = __ldg(p.offsets + i);
  }
  const long long total = f8_total_tiles(p);  // every warp counts for itself
  const int splits = f8_splits(total, p.pairs, p.k_blocks, p.max_units);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const Guard guard{p.ws, abort_flag, p.timeout_ns};
  F8Units units;
  F8Unit un;
  if (warp < 4) units.init(p, tab, total, splits);

  // 384 threads of 168 registers: the four role warps give some of theirs to the
  // eight epilogue warps (128 * 72 + 256 * 216 = 64512 = 384 * 168).
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (long long u = pair_id; ok && units.get(p, u, un); u += num_pairs) {
        const F8Tile& tl = un.tile;
        const int w_row = tl.n0 + (int)rank * 128;
        const int x_rows = tl.nmma >> 1;  // token rows this CTA holds
        const int x_row = tl.t0 + (int)rank * x_rows;
        const bool thin = x_rows <= 64;
        const int boxes = thin ? (x_rows + kF8ThinRows - 1) / kF8ThinRows : 1;
        const uint32_t tx = 2u * (uint32_t)(kF8WBytes + (thin ? boxes * kF8ThinRows * kF8BK : kF8XBytes));
        for (int kb = un.k0; kb < un.k1; ++kb) {
          if (!f8_wait<true>(guard, empty_bar(stage), phase ^ 1u, (kRoleProducer << 16) | stage)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), tx);
          const uint32_t fb = map_to_cta(full_bar(stage), 0);
          const int kx = kb * kF8BK;
          tma_load_3d_pair(smem_addr(smW + stage * kF8WBytes), &tmW, fb, kx, w_row, p.w_shared ? 0 : tl.g);
          const uint32_t xdst = smem_addr(smX + stage * kF8XBytes);
          if (thin) {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d_pair(xdst + i * kF8ThinRows * kF8BK, &tmXt, fb, kx, x_row + i * kF8ThinRows);
          } else {
            tma_load_2d_pair(xdst, &tmX, fb, kx, x_row);
          }
          if (++stage == kF8Stages) { stage = 0; phase ^= 1u; }
        }
      }
      for (int i = 0; i < kF8Stages && ok; ++i) {
        ok = f8_wait<true>(guard, empty_bar(stage), phase ^ 1u, (kRoleProducer << 16) | 0x100 | stage);
        if (++stage == kF8Stages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (leader)
    if (lane == 0 && rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (long long u = pair_id; ok && units.get(p, u, un); u += num_pairs) {
        const uint32_t idesc = p.idesc | ((uint32_t)(un.tile.nmma >> 3) << 17);
        for (int kb = un.k0; kb < un.k1; ++kb) {
          ok = f8_wait<true>(guard, acce_bar(acc), acc_phase ^ 1u, (kRoleMma << 16) | 0x100 | acc) &&
               f8_wait<false>(guard, full_bar(stage), phase, (kRoleMma << 16) | stage);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t wBase = smem_addr(smW + stage * kF8WBytes);
          const uint32_t xBase = smem_addr(smX + stage * kF8XBytes);
          const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kF8Tile);
#pragma unroll
          for (int k = 0; k < kF8BK / 32; ++k)
            umma_f8<2>(d_tmem, sdesc_sw128(wBase + k * 32, 16, 1024), sdesc_sw128(xBase + k * 32, 16, 1024), idesc,
                       k != 0 ? 1u : 0u);
          umma_commit_pair(empty_bar(stage), 0x3);
          umma_commit_pair(accf_bar(acc), 0x3);
          if (++stage == kF8Stages) { stage = 0; phase ^= 1u; }
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
    }
  } else if (warp == 2) {
    if (lane == 0 && blockIdx.x == 0 && p.offsets) f8_check_offsets(p.offsets, p.G, p.M_total, p.ws);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ scales
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (long long u = pair_id; ok && units.get(p, u, un); u += num_pairs) {
      const F8Tile& tl = un.tile;
      // 128 x 128 scales: this CTA's features share one per K block.
      const int block = min(tl.n0 + (int)rank * 128, p.N - 1) >> 7;
      const float* sb = p.sb + (long long)tl.g * p.strideSB + (long long)block * p.ldsb;
      const float* sa = p.sa + tl.t0 + lane;
      // The loads run kAhead blocks ahead of the stores.
      constexpr int kAhead = 4;
      float v[kAhead][8], w[kAhead];
      auto load = [&](int kb, float (&x)[8], float& y) {
        const bool in = kb < un.k1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          // columns past the group's rows get 0
          x[i] = in && i * 32 + (int)lane < tl.nt ? __ldg(sa + (long long)kb * p.ldsa + i * 32) : 0.0f;
        y = !SB_ROWS && in ? __ldg(sb + kb) : 1.0f;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(un.k0 + i, v[i], w[i]);
      for (int kb0 = un.k0; ok && kb0 < un.k1; kb0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (kb0 + i < un.k1 && ok) {
            ok = f8_wait<false>(guard, sce_bar(slot), phase ^ 1u, (kRoleProducer << 16) | 0x200 | slot);
            if (ok) {
              float* dst = smS + slot * kF8Tile + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (j * 32 < tl.nmma) dst[j * 32] = v[i][j] * w[i];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(scf_bar(slot));
            if (++slot == kF8ScaleStages) { slot = 0; phase ^= 1u; }
            load(kb0 + i + kAhead, v[i], w[i]);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
  }
  } else {
    // ------------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t stg = smem_addr(smStg + (warp - 4) * kF8StgBytes);
    int acc = 0;
    uint32_t acc_phase = 0;
    int slot = 0;
    uint32_t sc_phase = 0;
    bool ok = true;
    F8Place* place = reinterpret_cast<F8Place*>(reinterpret_cast<uint8_t*>(off_tab + kF8TabMax) + (warp - 4) * kF8WalkBytes);
    if (lane == 0) place->units.init(p, tab, total, splits);
    for (long long u = pair_id; ok; u += num_pairs) {
      __syncwarp();
      if (lane == 0) place->more = place->units.get(p, u, place->unit) ? 1 : 0;
      __syncwarp();
      if (!place->more) break;
      const F8Unit un = place->unit;
      const F8Tile tl = un.tile;
      // This warp's 32 features and its share of the token columns.
      const int n_base = tl.n0 + (int)rank * 128 + q * 32;
      const int n_lane = min(n_base + (int)lane, p.N - 1);
      const int share = ((tl.nmma >> 4) + kF8Parts - 1) / kF8Parts * 16;
      const int c_lo = part * share;
      const int c_n = max(0, min(share, tl.nmma - c_lo));
      const float* sb = p.sb + (long long)tl.g * p.strideSB + n_lane;
      float sb_next = SB_ROWS ? __ldg(sb + un.k0 * p.ldsb) : 1.0f;
      float sum[kF8PartCols];
#pragma unroll
      for (int i = 0; i < kF8PartCols; ++i) sum[i] = 0.0f;
      for (int kb = un.k0; kb < un.k1; ++kb) {
        const float w = sb_next;
        if (SB_ROWS && kb + 1 < un.k1) sb_next = __ldg(sb + (kb + 1) * p.ldsb);
        ok = f8_wait<false>(guard, scf_bar(slot), sc_phase, (kRoleEpilogue << 16) | 0x200 | slot) &&
             f8_wait<false>(guard, accf_bar(acc), acc_phase, (kRoleEpilogue << 16) | acc);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t xs = smem_addr(smS + slot * kF8Tile + c_lo);
        const uint32_t t_lane = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kF8Tile + c_lo);
        auto add = [&](int c, const uint32_t (&r)[16]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float4 s;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(s.x), "=f"(s.y), "=f"(s.z), "=f"(s.w)
                         : "r"(xs + c * 64 + i * 16));
            if constexpr (SB_ROWS) {
              s.x *= w;
              s.y *= w;
              s.z *= w;
              s.w *= w;
            }
            float* a = sum + c * 16 + i * 4;
            a[0] = fmaf(s.x, __uint_as_float(r[4 * i]), a[0]);
            a[1] = fmaf(s.y, __uint_as_float(r[4 * i + 1]), a[1]);
            a[2] = fmaf(s.z, __uint_as_float(r[4 * i + 2]), a[2]);
            a[3] = fmaf(s.w, __uint_as_float(r[4 * i + 3]), a[3]);
          }
        };
        // Sixteen columns are added while the next sixteen load.
        uint32_t r0[16], r1[16];
        if (c_n == kF8PartCols) {
          tmem_load16_async(t_lane, r0);
#pragma unroll
          for (int c = 0; c < kF8PartCols / 16; c += 2) {
            tmem_wait_ld(r0);
            tmem_load16_async(t_lane + c * 16 + 16, r1);
            add(c, r0);
            tmem_wait_ld(r1);
            if (c + 2 < kF8PartCols / 16) tmem_load16_async(t_lane + c * 16 + 32, r0);
            add(c + 1, r1);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kF8PartCols / 16; ++c)
            if (c * 16 < c_n) {
              tmem_load16_async(t_lane + c * 16, r0);
              tmem_wait_ld(r0);
              add(c, r0);
            }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(map_to_cta(acce_bar(acc), 0));
        __syncwarp();
        if (lane == 0) mbar_arrive(sce_bar(slot));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        if (++slot == kF8ScaleStages) { slot = 0; sc_phase ^= 1u; }
      }
      if (un.split >= 0) {
        // Store the sums, [token column][128 features], and count in.  (A pair
        // has one split unit at most; a warp that gave up waiting still takes
        // part in the barriers, and nothing is counted then.)
        float* slots = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.ws) + kWsHeaderBytes);
        const long long first = un.index * splits;
        float* mine = slots + ((first + un.split) * 2 + rank) * kF8SlotFloats + q * 32 + lane;
#pragma unroll
        for (int i = 0; i < kF8PartCols; ++i)
          if (i < c_n) __stcg(mine + (long long)(c_lo + i) * 128, sum[i]);
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kF8EpiWarps) : "memory");
        if (warp == 4 && lane == 0) {
          uint32_t last = 0u;
          if (!*abort_flag) {
            uint32_t* c = p.ws->pad + un.index;
            const uint32_t shift = 16u * rank;
            last = ((atomicAdd(c, 1u << shift) >> shift) & 0xffffu) == (uint32_t)splits - 1u ? 1u : 0u;
            if (last) atomicSub(c, (uint32_t)splits << shift);  // ready for the next call
          }
          *last_flag = last;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kF8EpiWarps) : "memory");
        if (!ok) break;
        if (!*last_flag) continue;
        __threadfence();
        const float* parts = slots + (first * 2 + rank) * kF8SlotFloats + q * 32 + lane;
#pragma unroll
        for (int i = 0; i < kF8PartCols; ++i) sum[i] = 0.0f;
#pragma unroll 1
        for (int s = 0; s < splits; ++s, parts += 2 * kF8SlotFloats) {
          // (sixteen loads in flight)
#pragma unroll
          for (int c = 0; c < kF8PartCols / 16; ++c) {
            if (c * 16 < c_n) {
              float v[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __ldcg(parts + (c_lo + c * 16 + i) * 128);
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c * 16 + i] += v[i];
            }
          }
        }
      }
      if (!ok) break;
      float bias_v = 0.0f;
      if (EPI && n_base + (int)lane < p.N) bias_v = __bfloat162float(p.bias[(long long)tl.g * p.bias_stride + n_lane]);
      constexpr int kTok = OUT_F32 ? 16 : 32;  // tokens per staged block
#pragma unroll
      for (int c = 0; c < kF8PartCols / kTok; ++c) {
        if (c * kTok < c_n) {
          const int width = min(kTok, c_n - c * kTok);
          const int col = c_lo + c * kTok;
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          // Transpose: lane (feature) writes column `lane` of the [token][feature] block.
#pragma unroll
          for (int j = 0; j < kTok; ++j) {
            if (j < width) {
              float v = sum[c * kTok + j];
              if constexpr (EPI) v = f8_act(p.epi, v + bias_v);
              if constexpr (OUT_F32) {
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(stg + j * 128u + lane * 4u), "f"(v) : "memory");
              } else {
                const __nv_bfloat16 h = __float2bfloat16_rn(v);
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(stg + j * 64u + lane * 2u),
                             "h"(*reinterpret_cast<const unsigned short*>(&h)) : "memory");
              }
            }
          }
          if (col + kTok <= tl.nt && width == kTok && n_base + 32 <= p.N) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmC, stg, n_base, tl.t0 + col);
              bulk_commit_group();
            }
            continue;
          }
          __syncwarp();
          // The group's last tokens or the last features: masked stores of row segments.
          constexpr int kSegs = OUT_F32 ? 8 : 4;
          constexpr int kElems = OUT_F32 ? 4 : 8;
          const int seg = (int)lane % kSegs;
          const int ncol = n_base + seg * kElems;
#pragma unroll
          for (int pass = 0; pass < kTok * kSegs / 32; ++pass) {
            const int row = (int)lane / kSegs + pass * (32 / kSegs);
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(stg + row * (OUT_F32 ? 128u : 64u) + seg * 16u));
            if (row < width && col + row < tl.nt && ncol < p.N) {
              const long long off = (long long)(tl.t0 + col + row) * p.ldc + ncol;
              if (ncol + kElems <= p.N) {
                if constexpr (OUT_F32) *reinterpret_cast<uint4*>(static_cast<float*>(p.C) + off) = w;
                else *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.C) + off) = w;
              } else {
                const uint32_t parts[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < kElems; ++e) {
                  if (ncol + e >= p.N) continue;
                  if constexpr (OUT_F32) static_cast<uint32_t*>(p.C)[off + e] = parts[e];
                  else static_cast<unsigned short*>(p.C)[off + e] = (unsigned short)(parts[e >> 1] >> ((e & 1) * 16));
                }
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
  }
  cluster_sync();
  tc_fence_after_sync();
  if (warp == 2) tmem_dealloc<2>(tmem_base, 512);
}

}  // namespace wst
