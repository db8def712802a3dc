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
// warps add it, scaled, to fp32 sums in registers while the tensor core fills the
// other one.
//
// A thread of the epilogue holds 4 features x 32 token columns (the 16x256b form
// of tcgen05.ld): a token scale is loaded from shared memory once for four
// products, two columns are one packed multiply-add, and bf16 results leave
// through transposing matrix stores.  (With one feature and 128 columns a thread,
// the scales alone took 32 16-byte shared loads per warp and K block, 1024 cycles
// of an SM's load path.)
//
// What bounds it: 8192^3 takes 546-563 us (2.0 PFLOP/s) call after call, under the
// power cap, and 388 us (2.8 PFLOP/s) without the scaled sums.  A K block of a
// 256 x 256 tile costs about 1050 cycles: the epilogue's chain of a barrier wait
// (about 200 cycles while products run, even on a phase long complete), four
// rounds of tensor-memory loads and packed multiply-adds, and the hand-back, at
// two warps per sub-core.  Measured and dropped (each against 527-531 us for this
// form, in runs of a few passes): testing the next barriers ahead of their use
// (617 us: a test holds the warp up as long as a wait); the weights' scale
// multiplied in by the epilogue (+50 us); two accumulators of 128 columns per K
// block (749 us), tiles of 128 tokens with four accumulators (820 us), sixteen
// epilogue warps with 96 registers each (840 us, sums spilled).
//
// Roles per CTA (persistent, one CTA per SM, pairs in clusters of 2):
//   warp 0     TMA producer: this CTA's 128 rows of B[g] and its half of the
//              token tile, 128 bytes of K each; both CTAs' copies complete on
//              the leader's full[s].
//   warps 1-2  MMA issuers (leader CTA only), kind::f8f6f4, M = 256: a unit's
//              even and odd K blocks, one accumulator each (either's two waits
//              per block take most of the 512 cycles of its products).  Warp 2
//              also allocates the tensor memory and checks the offsets.
//   warp 3     scales to shared memory, four K blocks at a time, in 4-byte
//              asynchronous copies (a group may start at any row; loads through
//              registers could not run far enough ahead); with 128 x 128 weight
//              scales it multiplies the token scales by the CTA's one.
//   warps 4-11 epilogue: two warps per 32 features, one for each half of the tokens.
//
// Few tiles (short token tiles of a decoding step): when the tiles fill less
// than half of the pairs, each tile's K blocks are split over several pairs;
// every pair stores its fp32 sums to the workspace, and the last one to arrive
// (a counter per tile and CTA, which it sets back to 0) adds them in the order
// of the splits, so the result does not depend on which one is last.
#pragma once

#include <type_traits>

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
constexpr int kF8ScaleBlocks = 4;  // K blocks per slot of scales
constexpr int kF8ScaleStages = 3;
constexpr int kF8ScaleFloats = kF8Tile + 128;  // of one K block: the tokens', the CTA's features'
constexpr int kF8StgBytes = 2048;  // 32 features x 32 tokens (bf16) or 16 tokens (fp32), two per warp
constexpr int kF8StgBufs = 2;
constexpr int kF8TabMax = 256;
constexpr int kF8WalkBytes = 128;  // an epilogue warp's place in the walk over the tiles
constexpr size_t kF8SmemBytes = (size_t)kF8Stages * kF8StageBytes + kF8ScaleStages * kF8ScaleBlocks * kF8ScaleFloats * 4 +
                                kF8EpiWarps * kF8StgBufs * kF8StgBytes + 512 + kF8TabMax * 4 + kF8EpiWarps * kF8WalkBytes + 1024;
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

// Splits of each tile's K loop: no more than keep every unit on a pair of its
// own, and no more than pay.  A K block costs a pair about 0.3 us, adding up one
// split's sums about 0.3 us and 1.1 us more for 256 token columns, so s splits
// of k blocks take about 0.3 (k / s + s (1 + width / 64)) us, least at
// s = sqrt(k / (1 + width / 64)); counting in and out costs 2 us more, so short
// loops stay whole.  Measured whole / as chosen / best of other splits, us:
// 16 x 256 x 8192 25.7 / 14.8 (7) / 14.6 (6), 128 x 1024 x 8192 42.6 / 25.1 (4) /
// 24.3 (5), 256 x 512 x 8192 42.6 / 28.4 (3) / 28.3, 64 x 2048 x 4096 18.5 / 16.1
// (4) / 15.7 (3), 512 x 2048 x 2048 16.3 (whole) / 20.7 (2), 16 x 256 x 1024 8.8
// (whole) / 10.4 (2).
__host__ __device__ inline int f8_splits(long long tiles, int pairs, int k_blocks, int max_units, int M) {
  const int room = pairs < max_units ? pairs : max_units;
  if (tiles <= 0 || tiles > room || k_blocks <= 12) return 1;
  const int most = room / (int)tiles;
  const int width = M < kF8Tile ? M : kF8Tile;
  int s = 1;
  while (s < most && (s + 1) * (s + 1) * (64 + width) <= 64 * k_blocks) ++s;
  return s;
}

struct F8Tile {
  int g, t0, nt, nmma, n0;
};
// The epilogue's two warps per 32 features take the first f8_half0 token columns
// and the rest.
__device__ __forceinline__ int f8_half0(int nmma) { return ((nmma >> 4) + 1) / 2 * 16; }
__device__ __forceinline__ int f8_token(int nmma, int half, int c) { return half ? f8_half0(nmma) + c : c; }
// Where the scale of column c lies among its half's 128: the columns
// 8 j + 2 q + {0, 1} and 8 (j + 1) + 2 q + {0, 1} of a thread are one 16-byte word.
__device__ __forceinline__ int f8_scale_at(int c) { return (c & ~15) | ((c & 6) << 1) | ((c & 8) >> 2) | (c & 1); }

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

// (a0, a1) += (s0, s1) * (v0, v1) in one packed instruction.
__device__ __forceinline__ void f8_fma2(float& a0, float& a1, float s0, float s1, uint32_t v0, uint32_t v1) {
  asm("{\n\t.reg .b64 a, s, v;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "fma.rn.f32x2 a, s, v, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(s0), "f"(s1), "r"(v0), "r"(v1));
}

// 32 fp32 columns of 16 TMEM lanes, valid after tmem_wait_ld: thread t gets, for
// j < 4, r[4j], r[4j+1] = lane t/4, columns 8j + 2(t%4) + {0, 1} and
// r[4j+2], r[4j+3] = lane t/4 + 8, the same columns.
__device__ __forceinline__ void tmem_load_16x32_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tensor-memory loads; naming the registers keeps
// their uses behind the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
}
// Four 8 x 8 matrices of bf16 in the layout of tmem_load_16x32_async (a register
// holds two columns of one row), stored transposed: lane i gives the address of
// 16-byte row i % 8 of matrix i / 8.
__device__ __forceinline__ void st_matrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
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
// THIN: tiles of at most 64 tokens have a loop of their own (see there).
template <bool OUT_F32, bool SB_ROWS, bool EPI, bool THIN>
__global__ void __launch_bounds__(kF8Threads, 1)
    k_gemm_fp8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmXt, const __grid_constant__ CUtensorMap tmC, const F8Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smW = smem;
  uint8_t* smX = smW + kF8Stages * kF8WBytes;
  float* smS = reinterpret_cast<float*>(smX + kF8Stages * kF8XBytes);
  uint8_t* smStg = reinterpret_cast<uint8_t*>(smS + kF8ScaleStages * kF8ScaleBlocks * kF8ScaleFloats);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smStg + kF8EpiWarps * kF8StgBufs * kF8StgBytes);
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
      mbar_init(scf_bar(s), SB_ROWS ? 32 : 1);
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
  const int splits = f8_splits(total, p.pairs, p.k_blocks, p.max_units, p.M_total);
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
    } else if (warp <= 2) {
      // ------------------------------------------------------------------ MMA issuers (leader)
      const int mine = warp - 1;
      if (lane == 0 && rank == 0) {
        int stage = 0;
        uint32_t phase = 0, acc_phase = 0;  // (acc_phase: this issuer's accumulator)
        bool ok = true;
        for (long long u = pair_id; ok && units.get(p, u, un); u += num_pairs) {
          const uint32_t idesc = p.idesc | ((uint32_t)(un.tile.nmma >> 3) << 17);
          for (int kb = un.k0; kb < un.k1; ++kb) {
            if (((kb - un.k0) & 1) == mine) {
              // The accumulator first: its hand-back means that the epilogue has added
              // this issuer's block before, hence every block up to it, so full[stage]
              // has completed the lap before this one.  (With three K blocks a unit an
              // issuer's blocks are three apart, and without that full[stage] could be
              // two laps behind, whose parity reads as complete.)
              ok = f8_wait<false>(guard, acce_bar(mine), acc_phase ^ 1u, (kRoleMma << 16) | 0x100 | mine) &&
                   f8_wait<false>(guard, full_bar(stage), phase, (kRoleMma << 16) | stage);
              if (!ok) break;
              tc_fence_after_sync();
              const uint32_t wBase = smem_addr(smW + stage * kF8WBytes);
              const uint32_t xBase = smem_addr(smX + stage * kF8XBytes);
              const uint32_t d_tmem = tmem_base + (uint32_t)(mine * kF8Tile);
#pragma unroll
              for (int k = 0; k < kF8BK / 32; ++k)
                umma_f8<2>(d_tmem, sdesc_sw128(wBase + k * 32, 16, 1024), sdesc_sw128(xBase + k * 32, 16, 1024), idesc,
                           k != 0 ? 1u : 0u);
              umma_commit_pair(accf_bar(mine), 0x3);
              umma_commit_pair(empty_bar(stage), 0x3);
              acc_phase ^= 1u;
            }
            if (++stage == kF8Stages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (warp == 2 && lane == 1 && blockIdx.x == 0 && p.offsets) f8_check_offsets(p.offsets, p.G, p.M_total, p.ws);
    } else if (warp == 3) {
      // ------------------------------------------------------------------ scales
      auto copy4 = [](uint32_t dst, const float* src, bool in) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
      };
      // 128 x 128 scales: a slot's token scales times the weights' one of each K
      // block.  (Blocks the slot does not hold are multiplied too: nothing reads them.)
      int before = -1;
      auto finish = [&](int filled) {
        __syncwarp();
        float* s = smS + filled * kF8ScaleBlocks * kF8ScaleFloats;
#pragma unroll
        for (int k = 0; k < kF8ScaleBlocks; ++k, s += kF8ScaleFloats) {
          const float w = s[kF8Tile];
          float4* v = reinterpret_cast<float4*>(s) + lane;
#pragma unroll
          for (int i = 0; i < kF8Tile / 128; ++i) {
            float4 x = v[i * 32];
            x.x *= w;
            x.y *= w;
            x.z *= w;
            x.w *= w;
            v[i * 32] = x;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(scf_bar(filled));
      };
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (long long u = pair_id; ok && units.get(p, u, un); u += num_pairs) {
        const F8Tile& tl = un.tile;
        // 128 x 128 scales: this CTA's features share one per K block.
        const int f0 = tl.n0 + (int)rank * 128;
        const float* sb = p.sb + (long long)tl.g * p.strideSB +
                          (SB_ROWS ? 0 : (long long)(min(f0, p.N - 1) >> 7) * p.ldsb);
        const float* sa = p.sa + tl.t0;
        int tok[8];
  #pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (i & 3) * 32 + (int)lane, n0 = f8_half0(tl.nmma);
          tok[i] = c < (i < 4 ? n0 : tl.nmma - n0) ? f8_token(tl.nmma, i >> 2, c) : kF8Tile;
        }
        for (int kb = un.k0; ok && kb < un.k1; kb += kF8ScaleBlocks) {
          ok = f8_wait<false>(guard, sce_bar(slot), phase ^ 1u, (kRoleProducer << 16) | 0x200 | slot);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
  #pragma unroll
          for (int k = 0; k < kF8ScaleBlocks; ++k) {
            if (kb + k >= un.k1) continue;
            const uint32_t dst = smem_addr(smS + (slot * kF8ScaleBlocks + k) * kF8ScaleFloats);
            const float* src = sa + (long long)(kb + k) * p.ldsa;
            // (columns past the group's rows get 0)
  #pragma unroll
            for (int i = 0; i < 8; ++i)
              copy4(dst + 4u * (i * 32 + f8_scale_at((int)lane)), src + (tok[i] < tl.nt ? tok[i] : 0), tok[i] < tl.nt);
            if constexpr (SB_ROWS) {
  #pragma unroll
              for (int i = 0; i < 4; ++i)
                copy4(dst + 4u * (kF8Tile + i * 32 + lane),
                      sb + (long long)(kb + k) * p.ldsb + min(f0 + i * 32 + (int)lane, p.N - 1), true);
            } else {
              if (lane == 0) copy4(dst + 4u * kF8Tile, sb + kb + k, true);
            }
          }
          if constexpr (SB_ROWS) {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(scf_bar(slot)) : "memory");
          } else {
            // The copies of the slot before are waited for and multiplied while
            // these are under way.
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (before >= 0) {
              asm volatile("cp.async.wait_group 1;" ::: "memory");
              finish(before);
            }
            before = slot;
          }
          if (++slot == kF8ScaleStages) { slot = 0; phase ^= 1u; }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!SB_ROWS && before >= 0) finish(before);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t stg0 = smem_addr(smStg + (warp - 4) * kF8StgBufs * kF8StgBytes);
    const int row = (int)lane >> 2, cq = (int)lane & 3;  // this thread's features row + 8 i and columns 8 j + 2 cq + {0, 1}
    uint32_t acc_phase = 0;  // (bit a: accumulator a's parity)
    int slot = 0;
    uint32_t sc_phase = 0;
    int sbuf = 0;
    bool ok = true;
    F8Place* place = reinterpret_cast<F8Place*>(reinterpret_cast<uint8_t*>(off_tab + kF8TabMax) + (warp - 4) * kF8WalkBytes);
    if (lane == 0) place->units.init(p, tab, total, splits);
    for (long long u = pair_id; ok; u += num_pairs) {
      __syncwarp();
      if (lane == 0) place->more = place->units.get(p, u, place->unit) ? 1 : 0;
      __syncwarp();
      if (!place->more) break;
      // (Read again where they are needed: the loop below has no registers left.)
      const volatile F8Unit& un = place->unit;
      const volatile F8Tile& tl = un.tile;
      // This warp's half of the token columns.
      const int c_n = half ? tl.nmma - f8_half0(tl.nmma) : f8_half0(tl.nmma);
      const uint32_t t_warp = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half ? f8_half0(tl.nmma) : 0);
      // This thread's scales in a slot: its columns', and its features'.
      const uint32_t sc_warp = smem_addr(smS) + (half * kF8PartCols + cq * 4) * 4u;
      const uint32_t sc_rows = (uint32_t)(kF8Tile + q * 32 + row - half * kF8PartCols - cq * 4) * 4u;
      const uint32_t acce_leader = map_to_cta(acce_bar(0), 0);
      int left = un.k1 - un.k0, kk = 0;
      // sum[h][j][i]: features row + 16 h + 8 (i / 2), columns 8 j + 2 cq + i % 2
      float sum[2][16][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[h][j][i] = 0.0f;
      // One K block, of accumulator ACC (a constant: its addresses cost no
      // instructions).  All of this warp's 128 columns are loaded and added; in a
      // tile of fewer tokens those behind c_n lie inside the accumulators and are
      // not stored.
      auto step = [&](auto acc_constant) -> bool {
        constexpr int ACC = decltype(acc_constant)::value;
        if (kk == 0) {
          ok = f8_wait<false>(guard, scf_bar(slot), sc_phase, (kRoleEpilogue << 16) | 0x200 | slot);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return false;
        }
        const uint32_t sc = sc_warp + (uint32_t)((slot * kF8ScaleBlocks + kk) * kF8ScaleFloats * 4);
        [[maybe_unused]] float w[4];  // this thread's features' scales
        if constexpr (SB_ROWS) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[i]) : "r"(sc + sc_rows + i * 32u));
        }
        // This thread's scales of 64 columns.
        float s[4][4];
        auto load_scales = [&](int c64) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(s[i][0]), "=f"(s[i][1]), "=f"(s[i][2]), "=f"(s[i][3])
                         : "r"(sc + (c64 * 64 + i * 16) * 4u));
        };
        load_scales(0);
        uint32_t r0[16], r1[16];
        // Step k: columns 32 (k / 2) .., features 16 (k % 2) ..
        auto fetch = [&](int k, uint32_t (&r)[16]) {
          tmem_load_16x32_async(t_warp + (uint32_t)(ACC * kF8Tile) + ((uint32_t)(k & 1) << 20) + (k >> 1) * 32, r);
        };
        ok = f8_wait<false>(guard, accf_bar(ACC), (acc_phase >> ACC) & 1u, (kRoleEpilogue << 16) | ACC);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        acc_phase ^= 1u << ACC;
        tc_fence_after_sync();
        fetch(0, r0);
        fetch(1, r1);
        auto add = [&](int k, const uint32_t (&r)[16]) {
          const int c = k >> 1, h = k & 1;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              float* a = sum[h][c * 4 + j] + i;
              float s0 = s[(c & 1) * 2 + j / 2][2 * (j & 1)], s1 = s[(c & 1) * 2 + j / 2][2 * (j & 1) + 1];
              if constexpr (SB_ROWS) {
                s0 *= w[2 * h + i / 2];
                s1 *= w[2 * h + i / 2];
              }
              f8_fma2(a[0], a[1], s0, s1, r[4 * j + i], r[4 * j + i + 1]);
            }
        };
        // 32 columns x 16 features are added while others load.
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          tmem_wait_ld(r0, r1);
          if (k == 6) {
            // Every load is complete: the accumulator goes back.
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_tmem(acce_leader + 8u * ACC);
          }
          add(k, r0);
          if (k < 6) fetch(k + 2, r0);
          add(k + 1, r1);
          if (k < 6) fetch(k + 3, r1);
          if (k == 2) load_scales(1);
        }
        if (++kk == kF8ScaleBlocks || left == 1) {
          if (lane == 0) mbar_arrive(sce_bar(slot));
          kk = 0;
          if (++slot == kF8ScaleStages) { slot = 0; sc_phase ^= 1u; }
        }
        return true;
      };
      using I0 = std::integral_constant<int, 0>;
      using I1 = std::integral_constant<int, 1>;
      if (!THIN || c_n > 32) {
#pragma unroll 1
        while (step(I0()) && --left > 0 && step(I1()) && --left > 0) {}
      } else {
        // At most 32 columns (tiles of up to 64 tokens, whose products wait for
        // the weights from HBM): one round of loads.  16 x 4096 x 8192 takes 18 us
        // with it and 20 us in the loop above; its mere presence costs large
        // products 2 % (8192^3 559 against 547 us), so they run a kernel without.
#pragma unroll 1
        for (int acc = 0; left > 0; --left, acc ^= 1) {
          if (kk == 0) {
            ok = f8_wait<false>(guard, scf_bar(slot), sc_phase, (kRoleEpilogue << 16) | 0x200 | slot);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          const uint32_t sc = sc_warp + (uint32_t)((slot * kF8ScaleBlocks + kk) * kF8ScaleFloats * 4);
          float w[4], s[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = 1.0f;
            if constexpr (SB_ROWS) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[i]) : "r"(sc + sc_rows + i * 32u));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(s[i][0]), "=f"(s[i][1]), "=f"(s[i][2]), "=f"(s[i][3])
                         : "r"(sc + i * 64u));
          ok = f8_wait<false>(guard, accf_bar(acc), (acc_phase >> acc) & 1u, (kRoleEpilogue << 16) | acc);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          acc_phase ^= 1u << acc;
          tc_fence_after_sync();
          uint32_t r[2][16];
          tmem_load_16x32_async(t_warp + (uint32_t)(acc * kF8Tile), r[0]);
          tmem_load_16x32_async(t_warp + (uint32_t)(acc * kF8Tile) + (16u << 16), r[1]);
          tmem_wait_ld(r[0], r[1]);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_tmem(acce_leader + 8u * acc);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                float s0 = s[j / 2][2 * (j & 1)], s1 = s[j / 2][2 * (j & 1) + 1];
                if constexpr (SB_ROWS) {
                  s0 *= w[2 * h + i / 2];
                  s1 *= w[2 * h + i / 2];
                }
                f8_fma2(sum[h][j][i], sum[h][j][i + 1], s0, s1, r[h][4 * j + i], r[h][4 * j + i + 1]);
              }
          if (++kk == kF8ScaleBlocks || left == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(sce_bar(slot));
            kk = 0;
            if (++slot == kF8ScaleStages) { slot = 0; sc_phase ^= 1u; }
          }
        }
      }

      const int n_base = tl.n0 + (int)rank * 128 + q * 32;
      if (un.split >= 0) {
        // Store the sums, 128 of each of the epilogue's threads, and count in.
        // (A warp that gave up waiting still takes part in the barriers; nothing
        // is counted then, and all warps leave together, or the others would wait
        // for it at the next unit's barrier.)
        float* slots = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.ws) + kWsHeaderBytes) + (threadIdx.x - 128);
        const long long first = un.index * splits;
        float* mine = slots + ((first + un.split) * 2 + rank) * kF8SlotFloats;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j * 8 < c_n) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) __stcg(mine + ((j * 2 + h) * 4 + i) * (32 * kF8EpiWarps), sum[h][j][i]);
          }
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kF8EpiWarps) : "memory");
        if (warp == 4 && lane == 0) {
          uint32_t last = 2u;  // 2: given up
          if (!*abort_flag) {
            uint32_t* c = p.ws->pad + un.index;
            const uint32_t shift = 16u * rank;
            last = ((atomicAdd(c, 1u << shift) >> shift) & 0xffffu) == (uint32_t)splits - 1u ? 1u : 0u;
            if (last) atomicSub(c, (uint32_t)splits << shift);  // ready for the next call
          }
          *last_flag = last;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kF8EpiWarps) : "memory");
        const uint32_t last = *last_flag;
        if (last == 2u) break;
        if (last == 0u) continue;
        __threadfence();
        const float* parts = slots + (first * 2 + rank) * kF8SlotFloats;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[h][j][i] = 0.0f;
#pragma unroll 1
        for (int s = 0; s < splits; ++s, parts += 2 * kF8SlotFloats) {
          // (thirty-two loads in flight)
#pragma unroll
          for (int j0 = 0; j0 < 16; j0 += 4)
            if (j0 * 8 < c_n) {
              float v[4][2][4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if ((j0 + j) * 8 < c_n) {
#pragma unroll
                  for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                      v[j][h][i] = __ldcg(parts + (((j0 + j) * 2 + h) * 4 + i) * (32 * kF8EpiWarps));
                }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if ((j0 + j) * 8 < c_n) {
#pragma unroll
                  for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[h][j0 + j][i] += v[j][h][i];
                }
            }
        }
      }
      if (!ok) break;

      if constexpr (EPI) {
        float bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n_base + row + 8 * i;
          bias[i] = n < p.N ? __bfloat162float(p.bias[(long long)tl.g * p.bias_stride + n]) : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[h][j][i] = f8_act(p.epi, sum[h][j][i] + bias[2 * h + i / 2]);
      }
      constexpr int kTok = OUT_F32 ? 16 : 32;  // tokens per staged block of [token][32 features]
      const bool whole = tl.nt == kF8Tile && n_base + 32 <= p.N;
#pragma unroll
      for (int c = 0; c < kF8PartCols / kTok; ++c) {
        if (c * kTok < c_n) {
          const uint32_t stg = stg0 + sbuf * kF8StgBytes;
          // The stores that read this buffer (all but the newest) are done with it.
          if (lane == 0) bulk_wait_group_read<kF8StgBufs - 1>();
          __syncwarp();
          // 16-byte words of a row are swizzled as the tensor map says, which
          // also keeps these stores free of bank conflicts.
          if constexpr (OUT_F32) {
#pragma unroll
            for (int j = 0; j < kTok / 8; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int tok = j * 8 + 2 * cq + (i & 1), f = row + 16 * h + 8 * (i >> 1);
                  asm volatile("st.shared.f32 [%0], %1;" ::"r"(stg + tok * 128u + (((f >> 2) ^ (tok & 7)) * 16u) + (f & 3) * 4u),
                               "f"(sum[h][c * 2 + j][i])
                               : "memory");
                }
          } else {
            const int tok = (int)lane & 7, m = (int)lane >> 3;  // the row this lane addresses
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float(&s0)[4] = sum[0][c * 4 + j];
              const float(&s1)[4] = sum[1][c * 4 + j];
              st_matrix4_trans(stg + (j * 8 + tok) * 64u + ((m ^ ((tok >> 1) & 3)) * 16u), pack_bf16x2(s0[0], s0[1]),
                               pack_bf16x2(s0[2], s0[3]), pack_bf16x2(s1[0], s1[1]), pack_bf16x2(s1[2], s1[3]));
            }
          }
          if (whole) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmC, stg, n_base, tl.t0 + f8_token(kF8Tile, half, c * kTok));
              bulk_commit_group();
            }
            sbuf = sbuf + 1 == kF8StgBufs ? 0 : sbuf + 1;
            continue;
          }
          __syncwarp();
          // A group's last tokens or the last features: masked stores of row segments.
          constexpr int kSegs = OUT_F32 ? 8 : 4;
          constexpr int kElems = OUT_F32 ? 4 : 8;
          const int seg = (int)lane % kSegs;
          const int ncol = n_base + seg * kElems;
#pragma unroll
          for (int pass = 0; pass < kTok * kSegs / 32; ++pass) {
            const int r = (int)lane / kSegs + pass * (32 / kSegs);  // column of the block
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(OUT_F32 ? stg + r * 128u + ((seg ^ (r & 7)) * 16u)
                                       : stg + r * 64u + ((seg ^ ((r >> 1) & 3)) * 16u)));
            const int tok = f8_token(tl.nmma, half, c * kTok + r);
            if (c * kTok + r < c_n && tok < tl.nt && ncol < p.N) {
              const long long off = (long long)(tl.t0 + tok) * p.ldc + ncol;
              if (ncol + kElems <= p.N) {
                if constexpr (OUT_F32) *reinterpret_cast<uint4*>(static_cast<float*>(p.C) + off) = v;
                else *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.C) + off) = v;
              } else {
                const uint32_t parts[4] = {v.x, v.y, v.z, v.w};
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
