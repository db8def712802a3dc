// wgrad_ws.cuh -- persistent, warp-specialized weight gradient of the grouped
// GEMM (bf16, tcgen05, CTA pairs).
//
//   dB[g][n][k] (+)= sum_{m in group g} dC[m][n] A[m][k]
//
// The contraction runs over the group's tokens, the rows of both operands, so
// both are MN-major: a K step of 16 tokens is 16 rows of 128 bytes (64 features)
// per 64-wide chunk, loaded as they lie in memory.  Tiles of 256 n x 256 k per
// CTA pair; the number of tiles does not depend on the group sizes, and an empty
// group's tiles are stored as zeros.
//
// A group ends inside a block of 64 tokens: the tensor core then takes only the
// 16-token steps that hold rows of the group, and the rows of the last step that
// belong to the next group (or to none) are overwritten with zeros in shared
// memory by warp 3 of both CTAs before that block is multiplied -- in both
// operands, since a NaN or an infinity there would survive a zero on one side.
// Such a block's copies complete on a barrier of each CTA's own, and the tensor
// core waits for both masks instead of the copies.  A group's blocks run
// backwards, so the one with masked rows is a tile's first: its copies land
// several blocks ahead of their use (as a tile's last block it held the tensor
// core up for about 2000 cycles a tile).
//
// What bounds it: per tile 2 (N + K) bytes a token in from L2, 256 x 256 outputs
// to HBM; at about 450 tokens a group the products (512 cycles per 64 tokens) and
// the fp32 output stream take about as long as each other.  On GB300: 64 groups of
// 512 rows, 1536 x 4096 fp32, 367 us (1.12 PFLOP/s and 4.4 TB/s of output),
// ragged ones 418 us; one group of 16384 rows, 4096 x 4096, 410 us (1.34
// PFLOP/s).  The ring's depth counts: four stages and deeper output staging took
// 624 us where six took 505.
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (leader), warp 2 tensor
// memory and offset check, warp 3 row masks, warps 4-11 epilogue (32 output rows
// by 128 columns each; through swizzled shared memory and TMA stores, or TMA adds
// when the gradient accumulates in fp32).
#pragma once

#include "wst_common.cuh"

namespace wst {

constexpr int kWgTile = 256;    // n and k per pair
constexpr int kWgBK = 64;       // tokens per block
constexpr int kWgStages = 6;
constexpr int kWgEpiWarps = 8;
constexpr int kWgStgBufs = 1;     // staging buffers per epilogue warp
constexpr int kWgThreads = 128 + 32 * kWgEpiWarps;
constexpr int kWgChunk = 64 * kWgBK * 2;        // 64 features x 64 tokens
constexpr int kWgOpBytes = 2 * kWgChunk;        // this CTA's 128 features of one operand
constexpr int kWgStageBytes = 2 * kWgOpBytes;
constexpr int kWgStgBytes = 32 * 128;           // 32 output rows of 128 bytes
constexpr int kWgTabMax = 256;                  // offsets kept in shared memory (fewer groups than that)
constexpr size_t kWgSmemBytes =
    (size_t)kWgStages * kWgStageBytes + kWgEpiWarps * kWgStgBufs * kWgStgBytes + 512 + kWgTabMax * 4 + 1024;
static_assert(kWgSmemBytes <= 232448, "shared memory per CTA");

struct WgArgs {
  int G, M_total, N, K;
  int n_tiles, k_tiles;
  const int* offsets;
  int accumulate;
  void* dB;
  long long lddb, stride_dB;
  WsHeader* ws;
  unsigned long long timeout_ns;
};

struct WgTile {
  int g, n0, k0;
  int r0, rows;    // the group's rows
  int blocks;      // of 64 tokens
  int last;        // rows in the last block
};

// Tile t: k fastest, so that consecutive pairs share the dC columns.
__device__ __forceinline__ WgTile wg_tile(const WgArgs& p, const int* offsets, int t) {
  WgTile x;
  const int per = p.n_tiles * p.k_tiles;
  x.g = t / per;
  const int r = t - x.g * per;
  const int ni = r / p.k_tiles;
  x.n0 = ni * kWgTile;
  x.k0 = (r - ni * p.k_tiles) * kWgTile;
  const int a = min(max(offsets[x.g], 0), p.M_total);
  const int b = min(max(offsets[x.g + 1], a), p.M_total);
  x.r0 = a;
  x.rows = b - a;
  x.blocks = (x.rows + kWgBK - 1) / kWgBK;
  x.last = x.rows - (x.blocks - 1) * kWgBK;
  return x;
}

static __device__ __noinline__ void wg_check_offsets(const WgArgs& p) {
  bool bad = __ldg(p.offsets) != 0;
  int prev = 0;
  for (int g = 0; g <= p.G && !bad; ++g) {
    const int v = __ldg(p.offsets + g);
    bad = v < prev || v > p.M_total;
    prev = v;
  }
  if (bad) latch_error(p.ws, kErrBadOffsets, 3);
}

// A ring position that every role advances by the same blocks.
struct WgRing {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kWgStages) { stage = 0; phase ^= 1u; }
  }
};

// ADD_BF16: the gradient is added to a bf16 dB (a form of its own: the registers
// of what dB holds slow the others down, 316 -> 320 us).
template <bool OUT_F32, bool ADD_BF16>
__global__ void __launch_bounds__(kWgThreads, 1)
    k_wgrad_ws(const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmA,
               const __grid_constant__ CUtensorMap tmOut, const WgArgs p, const int tiles) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smD = smem;
  uint8_t* smA = smD + kWgStages * kWgOpBytes;
  uint8_t* smStg = smA + kWgStages * kWgOpBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smStg + kWgEpiWarps * kWgStgBufs * kWgStgBytes);
  // bars: full[S] | empty[S] | acc_full[2] | acc_empty[2] | masked[S] | own[S]
  constexpr int kNumBars = 4 * kWgStages + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  static_assert(kNumBars * 8 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t bar_base = smem_addr(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kWgStages + s); };
  auto accf_bar = [&](int a) { return bar_base + 8u * (2 * kWgStages + a); };
  auto acce_bar = [&](int a) { return bar_base + 8u * (2 * kWgStages + 2 + a); };
  // One pair per stage: several groups may end within the ring at once.
  auto masked_bar = [&](int s) { return bar_base + 8u * (2 * kWgStages + 4 + s); };  // leader: both CTAs' rows are zeroed
  auto own_bar = [&](int s) { return bar_base + 8u * (3 * kWgStages + 4 + s); };     // this CTA's copies of a block to mask
  const uint32_t rank = cluster_ctarank();
  const int pair_id = (int)(blockIdx.x / 2), pairs = (int)(gridDim.x / 2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWgStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf_bar(a), 1);
      mbar_init(acce_bar(a), 2 * kWgEpiWarps);
    }
    for (int s = 0; s < kWgStages; ++s) {
      mbar_init(masked_bar(s), 2);
      mbar_init(own_bar(s), 1);
    }
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmD);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmOut);
  }
  if (warp == 2) {
    tmem_alloc<2>(smem_addr(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  // (a tile's rows are looked up by every role; a load from global memory there
  // holds up the start of each tile)
  int* tab = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
  const int* offsets = p.G < kWgTabMax ? tab : p.offsets;
  if (warp == 3 && p.G < kWgTabMax)
    for (int i = (int)lane; i <= p.G; i += 32) tab[i] = __ldg(p.offsets + i);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const Guard guard{p.ws, abort_flag, p.timeout_ns};

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      WgRing ring;
      bool ok = true;
      for (int t = pair_id; ok && t < tiles; t += pairs) {
        const WgTile tl = wg_tile(p, offsets, t);
        const int nx = tl.n0 + (int)rank * 128, kx = tl.k0 + (int)rank * 128;
        for (int b = 0; b < tl.blocks; ++b) {
          ok = wait_phase_cluster(guard, empty_bar(ring.stage), ring.phase ^ 1u, (kRoleProducer << 16) | ring.stage);
          if (!ok) break;
          const uint32_t d = smem_addr(smD + ring.stage * kWgOpBytes), a = smem_addr(smA + ring.stage * kWgOpBytes);
          const int y = tl.r0 + (tl.blocks - 1 - b) * kWgBK;
          if (b == 0 && (tl.last & 15)) {
            if (rank == 0) mbar_arrive(full_bar(ring.stage));  // (completes the phase; the masks stand for the copies)
            const uint32_t own = own_bar(ring.stage);
            mbar_arrive_expect_tx(own, kWgStageBytes);
            for (int c = 0; c < 2; ++c) {
              tma_load_2d(d + c * kWgChunk, &tmD, own, nx + c * 64, y);
              tma_load_2d(a + c * kWgChunk, &tmA, own, kx + c * 64, y);
            }
          } else {
            if (rank == 0) mbar_arrive_expect_tx(full_bar(ring.stage), 2u * kWgStageBytes);
            const uint32_t fb = map_to_cta(full_bar(ring.stage), 0);
            for (int c = 0; c < 2; ++c) {
              tma_load_2d_pair(d + c * kWgChunk, &tmD, fb, nx + c * 64, y);
              tma_load_2d_pair(a + c * kWgChunk, &tmA, fb, kx + c * 64, y);
            }
          }
          ring.next();
        }
      }
      for (int i = 0; i < kWgStages && ok; ++i) {
        ok = wait_phase_cluster(guard, empty_bar(ring.stage), ring.phase ^ 1u, (kRoleProducer << 16) | 0x100 | ring.stage);
        ring.next();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (leader)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, true, true);
      WgRing ring;
      int acc = 0;
      uint32_t acc_phase = 0, masked_phase = 0;  // (bit s: the parity of stage s)
      bool ok = true, full_ok = false;
      for (int t = pair_id; ok && t < tiles; t += pairs) {
        const WgTile tl = wg_tile(p, offsets, t);
        if (tl.blocks == 0) continue;
        ok = wait_phase_cluster(guard, acce_bar(acc), acc_phase ^ 1u, (kRoleMma << 16) | 0x100 | acc);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kWgTile);
        for (int b = 0; b < tl.blocks; ++b) {
          ok = full_ok || wait_phase(guard, full_bar(ring.stage), ring.phase, (kRoleMma << 16) | ring.stage);
          int steps = kWgBK / 16;
          if (ok && b == 0) {
            steps = (tl.last + 15) / 16;
            if (tl.last & 15) {
              ok = wait_phase_cluster(guard, masked_bar(ring.stage), (masked_phase >> ring.stage) & 1u, (kRoleMma << 16) | 0x200);
              masked_phase ^= 1u << ring.stage;
            }
          }
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t d = smem_addr(smD + ring.stage * kWgOpBytes), a = smem_addr(smA + ring.stage * kWgOpBytes);
          const uint32_t this_empty = empty_bar(ring.stage);
          ring.next();
          // (a barrier test takes long while products run: ahead of its use)
          full_ok = mbar_test_wait(full_bar(ring.stage), ring.phase);
          for (int k = 0; k < steps; ++k)
            umma_bf16<2>(d_tmem, sdesc_sw128(d + k * 2048, kWgChunk, 1024), sdesc_sw128(a + k * 2048, kWgChunk, 1024),
                         idesc, (b | k) != 0 ? 1u : 0u);
          umma_commit_pair(this_empty, 0x3);
        }
        if (!ok) break;
        umma_commit_pair(accf_bar(acc), 0x3);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
    }
  } else if (warp == 2) {
    if (lane == 0 && blockIdx.x == 0) wg_check_offsets(p);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ row masks
    WgRing ring;
    uint32_t own_phase = 0;  // (bit s: the parity of stage s)
    bool ok = true;
    for (int t = pair_id; ok && t < tiles; t += pairs) {
      const WgTile tl = wg_tile(p, offsets, t);
      if (tl.blocks > 0 && (tl.last & 15)) {
        ok = warp_wait_phase(guard, own_bar(ring.stage), (own_phase >> ring.stage) & 1u, (kRoleFlag << 16) | ring.stage);
        if (!ok) break;
        own_phase ^= 1u << ring.stage;
        // Rows last .. of the step, 128 bytes each, in the four chunks: eight
        // lanes per row (whole rows, so the swizzle does not matter).
        const int rows = 16 - (tl.last & 15);
        for (int i = (int)lane; i < rows * 4 * 8; i += 32) {
          const int unit = i & 7, chunk = (i >> 3) & 3, row = tl.last + (i >> 5);
          uint8_t* base = (chunk < 2 ? smD : smA) + ring.stage * kWgOpBytes + (chunk & 1) * kWgChunk;
          st_shared_v4(smem_addr(base) + row * 128u + unit * 16u, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_cta(masked_bar(ring.stage), 0));
      }
      for (int b = 0; b < tl.blocks; ++b) ring.next();
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;  // 32 rows, 128 columns of them
    const uint32_t stg0 = smem_addr(smStg + (warp - 4) * kWgStgBufs * kWgStgBytes);
    int sbuf = 0, acc = 0;
    uint32_t acc_phase = 0;
    for (int t = pair_id; t < tiles; t += pairs) {
      const WgTile tl = wg_tile(p, offsets, t);
      const bool empty = tl.blocks == 0;
      if (empty && p.accumulate) continue;
      constexpr int kCols = OUT_F32 ? 32 : 64;  // columns per 128-byte row
      const int n = tl.n0 + (int)rank * 128 + q * 32;  // first of this warp's rows
      // ADD_BF16: what dB holds is added to the fp32 sum and rounded once (a TMA add
      // would round the sum first and the result again).  It is fetched to L2 a
      // tile ahead, read ahead of the wait, eight lanes to a row of 128 bytes, and
      // goes through the staging buffer to the lanes that hold the rows.  64 groups
      // of 512 rows, 1536 x 4096: 369 us (without accumulation 316; with one
      // row a lane, read behind the wait, 521).
      [[maybe_unused]] uint4 held[8];
      [[maybe_unused]] auto read_old = [&](int c) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int row = n + u * 4 + (int)(lane >> 3), col = tl.k0 + c + (int)(lane & 7) * 8;
          const int cols = row < p.N ? p.K - col : 0;  // (rows begin on 16 bytes; this tile is no other CTA's)
          const unsigned short* src =
              static_cast<const unsigned short*>(p.dB) + tl.g * p.stride_dB + (long long)row * p.lddb + col;
          held[u] = make_uint4(0u, 0u, 0u, 0u);
          if (cols >= 8) {
            held[u] = *reinterpret_cast<const uint4*>(src);
          } else if (cols > 0) {
            uint32_t part[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < cols) part[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
            held[u] = make_uint4(part[0], part[1], part[2], part[3]);
          }
        }
      };
      if constexpr (ADD_BF16) {
        read_old(half * (kWgTile / 2));
        if (lane == 0 && t + pairs < tiles) {
          const WgTile next = wg_tile(p, offsets, t + pairs);
          const int row = next.n0 + (int)rank * 128 + q * 32, col = next.k0 + half * (kWgTile / 2);
          for (int c = 0; c < kWgTile / 2; c += kCols)
            if (row < p.N && col + c < p.K) tma_prefetch_3d(&tmOut, col + c, row, next.g);
        }
      }
      if (!empty) {
        if (!warp_wait_phase_cluster(guard, accf_bar(acc), acc_phase, (kRoleEpilogue << 16) | acc)) break;
        tc_fence_after_sync();
      }
      const uint32_t t_lane = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kWgTile);
#pragma unroll 1
      for (int c = half * (kWgTile / 2); c < (half + 1) * (kWgTile / 2); c += kCols) {
        if (n >= p.N || tl.k0 + c >= p.K) break;  // (warp-uniform; nothing of it is stored)
        uint32_t w[32];
        if constexpr (OUT_F32) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.0f;
          if (!empty) tmem_load32(t_lane + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j]);
        } else {
          [[maybe_unused]] uint4 old[8];  // what dB holds of this lane's row
          if constexpr (ADD_BF16) {
            const uint32_t stg = stg0 + sbuf * kWgStgBytes;
            if (lane == 0) bulk_wait_group_read<kWgStgBufs - 1>();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const uint32_t r = u * 4 + (lane >> 3);
              st_shared_v4(stg + r * 128u + (((lane ^ r) & 7) * 16u), held[u].x, held[u].y, held[u].z, held[u].w);
            }
            if (c + kCols < (half + 1) * (kWgTile / 2)) read_old(c + kCols);
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(old[u].x), "=r"(old[u].y), "=r"(old[u].z), "=r"(old[u].w)
                           : "r"(stg + lane * 128u + ((u ^ (lane & 7)) * 16u)));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            if (!empty) tmem_load32(t_lane + c + h * 32, v);
            if constexpr (ADD_BF16) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const uint4& word = old[h * 4 + (j >> 3)];
                const uint32_t two = (j & 6) == 0 ? word.x : (j & 6) == 2 ? word.y : (j & 6) == 4 ? word.z : word.w;
                v[j] += __uint_as_float(two << 16);
                v[j + 1] += __uint_as_float(two & 0xffff0000u);
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) w[h * 16 + j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
          }
        }
        if ((p.K & (16 / (OUT_F32 ? 4 : 2) - 1)) != 0 && tl.k0 + c + kCols > p.K) {
          // A TMA store writes whole 16-byte words: the last columns of a K that
          // ends inside one go by single elements.
          if (n + (int)lane < p.N) {
            const long long at = tl.g * p.stride_dB + (long long)(n + (int)lane) * p.lddb + tl.k0 + c;
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
              if (tl.k0 + c + j < p.K) {
                if constexpr (OUT_F32) {
                  float* o = static_cast<float*>(p.dB) + at + j;
                  *o = p.accumulate ? *o + __uint_as_float(w[j]) : __uint_as_float(w[j]);
                } else {
                  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.dB) + at + j;
                  *o = __float2bfloat16_rn(__uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16)));
                }
              }
            }
          }
          continue;
        }
        const uint32_t stg = stg0 + sbuf * kWgStgBytes;
        // the store that read this buffer (not the newest ones) is done with it
        if (lane == 0) bulk_wait_group_read<kWgStgBufs - 1>();
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          st_shared_v4(stg + lane * 128u + ((u ^ (lane & 7)) * 16u), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          // (columns and rows past K and N are not stored)
          if (OUT_F32 && p.accumulate) tma_add_3d(&tmOut, stg, tl.k0 + c, n, tl.g);
          else tma_store_3d(&tmOut, stg, tl.k0 + c, n, tl.g);
          bulk_commit_group();
        }
        sbuf = sbuf + 1 == kWgStgBufs ? 0 : sbuf + 1;
      }
      if (!empty) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(map_to_cta(acce_bar(acc), 0));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
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
