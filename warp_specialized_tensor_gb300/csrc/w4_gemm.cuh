// w4_gemm.cuh -- products of few bf16 rows with 4-bit weights and group scales,
// dense and grouped, for sm_103a.
//
//   C[m][n] = epi( sum_b s[b][n] sum_{k in b} A[m][k] (w[n][k] - 8) (+ bias[n]) )
//
// A decoding step's product reads its weights once for a few rows, so the weights'
// bytes bound it, and what has to be cheap is turning a byte of them into operands:
// about 90 instructions for the 1 KB that a warp takes at a time, against the 170
// clocks that HBM needs for four such (one for each scheduler).  So:
//  - A unit is 128 features x 128 k.  A TMA producer warp keeps a ring of units in
//    flight (weights as they lie in memory, the rows' 128 k, the scales).
//  - Sixteen warps in two sets (eight for 64 tokens) take the units in turn; a warp multiplies 16
//    features with mma.sync (features as the instruction's 16 rows, 8 tokens per
//    column tile).  tcgen05 wants 128 x 64-byte operand tiles in shared memory or
//    tensor memory: the unpacked weights would have to be stored there and read
//    again, four times the bytes of the packed ones, while a register fragment is
//    used where it was made.
//  - The sum over k may be taken in any order, so a fragment's k are the eight of one
//    32-bit word of weights: (w >> 4i) & 0x000f000f are the numbers k = i and k = i + 4
//    of it.  With 0x4300 over each they are the bf16 128 + w; minus 136, exact.  The
//    rows' eight values are paired the same way by byte permutes.
//  - Accumulators of one group are scaled and added in fp32 when the group ends.
//  - The tiles' units stand in one line and each CTA takes an equal share of it
//    (work_split.cuh).  A tile that is cut is added up by the CTA that finishes it
//    last, from fp32 partial sums in the workspace, in ascending order of k: the
//    result does not depend on which CTA that is.
#pragma once

#include "work_split.cuh"
#include "wst_common.cuh"

namespace wst {

constexpr int kW4Feats = 128;     // features of a tile: 8 warps x 16
constexpr int kW4K = 128;         // k of a unit
constexpr int kW4WBytes = kW4Feats * kW4K / 2;
constexpr int kW4SBytes = 1024;   // scales: 128 features x up to 4 groups, bf16
constexpr int kW4MaxCtas = 160;
constexpr int kW4Pitch = kW4Feats + 4;  // floats of a token's row of the output tile

template <int NT>
struct W4Cfg {
  // Sets of 8 warps that take the units in turn.  (64 tokens' accumulators leave
  // no room for the registers of a second set.)
  static constexpr int kSets = NT == 8 ? 1 : 2;
  static constexpr int kWarps = 8 * kSets;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kTokens = 8 * NT;
  static constexpr int kABytes = kTokens * kW4K * 2;  // four boxes of 32 k
  static constexpr int kStage = kW4WBytes + kABytes + kW4SBytes;
  static constexpr int kOut = kTokens * kW4Pitch * 4;
  static constexpr int kStages = (232448 - 1024 - 1024 - kOut) / kStage > 16 ? 16 : (232448 - 1024 - 1024 - kOut) / kStage;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kOut + 1024;
  static_assert(kStage % 1024 == 0 && kStages >= 4 && kSmem <= 232448, "shared memory");
};

// Workspace after the header: tickets[kW4MaxCtas] (8 bytes each), then two slots of
// partial sums per CTA: [64 tokens][128 features] fp32 each.
constexpr size_t kW4TicketOffset = kWsHeaderBytes;
constexpr size_t kW4SlotOffset = 256 * ((kW4TicketOffset + kW4MaxCtas * 8 + 255) / 256);
constexpr size_t kW4SlotFloats = 64 * kW4Feats;
constexpr size_t kW4WorkspaceBytes = kW4SlotOffset + 2 * (size_t)kW4MaxCtas * kW4SlotFloats * 4;

struct W4Args {
  int G, M, N, K;
  int k_units;        // ceil(K / 128)
  int n_tiles;        // ceil(N / 128)
  int steps;          // 32-k blocks per group: 1, 2 or 4
  int scale_bytes;    // of a unit: 256 * groups of it
  const int* offsets; // NULL: one group of M rows
  const __nv_bfloat16* bias;
  long long stride_bias;
  void* C;
  long long ldc;
  int c_f32;
  int epi;
  int split;          // the workspace holds tickets and slots
  uint32_t epoch;     // this call's value in the tickets
  WsHeader* ws;
  unsigned long long* tickets;
  float* slots;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ void w4_rows(const W4Args& p, int g, int& a, int& b) {
  if (!p.offsets) {
    a = 0;
    b = p.M;
    return;
  }
  a = min(max(__ldg(p.offsets + g), 0), p.M);
  b = min(max(__ldg(p.offsets + g + 1), a), p.M);
}

static __device__ __noinline__ void w4_check_offsets(const W4Args& p) {
  bool bad = __ldg(p.offsets) != 0;
  int prev = 0;
  for (int g = 0; g <= p.G && !bad; ++g) {
    const int v = __ldg(p.offsets + g);
    if (v < prev || v > p.M) bad = true;
    prev = v;
  }
  if (bad) latch_error(p.ws, kErrBadOffsets, 3);
}

// A CTA's share, one fragment (consecutive units of one tile) after another.
template <int NT>
struct W4Walker {
  long long x, hi;        // next unit, end of the share
  int g;
  long long base, count;  // group g's first unit and how many it has
  int a, b;               // its rows
  // the fragment
  long long item;         // its tile's first unit
  int tile, row0, rows, ua, ub;

  __device__ __forceinline__ static long long units(const W4Args& p, int a, int b) {
    return (long long)((b - a + 8 * NT - 1) / (8 * NT)) * p.n_tiles * p.k_units;
  }
  __device__ __forceinline__ void init(const W4Args& p, long long lo, long long hi_, int g_, long long base_) {
    x = lo;
    hi = hi_;
    g = g_;
    base = base_;
    count = 0;
    if (x < hi) {
      w4_rows(p, g, a, b);
      count = units(p, a, b);
    }
  }
  __device__ __forceinline__ bool next(const W4Args& p) {
    if (x >= hi) return false;
    while (x >= base + count) {
      base += count;
      ++g;  // (x < W: a group holds it)
      w4_rows(p, g, a, b);
      count = units(p, a, b);
    }
    // tiles of features, and inside one the row chunks: those read the same weights
    const int chunks = (b - a + 8 * NT - 1) / (8 * NT);
    const long long r = x - base;
    const long long t = r / p.k_units;
    ua = (int)(r - t * p.k_units);
    ub = (int)min((long long)p.k_units, ua + (hi - x));
    item = x - ua;
    tile = (int)(t / chunks);
    row0 = a + (int)(t - (long long)tile * chunks) * (8 * NT);
    rows = min(8 * NT, b - row0);
    x += ub - ua;
    return true;
  }
};

// Two 4-bit numbers (bits 4i.. and 16 + 4i.. of w) minus 8, as bf16.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {
  uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;  // 128 + w
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x43084308u));  // 136
  return v;
}
__device__ __forceinline__ void w4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t w4_lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 w4_lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float w4_lds_bf16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return __uint_as_float((uint32_t)v << 16);
}
// A barrier of the multiplying warps.
template <int THREADS>
__device__ __forceinline__ void w4_sync() {
  asm volatile("barrier.sync 1, %0;" ::"n"(THREADS) : "memory");
}

__device__ __forceinline__ float w4_activate(float v, int epi) {
  if (epi == 2) return v / (1.0f + expf(-v));
  if (epi == 3) return v * normcdff(v);
  return v;
}

// Writes features f, f + 1 of token `tok` of a finished tile.
__device__ __forceinline__ void w4_store(const W4Args& p, int g, int tile, int row, int f, float v0, float v1) {
  const int n = tile * kW4Feats + f;
  if (n >= p.N) return;
  const bool two = n + 1 < p.N;
  if (p.epi) {
    const __nv_bfloat16* bias = p.bias + g * p.stride_bias + n;
    v0 = w4_activate(v0 + __bfloat162float(bias[0]), p.epi);
    if (two) v1 = w4_activate(v1 + __bfloat162float(bias[1]), p.epi);
  }
  const long long at = (long long)row * p.ldc + n;
  if (p.c_f32) {
    float* c = static_cast<float*>(p.C) + at;
    if (two) *reinterpret_cast<float2*>(c) = make_float2(v0, v1);
    else *c = v0;
  } else {
    __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + at;
    if (two) *reinterpret_cast<uint32_t*>(c) = pack_bf16x2(v0, v1);
    else *c = __float2bfloat16_rn(v0);
  }
}

// Counts one finished piece of a cut tile; true for the last of `pieces`.  A ticket
// holds this call's value and the count: whatever an earlier operation left there
// counts as zero, and the last piece leaves zero.
__device__ __forceinline__ bool w4_last_piece(unsigned long long* ticket, uint32_t epoch, int pieces) {
  unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(ticket);
  while (true) {
    const uint32_t n = (uint32_t)(old >> 32) == epoch ? (uint32_t)old : 0u;
    const unsigned long long want = (int)n + 1 == pieces ? 0ull : ((unsigned long long)epoch << 32) | (n + 1u);
    const unsigned long long got = atomicCAS(ticket, old, want);
    if (got == old) return want == 0ull;
    old = got;  // another piece was counted: at most `pieces` times
  }
}

// tmW {ceil(K/2) bytes, N, G}, boxes of 64 bytes x 128 features, 64-byte swizzle;
// tmA {K, M}, boxes of 32 k x 8 NT rows, 64-byte swizzle; tmS {N, ceil(K/group), G},
// boxes of 128 features x the groups of a unit.
template <int NT>
__global__ void __launch_bounds__(W4Cfg<NT>::kThreads, 1)
    k_w4_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
              const __grid_constant__ CUtensorMap tmS, const W4Args p) {
  using Cfg = W4Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* tile_out = reinterpret_cast<float*>(smem + Cfg::kStages * Cfg::kStage);  // [token][kW4Pitch]
  __shared__ uint64_t bars[2 * 16];
  __shared__ long long scratch[33], found[2];
  __shared__ uint32_t abort_word, is_last;
  volatile uint32_t* abort_flag = &abort_word;
  const int warp = (int)threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (16 + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 8);
    }
    *abort_flag = 0u;
    found[0] = found[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmS);
  }
  // this CTA's share (block_total and block_locate end with barriers)
  auto count = [&](int g) -> long long {
    int a, b;
    w4_rows(p, g, a, b);
    return W4Walker<NT>::units(p, a, b);
  };
  const long long W = block_total<Cfg::kThreads>(p.G, count, scratch);
  // whole tiles where the workspace holds no partial sums
  const long long grain = p.split ? 1 : p.k_units;
  const Share share{W / grain, (int)max(1ll, min((long long)gridDim.x, W / (2 * grain)))};
  long long lo = 0, hi = 0;
  if ((int)blockIdx.x < share.G) {
    lo = share.lo((int)blockIdx.x) * grain;
    hi = share.lo((int)blockIdx.x + 1) * grain;
  }
  if (lo < hi) block_locate<Cfg::kThreads>(p.G, count, lo, scratch, found);
  __syncthreads();
  const Guard guard{p.ws, abort_flag, p.timeout_ns};
  W4Walker<NT> w;
  w.init(p, lo, hi, (int)found[0], found[1]);

  if (warp == Cfg::kWarps) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      const uint32_t bytes = (uint32_t)(kW4WBytes + Cfg::kABytes + p.scale_bytes);
      const int groups = p.scale_bytes / 256;
      while (ok && w.next(p)) {
        for (int u = w.ua; u < w.ub; ++u) {
          if (!wait_phase(guard, empty_bar(s), ph, (kRoleProducer << 16) | s)) {
            ok = false;
            break;
          }
          const uint32_t at = smem_addr(smem + s * Cfg::kStage);
          mbar_arrive_expect_tx(full_bar(s), bytes);
          tma_load_3d(at, &tmW, full_bar(s), u * (kW4K / 2), w.tile * kW4Feats, w.g);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            tma_load_2d(at + kW4WBytes + q * (Cfg::kABytes / 4), &tmA, full_bar(s), u * kW4K + 32 * q, w.row0);
          tma_load_3d(at + kW4WBytes + Cfg::kABytes, &tmS, full_bar(s), w.tile * kW4Feats, u * groups, w.g);
          if (++s == Cfg::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (lane == 1 && blockIdx.x == 0 && p.offsets) {
      w4_check_offsets(p);
    }
  } else {
    // ------------------------------------------------------------------ multiplying warps
    const int set = warp >> 3;
    const int f0 = (warp & 7) * 16;               // the warp's features of a tile
    const int fr = f0 + (int)(lane >> 2), t = (int)(lane & 3);
    const uint32_t swz = (uint32_t)((lane >> 3) & 3);  // (row >> 1) & 3 of every row that the lane reads
    const uint32_t w_at = (uint32_t)(fr * 64 + t * 4);
    const uint32_t a_at = (uint32_t)(kW4WBytes + (lane >> 2) * 64 + (((uint32_t)t ^ swz) << 4));
    const uint32_t s_at = (uint32_t)(kW4WBytes + Cfg::kABytes + fr * 2);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (w.next(p)) {
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
      for (int u = w.ua; u < w.ub; ++u) {
        // (a wait that gave up: the barriers and tickets below still count this CTA)
        if (turn == set && ok) ok = warp_wait_phase(guard, full_bar(s), ph, (kRoleMma << 16) | s);
        if (turn == set && ok) {
          const uint32_t at = smem_addr(smem + s * Cfg::kStage);
          float part[NT][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t wq = at + w_at + (((uint32_t)q ^ swz) << 4);
            const uint32_t w0 = w4_lds32(wq), w1 = w4_lds32(wq + 8 * 64);
            const uint32_t a0 = w4_pair(w0, 0), a1 = w4_pair(w1, 0), a2 = w4_pair(w0, 1), a3 = w4_pair(w1, 1);
            const uint32_t a4 = w4_pair(w0, 2), a5 = w4_pair(w1, 2), a6 = w4_pair(w0, 3), a7 = w4_pair(w1, 3);
            const bool first = p.steps == 1 || (p.steps == 2 ? (q & 1) == 0 : q == 0);
            if (first) {
#pragma unroll
              for (int i = 0; i < NT; ++i) part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const uint4 x = w4_lds128(at + a_at + (uint32_t)(q * (Cfg::kABytes / 4) + i * 512));
              w4_mma(part[i], a0, a1, a2, a3, __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
              w4_mma(part[i], a4, a5, a6, a7, __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            }
            const bool last = p.steps == 1 || (p.steps == 2 ? (q & 1) == 1 : q == 3);
            if (last) {
              const uint32_t sq = at + s_at + (uint32_t)((p.steps == 1 ? q : p.steps == 2 ? q >> 1 : 0) * 256);
              const float s0 = w4_lds_bf16(sq), s1 = w4_lds_bf16(sq + 16);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                acc[i][0] = fmaf(s0, part[i][0], acc[i][0]);
                acc[i][1] = fmaf(s0, part[i][1], acc[i][1]);
                acc[i][2] = fmaf(s1, part[i][2], acc[i][2]);
                acc[i][3] = fmaf(s1, part[i][3], acc[i][3]);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty_bar(s));
        }
        if (++turn == Cfg::kSets) turn = 0;
        if (++s == Cfg::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // The sets' sums: the last one's into shared memory, set 0 adds its own.
      float* mine = tile_out + (2 * t) * kW4Pitch + fr;
      w4_sync<32 * Cfg::kWarps>();  // the tile before this one has been read
      if (set == Cfg::kSets - 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float* o = mine + i * 8 * kW4Pitch;
          o[0] = acc[i][0];
          o[kW4Pitch] = acc[i][1];
          o[8] = acc[i][2];
          o[kW4Pitch + 8] = acc[i][3];
        }
      }
      if constexpr (Cfg::kSets == 2) {
        w4_sync<32 * Cfg::kWarps>();
        if (set == 0) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float* o = mine + i * 8 * kW4Pitch;
            o[0] += acc[i][0];
            o[kW4Pitch] += acc[i][1];
            o[8] += acc[i][2];
            o[kW4Pitch + 8] += acc[i][3];
          }
        }
      }
      w4_sync<32 * Cfg::kWarps>();
      const int f = 2 * (int)(threadIdx.x & 63), tok0 = (int)threadIdx.x >> 6;  // two features, every eighth token
      if (w.ub - w.ua == p.k_units) {
        for (int tok = tok0; tok < w.rows; tok += Cfg::kWarps / 2) {
          const float2 v = *reinterpret_cast<const float2*>(tile_out + tok * kW4Pitch + f);
          w4_store(p, w.g, w.tile, w.row0 + tok, f, v.x, v.y);
        }
      } else {
        // A piece of a cut tile: into this CTA's slot (the second one if the tile
        // begins in its share), then the last of the tile's CTAs adds them up.
        const int c0 = share.owner(w.item), c1 = share.owner(w.item + p.k_units - 1);
        float* slot = p.slots + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == c0 ? 1 : 0)) * kW4SlotFloats;
        for (int tok = tok0; tok < w.rows; tok += Cfg::kWarps / 2)
          __stcg(reinterpret_cast<float2*>(slot + tok * kW4Feats + f), *reinterpret_cast<const float2*>(tile_out + tok * kW4Pitch + f));
        w4_sync<32 * Cfg::kWarps>();
        if (threadIdx.x == 0) {
          __threadfence();  // (after the barrier: all the warps' stores)
          is_last = w4_last_piece(p.tickets + c0, p.epoch, c1 - c0 + 1) ? 1u : 0u;
          __threadfence();
        }
        w4_sync<32 * Cfg::kWarps>();
        if (is_last) {
          for (int tok = tok0; tok < w.rows; tok += Cfg::kWarps / 2) {
            float v0 = 0.0f, v1 = 0.0f;
            for (int c = c0; c <= c1; ++c) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(
                  p.slots + (size_t)(2 * c + (c == c0 ? 1 : 0)) * kW4SlotFloats + tok * kW4Feats + f));
              v0 += v.x;
              v1 += v.y;
            }
            w4_store(p, w.g, w.tile, w.row0 + tok, f, v0, v1);
          }
        }
      }
    }
  }
  __syncthreads();
  if (*abort_flag) {
    for (int i = 0; i < 200; ++i) __nanosleep(1000);  // copies still in flight land first
  }
}

}  // namespace wst
