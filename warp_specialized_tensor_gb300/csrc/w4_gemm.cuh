// w4_gemm.cuh -- products of few bf16 rows with 4-bit weights and group scales,
// dense and grouped, for sm_103a.
//
//   C[m][n] = epi( sum_b s[b][n] sum_{k in b} A[m][k] (w[n][k] - 8) (+ bias[n]) )
//
// A decoding step's product reads its weights once for a few rows, so the weights'
// bytes bound it: an SM's share of HBM brings a unit (128 features x 256 k, 16 KB) in 690
// clocks, and in that time its 32,768 numbers have to be unpacked and multiplied.
//  - The sum over k may be taken in any order, so a fragment's pairs are the numbers i
//    and i + 4 of a 32-bit word's eight, which a mask and one bf16 multiply-add unpack
//    (w4_pair): 9 instructions a word, five of them on the integer pipe, which takes one
//    every two clocks and bounds the rest (11 with shifts and 128 + w: 7 there).
//  - mma.sync takes them from the registers where they were unpacked: a warp has 32
//    features (two tiles of 16) and all the rows, 8 to a column tile.  (tcgen05 was built
//    and measured: unpacked numbers go to tensor memory at 174 bytes a clock, a product
//    of 16 k takes 45 clocks however few rows it has and 100 while other warps unpack
//    and store: 1,600 clocks a unit.)
//  - The rows' values are put in the weights' order by a warp of its own, where the
//    instruction's fragments are one 16-byte load.
//  - Accumulators of one group are scaled and added in fp32 when the group ends.
//  - The tiles' units stand in one line and each CTA takes an equal share of it
//    (work_split.cuh).  A tile that is cut is added up by the CTA that finishes it
//    last, from fp32 partial sums in the workspace, in ascending order of k: the
//    result does not depend on which CTA that is.
//
// Roles: sets of four multiplying warps, which take the units in turn (4 sets; 3 or 2
// where the rows' accumulators need the registers), then a warp that loads the weights,
// as they lie in memory, one that loads the rows' k and the scales (a copy and its
// barrier take the issuing thread about 200 clocks), one that adds the sets' sums of a
// tile and stores it while they multiply the next, and one or two that order the rows (a
// unit takes one 1,000 clocks at 8 rows, most of it latency).
// Measured (weights in L2, and out of it): 1 x 4,096 x 4,096 8.2 and 8.9 us, 16 x 8,192 x 8,192
// with bias and SiLU 16.2 and 17.4 us, 64 rows of 64 experts, 1,536 x 4,096, 32 us.  Where the
// time goes, in clocks of a CTA (2,070 a us) from the end of the kernel before:
//                                  1 x 4,096^2   16 x 8,192^2   experts
//   share found, roles start            2,250          1,960      5,750
//   first unit there and ordered        2,650          3,300      4,200
//   a set's units: wait + product   1 x 1,540      6 x 2,700  12 x 2,850
//   sums handed over, tiles out         1,400          2,100      8,100
//   last sums, merge (mean; last)  3,400; 5,500   4,900; 7,100  4,500; 7,100
// A set needs 1,500 to 2,500 clocks for a unit alone, so its CTA one in 750 (four sets, 8 rows)
// to 900 (three, 16 rows); the experts' sets also wait 850 of every 2,850 for their next one.
#pragma once

#include "work_split.cuh"
#include "wst_common.cuh"

namespace wst {

constexpr int kW4Feats = 128;  // features of a tile: 4 warps x 32
constexpr int kW4K = 256;      // k of a unit: two halves of 128
constexpr int kW4WBytes = kW4Feats * kW4K / 2;
constexpr int kW4SBytes = 2048;  // scales: 128 features x up to 8 groups, bf16
constexpr int kW4MaxCtas = 160;
constexpr int kW4Pitch = kW4Feats + 4;  // floats of a row of a set's sums

template <int NT>  // column tiles of 8 rows: 1, 2, 4
struct W4Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kSets = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int kOrder = NT <= 2 ? 2 : 1;  // ordering warps
  static constexpr int kThreads = 128 * kSets + 32 * (3 + kOrder);
  static constexpr int kABytes = kRows * kW4K * 2;
  static constexpr int kStage = kW4WBytes + kABytes + kW4SBytes;
  static constexpr int kBufs = NT == 1 ? 2 : 1;  // of the sets' sums
  static constexpr int kSums = kBufs * kSets * kRows * kW4Pitch * 4;
  static constexpr int kFit = (232448 - 2048 - kSums) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kSums + 1024;
  static_assert(kStage % 1024 == 0 && kSmem <= 232448 && kStages >= kSets, "shared memory");
};

// Workspace after the header: two slots of partial sums per CTA, [32 rows][128
// features] fp32 each.  The pieces of the cut tiles are counted in the header's spare
// words, which hold zeros between calls: a byte for each CTA (the tile that begins in
// its share and ends in another's).
constexpr size_t kW4SlotFloats = 32 * kW4Feats;
constexpr size_t kW4WorkspaceBytes = kWsHeaderBytes + 2 * (size_t)kW4MaxCtas * kW4SlotFloats * 4;
static_assert(kW4MaxCtas <= (int)sizeof(WsHeader::pad) && kW4MaxCtas < 256, "a byte for each CTA, counting up to all of them");

struct W4Args {
  int G, M, N, K;
  int k_units;        // ceil(K / 256)
  uint32_t k_mul, k_shift;  // x / k_units = (umulhi(x, k_mul) + x) >> k_shift for x < 2^31
  int n_tiles;        // ceil(N / 128)
  const int* offsets; // NULL: one group of M rows
  const __nv_bfloat16* bias;
  long long stride_bias;
  void* C;
  long long ldc;
  int c_f32;
  int epi;
  int split;          // the workspace holds the slots
  WsHeader* ws;
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
  // (the threads of one CTA, an offset each)
  for (int g = (int)threadIdx.x; g <= p.G; g += (int)blockDim.x) {
    const int v = __ldg(p.offsets + g);
    if (v < (g ? __ldg(p.offsets + g - 1) : 0) || v > p.M || (g == 0 && v != 0)) latch_error(p.ws, kErrBadOffsets, 3);
  }
}

// A CTA's share, one fragment (consecutive units of one tile) after another.
template <int NT>
struct W4Walker {
  int x, hi;          // next unit, end of the share
  int g;
  int base, count;    // group g's first unit and how many it has
  int a, b;           // its rows
  bool fresh;         // the tile of unit x has still to be found
  // the fragment
  int item;           // its tile's first unit
  int tile, chunk, row0, rows, ua, ub;

  __device__ __forceinline__ static int units(const W4Args& p, int a, int b) {
    return (b - a + 8 * NT - 1) / (8 * NT) * p.n_tiles * p.k_units;
  }
  __device__ __forceinline__ void init(const W4Args& p, int lo, int hi_, int g_, int base_) {
    x = lo;
    hi = hi_;
    g = g_;
    base = base_;
    fresh = true;
    if (x < hi) {
      w4_rows(p, g, a, b);
      count = units(p, a, b);
    }
  }
  __device__ __forceinline__ bool next(const W4Args& p) {
    if (x >= hi) return false;
    bool moved = false;
    while (x >= base + count) {
      base += count;
      ++g;  // (x < W: a group holds it)
      w4_rows(p, g, a, b);
      count = units(p, a, b);
      moved = true;
    }
    // tiles of features, and inside one the row chunks: those read the same weights
    const int chunks = (b - a + 8 * NT - 1) / (8 * NT);
    if (fresh) {
      const int t = (int)((__umulhi((uint32_t)(x - base), p.k_mul) + (uint32_t)(x - base)) >> p.k_shift);
      ua = x - base - t * p.k_units;
      tile = chunks == 1 ? t : t / chunks;
      chunk = t - tile * chunks;
      fresh = false;
    } else {  // the tile before this one has ended at x
      ua = 0;
      if (moved) tile = chunk = 0;
      else if (++chunk == chunks) {
        chunk = 0;
        ++tile;
      }
    }
    ub = min(p.k_units, ua + (hi - x));
    item = x - ua;
    row0 = a + chunk * (8 * NT);
    rows = min(8 * NT, b - row0);
    x += ub - ua;
    return true;
  }
};

// The numbers i and i + 4 of a word's eight, minus 8, in 64ths, as bf16.  Four bits at
// the bottom of a bf16 read n 2^-133, four above them n 2^-129 (below 8 a subnormal, from
// 8 on the first normals: the step is the same), so a mask and one multiplication and
// addition do it, exact: n 2^-133 2^127 - 8/64, n 2^-129 2^123 - 8/64.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {
  const uint32_t x = i < 2 ? w : w >> 8;
  uint32_t v = x & (i & 1 ? 0x00f000f0u : 0x000f000fu);
  asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(i & 1 ? 0x7d007d00u : 0x7f007f00u), "r"(0xbe00be00u));
  return v;
}
// d = a b (+ c): 16 features x 16 k, 16 k x 8 rows.
__device__ __forceinline__ void w4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint4 w4_lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// The four words that a lane unpacks of 128 k of the row of weights at `row` (its
// 16-byte words in the order that `swz` gives), where they hold GROUPS groups: lane t of
// four has the t-th part of each group.
template <int GROUPS>
__device__ __forceinline__ void w4_words(uint32_t row, uint32_t swz, uint32_t t, uint32_t (&w)[4]) {
  if constexpr (GROUPS == 1) {
    const uint4 v = w4_lds128(row + ((t ^ swz) << 4));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (GROUPS == 2) {
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(w[2 * h]), "=r"(w[2 * h + 1])
                   : "r"(row + (((2 * h + (t >> 1)) ^ swz) << 4) + 8 * (t & 1))
                   : "memory");
  } else {
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[q]) : "r"(row + ((q ^ swz) << 4) + 4 * t) : "memory");
  }
}
__device__ __forceinline__ float w4_lds_bf16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return __uint_as_float((uint32_t)v << 16);
}
// (a call: inlined at every store it made the code of a tile's end several times as long,
// and code that runs once a launch costs its fetching)
static __device__ __noinline__ float w4_activate(float v, int epi) {
  if (epi == 2) return v / (1.0f + expf(-v));
  if (epi == 3) return v * normcdff(v);
  return v;
}

// Stores features f, f + 1 of a finished tile, row by row.
struct W4Out {
  int n;        // the first feature
  int count;    // how many of the two there are
  float b0, b1;
  __device__ __forceinline__ W4Out(const W4Args& p, int g, int tile, int f) {
    n = tile * kW4Feats + f;
    count = min(max(p.N - n, 0), 2);
    b0 = b1 = 0.0f;
    if (p.epi) {
      const __nv_bfloat16* bias = p.bias + g * p.stride_bias + n;
      if (count > 0) b0 = __bfloat162float(bias[0]);
      if (count > 1) b1 = __bfloat162float(bias[1]);
    }
  }
  __device__ __forceinline__ void store(const W4Args& p, int row, float2 v) const {
    v.x += b0;
    v.y += b1;
    if (p.epi > 1) {
      v.x = w4_activate(v.x, p.epi);
      v.y = w4_activate(v.y, p.epi);
    }
    const long long at = (long long)row * p.ldc + n;
    if (p.c_f32) {
      float* c = static_cast<float*>(p.C) + at;
      if (count == 2) *reinterpret_cast<float2*>(c) = v;
      else if (count == 1) *c = v.x;
    } else {
      __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.C) + at;
      if (count == 2) *reinterpret_cast<uint32_t*>(c) = pack_bf16x2(v.x, v.y);
      else if (count == 1) *c = __float2bfloat16_rn(v.x);
    }
  }
};

// Counts one finished piece of the cut tile that begins in CTA c's share; true for the
// last of `pieces`, which leaves zero.
__device__ __forceinline__ bool w4_last_piece(WsHeader* ws, int c, int pieces) {
  uint32_t* word = ws->pad + (c >> 2);
  const int shift = 8 * (c & 3);
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(word), "r"(1u << shift) : "memory");
  if ((int)((old >> shift) & 255u) + 1 != pieces) return false;
  atomicSub(word, (uint32_t)pieces << shift);
  return true;
}

// CTAs that share W units.  Where every tile can have one, each has the same number of them
// (of at least two units): then no share spans two tiles, whose sums a CTA would hand over
// one after the other, and no tile is cut at odd places.  (1 x 4,096 x 4,096 8.0 us on 128
// CTAs against 10.8 on all, 16 x 8,192 x 8,192 17.2 against 21.0, 61 x 1,531 x 2,744 9.7
// against 13.2; of 13 sizes none became slower.)
__device__ __forceinline__ int w4_ctas(const W4Args& p, int W) {
  const int tiles = W / p.k_units, grid = (int)gridDim.x;
  if (!p.split || tiles == 0) return max(1, min(grid, tiles));
  if (tiles <= grid) return tiles * max(1, min(grid / tiles, p.k_units / 2));
  return min(grid, W / 2);
}

// What is left of a cut tile's piece when its sums are in the slot.
struct W4Piece {
  int c0, c1;  // the tile's first and last CTA
  int g, tile, row0, rows;
};

// tmW {ceil(K/2) bytes, N, G}, boxes of 64 bytes x 128 features, 64-byte swizzle;
// tmA {K, M}, boxes of 256 k x 8 NT rows; tmS {N, ceil(K/group), G}, boxes of 128
// features x 2 GROUPS (GROUPS: the groups of 128 k).
template <int NT, int GROUPS>
__global__ void __launch_bounds__(W4Cfg<NT>::kThreads, 1)
    k_w4_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
              const __grid_constant__ CUtensorMap tmS, const W4Args p) {
  using Cfg = W4Cfg<NT>;
  constexpr int ST = Cfg::kStages, SETS = Cfg::kSets;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_addr(smem);
  float* sums = reinterpret_cast<float*>(smem + ST * Cfg::kStage);  // [buffer][set][row][kW4Pitch]
  __shared__ uint64_t bars[3 * ST + 4];
  __shared__ long long scratch[32], found[2];
  __shared__ uint32_t abort_word, is_last[2];
  // the cut tiles' pieces (at most the first and the last fragment), the last fragment
  // among them whether it is cut or not
  __shared__ W4Piece piece[2];
  __shared__ int pieces, last_buf;
  volatile uint32_t* abort_flag = &abort_word;
  const int warp = (int)threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  // loaded, full (and the rows are in order), empty; sum_full, sum_empty of the sums'
  // buffers.  A barrier's parity tells two phases apart, so who waits for a stage has to
  // know that its last use is over.  The ordering warps hand the stages on one after the
  // other, whatever order they arrive in: a set that has had unit u - SETS knows that unit
  // u - ST was there.
  const uint32_t loaded = smem_addr(bars), full = loaded + 8 * ST, empty = full + 8 * ST;
  const uint32_t sum_full = empty + 8 * ST, sum_empty = sum_full + 16;
  if (warp == 4 * SETS && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(loaded + 8 * i, 2);
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sum_full + 8 * i, 4 * SETS);
      mbar_init(sum_empty + 8 * i, 1);
    }
    *abort_flag = 0u;
    found[0] = found[1] = 0;
    pieces = 0;
    fence_mbar_init();
  }
  if (warp == 4 * SETS + 1 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmS);
  }
  early_wait();
  // this CTA's share; whole tiles where the workspace holds no partial sums
  const int grain = p.split ? 1 : p.k_units;
  int W, lo = 0, hi = 0;
  if (p.offsets) {
    BlockCount<long long, Cfg::kThreads> counted;
    auto count = [&](int g) -> long long {
      int a, b;
      w4_rows(p, g, a, b);
      return W4Walker<NT>::units(p, a, b);
    };
    const long long all = counted.total(p.G, count, scratch);
    W = all > 0x7fffffff ? 0 : (int)all;  // (only offsets that go back and forth count so many: they are refused)
    const Share<int> s(W / grain, w4_ctas(p, W));
    if ((int)blockIdx.x < s.G) {
      lo = s.lo((int)blockIdx.x) * grain;
      hi = s.lo((int)blockIdx.x + 1) * grain;
    }
    if (lo < hi) counted.locate(p.G, count, (long long)lo, scratch, found);
    if (blockIdx.x == 0) w4_check_offsets(p);
  } else {
    W = W4Walker<NT>::units(p, 0, p.M);
  }
  const Share<int> share(W / grain, w4_ctas(p, W));
  if (!p.offsets && (int)blockIdx.x < share.G) {
    lo = share.lo((int)blockIdx.x) * grain;
    hi = share.lo((int)blockIdx.x + 1) * grain;
  }
  // (the warp that loads the weights set the barriers up itself: without groups to find
  // it need not wait for the others)
  if (warp == 4 * SETS && !p.offsets) {
    __syncwarp();
    asm volatile("barrier.arrive 2, %0;" ::"n"(Cfg::kThreads) : "memory");
  } else {
    asm volatile("barrier.sync 2, %0;" ::"n"(Cfg::kThreads) : "memory");
  }
  const Guard guard{p.ws, abort_flag, p.timeout_ns};
  W4Walker<NT> w;
  w.init(p, lo, hi, p.offsets ? (int)found[0] : 0, p.offsets ? (int)found[1] : 0);

  if (warp == 4 * SETS || warp == 4 * SETS + 1) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      const bool weights = warp == 4 * SETS;
      int s = 0;
      uint32_t ph = 1;
      bool ok = true;
      while (ok && w.next(p)) {
        for (int u = w.ua; u < w.ub; ++u) {
          if (!wait_phase(guard, empty + 8 * s, ph, (kRoleProducer << 16) | s)) {
            ok = false;
            break;
          }
          const uint32_t at = ring + s * Cfg::kStage;
          if (weights) {
            mbar_arrive_expect_tx(loaded + 8 * s, (uint32_t)kW4WBytes);
            tma_load_3d(at, &tmW, loaded + 8 * s, u * (kW4K / 2), w.tile * kW4Feats, w.g);
            tma_load_3d(at + kW4WBytes / 2, &tmW, loaded + 8 * s, u * (kW4K / 2) + 64, w.tile * kW4Feats, w.g);
          } else {
            mbar_arrive_expect_tx(loaded + 8 * s, (uint32_t)(Cfg::kABytes + 512 * GROUPS));
            tma_load_2d(at + kW4WBytes, &tmA, loaded + 8 * s, u * kW4K, w.row0);
            tma_load_3d(at + Cfg::kStage - kW4SBytes, &tmS, loaded + 8 * s, w.tile * kW4Feats, 2 * u * GROUPS, w.g);
          }
          if (++s == ST) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp >= 4 * SETS + 3) {
    // ------------------------------------------------------------------ the rows' order
    // Eight k of a row (16 bytes) are one lane's fragments for the eight numbers of a
    // word: 0 4 1 5 2 6 3 7.  They stay in their row of 512 bytes, [half][word q][lane t],
    // odd rows with neighbouring q exchanged: the four lanes' words of two rows fill the
    // banks once.
    const uint32_t kc = lane & 15u;
    const uint32_t q = GROUPS == 1 ? kc & 3u : GROUPS == 2 ? (kc >> 3) * 2 + (kc & 1u) : kc >> 2;
    const uint32_t t = GROUPS == 1 ? kc >> 2 : GROUPS == 2 ? (kc >> 1) & 3u : kc & 3u;
    const uint32_t place[2] = {((lane >> 4) * 16 + q * 4 + t) * 16, ((lane >> 4) * 16 + (q ^ 1u) * 4 + t) * 16};
    constexpr int ORDER = Cfg::kOrder;
    static_assert(ST > ORDER && ST >= SETS, "who waits for a unit knows that the stage's last one is over");
    const int total = hi - lo;
    int s = warp - (4 * SETS + 3), prev = s == 0 ? ST - 1 : s - 1;  // the stages of unit u and of the one before
    uint32_t ph = 0, prev_ph = s == 0 ? 1u : 0u;
    for (int u = s; u < total; u += ORDER) {
      bool there = mbar_try_wait(loaded + 8 * s, ph);  // (by each lane: it reads the copies)
      if (!__all_sync(0xffffffffu, there) &&
          !__all_sync(0xffffffffu, wait_phase(guard, loaded + 8 * s, ph, (kRoleEpilogue << 16) | 0x100 | s)))
        break;
      const uint32_t at = ring + s * Cfg::kStage + kW4WBytes;
#pragma unroll 1
      for (int i0 = 0; i0 < 8 * NT; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w4_lds128(at + (uint32_t)((i0 + i) * (kW4K * 2)) + lane * 16);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(at + (uint32_t)((i0 + i) * (kW4K * 2)) + place[i & 1], __byte_perm(v[i].x, v[i].z, 0x5410),
                       __byte_perm(v[i].x, v[i].z, 0x7632), __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
      }
      fence_proxy_async_smem();  // (the stage's next copy comes by the other proxy: barriers alone do not put these stores before it)
      __syncwarp();
      if (lane == 0) {
        // in the units' order: after the unit before this one
        if (ORDER > 1 && !wait_phase(guard, full + 8 * prev, prev_ph, (kRoleEpilogue << 16) | 0x180 | s)) there = false;
        else mbar_arrive(full + 8 * s), there = true;
      }
      if (!__shfl_sync(0xffffffffu, there ? 1 : 0, 0)) break;
      if ((s += ORDER) >= ST) {
        s -= ST;
        ph ^= 1u;
      }
      if ((prev += ORDER) >= ST) {
        prev -= ST;
        prev_ph ^= 1u;
      }
    }
  } else if (warp == 4 * SETS + 2) {
    // ------------------------------------------------------------------ tiles out
    // All but the share's last one.  (lane: four features)
    const int f = 4 * (int)lane;
    int buf = 0, cut = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (w.next(p)) {
      const bool whole = w.ub - w.ua == p.k_units;
      const int c0 = whole ? (int)blockIdx.x : share.owner(w.item);
      // A piece of a cut tile goes into this CTA's slot (the second one if the tile begins
      // in its share); it is counted when the share is done.
      if (!whole || w.x >= w.hi) {
        if (lane == 0)
          piece[cut] = W4Piece{c0, whole ? c0 : share.owner(w.item + p.k_units - 1), w.g, w.tile, w.row0, w.rows};
        ++cut;
        if (w.x >= w.hi) break;
      }
      float* slot = p.slots + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == c0 ? 1 : 0)) * kW4SlotFloats + f;
      const W4Out out0(p, w.g, w.tile, f), out1(p, w.g, w.tile, f + 2);
      // (a wait that gave up: the pieces are counted all the same)
      ok = ok && warp_wait_phase(guard, sum_full + 8 * buf, ph, (kRoleEpilogue << 16) | 0x200 | buf);
      if (ok) {
        const float* from = sums + buf * (SETS * Cfg::kRows * kW4Pitch) + f;
#pragma unroll 1
        for (int row0 = 0; row0 < w.rows; row0 += 8) {  // (the buffer holds whole eights)
          float4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const float4*>(from + (row0 + i) * kW4Pitch);
#pragma unroll
          for (int k = 1; k < SETS; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = *reinterpret_cast<const float4*>(from + (k * Cfg::kRows + row0 + i) * kW4Pitch);
              v[i].x += x.x;
              v[i].y += x.y;
              v[i].z += x.z;
              v[i].w += x.w;
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (row0 + i >= w.rows) break;
            if (whole) {
              out0.store(p, w.row0 + row0 + i, make_float2(v[i].x, v[i].y));
              out1.store(p, w.row0 + row0 + i, make_float2(v[i].z, v[i].w));
            } else {
              __stcg(reinterpret_cast<float4*>(slot + (row0 + i) * kW4Feats), v[i]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sum_empty + 8 * buf);
      }
      if (++buf == Cfg::kBufs) {
        buf = 0;
        ph ^= 1u;
      }
    }
    if (lane == 0) {
      pieces = cut;
      last_buf = buf;
    }
  } else {
    // ------------------------------------------------------------------ products
    const int set = warp >> 2, f0 = (warp & 3) * 32;
    const uint32_t g8 = lane >> 2, t = lane & 3;
    const uint32_t swz = (g8 >> 1) & 3u;  // (row >> 1) & 3 of every row that the lane reads
    const uint32_t w_at = ring + (uint32_t)((f0 + (int)g8) * 64), s_at = ring + (uint32_t)(Cfg::kStage - kW4SBytes + (f0 + (int)g8) * 2);
    uint32_t a_at[2];  // of even and odd q
#pragma unroll
    for (int q = 0; q < 2; ++q) a_at[q] = ring + (uint32_t)kW4WBytes + g8 * (kW4K * 2) + ((((uint32_t)q ^ (g8 & 1u)) * 4 + t) << 4);
    int left = set;      // units until this set's next one
    int s = set;         // its stage
    uint32_t ph = 0;
    int buf = 0;
    uint32_t sph = 1;
    bool ok = true;
    while (w.next(p)) {
      float acc[2][NT][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.0f;
      const int n = w.ub - w.ua;
      for (; left < n; left += SETS) {
        ok = ok && warp_wait_phase(guard, full + 8 * s, ph, (kRoleMma << 16) | s);
        if (!ok) continue;
#pragma unroll NT <= 2 ? 2 : 1
        for (uint32_t half = 0; half < 2; ++half) {
          const uint32_t at = (uint32_t)(s * Cfg::kStage);
          const uint32_t hw = w_at + at + half * (kW4WBytes / 2), ha = at + half * (kW4K * 2 / 2), hs = s_at + at + half * (256 * GROUPS);
          uint32_t word[2][2][4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            w4_words<GROUPS>(hw + m * 1024, swz, t, word[m][0]);
            w4_words<GROUPS>(hw + m * 1024 + 512, swz, t, word[m][1]);
          }
          float part[2][NT][4];
          constexpr float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool first = q % (4 / GROUPS) == 0, last = (q + 1) % (4 / GROUPS) == 0;
            uint32_t a[2][2][4];  // [tile][half of the word][fragment]
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                a[m][j][0] = w4_pair(word[m][0][q], 2 * j);
                a[m][j][1] = w4_pair(word[m][1][q], 2 * j);
                a[m][j][2] = w4_pair(word[m][0][q], 2 * j + 1);
                a[m][j][3] = w4_pair(word[m][1][q], 2 * j + 1);
              }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const uint4 x = w4_lds128(a_at[q & 1] + ha + (uint32_t)((q >> 1) * 128 + i * (8 * kW4K * 2)));
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                if (first) w4_mma(part[m][i], a[m][0], x.x, x.y, zero);
                else w4_mma(part[m][i], a[m][0], x.x, x.y, part[m][i]);
                w4_mma(part[m][i], a[m][1], x.z, x.w, part[m][i]);
              }
            }
            if (last) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const uint32_t sq = hs + (uint32_t)(q / (4 / GROUPS) * 256 + m * 32);
                const float s0 = w4_lds_bf16(sq), s1 = w4_lds_bf16(sq + 16);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                  acc[m][i][0] = fmaf(s0, part[m][i][0], acc[m][i][0]);
                  acc[m][i][1] = fmaf(s0, part[m][i][1], acc[m][i][1]);
                  acc[m][i][2] = fmaf(s1, part[m][i][2], acc[m][i][2]);
                  acc[m][i][3] = fmaf(s1, part[m][i][3], acc[m][i][3]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        s += SETS;
        if (s >= ST) {
          s -= ST;
          ph ^= 1u;
        }
      }
      left -= n;
      // The tile's sums of this set, for the warp that stores it.
      ok = ok && warp_wait_phase(guard, sum_empty + 8 * buf, sph, (kRoleMma << 16) | 0x400 | buf);
      if (ok) {
        float* o = sums + ((buf * SETS + set) * Cfg::kRows + 2 * (int)t) * kW4Pitch + f0 + (int)g8;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)  // (the weights were in 64ths)
              o[(8 * i + (j & 1)) * kW4Pitch + 16 * m + 8 * (j >> 1)] = 64.0f * acc[m][i][j];
        __syncwarp();
        if (lane == 0) mbar_arrive(sum_full + 8 * buf);
      }
      if (++buf == Cfg::kBufs) {
        buf = 0;
        sph ^= 1u;
      }
    }
  }
  __syncthreads();
  // All threads: the sums of the last fragment (piece[pieces - 1]), then the cut tiles
  // of which this CTA counts the last piece.  (thread: two features, every TR-th row)
  constexpr int TR = Cfg::kThreads / 64;
  constexpr int PER = (Cfg::kRows + TR - 1) / TR < 6 ? (Cfg::kRows + TR - 1) / TR : 6;  // rows of a thread at a time
  const int f = 2 * (int)(threadIdx.x & 63);
  const int first_row = (int)threadIdx.x < 64 * TR ? (int)threadIdx.x >> 6 : Cfg::kRows;
  if (pieces > 0) {
    const W4Piece x = piece[pieces - 1];
    const bool whole = x.c0 == x.c1;
    float* slot = p.slots + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == x.c0 ? 1 : 0)) * kW4SlotFloats + f;
    const float* from = sums + last_buf * (SETS * Cfg::kRows * kW4Pitch) + f;
    const W4Out out(p, x.g, x.tile, f);
#pragma unroll 1
    for (int row0 = first_row; row0 < x.rows; row0 += PER * TR) {
      float2 v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < SETS; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (row0 + i * TR < Cfg::kRows) {
            const float2 y = *reinterpret_cast<const float2*>(from + (k * Cfg::kRows + row0 + i * TR) * kW4Pitch);
            v[i].x += y.x;
            v[i].y += y.y;
          }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int row = row0 + i * TR;
        if (row >= x.rows) break;
        if (whole) out.store(p, x.row0 + row, v[i]);
        else __stcg(reinterpret_cast<float2*>(slot + row * kW4Feats), v[i]);
      }
    }
    if (pieces == 2 || !whole) {  // (of two pieces the first is one of a cut tile)
      __syncthreads();
      if ((int)threadIdx.x < pieces) {
        // (the count releases all threads' stores, which the barrier put before it)
        const W4Piece& y = piece[threadIdx.x];
        is_last[threadIdx.x] = y.c0 != y.c1 && w4_last_piece(p.ws, y.c0, y.c1 - y.c0 + 1) ? 1u : 0u;
      }
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < pieces; ++k) {
        if (!is_last[k]) continue;
        const W4Piece y = piece[k];
        const W4Out out(p, y.g, y.tile, f);
#pragma unroll 1
        for (int row0 = first_row; row0 < y.rows; row0 += PER * TR) {
          float2 v[PER];
          const float* at = p.slots + (size_t)row0 * kW4Feats + f;
#pragma unroll
          for (int i = 0; i < PER; ++i) v[i] = make_float2(0.0f, 0.0f);
#pragma unroll (PER == 1 ? 8 : 4)
          for (int c = y.c0; c <= y.c1; ++c) {
            const float* of = at + (size_t)(2 * c + (c == y.c0 ? 1 : 0)) * kW4SlotFloats;
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (row0 + i * TR < Cfg::kRows) {  // (rows behind the last one too)
                const float2 z = __ldcg(reinterpret_cast<const float2*>(of + i * TR * kW4Feats));
                v[i].x += z.x;
                v[i].y += z.y;
              }
          }
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (row0 + i * TR >= y.rows) break;
            out.store(p, y.row0 + row0 + i * TR, v[i]);
          }
        }
      }
    }
  }
  if (*abort_flag) {
    for (int i = 0; i < 200; ++i) __nanosleep(1000);  // copies still in flight land first
  }
}

}  // namespace wst
