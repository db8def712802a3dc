// tree_attn.cuh -- attention of a step's tokens (a drafted tree, a chain, one token
// for each sequence) over a paged cache, for sm_103a.
//
//   O[i][h] = sum_j p_ij V[j][h / group],  p = softmax over the j that i sees of
//             scale * Q[i][h] . K[j][h / group]
// Sequence b has context[b] cached tokens, which all of its n_b new tokens see, and
// the new tokens themselves, of which a token sees those in its mask (or those up
// to itself).  All of them lie in the cache, through the sequence's page table.
//
// The query rows of a sequence that share a key head (its tokens x the `group` heads
// of that key head) are stacked into tiles of 128 rows, and K and V are read once per
// tile: for a step of few tokens that read is the whole cost, and the 128-row products
// hide under it even where most rows are empty (S and PV of 128 keys take 1,000 clocks of
// the tensor core, their 64 KB 2,800 clocks of an SM's share of HBM).
//
// Schedule: an item is (sequence, key head, tile), a block 128 keys.  The items' blocks
// stand in one line, each CTA takes an equal share (work_split.cuh); the lengths are on the
// device, so every CTA counts them at its start.  The line holds the even tiles of all
// sequences, then the odd ones: the two tiles of a sequence are worked on by two CTAs at
// nearly the same time, and the later one finds K and V in L2.  The cut between the lines is
// shifted (Share's lead) so that the two are up to 24 blocks apart: at the same time both
// miss L2 and read HBM.  (16 trees of 64 tokens on up to 8,192, 400 MB of K and V, four draws of
// the lengths: 131, 124, 139, 138 us, without a lead 144, 119, 143, 143; 500 to 700 MB are read,
// 740 without one.  It makes no difference to 32 trees on up to 2,048, nor to batches whose
// sequences have no second tile, where it only makes shares unequal, by less than a block: 64
// sequences of one token 135 us both ways.  In the sequences' order one CTA took a tile after
// the other, 138 us and 800 MB.)  Two tiles of a sequence in one CTA read 400 MB but wait for
// each other's products, 129 us, with one S/P buffer for each of the two.
// A piece of a cut item leaves its un-normalised O, row maxima m and sums l in the
// workspace, and a second kernel adds an item's pieces in a fixed order:
//   m* = max m_i,  l* = sum l_i 2^(m_i - m*),  O = sum O_i 2^(m_i - m*) / l*
// (its launch overlaps the first kernel's end; it is spread over all SMs, where the
// last CTA of an item alone would read up to 152 pieces of 64 KB).
//
// Inside a CTA, per block (online softmax in base 2, cs = scale * log2 e):
//   MMA      S = Q . K^T        Q and K from shared memory, 128 x 128 x Dh
//   softmax  P = 2^(cs S - m) as bf16 over S's tensor memory; m is a whole number that
//            moves only when a score exceeds it by more than 8, which rescales O and l (fp32
//            output: the sums that take O over)
//            (P <= 2^8; l sums the unrounded P).  One bf16 is off by up to 2^-8 of P, which
//            a bf16 output's own rounding covers; for fp32 output P is three bf16, each what
//            the ones before leave, off by 2^-24 together
//   MMA      O += P . V         P from tensor memory, V from shared memory (for each part of P;
//            fp32 output, and bf16 output of long sequences, take O over into sums of their
//            own, see kTreeRun)
// From a score's product to the next in its buffer it is S, softmax, PV and three
// handshakes, 5,000 clocks, of which the softmax is a third: three S/P buffers (two of the
// wider ones of fp32 output) let S run ahead of PV.  (Two items at a time with one buffer
// each: 147 us for 32 sequences of 4,096 against 82.)  Two threads issue the products, so
// that one's run under the other's wait.
// Measured (32 heads on 8 of 128): one token on 262,144 keys 159 us, 1.07 GB at 6.7 TB/s;
// one token each of 32 sequences of up to 4,096, 77 us, 403 MB, of which 14 are start, the
// items' ends and the second kernel; 4 chunks of 500 tokens behind up to 2,000 (28 heads on
// 4) 103 us, 0.35 PFLOP/s: the softmax's chain, 3,300 clocks a block.  fp32 output of these:
// 269, 133, 151 us.
//
// A block that ends behind the context (a sequence's last one or two) takes another
// path: each row's visible keys come as 128 bits, scores outside them do not count
// whatever they hold, and the rows of V outside the sequence are cleared in shared
// memory, since 0 * NaN in the product would reach every row.  For the same reason a
// new token's V that is not finite is cleared too and added again, at the end, to the
// rows that see it.
//
// Roles (256 threads): warp 0 loads K, warp 3 V (a lane per page of a block); warp 1
// issues S, warp 2 PV (and owns the tensor memory); warps 4-7 are the softmax and the
// output, thread = row = tensor memory lane, and load Q.  Each role walks the share for
// itself; the loaders fetch the page numbers of their next item while they work on one
// (two dependent reads).
#pragma once

#include "work_split.cuh"
#include "wst_common.cuh"

namespace wst {

constexpr int kTreeBM = 128;
constexpr int kTreeBN = 128;
constexpr int kTreeMaxCtas = 160;
constexpr float kTreeGrow = 8.0f;       // log2 of how far P may exceed 1
constexpr float kTreeGrowSum = 256.0f;  // 2^kTreeGrow

constexpr int kTreeThreads = 256;
constexpr int kTreeLead = 24;  // blocks, of one line before the other
// A product into tensor memory cuts its sum off after 24 bits, always towards zero, with every
// 16 keys of every part of P: 0.65 of 2^-23 on the average.  Left to add up, fp32 output was off
// by 4e-5 on 8,000 keys in one CTA and by 2e-3 on 262,144.  So the softmax warps of fp32 output
// take O over after every block, into fp32 sums in registers (2e-7 on 8,000 keys, 9e-7 on
// 262,144; a plain fp32 form 1e-7.  One token each of 32 sequences of 4,096 115 -> 133 us, 16
// trees of 64 224 -> 236, chunks of 500 140 -> 151; four warps of their own for the sums, handed
// a block's O at a time, took 178, 332 and 188).  bf16 output, whose own rounding is off by up to
// 2^-8, takes O over after kTreeRun blocks (8 cuts a block: 2^-11 at most), in a form of the
// kernel apart, for tables that hold more than kTreeLong keys: the code for it makes the loop
// slower where the softmax bounds it (trees 132 -> 141 us), but not one token on 262,144 keys
// (158.5 -> 159.1).
constexpr int kTreeRun = 512;
constexpr int kTreeLong = kTreeRun * kTreeBN;

// PARTS: bf16 numbers that hold one P, 1 for bf16 output, 3 for fp32.
template <int DH, int PARTS>
struct TreeCfg {
  static constexpr int kTile = kTreeBN * DH * 2;  // bytes of a Q tile or a block of K or V
  static constexpr int kKStages = DH == 128 ? 3 : 6;
  static constexpr int kVStages = DH == 128 ? 2 : 5;
  // S/P buffers and their columns of tensor memory: the first two parts of P lie over S,
  // the third behind it
  static constexpr int kSBufs = PARTS == 1 ? 3 : 2;
  // keys of a step of the softmax (fp32 output keeps DH sums in registers: 32 at Dh 128, spilled,
  // takes 157 us where 16 takes 133, 32 sequences of 4,096; at Dh 64 111 against 121)
  static constexpr int kWidth = PARTS == 1 ? 64 : DH == 64 ? 32 : 16;
  static constexpr int kSCols = PARTS == 1 ? kTreeBN : kTreeBN + kTreeBN / 2;
  static constexpr int kBars = 2 * kKStages + 2 * kVStages + 2 + 3 * kSBufs + 1;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kKStages + kVStages) * kTile + 1024;
  static constexpr int kTmemO = kSBufs * kSCols;
  static_assert(kSmem <= 232448 && kTmemO + DH <= 512 && DH % 64 == 0, "shared memory, tensor memory");
};

// What the second kernel needs of a cut item; pieces 0: none.
struct TreeCut {
  int pieces;   // of CTAs c, c + 1, ...
  int token0;   // the first row's token
  int head0;    // the first row's head
  int ntok;     // the item's tokens
};

// Workspace after the header: TreeCut[kTreeMaxCtas], then two slots per CTA (the second
// for an item that begins in its share): O as [Dh / 4][128 rows][4] fp32, m[128], l[128].
constexpr size_t kTreeCutOffset = kWsHeaderBytes;
constexpr size_t kTreeSlotOffset = kTreeCutOffset + (size_t)kTreeMaxCtas * sizeof(TreeCut);
constexpr size_t kTreeSlotFloats = (size_t)128 * kTreeBM + 2 * kTreeBM;
constexpr size_t kTreeWorkspaceBytes = kTreeSlotOffset + 2 * (size_t)kTreeMaxCtas * kTreeSlotFloats * 4;
static_assert(kTreeSlotOffset % 16 == 0, "alignment of the slots");

struct TreeArgs {
  int B, T, H, Hkv, group;
  int tokens;             // of a tile: 128 / group
  int lines;              // 2: even tiles, then odd ones; 1: no sequence has two
  int page_size, max_pages;
  int num_pages;
  int chunk;              // keys of one copy: min(page_size, 128)
  const int* q_offsets;
  const int* context;
  const int* mask;        // [T][mask_words] or NULL
  int mask_words;
  long long ldm;
  const int* table;
  long long ldt;
  const __nv_bfloat16* v;  // for new tokens that are not finite
  long long page_stride, token_stride, head_stride;
  float cs;               // scale * log2(e)
  void* O;
  long long ldo;
  WsHeader* ws;
  int split;
  TreeCut* cuts;
  float* slots;
  unsigned long long timeout_ns;
};

// sum over i < n of floor((a i + b) / 128), n < 2^23, a <= 256, b < 2^31: whole parts are
// taken out, then the points under the line are counted along the other axis, until none
// are left (a logarithm of 128 steps; the quotients fit 32 bits).
__device__ __forceinline__ long long tree_floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  long long sum = (long long)(a >> 7) * ((long long)n * (n - 1) / 2) + (long long)(b >> 7) * n;
  a &= 127u;
  b &= 127u;
  uint32_t m = 128;
  while (true) {
    const uint32_t top = a * n + b;  // (the line's value behind the last point, times m)
    n = top / m;
    if (n == 0) return sum;
    b = top - n * m;
    const uint32_t whole = m / a;  // (a > 0: else top < m)
    const uint32_t rest = m - whole * a;
    m = a;
    a = rest;
    sum += (long long)whole * ((long long)n * (n - 1) / 2) + (long long)(b / m) * n;
    b %= m;
  }
}

// r / d, in 32 bits where both fit (nearly always)
__device__ __forceinline__ long long tree_div(long long r, long long d) {
  if (((r | d) >> 32) == 0) return (long long)((uint32_t)r / (uint32_t)d);
  return r / d;
}

// One sequence's even or odd tiles (v: all sequences' even ones, then their odd ones), as
// every role sees it (what breaks the rules is clamped; the checks report it).
struct TreeSeq {
  int b, odd;
  int a, n;            // its rows of Q: tokens [a, a + n)
  int ctx;
  int tiles;           // even (or odd) ones
  long long per_head;  // their blocks, of one key head

  __device__ __forceinline__ void load(const TreeArgs& p, int v) {
    odd = v >= p.B ? 1 : 0;
    b = v - odd * p.B;
    const int o0 = __ldg(p.q_offsets + b), o1 = __ldg(p.q_offsets + b + 1), c = __ldg(p.context + b);
    a = min(max(o0, 0), p.T);
    n = min(max(o1, a), p.T) - a;
    const long long most = (long long)p.max_pages * p.page_size - n;
    ctx = (int)min((long long)max(c, 0), max(most, 0ll));
    const int all = n <= p.tokens ? (n > 0 ? 1 : 0) : (n + p.tokens - 1) / p.tokens;
    tiles = p.lines == 1 ? all : (all - odd + 1) >> 1;
    per_head = tiles == 0 ? 0 : before(p, tiles - 1) + blocks(p, tiles - 1);
  }
  // the sequence's first token of its i-th tile here
  __device__ __forceinline__ int token(const TreeArgs& p, int i) const { return (p.lines * i + odd) * p.tokens; }
  // keys that some row of the tile may see, and their blocks
  __device__ __forceinline__ int keys(const TreeArgs& p, int i) const {
    return ctx + (p.mask ? n : min(n, token(p, i) + p.tokens));
  }
  __device__ __forceinline__ int blocks(const TreeArgs& p, int i) const { return (keys(p, i) + kTreeBN - 1) / kTreeBN; }
  // blocks of the tiles before the i-th
  __device__ __forceinline__ long long before(const TreeArgs& p, int i) const {
    if (i == 0) return 0;
    if (p.mask) return (long long)i * ((ctx + n + kTreeBN - 1) / kTreeBN);
    return tree_floor_sum((uint32_t)i, (uint32_t)(p.lines * p.tokens), (uint32_t)(ctx + (odd + 1) * p.tokens + kTreeBN - 1));
  }
};

// A CTA's share, one fragment (consecutive blocks of one item) after another.
struct TreeWalker {
  long long x, hi;
  int v, h, t;
  long long base;   // first block of v
  bool fresh;       // (v, h, t) hold the item of block x
  TreeSeq s;
  // the fragment
  long long item;   // the item's first block
  int jb, je, nb;   // its blocks of the item's nb
  int token0, ntok; // the tile's tokens
  int keys;         // keys that it may see

  __device__ __forceinline__ void init(const TreeArgs& p, long long lo, long long hi_, int v_, long long base_) {
    x = lo;
    hi = hi_;
    v = v_;
    base = base_;
    if (x >= hi) return;
    s.load(p, v);
    const long long r = x - base;
    h = (int)tree_div(r, s.per_head);
    const long long at = r - h * s.per_head;
    int lo_t = 0, hi_t = s.tiles - 1;  // the last tile with before(t) <= at
    while (lo_t < hi_t) {
      const int mid = (lo_t + hi_t + 1) / 2;
      if (s.before(p, mid) <= at) lo_t = mid;
      else hi_t = mid - 1;
    }
    t = lo_t;
    item = base + h * s.per_head + s.before(p, t);
    fresh = true;
  }
  __device__ __forceinline__ bool next(const TreeArgs& p) {
    if (x >= hi) return false;
    if (!fresh) {  // the item before this one has ended at x
      if (++t == s.tiles) {
        t = 0;
        if (++h == p.Hkv) {
          h = 0;
          base += s.per_head * p.Hkv;
          do s.load(p, ++v);  // (x < W: a sequence holds it)
          while (s.tiles == 0);
        }
      }
      item = x;
    }
    nb = s.blocks(p, t);
    jb = (int)(x - item);
    je = (int)min((long long)nb, jb + (hi - x));
    token0 = s.a + s.token(p, t);
    ntok = min(p.tokens, s.n - s.token(p, t));
    keys = s.keys(p, t);
    x += je - jb;
    fresh = false;
    return true;
  }
};

static __device__ __noinline__ void tree_check(const TreeArgs& p) {
  // (the threads of one CTA, a sequence each)
  for (int b = (int)threadIdx.x; b < p.B; b += (int)blockDim.x) {
    const int o0 = __ldg(p.q_offsets + b), o1 = __ldg(p.q_offsets + b + 1), c = __ldg(p.context + b);
    const long long n = (long long)o1 - o0;
    if ((b == 0 && o0 != 0) || n < 0 || o0 < 0 || o1 > p.T || c < 0 || c + n > (long long)p.max_pages * p.page_size ||
        (p.mask && n > 32ll * p.mask_words))
      latch_error(p.ws, kErrBadOffsets, 5);
  }
}

// Bits 0..31: whether row `ti` of a sequence (its token's index there) sees keys
// e .. e + 31 behind the context (e < 0: keys of the context).
__device__ __forceinline__ uint32_t tree_visible(const TreeArgs& p, const TreeSeq& s, int ti, int e) {
  const int end = p.mask ? s.n : ti + 1;  // no key from here on
  const int left = end - e;
  if (left <= 0) return 0u;
  uint32_t bits = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
  if (p.mask && e + 31 >= 0) {
    const int* row = p.mask + (long long)(s.a + ti) * p.ldm;
    auto word = [&](int i) -> uint32_t { return i >= 0 && i < p.mask_words ? (uint32_t)__ldg(row + i) : 0u; };
    const int at = e >> 5;  // floor
    const uint32_t lo = at < 0 ? 0xffffffffu : word(at);
    bits &= __funnelshift_r(lo, word(at + 1), (uint32_t)(e & 31));
  }
  return bits;
}

// 32 consecutive columns of this thread's lane of tensor memory, without the wait.
__device__ __forceinline__ void tree_tmem_load32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tree_tmem_load16(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
// Waits for the thread's loads; v passes through, so that no use of it moves ahead.
template <int N>
__device__ __forceinline__ void tree_tmem_load_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tree_tmem_store16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tree_tmem_store8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Waits for a phase: tests for a while (a suspended wait takes longer to wake), then as
// the others do.
__device__ __forceinline__ bool tree_wait(const Guard& g, uint32_t bar, uint32_t parity, uint32_t info) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_test_wait(bar, parity)) return true;
  return wait_slow(g, bar, parity, info, false);
}

// The blocks of the share's K or V, for the warp that loads them: lane c of a block's
// copies takes chunk c (a page, or 128 keys of one).
template <int DH>
struct TreeLoads {
  TreeWalker w, nx;
  bool has, has_next;
  int ids, ids_next, ids_first;  // page of this lane's chunk, `batch` blocks at a time; -1: nothing to load
  int i, j, in_page;

  __device__ __forceinline__ static int fetch(const TreeArgs& p, const TreeWalker& f, int j0) {
    const int per_block = kTreeBN / p.chunk, page_blocks = p.page_size / kTreeBN;
    const int block = (int)lane_id() / per_block, chunk = (int)lane_id() - block * per_block;
    const int j = j0 + block;
    if (j >= f.je || j * kTreeBN + chunk * p.chunk >= f.keys) return -1;
    const int i = page_blocks ? j / page_blocks : j * per_block + chunk;
    return i < p.max_pages ? __ldg(p.table + (long long)f.s.b * p.ldt + i) : -1;
  }
  __device__ __forceinline__ void enter(const TreeArgs& p) {
    const int page_blocks = p.page_size / kTreeBN;
    ids = ids_first;
    ids_next = fetch(p, w, w.jb + 32 / (kTreeBN / p.chunk));
    i = 0;
    j = w.jb;
    in_page = page_blocks ? j % page_blocks : 0;
  }
  __device__ __forceinline__ void start(const TreeArgs& p, const TreeWalker& from) {
    w = from;
    has = w.next(p);
    if (!has) return;
    ids_first = fetch(p, w, w.jb);
    enter(p);
  }
  // One block into stage `st` (whose barriers are full and empty); false: gave up.
  __device__ __forceinline__ bool step(const TreeArgs& p, const Guard& guard, const CUtensorMap* tm, uint32_t dst, uint32_t full,
                                       uint32_t empty, uint32_t parity, uint32_t info) {
    const uint32_t lane = lane_id();
    const int per_block = kTreeBN / p.chunk, batch = 32 / per_block;  // chunks of a block: 1 .. 16
    if (i == batch) {
      i = 0;
      ids = ids_next;
      ids_next = fetch(p, w, j + batch);
    }
    const int left = w.keys - j * kTreeBN;
    const int chunks = left >= kTreeBN ? per_block : (left + p.chunk - 1) / p.chunk;
    const int page = __shfl_sync(0xffffffffu, ids, (i * per_block + (int)(lane & (uint32_t)(per_block - 1))) & 31);
    ++i;
    bool ok = true;
    if (lane == 0) {
      ok = wait_phase(guard, empty, parity, info);
      if (ok) mbar_arrive_expect_tx(full, (uint32_t)(chunks * p.chunk * DH * 2));
    }
    if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) return false;
    if ((int)lane < chunks) {
      // (a page outside the cache reads as zeros)
      if (page < 0 || page >= p.num_pages) latch_error(p.ws, 1u, (kRoleProducer << 16) | 0x20);
      const uint32_t to = dst + (uint32_t)((int)lane * p.chunk * 128);
      for (int hf = 0; hf < DH / 64; ++hf)
        tma_load_4d(to + hf * (kTreeBN * 128), tm, full, hf * 64, in_page * kTreeBN, w.h, page);
    }
    if (++in_page >= p.page_size / kTreeBN) in_page = 0;
    if (j == min(w.jb + 1, w.je - 1)) {  // the next item, while copies of this one are in flight
      nx = w;
      has_next = nx.next(p);
      ids_first = has_next ? fetch(p, nx, nx.jb) : -1;
    }
    if (++j == w.je) {
      w = nx;
      has = has_next;
      if (has) enter(p);
    }
    return true;
  }
};

template <int DH, int STAGES>
__device__ __forceinline__ void tree_load(const TreeArgs& p, const TreeWalker& w, const Guard& guard, const CUtensorMap* tm,
                                          uint32_t ring, uint32_t full0, uint32_t empty0, uint32_t info) {
  TreeLoads<DH> s;
  s.start(p, w);
  int st = 0;
  uint32_t ph = 1;
  while (s.has) {
    if (!s.step(p, guard, tm, ring + st * (kTreeBN * DH * 2), full0 + 8u * st, empty0 + 8u * st, ph, info | (uint32_t)st)) return;
    if (++st == STAGES) {
      st = 0;
      ph ^= 1u;
    }
  }
}

// A run's O, taken over: total = a total + O (a 0: total holds nothing yet), and those of the
// runs before an item's last one, put back: O += a total.
template <int DH>
static __device__ __noinline__ void tree_take_run(uint32_t t_o, float* total, float a) {
#pragma unroll 1
  for (int c = 0; c < DH; c += 32) {
    float v[32];
    tmem_load32(t_o + c, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) total[c + i] = a == 0.0f ? v[i] : fmaf(total[c + i], a, v[i]);
  }
}
template <int DH>
static __device__ __noinline__ void tree_add_runs(uint32_t t_o, const float* total, float a) {
#pragma unroll 1
  for (int c = 0; c < DH; c += 32) {
    float v[32];
    tmem_load32(t_o + c, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaf(total[c + i], a, v[i]);
    tmem_store32(t_o + c, v);
  }
  tmem_store_wait();
}

// tmQ {Dh, H, T}, boxes of 64 x group x (tokens of a tile); tmK, tmV {Dh, page_size,
// Hkv, pages}, boxes of 64 x chunk x 1 x 1; 128-byte swizzle.
// LONG: bf16 output, where a sequence may have more than kTreeLong keys.
template <int DH, bool OUT_F32, bool LONG>
__global__ void __launch_bounds__(kTreeThreads, 1)
    k_tree_attn(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const TreeArgs p) {
  constexpr int PARTS = OUT_F32 ? 3 : 1;
  using Cfg = TreeCfg<DH, PARTS>;
  constexpr int KS = Cfg::kKStages, VS = Cfg::kVStages, SB = Cfg::kSBufs, COLS = Cfg::kSCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_addr(smem), sK = sQ + 2 * Cfg::kTile, sV = sK + KS * Cfg::kTile;
  uint8_t* tail = smem + (2 + KS + VS) * Cfg::kTile;  // 1 KB
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  long long* scratch = reinterpret_cast<long long*>(tail + 320);
  long long* found = scratch + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(found + 2);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  // [4]: it + 1 where the share's item `it`, in place it & 3, met new tokens whose V is not
  // finite
  volatile uint32_t* odd_v = tmem_slot + 2;
  static_assert(Cfg::kBars * 8 <= 320 && 320 + 34 * 8 + 24 <= 1024, "the last kilobyte");
  const int warp = (int)threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  // k_full, k_empty, v_full, v_empty, q_full[2] (of items in turn), then of the S/P buffers
  // s_full, p_full, pv_done, then o_empty
  const uint32_t bar0 = smem_addr(bars);
  const uint32_t k_full = bar0, k_empty = k_full + 8 * KS, v_full = k_empty + 8 * KS, v_empty = v_full + 8 * VS;
  const uint32_t q_full = v_empty + 8 * VS, s_full = q_full + 16, p_full = s_full + 8 * SB, pv_done = p_full + 8 * SB;
  const uint32_t o_empty = pv_done + 8 * SB;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(q_full + 8 * i, 1);
    for (int i = 0; i < SB; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);  // the softmax warps
      mbar_init(pv_done + 8 * i, 1);
    }
    mbar_init(o_empty, 4);
    *abort_flag = 0u;
    for (int i = 0; i < 4; ++i) odd_v[i] = 0u;
    found[0] = found[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 2) {
    tmem_alloc<1>(smem_addr(tmem_slot), 512);
    tmem_relinquish<1>();
  }
  early_wait();
  if (blockIdx.x == 0) tree_check(p);
  // this CTA's share
  auto count = [&](int v) -> long long {
    TreeSeq s;
    s.load(p, v);
    return s.per_head * p.Hkv;
  };
  tc_fence_before_sync();
  BlockCount<long long, kTreeThreads> counted;
  const long long W = counted.total(p.lines * p.B, count, scratch);
  tc_fence_after_sync();
  const int G = (int)max(1ll, min((long long)gridDim.x, W));
  const Share<long long> share(W, G, p.lines == 2 ? (int)min((long long)kTreeLead, W / G / 2) : 0);
  long long lo = 0, hi = 0;
  if ((int)blockIdx.x < share.G) {
    lo = share.lo((int)blockIdx.x);
    hi = share.lo((int)blockIdx.x + 1);
  }
  if (lo < hi) counted.locate(p.lines * p.B, count, lo, scratch, found);
  __syncthreads();
  const uint32_t tmem_base = *tmem_slot;
  const Guard guard{p.ws, abort_flag, p.timeout_ns};
  TreeWalker w;
  w.init(p, lo, hi, (int)found[0], found[1]);
  if (!p.split && lo < hi) {
    // Whole items only: those that begin in the share.
    TreeWalker e = w;
    if (w.item < w.x) {  // the first one began earlier
      e.next(p);
      e.x = e.item + e.nb;
      w = e;
    }
    // the end: where the item that holds block hi - 1 ends
    long long end = hi;
    if (w.x < hi) {
      e = w;
      while (e.next(p)) end = e.item + e.nb;
    }
    w.hi = w.x < hi ? end : w.x;
  }

  if (warp == 0) {
    tree_load<DH, KS>(p, w, guard, &tmK, sK, k_full, k_empty, kRoleProducer << 16);
  } else if (warp == 3) {
    tree_load<DH, VS>(p, w, guard, &tmV, sV, v_full, v_empty, (kRoleProducer << 16) | 0x10);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kTreeBM, kTreeBN, false, false);
      int ks = 0, b = 0;
      uint32_t kph = 0, bph = 0, it = 0;
      bool used = false, ok = true;  // used: every buffer has been
      for (; ok && w.next(p); ++it) {
        const uint32_t qb = it & 1u;
        if (!tree_wait(guard, q_full + 8 * qb, (it >> 1) & 1u, (kRoleMma << 16) | 0x800 | qb)) break;
        const uint32_t q_at = sQ + qb * Cfg::kTile;
        for (int j = w.jb; j < w.je; ++j) {
          // the buffer's last P has been read, and K is there
          if ((used && !tree_wait(guard, pv_done + 8 * b, bph ^ 1u, (kRoleMma << 16) | 0x400 | b)) ||
              !tree_wait(guard, k_full + 8 * ks, kph, (kRoleMma << 16) | ks)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t k_at = sK + ks * Cfg::kTile, d = tmem_base + (uint32_t)(COLS * b);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t o = (uint32_t)((kk >> 2) * (kTreeBN * 128) + (kk & 3) * 32);
            umma_bf16<1>(d, sdesc_sw128(q_at + o, 16, 1024), sdesc_sw128(k_at + o, 16, 1024), idesc, kk != 0 ? 1u : 0u);
          }
          umma_commit(s_full + 8 * b);
          umma_commit(k_empty + 8 * ks);
          if (++ks == KS) {
            ks = 0;
            kph ^= 1u;
          }
          if (++b == SB) {
            b = 0;
            bph ^= 1u;
            used = true;
          }
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ O += P V
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kTreeBM, DH, false, true);
      int vs = 0, b = 0;
      uint32_t vph = 0, bph = 0, oph = 1;
      bool ok = true;
      while (ok && w.next(p)) {
        for (int j = w.jb; j < w.je; ++j) {
          if (!tree_wait(guard, v_full + 8 * vs, vph, (kRoleMma << 16) | 0x10 | vs) ||
              (j == w.jb && !tree_wait(guard, o_empty, oph, (kRoleMma << 16) | 0x300)) ||
              !tree_wait(guard, p_full + 8 * b, bph, (kRoleMma << 16) | 0x200 | b)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // 16 keys: 8 columns of P, 2 KB of V
          const uint64_t vd = sdesc_sw128(sV + vs * Cfg::kTile, kTreeBN * 128, 1024);
          const uint32_t a = tmem_base + (uint32_t)(COLS * b), d = tmem_base + Cfg::kTmemO;
          if constexpr (PARTS == 3) {  // the smallest parts first: what is cut off goes by the sum so far
#pragma unroll
            for (int kk = 0; kk < kTreeBN / 16; ++kk)
              umma_bf16_ts(d, a + (uint32_t)(kTreeBN + kk * 8), vd + (uint32_t)(kk * 128), idesc, kk != 0 ? 1u : 0u);
#pragma unroll
            for (int kk = 0; kk < kTreeBN / 16; ++kk)
              umma_bf16_ts(d, a + (uint32_t)(kk * 16 + 8), vd + (uint32_t)(kk * 128), idesc, 1u);
          }
#pragma unroll
          for (int kk = 0; kk < kTreeBN / 16; ++kk)
            umma_bf16_ts(d, a + (uint32_t)(PARTS == 3 ? kk * 16 : (kk >> 1) * 32 + (kk & 1) * 8), vd + (uint32_t)(kk * 128), idesc,
                        (PARTS == 3 || (LONG ? (j - w.jb) % kTreeRun != 0 : j > w.jb) || kk != 0) ? 1u : 0u);
          umma_commit(pv_done + 8 * b);
          umma_commit(v_empty + 8 * vs);
          if (++vs == VS) {
            vs = 0;
            vph ^= 1u;
          }
          if (++b == SB) {
            b = 0;
            bph ^= 1u;
          }
        }
        oph ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, output
    const int q = warp & 3;
    const int row = q * 32 + (int)lane;
    const uint32_t t_lane = tmem_base + ((uint32_t)(q * 32) << 16);
    const uint32_t t_o = t_lane + Cfg::kTmemO;
    const int my_tok = row / p.group, my_head = row - my_tok * p.group;
    const float cs = p.cs;
    const long long x_first = w.x;
    int b = 0;                     // S/P buffer of the next product,
    uint32_t bph = 0;              // its parity,
    int last_b = 0;                // and those of the product before
    uint32_t last_ph = 0, it = 0;  // (it: items of the share)
    bool wrote_cut = false, ok = true;
    auto load_q = [&](const TreeWalker& x, uint32_t qb) {
      if (q == 0 && lane == 0) {
        mbar_arrive_expect_tx(q_full + 8 * qb, (uint32_t)(DH / 64 * 128 * p.group * p.tokens));
        for (int hf = 0; hf < DH / 64; ++hf)
          tma_load_3d(sQ + qb * Cfg::kTile + hf * (kTreeBM * 128), &tmQ, q_full + 8 * qb, hf * 64, x.h * p.group, x.token0);
      }
    };
    bool has = w.next(p);
    if (has) load_q(w, 0);
    TreeWalker nx = w;
    bool has_next = false;
    for (; ok && has; w = nx, has = has_next, ++it) {
      const int rows = w.ntok * p.group;
      // the next item's Q, into the other buffer: the item before this one is over
      nx = w;
      has_next = nx.next(p);
      if (has_next) load_q(nx, (it + 1u) & 1u);
      const bool active = q * 32 < rows;  // (of the whole warp)
      const int ti = w.s.token(p, w.t) + my_tok;
      float m = -INFINITY, l = 0.0f;
      // what has been taken from O so far, relative to the maximum m_total (fp32: in registers;
      // runs: in local memory)
      float total[PARTS == 3 || LONG ? DH : 1];
      float m_total = -INFINITY;
      if constexpr (PARTS == 3) {
#pragma unroll
        for (int i = 0; i < DH; ++i) total[i] = 0.0f;
      }
      int run = w.jb;
    next_run:
      for (int j = LONG ? run : w.jb; j < (LONG ? min(run + kTreeRun, w.je) : w.je); ++j) {
        const bool inner = (j + 1) * kTreeBN <= w.s.ctx;  // every row sees every key
        if (!__all_sync(0xffffffffu, tree_wait(guard, s_full + 8 * b, bph, (kRoleEpilogue << 16) | b))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t t_s = t_lane + (uint32_t)(COLS * b);
        if (active) {
          // 64 keys at a time (fp32 output: fewer, for the registers of its parts and sums), in
          // a loop: code that fits the instruction cache's first level (unrolled over the block,
          // a warp waited for instructions a fourth of the time).  P goes over the scores: of
          // 32 keys the first 16 columns are bf16 pairs; for fp32 output of 16 keys the first
          // 8, then 8 of what those leave, and what both leave goes behind the scores.
          constexpr int WIDTH = Cfg::kWidth;
          uint32_t vis[4] = {0u, 0u, 0u, 0u};
          if (!inner && row < rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i) vis[i] = tree_visible(p, w.s, ti, j * kTreeBN - w.s.ctx + 32 * i);
          }
          float sum = 0.0f;
#pragma unroll 1
          for (int c = 0; c < kTreeBN / WIDTH; ++c) {
            const uint32_t t_c = t_s + WIDTH * c;
            uint32_t v0 = c == 0 ? vis[0] : vis[2], v1 = c == 0 ? vis[1] : vis[3];
            if constexpr (PARTS == 3) {
              const int key = WIDTH * c;
              v0 = (key < 64 ? key < 32 ? vis[0] : vis[1] : key < 96 ? vis[2] : vis[3]) >> (key & 31);
            }
            float x[WIDTH];
            auto load = [&]() {
              if constexpr (WIDTH == 16) tree_tmem_load16(t_c, x);
#pragma unroll
              for (int d = 0; d < WIDTH / 32; ++d) tree_tmem_load32(t_c + 32 * d, x + 32 * d);
              tree_tmem_load_wait<WIDTH>(x);
            };
            // the largest cs S that the row sees of these keys, rounded up: maxima are whole
            // numbers, so that a change of one scales by a power of two, exactly
            auto maximum = [&]() {
              float e[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              if (inner) {
#pragma unroll
                for (int i = 0; i < WIDTH; ++i) e[i & 3] = fmaxf(e[i & 3], __fmul_rn(x[i], cs));
              } else {
#pragma unroll
                for (int i = 0; i < WIDTH; ++i) e[i & 3] = (i < 32 ? v0 : v1) & (1u << (i & 31)) ? fmaxf(e[i & 3], __fmul_rn(x[i], cs)) : e[i & 3];
              }
              return ceilf(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])));
            };
            load();
            // A row without a maximum yet (its first keys): theirs.  Its O is zero so far, or
            // is overwritten.
            if (__any_sync(0xffffffffu, m == -INFINITY && row < rows)) {
              const float mx = maximum();
              if (m == -INFINITY) m = mx;
            }
            uint32_t hi[PARTS == 3 ? WIDTH : WIDTH / 2], lo[WIDTH / 2];
            auto probabilities = [&]() -> float {
              // (no key seen yet, or none whose score is above -inf: P zero)
              const float top = m == -INFINITY ? 0.0f : m;
              float rs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              if (__all_sync(0xffffffffu, fabsf(top) < 1.0e6f || row >= rows)) {
#pragma unroll
                for (int i = 0; i < WIDTH / 2; ++i) fma_f32x2(x[2 * i], x[2 * i + 1], cs, -top);
              } else {
                // scores that pass 2^24 take the rounded product, so that the largest one's difference
                // is 0: a choice of the row, or its bits would depend on the other rows of its warp
                const bool far = !(fabsf(top) < 1.0e6f);
                const float by = far ? cs : 1.0f, rest = far ? 1.0f : cs;
#pragma unroll
                for (int i = 0; i < WIDTH; ++i) x[i] = __fmaf_rn(__fmul_rn(x[i], by), rest, -top);
              }
              if (!inner) {
#pragma unroll
                for (int i = 0; i < WIDTH; ++i) x[i] = (i < 32 ? v0 : v1) & (1u << (i & 31)) ? x[i] : -INFINITY;
              }
#pragma unroll
              for (int i = 0; i < WIDTH / 2; ++i) {
                float& x0 = x[2 * i];
                float& x1 = x[2 * i + 1];
                x0 = ex2_ftz(x0);
                x1 = ex2_ftz(x1);
                add_f32x2(rs[2 * (i & 1)], rs[2 * (i & 1) + 1], x0, x1);
                if constexpr (PARTS == 3) {  // (the differences are exact; of 16 keys eight first parts, then eight second ones)
                  uint32_t &y = hi[i + (i & 8)], &z = hi[i + (i & 8) + 8];
                  y = pack_bf16x2(x0, x1);
                  const float r0 = x0 - __uint_as_float(y << 16), r1 = x1 - __uint_as_float(y & 0xffff0000u);
                  z = pack_bf16x2(r0, r1);
                  lo[i] = pack_bf16x2(r0 - __uint_as_float(z << 16), r1 - __uint_as_float(z & 0xffff0000u));
                } else {
                  hi[i] = pack_bf16x2(x0, x1);
                }
              }
              return (rs[0] + rs[1]) + (rs[2] + rs[3]);
            };
            float part = probabilities();
            // Every P is positive: a sum of at most 2^8 proves that none exceeds it and the
            // maximum need not be looked for.
            if (!__all_sync(0xffffffffu, part <= kTreeGrowSum || row >= rows)) {
              load();
              const float mx = maximum();
              const bool grow = mx > m + kTreeGrow && row < rows;
              if (__any_sync(0xffffffffu, grow)) {
                const float alpha = grow ? ex2_ftz(m - mx) : 1.0f;
                if (grow) {
                  l *= alpha;
                  sum *= alpha;
                  m = mx;
                }
                if (PARTS == 1 && j > (LONG ? run : w.jb)) {  // (a run's first PV product overwrites O)
                  if (!__all_sync(0xffffffffu, tree_wait(guard, pv_done + 8 * last_b, last_ph, (kRoleEpilogue << 16) | 0x100))) {
                    ok = false;
                    break;
                  }
                  tc_fence_after_sync();
#pragma unroll 1
                  for (int d = 0; d < DH / 32; ++d) {
                    float v[32];
                    tmem_load32(t_o + d * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= alpha;
                    tmem_store32(t_o + d * 32, v);
                  }
                }
                // the block's P so far, with the old maximum: the columns of every step (of which
                // bf16 output uses half), and of the third parts half as many.  The steps before
                // have stored it, and only this wait puts those stores before the loads.
                if (c > 0) tmem_store_wait();
                if constexpr (PARTS == 1) {
                  auto rescale = [&](uint32_t at) {
                    float v[32];
                    tmem_load32(at, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                      const uint32_t y = __float_as_uint(v[i]);
                      v[i] = __uint_as_float(pack_bf16x2(__uint_as_float(y << 16) * alpha, __uint_as_float(y & 0xffff0000u) * alpha));
                    }
                    tmem_store32(at, v);
                  };
#pragma unroll 1
                  for (int d = 0; d < c * (WIDTH / 32); ++d) rescale(t_s + 32 * d);
                } else {
                  auto rescale = [&](uint32_t at) {
                    float v[16];
                    tree_tmem_load16(at, v);
                    tree_tmem_load_wait<16>(v);
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      y[i] = pack_bf16x2(__uint_as_float(__float_as_uint(v[i]) << 16) * alpha, __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u) * alpha);
                    tree_tmem_store16(at, y);
                  };
#pragma unroll 1
                  for (int d = 0; d < c * (WIDTH / 16); ++d) rescale(t_s + 16 * d);
#pragma unroll 1
                  for (int d = 0; 2 * d < c * (WIDTH / 16); ++d) rescale(t_s + kTreeBN + 16 * d);  // (of this step too, which are written anew)
                }
                tmem_store_wait();
              }
              part = probabilities();
            }
            sum += part;
            if constexpr (PARTS == 3) {
#pragma unroll
              for (int d = 0; d < WIDTH / 16; ++d) tree_tmem_store16(t_c + 16 * d, hi + 16 * d);
              if constexpr (WIDTH == 16) tree_tmem_store8(t_s + kTreeBN + 8 * c, lo);
              else tree_tmem_store16(t_s + kTreeBN + 16 * c, lo);
            } else {
#pragma unroll
              for (int d = 0; d < WIDTH / 32; ++d) tree_tmem_store16(t_c + 32 * d, hi + 16 * d);
            }
          }
          if (!ok) break;
          l += sum;
          tmem_store_wait();
          if constexpr (PARTS == 3) {
            // O of the block before this one, relative to m_total as what it is added to is; the
            // next product, which overwrites it, waits for this warp
            if (j > w.jb) {
              if (!__all_sync(0xffffffffu, tree_wait(guard, pv_done + 8 * last_b, last_ph, (kRoleEpilogue << 16) | 0x700))) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
#pragma unroll
              for (int c = 0; c < DH / 32; ++c) {
                float v[32];
                tree_tmem_load32(t_o + c * 32, v);
                tree_tmem_load_wait<32>(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) add_f32x2(total[c * 32 + 2 * i], total[c * 32 + 2 * i + 1], v[2 * i], v[2 * i + 1]);
              }
              if (__any_sync(0xffffffffu, m != m_total)) {
                const float a = m == m_total ? 1.0f : ex2_ftz(m_total - m);
#pragma unroll
                for (int i = 0; i < DH; ++i) total[i] *= a;
              }
            }
            m_total = m;
          }
        }
        if (!inner) {
          // V: clear the block's keys behind the sequence and what is not finite of the new
          // tokens; thread = key.  These warps wait for V here only, and a parity tells two
          // phases apart: the stage's last use has to be over.  PV of SB blocks ago is (its
          // buffer holds this S), and two stages need that of two.
          const long long g = w.item + j - x_first;  // the share's blocks use the stages in turn
          static_assert(VS >= 2 && (VS == 2 || VS >= SB), "stages of V");
          if (VS == 2 && g >= 2 &&
              !__all_sync(0xffffffffu, tree_wait(guard, pv_done + 8 * (int)((g - 2) % SB), (uint32_t)((g - 2) / SB) & 1u, (kRoleEpilogue << 16) | 0x600))) {
            ok = false;
            break;
          }
          const int vs = (int)(g % VS);
          if (!__all_sync(0xffffffffu, tree_wait(guard, v_full + 8 * vs, (uint32_t)(g / VS) & 1u, (kRoleEpilogue << 16) | 0x500 | vs))) {
            ok = false;
            break;
          }
          const int key = j * kTreeBN + row;
          if (key >= w.s.ctx) {
            const bool out = key >= w.keys;
            bool odd = false;
            for (int hf = 0; hf < DH / 64; ++hf) {
              const uint32_t at = sV + vs * Cfg::kTile + (uint32_t)(hf * (kTreeBN * 128) + row * 128);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint32_t a16 = at + (uint32_t)((c ^ (row & 7)) << 4);  // (the eight words in an order without bank conflicts)
                if (out) {
                  st_shared_v4(a16, 0u, 0u, 0u, 0u);
                } else {
                  uint32_t x[4];
                  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                               : "r"(a16)
                               : "memory");
                  bool bad = false;
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    if ((x[i] & 0x7f80u) == 0x7f80u) {
                      x[i] &= 0xffff0000u;
                      bad = true;
                    }
                    if ((x[i] & 0x7f800000u) == 0x7f800000u) {
                      x[i] &= 0x0000ffffu;
                      bad = true;
                    }
                  }
                  if (bad) st_shared_v4(a16, x[0], x[1], x[2], x[3]);
                  odd |= bad;
                }
              }
            }
            if (odd) odd_v[it & 3u] = it + 1u;
          }
          fence_proxy_async_smem();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * b);
        last_b = b;
        last_ph = bph;
        if (++b == SB) {
          b = 0;
          bph ^= 1u;
        }
      }
      if (!ok) break;
      // (each lane: odd_v was written before the products were issued)
      if (!__all_sync(0xffffffffu, tree_wait(guard, pv_done + 8 * last_b, last_ph, (kRoleEpilogue << 16) | 0x300 | last_b))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if constexpr (LONG) {
        if (run + kTreeRun < w.je) {
          if (active) {
            tree_take_run<DH>(t_o, total, run == w.jb ? 0.0f : m_total == m ? 1.0f : ex2_ftz(m_total - m));
            m_total = m;
          }
          run += kTreeRun;
          goto next_run;
        }
        if (active && run > w.jb) tree_add_runs<DH>(t_o, total, m_total == m ? 1.0f : ex2_ftz(m_total - m));
      }
      if (PARTS == 3 && active && w.je - w.jb > 1) {
#pragma unroll
        for (int c = 0; c < (PARTS == 3 ? DH / 32 : 0); ++c) {
          float v[32];
          tmem_load32(t_o + c * 32, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += total[c * 32 + i];
          tmem_store32(t_o + c * 32, v);
        }
        tmem_store_wait();
      }
      if (active) {
        const bool whole = w.jb == 0 && w.je == w.nb;
        const bool odd = odd_v[it & 3u] > it;  // (a later item's: looked into too)
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const long long at = (long long)(w.token0 + my_tok) * p.ldo + (long long)(w.h * p.group + my_head) * DH;
        float* slot = whole ? nullptr : p.slots + (size_t)(2 * blockIdx.x + (w.jb == 0 ? 1 : 0)) * kTreeSlotFloats;
#pragma unroll 1
        for (int c = 0; c < DH / 32; ++c) {
          float v[32];
          tmem_load32(t_o + c * 32, v);
          if (row < rows) {
            if (odd) {
              // new tokens of this fragment's blocks whose V is not finite, where the row sees them
              for (int key = max(w.s.ctx, w.jb * kTreeBN); key < min(w.keys, w.je * kTreeBN); ++key) {
                if (!(tree_visible(p, w.s, ti, key - w.s.ctx) & 1u)) continue;
                const int pg = __ldg(p.table + (long long)w.s.b * p.ldt + min(key / p.page_size, p.max_pages - 1));
                if (pg < 0 || pg >= p.num_pages) continue;
                const __nv_bfloat16* vr = p.v + pg * p.page_stride + (key % p.page_size) * p.token_stride + w.h * p.head_stride + c * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float y = __bfloat162float(vr[i]);
                  if (!(fabsf(y) <= 3.4e38f)) v[i] += y;
                }
              }
            }
            if (whole) {
              if (l == 0.0f) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.0f;  // the row sees nothing
              }
              if constexpr (OUT_F32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.O) + at + c * 32);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + at + c * 32);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  dst[i] = make_uint4(pack_bf16x2(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16x2(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                      pack_bf16x2(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack_bf16x2(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
              }
            } else {
              float4* part = reinterpret_cast<float4*>(slot);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                __stcg(part + (c * 8 + i) * kTreeBM + row, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
            }
          }
        }
        if (!whole && row < rows) {
          __stcg(slot + 128 * kTreeBM + row, m);
          __stcg(slot + 128 * kTreeBM + kTreeBM + row, l);
        }
        if (!whole && w.jb == 0 && row == 0) {
          p.cuts[blockIdx.x] = TreeCut{share.owner(w.item + w.nb - 1) - (int)blockIdx.x + 1, w.token0, w.h * p.group, w.ntok};
          wrote_cut = true;
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_empty);
      }
    }
    if (p.split && row == 0 && !wrote_cut) p.cuts[blockIdx.x].pieces = 0;
  }
  tc_fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    for (int i = 0; i < 200; ++i) __nanosleep(1000);  // copies and products still in flight land first
  }
  tc_fence_after_sync();
  if (warp == 2) tmem_dealloc<1>(tmem_base, 512);
}

// The cut items' pieces added up: blockIdx.x is the CTA in whose share an item begins.  A
// thread takes four components of a row and every `ways`-th piece (all of them, where the
// rows alone fill the blocks), then the first of them adds up what the ways have found.
template <int DH, bool OUT_F32>
__global__ void __launch_bounds__(256) k_tree_merge(const TreeArgs p) {
  early_wait();
  const TreeCut cut = p.cuts[blockIdx.x];
  const int rows = cut.ntok * p.group;
  if (cut.pieces == 0) return;
  int ways = 1;
  while (ways < 8 && 2 * ways * rows <= kTreeBM && ways < cut.pieces) ways *= 2;
  const int per = 32 / ways;  // quads of rows of a warp
  const int way = (int)lane_id() / per, i = (int)(blockIdx.y * 8 + threadIdx.x / 32) * per + (int)lane_id() % per;
  const int quad = i / rows, row = i - quad * rows;
  const bool on = quad < DH / 4;
  auto slot = [&](int k) { return p.slots + (size_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * kTreeSlotFloats; };
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (on) {
    // four pieces' numbers in flight
    for (int k0 = way; k0 < cut.pieces; k0 += 4 * ways) {
      float mk[4], lk[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mk[k] = -INFINITY;
        lk[k] = 0.0f;
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k0 + k * ways < cut.pieces) {
          const float* s = slot(k0 + k * ways);
          mk[k] = __ldcg(s + 128 * kTreeBM + row);
          lk[k] = __ldcg(s + 128 * kTreeBM + kTreeBM + row);
          v[k] = __ldcg(reinterpret_cast<const float4*>(s) + quad * kTreeBM + row);
        }
      }
      const float top = fmaxf(fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])), m);
      const float ms = top == -INFINITY ? 0.0f : top;
      const float self = ex2_ftz(m - ms);
      l *= self;
      o.x *= self;
      o.y *= self;
      o.z *= self;
      o.w *= self;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = ex2_ftz(mk[k] - ms);
        l = fmaf(a, lk[k], l);
        o.x = fmaf(a, v[k].x, o.x);
        o.y = fmaf(a, v[k].y, o.y);
        o.z = fmaf(a, v[k].z, o.z);
        o.w = fmaf(a, v[k].w, o.w);
      }
      m = top;
    }
  }
  for (int d = per; d < 32; d *= 2) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, d), lo = __shfl_xor_sync(0xffffffffu, l, d);
    const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, o.x, d), __shfl_xor_sync(0xffffffffu, o.y, d),
                                 __shfl_xor_sync(0xffffffffu, o.z, d), __shfl_xor_sync(0xffffffffu, o.w, d));
    const float top = fmaxf(m, mo), ms = top == -INFINITY ? 0.0f : top;
    const float a = ex2_ftz(m - ms), c = ex2_ftz(mo - ms);
    m = top;
    l = l * a + lo * c;
    o = make_float4(o.x * a + y.x * c, o.y * a + y.y * c, o.z * a + y.z * c, o.w * a + y.w * c);
  }
  if (!on || way > 0) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const bool none = l == 0.0f;
  const int tok = row / p.group, head = row - tok * p.group;
  const long long at = (long long)(cut.token0 + tok) * p.ldo + (long long)(cut.head0 + head) * DH + quad * 4;
  const float y0 = none ? 0.0f : o.x * inv, y1 = none ? 0.0f : o.y * inv, y2 = none ? 0.0f : o.z * inv, y3 = none ? 0.0f : o.w * inv;
  if constexpr (OUT_F32) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = make_float4(y0, y1, y2, y3);
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) = make_uint2(pack_bf16x2(y0, y1), pack_bf16x2(y2, y3));
}

}  // namespace wst
