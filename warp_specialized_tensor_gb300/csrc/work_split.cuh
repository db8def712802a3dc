// work_split.cuh -- equal shares of a sequence of blocks, for kernels whose items
// (tiles, heads of a sequence) have lengths that only the device knows.
//
// The items' blocks stand in one line of W blocks, of which CTA c of G takes those from
// floor(c W / G) on: the shares that are one longer are spread evenly, so that with an even
// G the line's second half is cut where its first one is.  An item that lies in several
// shares is worked on in pieces, one per CTA, in ascending order of both.
#pragma once

#include <cstdint>

namespace wst {

template <class I>
struct Share {
  I W;
  int G;  // at most W (1 if W is 0)
  I q, r;
  int lead;  // blocks that the cut in the middle is late by, the ones around it in proportion; q > lead
  __device__ __forceinline__ Share(I w, int g, int lead_ = 0) : W(w), G(g), q(w / g), r(w - (w / g) * g), lead(lead_) {}
  // (r < G: 32 bits hold the product)
  __device__ __forceinline__ I lo(int c) const {
    return c * q + (I)(((uint32_t)c * (uint32_t)r + 2u * (uint32_t)lead * (uint32_t)(c < G - c ? c : G - c)) / (uint32_t)G);
  }
  // the CTA that holds block x < W: the last c with lo(c) <= x (c W <= (x + 1) G - 1)
  __device__ __forceinline__ int owner(I x) const {
    if (sizeof(I) == 4 && lead == 0) return (int)(((uint64_t)((uint32_t)x + 1u) * (uint32_t)G - 1u) / (uint32_t)W);
    int c = 0, last = G - 1;
    while (c < last) {
      const int mid = (c + last + 1) / 2;
      if (lo(mid) <= x) c = mid;
      else last = mid - 1;
    }
    return c;
  }
};

// count(i) summed over i < n by the whole block, for a share of the sum.
// scratch: 32 words of shared memory, found: two.  All threads take part.
template <class I, int THREADS>
struct BlockCount {
  static_assert(THREADS % 32 == 0 && THREADS <= 1024, "whole warps");
  I mine;  // count(threadIdx.x)

  template <class Count>
  __device__ __forceinline__ I total(int n, const Count& count, I* scratch) {
    I v = 0;
    mine = (int)threadIdx.x < n ? count((int)threadIdx.x) : (I)0;
    for (int i = (int)threadIdx.x + THREADS; i < n; i += THREADS) v += count(i);
    v += mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    I sum = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) sum += scratch[w];
    return sum;
  }

  // The i whose blocks hold block x < total, and the sum of the counts before it, into
  // `found`.  Ends with a barrier.
  template <class Count>
  __device__ __forceinline__ void locate(int n, const Count& count, I x, I* scratch, I* found) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    I before = 0;
    for (int base = 0; base < n && before <= x; base += THREADS) {
      const int i = base + (int)threadIdx.x;
      const I v = base == 0 ? mine : i < n ? count(i) : (I)0;
      I sum = v;  // inclusive, inside the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const I other = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += other;
      }
      __syncthreads();  // scratch has been read
      if (lane == 31) scratch[warp] = sum;
      __syncthreads();
      I ahead = before, all = before;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) ahead += scratch[w];
        all += scratch[w];
      }
      const I at = ahead + sum - v;
      if (at <= x && x < at + v) {
        found[0] = i;
        found[1] = at;
      }
      before = all;
    }
    __syncthreads();
  }
};

}  // namespace wst
