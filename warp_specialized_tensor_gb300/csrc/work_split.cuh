// work_split.cuh -- equal shares of a sequence of blocks, for kernels whose items
// (tiles, heads of a sequence) have lengths that only the device knows.
//
// The items' blocks stand in one line of W blocks; CTA c of G takes blocks
// [floor(c W / G), floor((c + 1) W / G)).  An item that lies in several shares is
// worked on in pieces, one per CTA, in ascending order of both.
#pragma once

#include <cstdint>

namespace wst {

struct Share {
  long long W;
  int G;
  __device__ __forceinline__ long long lo(int c) const { return (long long)c * W / G; }
  // the CTA that holds block x
  __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * G - 1) / W); }
};

// The sum of count(i) over i < n, by the whole block (all threads; scratch: 33
// words of shared memory).  Ends with a barrier.
template <int THREADS, class Count>
__device__ __forceinline__ long long block_total(int n, const Count& count, long long* scratch) {
  static_assert(THREADS % 32 == 0 && THREADS <= 1024, "whole warps");
  long long v = 0;
  for (int i = (int)threadIdx.x; i < n; i += THREADS) v += count(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) total += scratch[w];
  __syncthreads();
  return total;
}

// The i whose blocks hold block x (0 <= x < total), and the sum of the counts
// before it.  All threads; found: two words of shared memory.  Ends with a barrier.
template <int THREADS, class Count>
__device__ __forceinline__ void block_locate(int n, const Count& count, long long x, long long* scratch, long long* found) {
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  long long before = 0;
  for (int base = 0; base < n && before <= x; base += THREADS) {
    const int i = base + (int)threadIdx.x;
    const long long v = i < n ? count(i) : 0;
    long long sum = v;  // inclusive, inside the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long other = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += other;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    long long ahead = before, all = before;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) ahead += scratch[w];
      all += scratch[w];
    }
    const long long at = ahead + sum - v;
    if (at <= x && x < at + v) {
      found[0] = i;
      found[1] = at;
    }
    before = all;
    __syncthreads();
  }
}

}  // namespace wst
