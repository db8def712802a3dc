// moe_plan.cu -- the rows of a grouped product from a routing table on the
// GPU: a stable counting sort of the (token, slot) pairs by expert.
//
// Pair p = t * top_k + i goes to expert experts[p] (-1: to none).  Row r of the
// expert-major order holds pair row_pair[r] of token row_token[r]; position[p]
// is the row of pair p (-1: none); rows of expert e are
// [offsets[e], offsets[e+1]), pair ids ascending inside an expert, so the
// result does not depend on the order in which blocks run.
//
// Up to kPlanOne pairs one block does everything.  More pairs are cut into at
// most kPlanChunks chunks: one launch counts each chunk's pairs per expert, a
// second one adds the counts of the chunks before its own (each block reads
// the whole table of chunks x experts, at most 128 x 1024 counts from L2) and
// places its pairs.  Inside a block every warp owns a consecutive part of the
// chunk and ranks 32 pairs at a time by ballots over the warp.  A chain of
// dependent reads bounds it: 131072 pairs and 256 experts take 15 us on GB300,
// 256 pairs (one block) 3.4 us.
#include <algorithm>

#include "wst.h"
#include "wst_common.cuh"
#include "wst_host.h"

namespace wst {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanOne = 2048;
constexpr int kPlanChunk = 1024;
constexpr int kPlanChunks = 128;
constexpr int kPlanMaxExperts = 1024;

struct PlanArgs {
  int pairs, top_k, E;
  int bits;          // of an expert id
  int chunk;         // pairs per block, a multiple of 32 * kPlanWarps
  const int* experts;
  int* offsets;
  int* row_pair;
  int* row_token;
  int* position;
  int* counts;       // [blocks][E], NULL with one block
  WsHeader* ws;
};

// Expert of pair p, -1 for none; a bad id counts as none.
__device__ __forceinline__ int plan_expert(const PlanArgs& a, int p, int end, bool latch) {
  if (p >= end) return -1;
  const int e = __ldg(a.experts + p);
  if (e >= 0 && e < a.E) return e;
  if (latch && e != -1) latch_error(a.ws, 1u /*WST_ERR_INVALID_ARG*/, 0x60000u);
  return -1;
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_count(const PlanArgs a) {
  extern __shared__ int sm[];
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) sm[e] = 0;
  __syncthreads();
  const int p0 = (int)blockIdx.x * a.chunk;  // (pairs + chunk fits 32 bits)
  const int p1 = min(p0 + a.chunk, a.pairs);
#pragma unroll 4
  for (int p = p0 + (int)threadIdx.x; p < p1; p += kPlanThreads) {
    const int e = plan_expert(a, p, p1, false);
    if (e >= 0) atomicAdd(&sm[e], 1);  // integers: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.counts[(long long)blockIdx.x * a.E + e] = sm[e];
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_place(const PlanArgs a) {
  // [kPlanWarps][E] counts, then first rows, of each warp's part; [E] offsets
  extern __shared__ int sm[];
  __shared__ int warp_total[kPlanWarps];
  int* offs = sm + kPlanWarps * a.E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = (int)blockIdx.x * a.chunk;
  const int p1 = min(p0 + a.chunk, a.pairs);
  const int part = a.chunk / kPlanWarps;
  const int w0 = p0 + warp * part;
  const int w1 = min(w0 + part, p1);
  for (int i = threadIdx.x; i < kPlanWarps * a.E; i += kPlanThreads) sm[i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int p = w0 + lane; p < w1; p += 32) {
    const int e = plan_expert(a, p, w1, true);
    if (e >= 0) atomicAdd(&sm[warp * a.E + e], 1);
  }
  __syncthreads();
  // Total of each expert, and of the chunks before this one: `per` threads share
  // an expert's chunks (all threads where there are few experts).
  int per = 1;
  while (per < 8 && per * 2 * a.E <= kPlanThreads) per *= 2;
  for (int i0 = warp * 32; i0 < a.E * per; i0 += kPlanThreads) {
    // (whole warps; the threads of an expert are neighbours)
    const int e = (i0 + lane) / per, part_of = lane & (per - 1);
    int before = 0, total = 0;
    if (e < a.E) {
      if (a.counts) {
#pragma unroll 16
        for (int c = part_of; c < (int)gridDim.x; c += per) {
          const int n = __ldg(a.counts + c * a.E + e);
          total += n;
          if (c < (int)blockIdx.x) before += n;
        }
      } else if (part_of == 0) {
        for (int w = 0; w < kPlanWarps; ++w) total += sm[w * a.E + e];
      }
    }
    __syncwarp();
    for (int o = 1; o < per; o <<= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if (e < a.E && part_of == 0) {
      offs[e] = total;
      for (int w = 0; w < kPlanWarps; ++w) {
        const int n = sm[w * a.E + e];
        sm[w * a.E + e] = before;
        before += n;
      }
    }
  }
  __syncthreads();
  // Exclusive scan of the totals, kPlanThreads experts at a time.
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += kPlanThreads) {
    const int e = e0 + (int)threadIdx.x;
    const int n = e < a.E ? offs[e] : 0;
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_total[warp] = v;
    __syncthreads();
    int base = carry;
    for (int w = 0; w < warp; ++w) base += warp_total[w];
    if (e < a.E) offs[e] = base + v - n;
    for (int w = 0; w < kPlanWarps; ++w) carry += warp_total[w];
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.offsets[e] = offs[e];
    if (threadIdx.x == 0) a.offsets[a.E] = carry;
  }
  // Rows behind the last expert's hold nothing.
  for (long long r = (long long)carry + blockIdx.x * kPlanThreads + threadIdx.x; r < a.pairs;
       r += (long long)gridDim.x * kPlanThreads) {
    a.row_pair[r] = -1;
    a.row_token[r] = -1;
  }
  // Place this warp's pairs in order, 32 at a time.  The lanes with the same
  // expert are found bit by bit (ten ballots at most; a match instruction takes a
  // step for each different expert).
  int* first = sm + warp * a.E;
  for (int p = w0 + lane; p - lane < w1; p += 32) {
    const int e = plan_expert(a, p, w1, false);
    uint32_t same = __ballot_sync(0xffffffffu, e >= 0);
    for (int bit = 0; bit < a.bits; ++bit) {
      const uint32_t ones = __ballot_sync(0xffffffffu, (e >> bit) & 1);
      same &= (e >> bit) & 1 ? ones : ~ones;
    }
    const int rank = __popc(same & ((1u << lane) - 1u));
    int row = -1;
    if (e >= 0) row = offs[e] + first[e] + rank;
    __syncwarp();
    if (e >= 0 && rank == 0) first[e] += __popc(same);
    __syncwarp();
    if (p < w1) a.position[p] = row;
    if (row >= 0) {
      a.row_pair[row] = p;
      a.row_token[row] = (int)((unsigned)p / (unsigned)a.top_k);
    }
  }
}

int plan_blocks(long long pairs, int* chunk) {
  if (pairs <= kPlanOne) {
    constexpr long long unit = 32 * kPlanWarps;
    *chunk = (int)std::max(unit, (pairs + unit - 1) / unit * unit);
    return 1;
  }
  constexpr long long unit = 32 * kPlanWarps;
  const long long c = std::max<long long>(kPlanChunk, (pairs + kPlanChunks - 1) / kPlanChunks);
  *chunk = (int)((c + unit - 1) / unit * unit);
  return (int)((pairs + *chunk - 1) / *chunk);
}

}  // namespace

}  // namespace wst

using namespace wst;

#define WST_TRY(expr)                  \
  do {                                 \
    int st__ = (expr);                 \
    if (st__) return (wst_status)st__; \
  } while (0)

extern "C" {

size_t wst_moe_plan_workspace_size(int num_pairs, int num_experts) {
  if (num_pairs < 0 || num_experts < 1 || num_experts > kPlanMaxExperts) return 0;
  if (num_pairs <= kPlanOne) return kWsHeaderBytes;
  // (no fewer blocks than any smaller number of pairs takes, so that a workspace
  // serves every call up to its size)
  const long long blocks = std::min<long long>(kPlanChunks, ((long long)num_pairs + kPlanChunk - 1) / kPlanChunk);
  return kWsHeaderBytes + (size_t)blocks * num_experts * 4;
}

wst_status wst_moe_plan(int num_tokens, int top_k, const int* experts, int num_experts, int* offsets, int* row_pair,
                        int* row_token, int* position, void* workspace, size_t workspace_bytes, void* stream) {
  set_error("%s", "");
  if (num_tokens < 0 || top_k < 1 || num_experts < 1)
    return (wst_status)reject(ST_INVALID_ARG, "plan: sizes out of range (tokens=%d top_k=%d experts=%d)", num_tokens,
                              top_k, num_experts);
  if (num_experts > kPlanMaxExperts)
    return (wst_status)reject(ST_UNSUPPORTED, "plan: %d experts: this build supports up to %d", num_experts, kPlanMaxExperts);
  const long long pairs = (long long)num_tokens * top_k;
  if (pairs > 0x7fffffffLL - (1 << 25)) return (wst_status)reject(ST_INVALID_ARG, "plan: too many pairs");
  if (!offsets || !workspace || (pairs && (!experts || !row_pair || !row_token || !position)))
    return (wst_status)reject(ST_INVALID_ARG, "plan: NULL array");
  const size_t need = wst_moe_plan_workspace_size((int)pairs, num_experts);
  if (workspace_bytes < need)
    return (wst_status)reject(ST_INVALID_ARG, "plan: workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (!aligned_to(experts, 4) || !aligned_to(offsets, 4) || !aligned_to(row_pair, 4) || !aligned_to(row_token, 4) ||
      !aligned_to(position, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "plan: arrays must be 4-byte and the workspace 16-byte aligned");
  WST_TRY(check_operand(offsets, "offsets"));
  WST_TRY(check_operand(workspace, "workspace"));
  if (pairs) {
    WST_TRY(check_operand(experts, "experts"));
    WST_TRY(check_operand(row_pair, "row_pair"));
    WST_TRY(check_operand(row_token, "row_token"));
    WST_TRY(check_operand(position, "position"));
  }
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  PlanArgs a{};
  a.pairs = (int)pairs;
  a.top_k = top_k;
  a.E = num_experts;
  a.experts = experts;
  a.offsets = offsets;
  a.row_pair = row_pair;
  a.row_token = row_token;
  a.position = position;
  a.ws = static_cast<WsHeader*>(workspace);
  while ((1 << a.bits) < num_experts) ++a.bits;
  const int blocks = plan_blocks(pairs, &a.chunk);
  a.counts = blocks > 1 ? reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + kWsHeaderBytes) : nullptr;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = (size_t)(kPlanWarps + 1) * num_experts * 4;
  WST_TRY(ensure_smem_attr((const void*)k_plan_place, smem));
  if (blocks > 1) k_plan_count<<<blocks, kPlanThreads, (size_t)num_experts * 4, s>>>(a);
  k_plan_place<<<blocks, kPlanThreads, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_plan");
}

}  // extern "C"
