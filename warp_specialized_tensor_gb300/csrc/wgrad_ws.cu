// wgrad_ws.cu -- launcher and C ABI of the grouped GEMM's weight gradient.
#include <algorithm>
#include <atomic>

#include "wgrad_ws.cuh"
#include "wst.h"
#include "wst_host.h"

namespace wst {

namespace {

template <bool OUT_F32, bool ADD_BF16>
int launch_wgrad(const WgArgs& a, const void* dC, long lddc, const void* A, long lda, void* dB, long lddb, long stride_dB,
                 const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = k_wgrad_ws<OUT_F32, ADD_BF16>;
  CUtensorMap tmD, tmA, tmOut;
  int st;
  // Without a row there is nothing to load (every group is empty): the maps
  // only have to be valid.
  const bool none = a.M_total == 0;
  const uint32_t box[2] = {64, kWgBK};
  const uint64_t rows = none ? 1 : (uint64_t)a.M_total;
  uint64_t dimsD[2] = {(uint64_t)a.N, rows}, strD[1] = {(uint64_t)lddc * 2};
  uint64_t dimsA[2] = {(uint64_t)a.K, rows}, strA[1] = {(uint64_t)lda * 2};
  if ((st = encode_map(&tmD, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, none ? dB : dC, dimsD, strD, box,
                       CU_TENSOR_MAP_SWIZZLE_128B)) ||
      (st = encode_map(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, none ? dB : A, dimsA, strA, box,
                       CU_TENSOR_MAP_SWIZZLE_128B)))
    return st;
  const uint64_t es = OUT_F32 ? 4 : 2;
  uint64_t dimsO[3] = {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.G};
  uint64_t strO[2] = {(uint64_t)lddb * es, (uint64_t)(a.G > 1 ? stride_dB : (long)a.N * lddb) * es};
  const uint32_t boxO[3] = {OUT_F32 ? 32u : 64u, 32, 1};
  if ((st = encode_map(&tmOut, OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dB,
                       dimsO, strO, boxO, CU_TENSOR_MAP_SWIZZLE_128B)))
    return st;
  if ((st = ensure_smem_attr((const void*)kern, kWgSmemBytes))) return st;
  const long long tiles = (long long)a.G * a.n_tiles * a.k_tiles;
  if (tiles > 0x7fffffffLL - 4096) return reject(ST_UNSUPPORTED, "wgrad: %lld output tiles are too many", tiles);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kWgThreads, 1, 1);
  cfg.dynamicSmemBytes = kWgSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> max_clusters[64];
  int mc = max_clusters[dev.device & 63].load(std::memory_order_relaxed);
  if (mc == 0) {
    cfg.gridDim = dim3((unsigned)(dev.num_sms & ~1), 1, 1);
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = dev.num_sms / 2;
    }
    mc = n;
    max_clusters[dev.device & 63].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(mc, tiles)), 1, 1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmD, tmA, tmOut, a, (int)tiles);
  return e == cudaSuccess ? ST_OK : cuda_fail(e, "launch k_wgrad_ws");
}

}  // namespace
}  // namespace wst

using namespace wst;

extern "C" wst_status wst_grouped_gemm_wgrad_bf16(int G, int M_total, int N, int K, const void* dC, long lddc,
                                                  const void* A, long lda, const int* d_offsets, void* dB, long lddb,
                                                  long stride_dB, wst_dtype db_type, int accumulate, void* workspace,
                                                  void* stream) {
  set_error("%s", "");
  if (G < 1 || M_total < 0 || N < 1 || K < 1)
    return (wst_status)reject(ST_INVALID_ARG, "wgrad: sizes out of range (G=%d M_total=%d N=%d K=%d)", G, M_total, N, K);
  if (M_total > 0x7fffffff - 1024 || N > 0x7fffffff - 1024 || K > 0x7fffffff - 1024)
    return (wst_status)reject(ST_UNSUPPORTED, "wgrad: M_total=%d N=%d K=%d: too large", M_total, N, K);
  if (db_type != WST_F32 && db_type != WST_BF16)
    return (wst_status)reject(ST_INVALID_ARG, "wgrad: unknown db_type %d", (int)db_type);
  if (lddc < N || lda < K || lddb < K || (G > 1 && stride_dB < (long)(N - 1) * lddb + K))
    return (wst_status)reject(ST_INVALID_ARG,
                              "wgrad: leading dimensions too small or groups overlap (lddc=%ld lda=%ld lddb=%ld stride=%ld)",
                              lddc, lda, lddb, stride_dB);
  if (!dB || !d_offsets || !workspace || (M_total && (!dC || !A)))
    return (wst_status)reject(ST_INVALID_ARG, "wgrad: NULL array");
  const long es = db_type == WST_F32 ? 4 : 2;
  if ((M_total && (!aligned_to(dC, 16) || !aligned_to(A, 16))) || !aligned_to(dB, 16) || !aligned_to(d_offsets, 4) ||
      !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "wgrad: dC, A, dB and the workspace must be 16-byte aligned, offsets 4-byte");
  if (lddc * 2 % 16 || lda * 2 % 16 || lddb * es % 16 || (G > 1 && stride_dB * es % 16))
    return (wst_status)reject(ST_ALIGNMENT, "wgrad: leading dimensions and strides must be multiples of 16 bytes");
  int st;
  if ((M_total && ((st = check_operand(dC, "dC")) || (st = check_operand(A, "A")))) || (st = check_operand(dB, "dB")) ||
      (st = check_operand(d_offsets, "d_offsets")) || (st = check_operand(workspace, "workspace")))
    return (wst_status)st;
  DeviceInfo dev;
  if ((st = current_device_info(&dev))) return (wst_status)st;
  WgArgs a{};
  a.G = G;
  a.M_total = M_total;
  a.N = N;
  a.K = K;
  a.n_tiles = (N + kWgTile - 1) / kWgTile;
  a.k_tiles = (K + kWgTile - 1) / kWgTile;
  a.offsets = d_offsets;
  a.accumulate = accumulate != 0;
  a.dB = dB;
  a.lddb = lddb;
  a.stride_dB = G > 1 ? stride_dB : 0;
  a.ws = static_cast<WsHeader*>(workspace);
  a.timeout_ns = wait_timeout_ns();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = db_type == WST_F32 ? launch_wgrad<true, false> : a.accumulate ? launch_wgrad<false, true> : launch_wgrad<false, false>;
  return (wst_status)launch(a, dC, lddc, A, lda, dB, lddb, stride_dB, dev, s);
}
