// fp8_gemm.cu -- launcher and C ABI of the 8-bit products (dense and grouped).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp8_gemm.cuh"
#include "wst.h"
#include "wst_host.h"

namespace wst {

namespace {

struct F8Problem {
  int G, M, N, K;
  const void* A;
  long long lda;
  int a_type;
  const void* B;
  long long ldb, strideB;
  int b_type;
  void* C;
  long long ldc;
};

template <bool OUT_F32, bool SB_ROWS, bool EPI, bool THIN>
int launch_fp8(const F8Problem& pr, F8Args& a, const DeviceInfo& dev, cudaStream_t stream) {
  auto kern = k_gemm_fp8<OUT_F32, SB_ROWS, EPI, THIN>;
  CUtensorMap tmW, tmX, tmXt, tmC;
  int st;
  a.w_shared = pr.strideB == 0 ? 1 : 0;
  {
    uint64_t dims[3] = {(uint64_t)pr.K, (uint64_t)pr.N, (uint64_t)(a.w_shared ? 1 : pr.G)};
    uint64_t str[2] = {(uint64_t)pr.ldb, (uint64_t)(a.w_shared ? (long long)pr.N * pr.ldb : pr.strideB)};
    uint32_t box[3] = {kF8BK, 128, 1};
    if ((st = encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pr.B, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B)))
      return st;
  }
  {
    uint64_t dims[2] = {(uint64_t)pr.K, (uint64_t)pr.M};
    uint64_t str[1] = {(uint64_t)pr.lda};
    uint32_t box[2] = {kF8BK, 128};
    if ((st = encode_map(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pr.A, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B)))
      return st;
    box[1] = kF8ThinRows;
    if ((st = encode_map(&tmXt, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, pr.A, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B)))
      return st;
  }
  {
    const uint64_t es = OUT_F32 ? 4 : 2;
    uint64_t dims[2] = {(uint64_t)pr.N, (uint64_t)pr.M};
    uint64_t str[1] = {(uint64_t)pr.ldc * es};
    uint32_t box[2] = {32, OUT_F32 ? 16u : 32u};
    if ((st = encode_map(&tmC, OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pr.C,
                         dims, str, box, OUT_F32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)))
      return st;
  }
  if ((st = ensure_smem_attr((const void*)kern, kF8SmemBytes))) return st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kF8Threads, 1, 1);
  cfg.dynamicSmemBytes = kF8SmemBytes;
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
  a.pairs = mc;
  // Persistent grid, no larger than the units of work (an upper bound where
  // the group sizes are on the device).
  const long long tiles =
      (long long)a.n_tiles * ((long long)pr.M / kF8Tile + (a.offsets ? std::min<long long>(pr.G, pr.M) : 1));
  const long long units = tiles * std::max(1, a.k_blocks);
  cfg.gridDim = dim3((unsigned)(2 * std::min<long long>(mc, units)), 1, 1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmW, tmX, tmXt, tmC, a);
  return e == cudaSuccess ? ST_OK : cuda_fail(e, "launch k_gemm_fp8");
}

int fp8_product(const char* what, bool grouped, int G, int M, int N, int K, const void* A, long lda, int a_type,
                const float* scaleA, long ldsa, const void* B, long ldb, long strideB, int b_type, const float* scaleB,
                long ldsb, long strideSB, int b_scaling, const int* offsets, const void* bias, long strideBias, void* C,
                long ldc, int c_type, int epi, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (G < 1 || M < 0 || N < 1 || K < 1)
    return reject(ST_INVALID_ARG, "%s: sizes out of range (G=%d M=%d N=%d K=%d)", what, G, M, N, K);
  if (M > 0x7fffffff - 1024 || N > 0x7fffffff - 1024 || K > 0x7fffffff - 1024)
    return reject(ST_UNSUPPORTED, "%s: M=%d N=%d K=%d: too large", what, M, N, K);
  if ((a_type != WST_E4M3 && a_type != WST_E5M2) || (b_type != WST_E4M3 && b_type != WST_E5M2))
    return reject(ST_INVALID_ARG, "%s: unknown 8-bit type", what);
  if (c_type != WST_F32 && c_type != WST_BF16) return reject(ST_INVALID_ARG, "%s: unknown c_type %d", what, c_type);
  if (epi < 0 || epi > 3) return reject(ST_INVALID_ARG, "%s: unknown epilogue %d", what, epi);
  if (b_scaling != WST_FP8_ROWS && b_scaling != WST_FP8_BLOCKS)
    return reject(ST_INVALID_ARG, "%s: the scales of B are WST_FP8_ROWS or WST_FP8_BLOCKS", what);
  if (!workspace || workspace_bytes < kWsHeaderBytes)
    return reject(ST_INVALID_ARG, "%s: needs a workspace of at least %zu bytes", what, kWsHeaderBytes);
  const long kb = ((long)K + 127) / 128;
  const long sb_cols = b_scaling == WST_FP8_ROWS ? N : kb;
  if (lda < K || ldb < K || ldc < N || ldsa < M || ldsb < sb_cols)
    return reject(ST_INVALID_ARG, "%s: leading dimensions too small (lda=%ld ldb=%ld ldc=%ld ldsa=%ld ldsb=%ld)", what, lda,
                  ldb, ldc, ldsa, ldsb);
  if (G > 1 && (strideB < 0 || strideBias < 0 || strideSB < 0))  // (one group has no stride)
    return reject(ST_INVALID_ARG, "%s: negative group stride", what);
  if (M == 0) return ST_OK;  // no rows: nothing to compute or store
  if (!A || !B || !C || !scaleA || !scaleB || (grouped && !offsets) || (epi && !bias))
    return reject(ST_INVALID_ARG, "%s: NULL array", what);
  const long es = c_type == WST_F32 ? 4 : 2;
  if (!aligned_to(A, 16) || !aligned_to(B, 16) || !aligned_to(C, 16) || (epi && !aligned_to(bias, 2)) ||
      !aligned_to(workspace, 16) || !aligned_to(scaleA, 4) || !aligned_to(scaleB, 4) || !aligned_to(offsets, 4))
    return reject(ST_ALIGNMENT, "%s: A, B, C and the workspace must be 16-byte aligned, scales and offsets 4-byte", what);
  if (lda % 16 || ldb % 16 || ldc * es % 16 || (G > 1 && strideB % 16))
    return reject(ST_ALIGNMENT, "%s: leading dimensions and strides must be multiples of 16 bytes", what);
  int st;
  if ((st = check_operand(A, "A")) || (st = check_operand(B, "B")) || (st = check_operand(C, "C")) ||
      (st = check_operand(scaleA, "scaleA")) || (st = check_operand(scaleB, "scaleB")) ||
      (grouped && (st = check_operand(offsets, "d_offsets"))) || (epi && (st = check_operand(bias, "bias"))) ||
      (st = check_operand(workspace, "workspace")))
    return st;
  DeviceInfo dev;
  if ((st = current_device_info(&dev))) return st;
  F8Problem pr{G, M, N, K, A, lda, a_type, B, ldb, G > 1 ? strideB : 0, b_type, C, ldc};
  F8Args a{};
  a.G = G;
  a.M_total = M;
  a.N = N;
  a.K = K;
  a.n_tiles = (N + kF8Tile - 1) / kF8Tile;
  a.k_blocks = (K + kF8BK - 1) / kF8BK;
  a.offsets = offsets;
  a.sa = scaleA;
  a.ldsa = ldsa;
  a.sb = scaleB;
  a.ldsb = ldsb;
  a.strideSB = strideSB;
  a.idesc = idesc_f8_f32(256, b_type, a_type);
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.bias_stride = strideBias;
  a.epi = epi;
  a.C = C;
  a.ldc = ldc;
  a.max_units = workspace_bytes >= kF8WorkspaceBytes ? kF8MaxUnits : 0;
  a.ws = static_cast<WsHeader*>(workspace);
  a.timeout_ns = wait_timeout_ns();
  auto go = [&](auto out_f32, auto sb_rows) {
    constexpr bool F = decltype(out_f32)::value, R = decltype(sb_rows)::value;
    // Groups of at most 64 rows on average: most tiles are thin.
    if (M <= 64LL * G)
      return epi ? launch_fp8<F, R, true, true>(pr, a, dev, stream) : launch_fp8<F, R, false, true>(pr, a, dev, stream);
    return epi ? launch_fp8<F, R, true, false>(pr, a, dev, stream) : launch_fp8<F, R, false, false>(pr, a, dev, stream);
  };
  const bool rows = b_scaling == WST_FP8_ROWS;
  if (c_type == WST_F32)
    return rows ? go(std::true_type(), std::true_type()) : go(std::true_type(), std::false_type());
  return rows ? go(std::false_type(), std::true_type()) : go(std::false_type(), std::false_type());
}

}  // namespace
}  // namespace wst

using namespace wst;

extern "C" {

size_t wst_gemm_fp8_workspace_size(void) { return kF8WorkspaceBytes; }

wst_status wst_gemm_fp8(int M, int N, int K, const void* A, long lda, wst_fp8 a_type, const float* scaleA, long ldsa,
                        const void* B, long ldb, wst_fp8 b_type, const float* scaleB, long ldsb, wst_fp8_mode b_scaling,
                        const void* bias, void* C, long ldc, wst_dtype c_type, wst_epilogue epi, void* workspace,
                        size_t workspace_bytes, void* stream) {
  set_error("%s", "");
  return (wst_status)fp8_product("fp8 gemm", false, 1, M, N, K, A, lda, a_type, scaleA, ldsa, B, ldb, 0, b_type, scaleB,
                                 ldsb, 0, b_scaling, nullptr, bias, 0, C, ldc, c_type, epi, workspace, workspace_bytes,
                                 static_cast<cudaStream_t>(stream));
}

wst_status wst_grouped_gemm_fp8(int G, int M_total, int N, int K, const void* A, long lda, wst_fp8 a_type,
                                const float* scaleA, long ldsa, const void* B, long ldb, long strideB_group,
                                wst_fp8 b_type, const float* scaleB, long ldsb, long strideSB_group,
                                wst_fp8_mode b_scaling, const int* d_offsets, const void* bias, long strideBias, void* C,
                                long ldc, wst_dtype c_type, wst_epilogue epi, void* workspace, size_t workspace_bytes,
                                void* stream) {
  set_error("%s", "");
  return (wst_status)fp8_product("grouped fp8 gemm", true, G, M_total, N, K, A, lda, a_type, scaleA, ldsa, B, ldb,
                                 strideB_group, b_type, scaleB, ldsb, strideSB_group, b_scaling, d_offsets, bias,
                                 strideBias, C, ldc, c_type, epi, workspace, workspace_bytes,
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"
