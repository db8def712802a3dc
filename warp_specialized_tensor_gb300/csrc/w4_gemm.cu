// w4_gemm.cu -- C entry points and launcher of the products with 4-bit weights:
// argument checks, tensor maps, the number of column tiles, launch.
#include <algorithm>

#include "w4_gemm.cuh"
#include "wst.h"
#include "wst_host.h"

namespace wst {

namespace {

struct W4Problem {
  W4Args a;
  const void* A;
  long long lda;
  const void* W;
  long long ldw, strideW;
  const void* scales;
  long long lds, strideS;
  int group;
};

template <int NT, int GROUPS>
int launch_w4(W4Problem& pr, const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = W4Cfg<NT>;
  W4Args& a = pr.a;
  int st;
  CUtensorMap tmW, tmA, tmS;
  const int kb = (a.K + pr.group - 1) / pr.group;
  {
    // a stride of a dimension of one is never used, but has to be one that a map takes
    const uint64_t dims[3] = {(uint64_t)(a.K + 1) / 2, (uint64_t)a.N, (uint64_t)a.G};
    const uint64_t str[2] = {(uint64_t)pr.ldw, (uint64_t)(a.G > 1 ? pr.strideW : pr.ldw)};
    const uint32_t box[3] = {64, kW4Feats, 1};
    if ((st = encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pr.W, dims, str, box, CU_TENSOR_MAP_SWIZZLE_64B))) return st;
  }
  {
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)a.M};
    const uint64_t str[1] = {(uint64_t)pr.lda * 2};
    const uint32_t box[2] = {kW4K, (uint32_t)Cfg::kRows};
    if ((st = encode_map(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pr.A, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE))) return st;
  }
  {
    const uint64_t dims[3] = {(uint64_t)a.N, (uint64_t)kb, (uint64_t)a.G};
    const uint64_t str[2] = {(uint64_t)pr.lds * 2, (uint64_t)(a.G > 1 ? pr.strideS : pr.lds) * 2};
    const uint32_t box[3] = {kW4Feats, 2 * GROUPS, 1};
    if ((st = encode_map(&tmS, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, pr.scales, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE))) return st;
  }
  auto kern = k_w4_gemm<NT, GROUPS>;
  if ((st = ensure_smem_attr((const void*)kern, Cfg::kSmem))) return st;
  const int grid = std::min(dev.num_sms, kW4MaxCtas);
  const cudaError_t e = launch_early(kern, dim3((unsigned)grid), Cfg::kThreads, Cfg::kSmem, stream, tmW, tmA, tmS, a);
  return e == cudaSuccess ? ST_OK : cuda_fail(e, "launch k_w4_gemm");
}

template <int NT>
int launch_w4_group(W4Problem& pr, const DeviceInfo& dev, cudaStream_t stream) {
  if (pr.group == 128) return launch_w4<NT, 1>(pr, dev, stream);
  if (pr.group == 64) return launch_w4<NT, 2>(pr, dev, stream);
  return launch_w4<NT, 4>(pr, dev, stream);
}

// Tiles of 8 nt rows, at most (G: groups of rows, 0 for the dense product).
long long w4_tiles(int G, int M, int n_tiles, int nt) { return (((long long)M + 8 * nt - 1) / (8 * nt) + G) * n_tiles; }

// Column tiles of 8 rows in a tile: as many as the rows need (twice the mean of a group's),
// up to 4; fewer while that leaves a CTA at most 14 units, whose length then counts for
// less than the sums that are merged.  (64 x 2,048 x 2,048 7.7, 9.1, 9.0 us with 1, 2, 4;
// 64 x 4,096 x 4,096 22.6, 13.5, 14.2; 32 x 8,192 x 8,192 34.9, 22.3, 22.1.  Tiles of 64
// rows, 8, took 48 us for 64 x 8,192 x 8,192 where 4 takes 38.)
int w4_column_tiles(int G, int M, int N, int K, int num_sms) {
  const int n_tiles = (N + kW4Feats - 1) / kW4Feats, k_units = (K + kW4K - 1) / kW4K;
  const long long rows = G ? 2 * (((long long)M + G - 1) / G) : M;
  int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  while (nt > 1 && w4_tiles(G, M, n_tiles, nt / 2) <= 14ll * num_sms / k_units) nt /= 2;
  return nt;
}

int run_w4(const char* what, W4Problem& pr, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  W4Args& a = pr.a;
  if (a.N < 1 || a.K < 1 || a.M < 0 || a.G < 1)
    return reject(ST_INVALID_ARG, "%s: sizes out of range (G=%d M=%d N=%d K=%d)", what, a.G, a.M, a.N, a.K);
  if (a.N > 0x7fffffff - 1024 || a.K > 0x7fffffff - 1024 || a.M > 0x7fffffff - 1024 || a.G > 0x7fffffff - 1024)
    return reject(ST_UNSUPPORTED, "%s: G=%d M=%d N=%d K=%d: too large", what, a.G, a.M, a.N, a.K);
  if (pr.group != 32 && pr.group != 64 && pr.group != 128)
    return reject(ST_UNSUPPORTED, "%s: group=%d: this build supports 32, 64 and 128", what, pr.group);
  if (a.epi < 0 || a.epi > 3) return reject(ST_INVALID_ARG, "%s: unknown epilogue %d", what, a.epi);
  if (a.M && (!pr.A || !a.C)) return reject(ST_INVALID_ARG, "%s: NULL array", what);
  if (!pr.W || !pr.scales || (a.epi && !a.bias) || !workspace) return reject(ST_INVALID_ARG, "%s: NULL array", what);
  if (pr.lda < a.K || pr.ldw < ((long long)a.K + 1) / 2 || pr.lds < a.N || a.ldc < a.N)
    return reject(ST_INVALID_ARG, "%s: leading dimensions too small (lda=%lld ldw=%lld lds=%lld ldc=%lld)", what, pr.lda, pr.ldw, pr.lds, a.ldc);
  const long long kb = ((long long)a.K + pr.group - 1) / pr.group;
  if (a.G > 1 && (pr.strideW < 0 || pr.strideS < 0 || a.stride_bias < 0))
    return reject(ST_INVALID_ARG, "%s: negative stride", what);
  const int es = a.c_f32 ? 4 : 2;
  if (!aligned_to(pr.A, 16) || !aligned_to(pr.W, 16) || !aligned_to(pr.scales, 16) || !aligned_to(a.C, 16) || !aligned_to(workspace, 16) ||
      !aligned_to(a.bias, 2) || pr.lda % 8 || pr.ldw % 16 || pr.lds % 8 || a.ldc * es % 16 || (a.G > 1 && (pr.strideW % 16 || pr.strideS % 8)))
    return reject(ST_ALIGNMENT, "%s: arrays must be 16-byte aligned, leading dimensions and strides multiples of 16 bytes", what);
  if (workspace_bytes < kWsHeaderBytes) return reject(ST_INVALID_ARG, "%s: workspace of %zu bytes", what, workspace_bytes);
  if ((long long)a.N * kb > (1ll << 46)) return reject(ST_UNSUPPORTED, "%s: N=%d K=%d: too large", what, a.N, a.K);
  if (a.M == 0) return ST_OK;
  int st;
  if ((st = check_operand(pr.A, "A")) || (st = check_operand(pr.W, "W")) || (st = check_operand(pr.scales, "scales")) ||
      (st = check_operand(a.C, "C")) || (st = check_operand(workspace, "workspace")))
    return st;
  if (a.epi && (st = check_operand(a.bias, "bias"))) return st;
  if (a.offsets && (st = check_operand(a.offsets, "d_offsets"))) return st;
  DeviceInfo dev;
  if ((st = current_device_info(&dev))) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.k_units = (a.K + kW4K - 1) / kW4K;
  while ((1ll << a.k_shift) < a.k_units) ++a.k_shift;
  a.k_mul = (uint32_t)(((1ull << 32) * ((1ull << a.k_shift) - (uint64_t)a.k_units)) / (uint64_t)a.k_units + 1);
  a.n_tiles = (a.N + kW4Feats - 1) / kW4Feats;
  a.split = workspace_bytes >= kW4WorkspaceBytes ? 1 : 0;
  a.ws = reinterpret_cast<WsHeader*>(ws);
  a.slots = reinterpret_cast<float*>(ws + kWsHeaderBytes);
  a.timeout_ns = wait_timeout_ns();
  const int nt = w4_column_tiles(a.offsets ? a.G : 0, a.M, a.N, a.K, dev.num_sms);
  const long long units = w4_tiles(a.offsets ? a.G : 0, a.M, a.n_tiles, nt);
  if (units > 0x7fffffffll / a.k_units) return reject(ST_UNSUPPORTED, "%s: G=%d M=%d N=%d K=%d: too large", what, a.G, a.M, a.N, a.K);
  if (nt == 1) return launch_w4_group<1>(pr, dev, stream);
  if (nt == 2) return launch_w4_group<2>(pr, dev, stream);
  return launch_w4_group<4>(pr, dev, stream);
}

}  // namespace
}  // namespace wst

using namespace wst;

extern "C" {

size_t wst_gemm_w4_workspace_size(void) { return kW4WorkspaceBytes; }

int wst_gemm_w4_tile_rows(int G, int M, int N, int K, int num_sms) {
  const int most = 0x7fffffff - 1024;
  if (G < 0 || M < 0 || N < 1 || K < 1 || num_sms < 1 || G > most || M > most || N > most || K > most) return 0;
  return 8 * w4_column_tiles(G, M, N, K, num_sms);
}

wst_status wst_gemm_w4(int M, int N, int K, const void* A, long lda, const void* W, long ldw, const void* scales,
                       long lds, int group, const void* bias, void* C, long ldc, wst_dtype c_type,
                       wst_epilogue epi, void* workspace, size_t workspace_bytes, void* stream) {
  set_error("%s", "");
  if (c_type != WST_F32 && c_type != WST_BF16) return (wst_status)reject(ST_INVALID_ARG, "gemm_w4: unknown c_type %d", (int)c_type);
  W4Problem pr{};
  pr.a.G = 1;
  pr.a.M = M;
  pr.a.N = N;
  pr.a.K = K;
  pr.a.bias = epi ? static_cast<const __nv_bfloat16*>(bias) : nullptr;
  pr.a.C = C;
  pr.a.ldc = ldc;
  pr.a.c_f32 = c_type == WST_F32;
  pr.a.epi = (int)epi;
  pr.A = A;
  pr.lda = lda;
  pr.W = W;
  pr.ldw = ldw;
  pr.scales = scales;
  pr.lds = lds;
  pr.group = group;
  return (wst_status)run_w4("gemm_w4", pr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

wst_status wst_grouped_gemm_w4(int G, int M_total, int N, int K, const void* A, long lda, const void* W, long ldw,
                               long strideW_group, const void* scales, long lds, long strideS_group, int group,
                               const int* d_offsets, const void* bias, long strideBias, void* C, long ldc,
                               wst_dtype c_type, wst_epilogue epi, void* workspace, size_t workspace_bytes,
                               void* stream) {
  set_error("%s", "");
  if (c_type != WST_F32 && c_type != WST_BF16)
    return (wst_status)reject(ST_INVALID_ARG, "grouped_gemm_w4: unknown c_type %d", (int)c_type);
  if (!d_offsets) return (wst_status)reject(ST_INVALID_ARG, "grouped_gemm_w4: d_offsets is NULL");
  if (!aligned_to(d_offsets, 4)) return (wst_status)reject(ST_ALIGNMENT, "grouped_gemm_w4: d_offsets must be 4-byte aligned");
  W4Problem pr{};
  pr.a.G = G;
  pr.a.M = M_total;
  pr.a.N = N;
  pr.a.K = K;
  pr.a.offsets = d_offsets;
  pr.a.bias = epi ? static_cast<const __nv_bfloat16*>(bias) : nullptr;
  pr.a.stride_bias = strideBias;
  pr.a.C = C;
  pr.a.ldc = ldc;
  pr.a.c_f32 = c_type == WST_F32;
  pr.a.epi = (int)epi;
  pr.A = A;
  pr.lda = lda;
  pr.W = W;
  pr.ldw = ldw;
  pr.strideW = strideW_group;
  pr.scales = scales;
  pr.lds = lds;
  pr.strideS = strideS_group;
  pr.group = group;
  return (wst_status)run_w4("grouped_gemm_w4", pr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
