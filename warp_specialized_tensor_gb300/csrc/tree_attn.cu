// tree_attn.cu -- C entry point and launcher of the attention over a paged cache:
// argument checks, tensor maps, the two launches.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tree_attn.cuh"
#include "wst.h"
#include "wst_host.h"

namespace wst {

namespace {

template <int DH, bool OUT_F32, bool LONG>
int launch_tree(const TreeArgs& a, const void* Q, long long ldq, const void* K, const void* V, const DeviceInfo& dev,
                cudaStream_t stream) {
  using Cfg = TreeCfg<DH, OUT_F32 ? 3 : 1>;
  int st;
  CUtensorMap tmQ, tmK, tmV;
  {
    const uint64_t dims[3] = {(uint64_t)DH, (uint64_t)a.H, (uint64_t)a.T};
    const uint64_t str[2] = {(uint64_t)DH * 2, (uint64_t)ldq * 2};
    const uint32_t box[3] = {64, (uint32_t)a.group, (uint32_t)a.tokens};
    if ((st = encode_map(&tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, Q, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  }
  const uint64_t dims[4] = {(uint64_t)DH, (uint64_t)a.page_size, (uint64_t)a.Hkv, (uint64_t)a.num_pages};
  const uint64_t str[3] = {(uint64_t)a.token_stride * 2, (uint64_t)a.head_stride * 2, (uint64_t)a.page_stride * 2};
  const uint32_t box[4] = {64, (uint32_t)a.chunk, 1, 1};
  if ((st = encode_map(&tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, K, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  if ((st = encode_map(&tmV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, V, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))) return st;
  auto kern = k_tree_attn<DH, OUT_F32, LONG>;
  if ((st = ensure_smem_attr((const void*)kern, Cfg::kSmem))) return st;
  const int grid = std::min(dev.num_sms, kTreeMaxCtas);
  cudaError_t e = launch_early(kern, dim3((unsigned)grid), kTreeThreads, Cfg::kSmem, stream, tmQ, tmK, tmV, a);
  if (e != cudaSuccess) return cuda_fail(e, "launch k_tree_attn");
  if (!a.split) return ST_OK;
  e = launch_early(k_tree_merge<DH, OUT_F32>, dim3((unsigned)grid, (unsigned)(DH / 4 * kTreeBM / 256)), 256, 0, stream, a);
  return e == cudaSuccess ? ST_OK : cuda_fail(e, "launch k_tree_merge");
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

size_t wst_tree_attention_workspace_size(void) { return kTreeWorkspaceBytes; }

wst_status wst_tree_attention_bf16(int B, int T, int H, int Hkv, int Dh, const void* Q, long ldq,
                                   const int* d_q_offsets, const int* d_context, const int* mask, int mask_words,
                                   long ldm, const void* k_cache, const void* v_cache, int num_pages, int page_size,
                                   long page_stride, long token_stride, long head_stride, const int* page_table,
                                   int max_pages, long ldt, float scale, void* O, long ldo, wst_dtype o_type,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  set_error("%s", "");
  if (B < 0 || T < 0 || Hkv < 1 || H < 1 || H % Hkv || Dh < 1)
    return (wst_status)reject(ST_INVALID_ARG, "tree attention: sizes out of range (B=%d T=%d H=%d Hkv=%d Dh=%d)", B, T, H, Hkv, Dh);
  const int group = H / Hkv;
  if (Dh != 64 && Dh != 128) return (wst_status)reject(ST_UNSUPPORTED, "tree attention: Dh=%d: this build supports 64 and 128", Dh);
  if (group > kTreeBM)
    return (wst_status)reject(ST_UNSUPPORTED, "tree attention: %d heads to a key head: this build supports up to %d", group, kTreeBM);
  WST_TRY(check_cache("tree attention", k_cache, v_cache, num_pages, page_size, page_stride, token_stride, head_stride));
  if (page_size % 128 && page_size != 8 && page_size != 16 && page_size != 32 && page_size != 64)
    return (wst_status)reject(ST_UNSUPPORTED, "tree attention: page_size=%d: this build supports 8, 16, 32, 64 and multiples of 128", page_size);
  if (page_stride < 1 || token_stride < 1 || head_stride < 1)
    return (wst_status)reject(ST_INVALID_ARG, "tree attention: the cache's strides must be positive");
  if (max_pages < 1 && B > 0) return (wst_status)reject(ST_INVALID_ARG, "tree attention: max_pages=%d", max_pages);
  if ((long long)max_pages * page_size > (1ll << 30) || T > (1 << 30) || B > (1 << 29))
    return (wst_status)reject(ST_UNSUPPORTED, "tree attention: B=%d T=%d, %d pages of %d a sequence: too large", B, T, max_pages, page_size);
  if (o_type != WST_F32 && o_type != WST_BF16) return (wst_status)reject(ST_INVALID_ARG, "tree attention: unknown o_type %d", (int)o_type);
  if (!(std::fabs(scale) <= 2.0e38f))  // (times log2(e) it has to be finite too)
    return (wst_status)reject(ST_INVALID_ARG, "tree attention: scale must be finite, at most 2e38");
  const bool any = B > 0 && T > 0;
  if ((any && (!Q || !O || !d_q_offsets || !d_context || !page_table)) || !workspace)
    return (wst_status)reject(ST_INVALID_ARG, "tree attention: NULL array");
  if (ldq < (long)H * Dh || ldo < (long)H * Dh || (B > 1 && ldt < max_pages) || (mask && (mask_words < 1 || (T > 1 && ldm < mask_words))))
    return (wst_status)reject(ST_INVALID_ARG, "tree attention: leading dimensions too small (ldq=%ld ldo=%ld ldt=%ld ldm=%ld mask_words=%d)",
                              ldq, ldo, ldt, ldm, mask_words);
  const long es = o_type == WST_F32 ? 4 : 2;
  if (!aligned_to(Q, 16) || !aligned_to(O, 16) || ldq % 8 || ldo * es % 16)
    return (wst_status)reject(ST_ALIGNMENT, "tree attention: Q and O must be 16-byte aligned, leading dimensions multiples of 16 bytes");
  if (!aligned_to(d_q_offsets, 4) || !aligned_to(d_context, 4) || !aligned_to(mask, 4) || !aligned_to(page_table, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "tree attention: index arrays must be 4-byte, the workspace 16-byte aligned");
  if (workspace_bytes < kWsHeaderBytes) return (wst_status)reject(ST_INVALID_ARG, "tree attention: workspace of %zu bytes", workspace_bytes);
  if (!any) return WST_OK;
  WST_TRY(check_operand(Q, "Q"));
  WST_TRY(check_operand(d_q_offsets, "d_q_offsets"));
  WST_TRY(check_operand(d_context, "d_context"));
  if (mask) WST_TRY(check_operand(mask, "mask"));
  WST_TRY(check_operand(k_cache, "k_cache"));
  WST_TRY(check_operand(v_cache, "v_cache"));
  WST_TRY(check_operand(page_table, "page_table"));
  WST_TRY(check_operand(O, "O"));
  WST_TRY(check_operand(workspace, "workspace"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  TreeArgs a{};
  a.B = B;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.group = group;
  a.tokens = kTreeBM / group;
  a.lines = T > a.tokens ? 2 : 1;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.chunk = std::min(page_size, kTreeBN);
  a.q_offsets = d_q_offsets;
  a.context = d_context;
  a.mask = mask;
  a.mask_words = mask_words;
  a.ldm = ldm;
  a.table = page_table;
  a.ldt = ldt;
  a.v = static_cast<const __nv_bfloat16*>(v_cache);
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.cs = (float)((double)scale * 1.4426950408889634);  // log2(e)
  a.O = O;
  a.ldo = ldo;
  a.ws = reinterpret_cast<WsHeader*>(ws);
  a.split = workspace_bytes >= kTreeWorkspaceBytes ? 1 : 0;
  a.cuts = reinterpret_cast<TreeCut*>(ws + kTreeCutOffset);
  a.slots = reinterpret_cast<float*>(ws + kTreeSlotOffset);
  a.timeout_ns = wait_timeout_ns();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool is_long = (long long)max_pages * page_size > kTreeLong;
  auto launch = [&](auto dh) {
    constexpr int DH = decltype(dh)::value;
    if (o_type == WST_F32) return launch_tree<DH, true, false>(a, Q, ldq, k_cache, v_cache, dev, s);
    return is_long ? launch_tree<DH, false, true>(a, Q, ldq, k_cache, v_cache, dev, s) : launch_tree<DH, false, false>(a, Q, ldq, k_cache, v_cache, dev, s);
  };
  return (wst_status)(Dh == 128 ? launch(std::integral_constant<int, 128>()) : launch(std::integral_constant<int, 64>()));
}

}  // extern "C"
