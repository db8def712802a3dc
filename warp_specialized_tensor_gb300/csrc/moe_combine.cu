// moe_combine.cu -- the weighted sum of the experts' rows of each token, and
// its gradients.
//
//   out[t]      = sum_i w[t][i] y[pos[t][i]]          (pos -1: no row; w NULL: 1)
//   dy[pos]     = w[t][i] dout[t]
//   dw[t][i]    = <dout[t], y[pos[t][i]]>             (0 where there is no row)
//
// Both are bound by HBM: every row of y and of out moves once.  A thread holds
// eight neighbouring columns and adds a token's rows in slot order in fp32
// (one rounding, at the store); eight 16-byte words of rows are in flight per
// thread.  The gradient's block holds one or more whole tokens, so dout is
// read once for all of a token's rows and the dot products are summed inside
// the block, in a fixed order.  On GB300 16384 x 2 rows of 4096 (bf16) take 65 us
// (6.2 TB/s), the gradients of 5003 x 4 rows of 1531 27 us (4.9 TB/s: a warp's
// loads wait for its position reads, and the registers of five rows per lane
// leave room for few warps).
#include "wst.h"
#include "wst_common.cuh"
#include "wst_host.h"

namespace wst {

namespace {

constexpr int kCombThreads = 128;  // (256: 72 against 65 us for 16384 x 2 x 4096, a longer last wave)
constexpr int kCombMaxTopK = 32;
constexpr int kCombMaxVecs = 8;    // vectors of eight columns a thread takes at a time, at most

struct CombineArgs {
  int T, top_k, N, n_rows;
  const void* y;
  long long ldy;
  const int* position;
  const float* weights;
  void* out;  // forward: out; backward: dout
  long long ldo;
  void* dy;
  long long lddy;
  float* dweights;
  WsHeader* ws;
};

// Eight columns as loaded (one 16-byte word of bf16, two of fp32); columns from n
// on read as 0 and are not stored.
template <typename X>
struct Eight {
  uint4 w[sizeof(X) / 2];
};
template <typename X>
__device__ __forceinline__ Eight<X> load8(const X* p, int n) {
  Eight<X> r;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(X) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  } else {
    uint32_t u[sizeof(X) * 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(X) * 2; ++i) u[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (sizeof(X) == 4) u[i] = __float_as_uint(__ldg(reinterpret_cast<const float*>(p) + i));
        else u[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i & 1));
      }
#pragma unroll
    for (int i = 0; i < (int)sizeof(X) / 2; ++i) r.w[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
  }
  return r;
}
__device__ __forceinline__ void unpack8(const Eight<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void unpack8(const Eight<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}

// Row of slot i of token t, -1 for none; a row past the end counts as none.
__device__ __forceinline__ int combine_row(const CombineArgs& a, int t, int i, bool latch) {
  const int p = __ldg(a.position + (long long)t * a.top_k + i);
  if (p < a.n_rows) return p;
  if (latch) latch_error(a.ws, 1u /*WST_ERR_INVALID_ARG*/, 0x70000u);
  return -1;
}

// tpt threads per token (a power of two from 32 to kCombThreads); each takes V
// vectors of eight columns at a time, KC rows of each in flight.
template <typename Y, typename O, int KC, int V>
__global__ void __launch_bounds__(kCombThreads) k_combine(const CombineArgs a, int tpt) {
  static_assert(V <= kCombMaxVecs, "columns fit 32 bits");
  const int t = blockIdx.x * (kCombThreads / tpt) + (int)threadIdx.x / tpt;
  const int me = (int)threadIdx.x & (tpt - 1);
  if (t >= a.T) return;
  const Y* y = static_cast<const Y*>(a.y);
  O* out = static_cast<O*>(a.out) + (long long)t * a.ldo;
  for (int c0 = me * 8; c0 < a.N; c0 += tpt * 8 * V) {
    float acc[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[v][c] = 0.0f;
    for (int i0 = 0; i0 < a.top_k; i0 += KC) {
      long long row[KC];
      float w[KC];
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        const int r = i0 + i < a.top_k ? combine_row(a, t, i0 + i, c0 == 0) : -1;
        w[i] = r >= 0 && a.weights ? __ldg(a.weights + (long long)t * a.top_k + i0 + i) : 1.0f;
        row[i] = r >= 0 ? (long long)r * a.ldy : -1;
      }
      Eight<Y> raw[V][KC];
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const int c = c0 + v * tpt * 8;
          if (row[i] >= 0 && c < a.N) raw[v][i] = load8(y + row[i] + c, a.N - c);
        }
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < KC; ++i)
          if (row[i] >= 0) {
            float x[8];
            unpack8(raw[v][i], x);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[v][c] = fmaf(w[i], x[c], acc[v][c]);
          }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * tpt * 8;
      if (c < a.N) store8(out + c, a.N - c, acc[v]);
    }
  }
}

// KC slots at a time (more slots take further passes over dout).
template <typename Y, typename O, int KC>
__global__ void __launch_bounds__(kCombThreads) k_combine_backward(const CombineArgs a, int tpt) {
  __shared__ float part[kCombThreads / 32][KC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (kCombThreads / tpt) + (int)threadIdx.x / tpt;
  const int me = (int)threadIdx.x & (tpt - 1);
  const bool there = t < a.T;
  const O* dout = static_cast<const O*>(a.out) + (long long)(there ? t : 0) * a.ldo;
  for (int i0 = 0; i0 < a.top_k; i0 += KC) {
    int row[KC];
    float w[KC], dot[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      row[i] = there && i0 + i < a.top_k ? combine_row(a, t, i0 + i, me == 0) : -1;
      w[i] = row[i] >= 0 && a.weights ? __ldg(a.weights + (long long)t * a.top_k + i0 + i) : 1.0f;
      dot[i] = 0.0f;
    }
    for (int c = me * 8; there && c < a.N; c += tpt * 8) {
      const Eight<O> draw = load8(dout + c, a.N - c);
      Eight<Y> raw[KC];
      if (a.dweights) {
#pragma unroll
        for (int i = 0; i < KC; ++i)
          if (row[i] >= 0) raw[i] = load8(static_cast<const Y*>(a.y) + (long long)row[i] * a.ldy + c, a.N - c);
      }
      float d[8];
      unpack8(draw, d);
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        if (row[i] < 0) continue;
        if (a.dweights) {
          float x[8];
          unpack8(raw[i], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) dot[i] = fmaf(d[j], x[j], dot[i]);
        }
        if (a.dy) {
          float g[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = w[i] * d[j];
          store8(static_cast<Y*>(a.dy) + (long long)row[i] * a.lddy + c, a.N - c, g);
        }
      }
    }
    if (a.dweights) {
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
      if (tpt > 32) {
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < KC; ++i) part[warp][i] = dot[i];
        }
        __syncthreads();
        if (there && me < KC && i0 + me < a.top_k) {
          float sum = 0.0f;
          for (int k = 0; k < tpt / 32; ++k) sum += part[warp + k][me];
          a.dweights[(long long)t * a.top_k + i0 + me] = sum;
        }
        __syncthreads();
      } else if (there && lane == 0) {
#pragma unroll
        for (int i = 0; i < KC; ++i)
          if (i0 + i < a.top_k) a.dweights[(long long)t * a.top_k + i0 + i] = dot[i];
      }
    }
  }
}

// One warp per token where there are tokens enough to fill the SMs with warps
// (each warp then has more loads in flight and needs no barrier); more threads
// per token for few tokens.
int threads_per_token(int T, int N, int sms) {
  int tpt = 32;
  while (tpt < kCombThreads && tpt * 8 < N && (long long)T * tpt < 512LL * sms) tpt *= 2;
  return tpt;
}

template <typename Y, typename O>
void launch_combine(const CombineArgs& a, int sms, cudaStream_t s) {
  const int tpt = threads_per_token(a.T, a.N, sms), per = kCombThreads / tpt;
  const unsigned grid = (unsigned)((a.T + per - 1) / per);
  if (a.top_k == 1) k_combine<Y, O, 1, 8><<<grid, kCombThreads, 0, s>>>(a, tpt);
  else if (a.top_k == 2) k_combine<Y, O, 2, 4><<<grid, kCombThreads, 0, s>>>(a, tpt);
  else k_combine<Y, O, 4, 2><<<grid, kCombThreads, 0, s>>>(a, tpt);
}

template <typename Y, typename O>
void launch_combine_backward(const CombineArgs& a, int sms, cudaStream_t s) {
  const int tpt = threads_per_token(a.T, a.N, sms), per = kCombThreads / tpt;
  const unsigned grid = (unsigned)((a.T + per - 1) / per);
  if (a.top_k == 1) k_combine_backward<Y, O, 1><<<grid, kCombThreads, 0, s>>>(a, tpt);
  else if (a.top_k == 2) k_combine_backward<Y, O, 2><<<grid, kCombThreads, 0, s>>>(a, tpt);
  else if (a.top_k <= 4) k_combine_backward<Y, O, 4><<<grid, kCombThreads, 0, s>>>(a, tpt);
  else k_combine_backward<Y, O, 8><<<grid, kCombThreads, 0, s>>>(a, tpt);
}

int check_combine(const char* what, int T, int top_k, int N, int y_type, int n_rows, int out_type) {
  if (T < 0 || top_k < 1 || N < 1 || n_rows < 0)
    return reject(ST_INVALID_ARG, "%s: sizes out of range (T=%d top_k=%d N=%d n_rows=%d)", what, T, top_k, N, n_rows);
  if (top_k > kCombMaxTopK)
    return reject(ST_UNSUPPORTED, "%s: top_k=%d: this build supports up to %d", what, top_k, kCombMaxTopK);
  // (a step past the last column, and a block of tokens past the last one, fit 32 bits)
  if (N > 0x7fffffff - 8 * kCombThreads * kCombMaxVecs) return reject(ST_UNSUPPORTED, "%s: N=%d is too wide", what, N);
  if (T > 0x7fffffff - 1024) return reject(ST_UNSUPPORTED, "%s: T=%d: too many tokens", what, T);
  if ((y_type != WST_F32 && y_type != WST_BF16) || (out_type != WST_F32 && out_type != WST_BF16))
    return reject(ST_INVALID_ARG, "%s: unknown type", what);
  return ST_OK;
}

int check_rows(const char* what, const char* name, const void* p, long ld, int type, int N) {
  const long es = type == WST_F32 ? 4 : 2;
  if (ld < N) return reject(ST_INVALID_ARG, "%s: leading dimension %ld of %s < N", what, ld, name);
  if (!aligned_to(p, 16) || ld * es % 16)
    return reject(ST_ALIGNMENT, "%s: %s must be 16-byte aligned, its leading dimension a multiple of 16 bytes", what, name);
  return ST_OK;
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

wst_status wst_moe_combine(int T, int top_k, int N, const void* y, long ldy, wst_dtype y_type, int n_rows,
                           const int* position, const float* weights, void* out, long ldo, wst_dtype out_type,
                           void* workspace, void* stream) {
  set_error("%s", "");
  WST_TRY(check_combine("combine", T, top_k, N, y_type, n_rows, out_type));
  if ((n_rows && T && !y) || (T && (!position || !out)) || !workspace)
    return (wst_status)reject(ST_INVALID_ARG, "combine: NULL array");
  WST_TRY(check_rows("combine", "y", y, ldy, y_type, N));
  WST_TRY(check_rows("combine", "out", out, ldo, out_type, N));
  if (!aligned_to(position, 4) || !aligned_to(weights, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "combine: position and weights must be 4-byte, the workspace 16-byte aligned");
  if (T == 0) return WST_OK;
  if (n_rows) WST_TRY(check_operand(y, "y"));
  WST_TRY(check_operand(position, "position"));
  if (weights) WST_TRY(check_operand(weights, "weights"));
  WST_TRY(check_operand(out, "out"));
  WST_TRY(check_operand(workspace, "workspace"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  CombineArgs a{};
  a.T = T;
  a.top_k = top_k;
  a.N = N;
  a.n_rows = n_rows;
  a.y = y;
  a.ldy = ldy;
  a.position = position;
  a.weights = weights;
  a.out = out;
  a.ldo = ldo;
  a.ws = static_cast<WsHeader*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (y_type == WST_F32) {
    if (out_type == WST_F32) launch_combine<float, float>(a, dev.num_sms, s);
    else launch_combine<float, __nv_bfloat16>(a, dev.num_sms, s);
  } else {
    if (out_type == WST_F32) launch_combine<__nv_bfloat16, float>(a, dev.num_sms, s);
    else launch_combine<__nv_bfloat16, __nv_bfloat16>(a, dev.num_sms, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_combine");
}

wst_status wst_moe_combine_backward(int T, int top_k, int N, const void* dout, long ldo, wst_dtype out_type,
                                    const void* y, long ldy, wst_dtype y_type, int n_rows, const int* position,
                                    const float* weights, void* dy, long lddy, float* dweights, void* workspace,
                                    void* stream) {
  set_error("%s", "");
  WST_TRY(check_combine("combine backward", T, top_k, N, y_type, n_rows, out_type));
  if ((T && (!dout || !position)) || !workspace) return (wst_status)reject(ST_INVALID_ARG, "combine backward: NULL array");
  // (a dy without a row may be NULL: only the positions are looked at)
  if (!dy && !dweights && n_rows)
    return (wst_status)reject(ST_INVALID_ARG, "combine backward: neither dy nor dweights is asked for");
  if (T && dweights && n_rows && !y) return (wst_status)reject(ST_INVALID_ARG, "combine backward: dweights needs y");
  WST_TRY(check_rows("combine backward", "dout", dout, ldo, out_type, N));
  if (dweights && n_rows) WST_TRY(check_rows("combine backward", "y", y, ldy, y_type, N));
  if (dy) WST_TRY(check_rows("combine backward", "dy", dy, lddy, y_type, N));
  if (!aligned_to(position, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT,
                              "combine backward: position and weights must be 4-byte, the workspace 16-byte aligned");
  if (T == 0) return WST_OK;
  WST_TRY(check_operand(dout, "dout"));
  WST_TRY(check_operand(position, "position"));
  if (dweights && n_rows) WST_TRY(check_operand(y, "y"));
  if (weights) WST_TRY(check_operand(weights, "weights"));
  if (dy) WST_TRY(check_operand(dy, "dy"));
  if (dweights) WST_TRY(check_operand(dweights, "dweights"));
  WST_TRY(check_operand(workspace, "workspace"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  CombineArgs a{};
  a.T = T;
  a.top_k = top_k;
  a.N = N;
  a.n_rows = n_rows;
  a.y = y;
  a.ldy = ldy;
  a.position = position;
  a.weights = weights;
  a.out = const_cast<void*>(dout);
  a.ldo = ldo;
  a.dy = dy;
  a.lddy = lddy;
  a.dweights = dweights;
  a.ws = static_cast<WsHeader*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (y_type == WST_F32) {
    if (out_type == WST_F32) launch_combine_backward<float, float>(a, dev.num_sms, s);
    else launch_combine_backward<float, __nv_bfloat16>(a, dev.num_sms, s);
  } else {
    if (out_type == WST_F32) launch_combine_backward<__nv_bfloat16, float>(a, dev.num_sms, s);
    else launch_combine_backward<__nv_bfloat16, __nv_bfloat16>(a, dev.num_sms, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_combine_backward");
}

}  // extern "C"
