// fp8_quant.cu -- quantisation to 8-bit floating point with one fp32 scale for
// each block of 128.
//
//   amax  = max |x| over the block, at least 2^-100
//   scale = amax * (1 / largest)        (largest: 448 for e4m3, 57344 for e5m2)
//           or, with pow2, the smallest power of two with amax <= largest * scale
//   q     = rn(x * (1 / scale)),        so x ~ q * scale
// in fp32, each operation rounded once.  The largest value of a block maps to
// `largest` up to two roundings, which the 8-bit rounding absorbs.  A block
// that holds a NaN or an infinity gets it as its scale.
//
// Blocks: ROWS 1 x 128 along a row; COLS 128 x 1 down a column, values
// transposed; BLOCKS 128 x 128; BLOCKS_T 128 x 128, values and scales
// transposed.
//
// All forms are bound by HBM (2 or 4 bytes in, 1 byte out).  ROWS: eight
// lanes hold one block, 16 values each, and find its largest by shuffles; with a
// row index each block is quantised once and stored to every row that wants
// it.  The others: one 128 x 128 tile per block of threads, an 8 x 8 patch in
// each thread's registers, so a transposed patch leaves as eight 8-byte words
// through shared memory (words XOR-swizzled by the column group: no bank
// conflicts either way).  On GB300: 16384 x 4096 bf16 to two rows each 51 us
// (5.3 TB/s), 16 x 1536 x 4096 bf16 in transposed 128 x 128 blocks 50 us (6.0
// TB/s; 98 us with the patch unpacked to fp32, at half the resident warps).
#include <type_traits>

#include <cuda_fp8.h>

#include "wst.h"
#include "wst_common.cuh"
#include "wst_host.h"

namespace wst {

namespace {

constexpr int kQThreads = 256;

template <bool E5>
struct Fp8 {
  static constexpr float kInvLargest = (float)(1.0 / (E5 ? 57344.0 : 448.0));
  // largest = 1.75 * 2^kExp
  static constexpr int kExp = E5 ? 15 : 8;
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, E5 ? __NV_E5M2 : __NV_E4M3);
  }
  static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    return pack2(a, b) | (pack2(c, d) << 16);
  }
};

// |x| as an integer: ordered like the values, NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <bool E5, bool POW2>
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const uint32_t b = max(amax_bits, 0x0d800000u);  // 2^-100
  if (b >= 0x7f800000u) return __uint_as_float(b);
  if constexpr (POW2) {
    // amax = m 2^e, 1 <= m < 2: 2^(e - kExp) holds m <= 1.75, else one more
    const uint32_t up = (b + 0x1fffffu) & 0x7f800000u;
    return __uint_as_float(up - ((uint32_t)Fp8<E5>::kExp << 23));
  } else {
    return __fmul_rn(__uint_as_float(b), Fp8<E5>::kInvLargest);
  }
}

struct QuantArgs {
  int M, K;
  const void* x;
  long long ldx, strideX;
  uint8_t* q;
  long long ldq, strideQ;
  float* scales;
  long long lds, strideS;
  const int* position;  // ROWS: rows of q for each row of x, or NULL
  int copies, n_rows;
  WsHeader* ws;
};

// Values held per 16-byte load of X.
template <typename X>
constexpr int vec_of() { return 16 / (int)sizeof(X); }

// The largest |x| of 16 raw bytes of X as fp32 bits (NaN above infinity).
__device__ __forceinline__ uint32_t vec_amax(uint4 r, uint32_t so_far, float) {
  return max(max(so_far, max(r.x & 0x7fffffffu, r.y & 0x7fffffffu)), max(r.z & 0x7fffffffu, r.w & 0x7fffffffu));
}
__device__ __forceinline__ uint32_t vec_amax(uint4 r, uint32_t so_far, __nv_bfloat16) {
  // two at a time: |x| of bf16 is ordered like 16-bit integers, too
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
  return max(so_far, max(a & 0xffff0000u, a << 16));
}
__device__ __forceinline__ void unpack(uint4 r, float (&v)[4]) {
  v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// 16 bytes of a row from element k on; what lies behind the row's K is 0.
template <typename X>
__device__ __forceinline__ uint4 load_raw(const X* x, int k, int K) {
  constexpr int V = vec_of<X>();
  if (k + V <= K) return __ldg(reinterpret_cast<const uint4*>(x + k));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (k + i < K) {
      if constexpr (V == 4) w[i] = __float_as_uint(__ldg(x + k + i));
      else w[i >> 1] |= (uint32_t)__bfloat16_as_ushort(__ldg(x + k + i)) << (16 * (i & 1));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One warp per four blocks of a row, eight lanes and 16 values a lane each; bf16
// as two 16-byte loads of eight, fp32 as four of four.
template <typename X, bool E5, bool POW2>
__global__ void __launch_bounds__(kQThreads, 6) k_quant_rows(const QuantArgs a) {
  constexpr int V = vec_of<X>(), P = 16 / V;  // values per load, loads per lane
  const int lane = threadIdx.x & 31, l8 = lane & 7;
  const int m = (int)blockIdx.x * (kQThreads / 32) + (int)(threadIdx.x >> 5);
  if (m >= a.M) return;
  const X* x = static_cast<const X*>(a.x) + blockIdx.z * a.strideX + (long long)m * a.ldx;
  const int copies = a.position ? a.copies : 1;
  const int blocks = (a.K + 127) >> 7;
  // blockIdx.y shares a row's strips between blocks of threads (few rows)
  for (int kb0 = (int)blockIdx.y * 4; kb0 < blocks; kb0 += (int)gridDim.y * 4) {
    const int kb = kb0 + (lane >> 3), k0 = kb * 128 + l8 * V;
    uint4 raw[P];
    uint32_t amax = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) raw[p] = load_raw(x, k0 + p * 8 * V, a.K);
#pragma unroll
    for (int p = 0; p < P; ++p) amax = vec_amax(raw[p], amax, X());
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (kb >= blocks) continue;
    const float scale = block_scale<E5, POW2>(amax);
    const float inv = 1.0f / scale;
    uint32_t out[P][V / 4];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float v[V];
      unpack(raw[p], v);
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        out[p][i] = Fp8<E5>::pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    }
#pragma unroll 1
    for (int c = 0; c < copies; ++c) {
      int row = m;
      if (a.position) {
        row = __ldg(a.position + (long long)m * copies + c);
        if (row < 0) continue;
        if (row >= a.n_rows) {
          if (lane == 0) latch_error(a.ws, 1u /*WST_ERR_INVALID_ARG*/, 0x80000u);
          continue;
        }
      }
      uint8_t* q = a.q + blockIdx.z * a.strideQ + (long long)row * a.ldq;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int k = k0 + p * 8 * V;
        if (k + V <= a.K) {
          if constexpr (V == 8) *reinterpret_cast<uint2*>(q + k) = make_uint2(out[p][0], out[p][1]);
          else *reinterpret_cast<uint32_t*>(q + k) = out[p][0];
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (k + i < a.K) q[k + i] = (uint8_t)(out[p][i >> 2] >> (8 * (i & 3)));
        }
      }
      if (l8 == 0) a.scales[blockIdx.z * a.strideS + (long long)kb * a.lds + row] = scale;
    }
  }
}

// One 128 x 128 tile per block of threads; thread t holds rows (t / 16) * 8 ..
// and columns (t % 16) * 8 .. of it.
template <typename X, bool E5, bool POW2, bool COLS, bool TRANS>
__global__ void __launch_bounds__(kQThreads) k_quant_tile(const QuantArgs a) {
  constexpr int V = vec_of<X>(), P = 8 / V;
  __shared__ uint32_t part[COLS ? 16 : 1][128];
  __shared__ float col_scale[128];
  __shared__ __align__(16) uint2 tile[TRANS ? 128 : 1][16];  // [column][8-row word]
  const int t = threadIdx.x, r8 = t >> 4, c8 = t & 15;
  const int m0 = (int)blockIdx.y * 128, k0 = (int)blockIdx.x * 128;
  const X* x = static_cast<const X*>(a.x) + blockIdx.z * a.strideX;
  // (held as loaded: unpacked, bf16 would take twice the registers)
  uint4 raw[8][P];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + r8 * 8 + i;
#pragma unroll
    for (int p = 0; p < P; ++p)
      raw[i][p] = m < a.M ? load_raw(x + (long long)m * a.ldx, k0 + c8 * 8 + p * V, a.K) : make_uint4(0, 0, 0, 0);
  }
  float inv[8];
  if constexpr (COLS) {
    uint32_t b[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float v[V];
        unpack(raw[i][p], v);
#pragma unroll
        for (int j = 0; j < V; ++j) b[p * V + j] = max(b[p * V + j], abs_bits(v[j]));
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[r8][c8 * 8 + j] = b[j];
    __syncthreads();
    if (t < 128) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, part[i][t]);
      const float s = block_scale<E5, POW2>(m);
      col_scale[t] = 1.0f / s;
      if (k0 + t < a.K) a.scales[blockIdx.z * a.strideS + (long long)blockIdx.y * a.lds + k0 + t] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = col_scale[c8 * 8 + j];
  } else {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) b = vec_amax(raw[i][p], b, X());
    b = __reduce_max_sync(0xffffffffu, b);
    if ((t & 31) == 0) part[0][t >> 5] = b;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 32; ++i) b = max(b, part[0][i]);
    const float s = block_scale<E5, POW2>(b);
    if (t == 0) {
      const long long mb = blockIdx.y, kb = blockIdx.x;
      a.scales[blockIdx.z * a.strideS + (TRANS ? kb * a.lds + mb : mb * a.lds + kb)] = s;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = 1.0f / s;
  }
  // Value (row i, column j) of the patch.
  auto at = [&](int i, int j) {
    const uint4& r = raw[i][j / V];
    if constexpr (V == 4) {
      return __uint_as_float((j & 3) == 0 ? r.x : (j & 3) == 1 ? r.y : (j & 3) == 2 ? r.z : r.w);
    } else {
      const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
      return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
    }
  };
  uint8_t* q = a.q + blockIdx.z * a.strideQ;
  if constexpr (TRANS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = inv[j];
      tile[c8 * 8 + j][r8 ^ c8] = make_uint2(
          Fp8<E5>::pack4(at(0, j) * f, at(1, j) * f, at(2, j) * f, at(3, j) * f),
          Fp8<E5>::pack4(at(4, j) * f, at(5, j) * f, at(6, j) * f, at(7, j) * f));
    }
    __syncthreads();
    // 16 lanes per transposed row: 128 consecutive bytes.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 16 + r8, k = k0 + c, m = m0 + c8 * 8;
      if (k >= a.K || m >= a.M) continue;
      const uint2 word = tile[c][c8 ^ (c >> 3)];
      uint8_t* dst = q + (long long)k * a.ldq + m;
      if (m + 8 <= a.M) {
        *reinterpret_cast<uint2*>(dst) = word;
      } else {
        for (int j = 0; j < 8 && m + j < a.M; ++j) dst[j] = (uint8_t)((j < 4 ? word.x : word.y) >> (8 * (j & 3)));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = m0 + r8 * 8 + i, k = k0 + c8 * 8;
      if (m >= a.M || k >= a.K) continue;
      const uint2 word = make_uint2(
          Fp8<E5>::pack4(at(i, 0) * inv[0], at(i, 1) * inv[1], at(i, 2) * inv[2], at(i, 3) * inv[3]),
          Fp8<E5>::pack4(at(i, 4) * inv[4], at(i, 5) * inv[5], at(i, 6) * inv[6], at(i, 7) * inv[7]));
      uint8_t* dst = q + (long long)m * a.ldq + k;
      if (k + 8 <= a.K) {
        *reinterpret_cast<uint2*>(dst) = word;
      } else {
        for (int j = 0; j < 8 && k + j < a.K; ++j) dst[j] = (uint8_t)((j < 4 ? word.x : word.y) >> (8 * (j & 3)));
      }
    }
  }
}

template <typename X, bool E5, bool POW2>
void launch_quant(int mode, const QuantArgs& a, int batch, cudaStream_t s) {
  if (mode == WST_FP8_ROWS) {
    // One warp per row, or per strip of four blocks where there are few rows.
    const unsigned strips = (unsigned)((a.K + 511) / 512);
    const unsigned rows = (unsigned)((a.M + 7) / 8);
    const unsigned share = rows >= 1024 ? 1 : strips < 1024 / rows + 1 ? strips : 1024 / rows + 1;
    k_quant_rows<X, E5, POW2><<<dim3(rows, share, (unsigned)batch), kQThreads, 0, s>>>(a);
    return;
  }
  const dim3 grid((unsigned)((a.K + 127) / 128), (unsigned)((a.M + 127) / 128), (unsigned)batch);
  if (mode == WST_FP8_COLS) k_quant_tile<X, E5, POW2, true, true><<<grid, kQThreads, 0, s>>>(a);
  else if (mode == WST_FP8_BLOCKS) k_quant_tile<X, E5, POW2, false, false><<<grid, kQThreads, 0, s>>>(a);
  else k_quant_tile<X, E5, POW2, false, true><<<grid, kQThreads, 0, s>>>(a);
}

int run_quant(int mode, const QuantArgs& a, int batch, int x_type, int q_type, bool pow2, cudaStream_t s) {
  DeviceInfo dev;
  const int st = current_device_info(&dev);
  if (st) return st;
  auto go = [&](auto x, auto e5) {
    using X = decltype(x);
    constexpr bool E5 = decltype(e5)::value;
    if (pow2) launch_quant<X, E5, true>(mode, a, batch, s);
    else launch_quant<X, E5, false>(mode, a, batch, s);
  };
  auto by_q = [&](auto x) {
    if (q_type == WST_E5M2) go(x, std::true_type());
    else go(x, std::false_type());
  };
  if (x_type == WST_F32) by_q(float());
  else by_q(__nv_bfloat16());
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ST_OK : cuda_fail(e, "launch k_quant");
}

int check_quant(const char* what, int M, int K, const void* x, long ldx, int x_type, const void* q, long ldq, long q_cols,
                int q_type, const void* scales, bool stores = true) {
  if (M > 0x7fffffff - 1024 || K > 0x7fffffff - 1024)
    return reject(ST_UNSUPPORTED, "%s: M=%d K=%d: too large", what, M, K);
  if (M < 0 || K < 1) return reject(ST_INVALID_ARG, "%s: sizes out of range (M=%d K=%d)", what, M, K);
  if (x_type != WST_F32 && x_type != WST_BF16) return reject(ST_INVALID_ARG, "%s: unknown type %d", what, x_type);
  if (q_type != WST_E4M3 && q_type != WST_E5M2) return reject(ST_INVALID_ARG, "%s: unknown 8-bit type %d", what, q_type);
  if (M && (!x || (stores && (!q || !scales)))) return reject(ST_INVALID_ARG, "%s: NULL array", what);
  if (ldx < K || ldq < q_cols)
    return reject(ST_INVALID_ARG, "%s: leading dimensions too small (ldx=%ld ldq=%ld)", what, ldx, ldq);
  const long es = x_type == WST_F32 ? 4 : 2;
  if (!aligned_to(x, 16) || !aligned_to(q, 16) || !aligned_to(scales, 4) || ldx * es % 16 || ldq % 16)
    return reject(ST_ALIGNMENT, "%s: x and q must be 16-byte aligned, leading dimensions multiples of 16 bytes", what);
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

wst_status wst_quantize_fp8(wst_fp8_mode mode, int batch, int M, int K, const void* x, long ldx, long strideX,
                            wst_dtype x_type, void* q, long ldq, long strideQ, wst_fp8 q_type, float* scales, long lds,
                            long strideS, int pow2, void* stream) {
  set_error("%s", "");
  if ((int)mode < WST_FP8_ROWS || (int)mode > WST_FP8_BLOCKS_T)
    return (wst_status)reject(ST_INVALID_ARG, "quantize: unknown mode %d", (int)mode);
  if (batch < 1 || batch > 65535) return (wst_status)reject(ST_INVALID_ARG, "quantize: batch=%d outside [1, 65535]", batch);
  const bool trans = mode == WST_FP8_COLS || mode == WST_FP8_BLOCKS_T;
  WST_TRY(check_quant("quantize", M, K, x, ldx, x_type, q, ldq, trans ? M : K, q_type, scales));
  const long mb = ((long)M + 127) / 128, kb = ((long)K + 127) / 128;
  const long s_cols = mode == WST_FP8_ROWS ? M : mode == WST_FP8_COLS ? K : mode == WST_FP8_BLOCKS ? kb : mb;
  const long s_rows = mode == WST_FP8_ROWS ? kb : mode == WST_FP8_COLS ? mb : mode == WST_FP8_BLOCKS ? mb : kb;
  if (lds < s_cols) return (wst_status)reject(ST_INVALID_ARG, "quantize: leading dimension %ld of the scales < %ld", lds, s_cols);
  if (mb > 65535) return (wst_status)reject(ST_UNSUPPORTED, "quantize: M=%d: this build supports up to %d", M, 65535 * 128);
  const long es = x_type == WST_F32 ? 4 : 2;
  if (batch > 1) {
    const long q_rows = trans ? K : M, q_cols = trans ? M : K;
    if (strideX < 0 || strideQ < (q_rows - 1) * ldq + q_cols || strideS < (s_rows - 1) * lds + s_cols)
      return (wst_status)reject(ST_INVALID_ARG, "quantize: batch strides overlap (strideQ=%ld strideS=%ld)", strideQ, strideS);
    if (strideX * es % 16 || strideQ % 16)
      return (wst_status)reject(ST_ALIGNMENT, "quantize: batch strides must be multiples of 16 bytes");
  }
  if (M == 0) return WST_OK;
  WST_TRY(check_operand(x, "x"));
  WST_TRY(check_operand(q, "q"));
  WST_TRY(check_operand(scales, "scales"));
  QuantArgs a{};
  a.M = M;
  a.K = K;
  a.x = x;
  a.ldx = ldx;
  a.strideX = batch > 1 ? strideX : 0;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.strideQ = batch > 1 ? strideQ : 0;
  a.scales = scales;
  a.lds = lds;
  a.strideS = batch > 1 ? strideS : 0;
  return (wst_status)run_quant(mode, a, batch, x_type, q_type, pow2 != 0, static_cast<cudaStream_t>(stream));
}

wst_status wst_quantize_fp8_dispatch(int M, int K, int copies, const void* x, long ldx, wst_dtype x_type,
                                     const int* position, int n_rows, void* q, long ldq, wst_fp8 q_type, float* scales,
                                     long lds, int pow2, void* workspace, void* stream) {
  set_error("%s", "");
  // (without a row nothing is stored, and q and the scales may be NULL)
  WST_TRY(check_quant("quantize dispatch", M, K, x, ldx, x_type, q, ldq, K, q_type, scales, n_rows > 0));
  if (copies < 1 || n_rows < 0 || (M && !position) || !workspace)
    return (wst_status)reject(ST_INVALID_ARG, "quantize dispatch: copies=%d n_rows=%d, or a NULL array", copies, n_rows);
  if (lds < n_rows)
    return (wst_status)reject(ST_INVALID_ARG, "quantize dispatch: leading dimension %ld of the scales < %d", lds, n_rows);
  if (!aligned_to(position, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "quantize dispatch: position must be 4-byte, the workspace 16-byte aligned");
  if (M == 0) return WST_OK;
  WST_TRY(check_operand(x, "x"));
  WST_TRY(check_operand(position, "position"));
  if (n_rows > 0) {
    WST_TRY(check_operand(q, "q"));
    WST_TRY(check_operand(scales, "scales"));
  }
  WST_TRY(check_operand(workspace, "workspace"));
  QuantArgs a{};
  a.M = M;
  a.K = K;
  a.x = x;
  a.ldx = ldx;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.scales = scales;
  a.lds = lds;
  a.position = position;
  a.copies = copies;
  a.n_rows = n_rows;
  a.ws = static_cast<WsHeader*>(workspace);
  return (wst_status)run_quant(WST_FP8_ROWS, a, 1, x_type, q_type, pow2 != 0, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
