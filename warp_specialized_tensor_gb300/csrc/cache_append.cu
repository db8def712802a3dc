// cache_append.cu -- new keys and values into a paged cache, the position
// rotation applied on the way (and to the queries).
//
//   (a, b) -> (a cos x - b sin x, b cos x + a sin x),  x = position * inv_freq[j]
//
// The angle matters modulo one turn only.  inv_freq / 2 pi is kept as a 64-bit
// fraction of a turn, so its product with an integer position modulo 2^64 IS the
// reduction: exact, for near and far positions alike, one integer multiplication
// per angle (the fraction itself is rounded to about 2^-52 relative: 5e-7 radians at
// position 2^31 and inv_freq 1, 2e-10 at a million).
//
// Bound by HBM: every component moves in and out once.  A block takes a step of one token
// at a time, or of several small ones (two units to a thread); its threads compute the
// step's sines and cosines into shared memory while their first two units of data are in
// flight.  A unit is 16 components of a head: two 16-byte words of bf16, the two halves of
// eight pairs.  Measured: 16,384 tokens of 32 + 2 x 8 heads of 128, bf16: 71.6 us, 403 MB at
// 5.6 TB/s (a plain copy reaches 6.8); 5,003 of 14 + 2 x 2 heads of 64, fp32: 10.0 us, 33 MB (a
// token to a step 19.8 us, three of four threads without a unit); 32 tokens 2.6 us, of which a
// launch is 2.
#include <algorithm>

#include "wst.h"
#include "wst_common.cuh"
#include "wst_host.h"

namespace wst {

namespace {

constexpr int kAppendThreads = 192;  // two units each for 48 heads of 128
constexpr int kAppendMaxDh = 256;    // rot / 2 <= 128 angles
constexpr int kAppendAngles = 1024;  // of a step
// blocks that fit an SM by their registers
template <typename X>
constexpr int kAppendBlocks = sizeof(X) == 2 ? 5 : 4;

struct AppendArgs {
  int tokens;  // of a step
  int T, H, Hkv, Dh, rot;
  const void* q;
  long long ldq;
  const void* k;
  long long ldk;
  const void* v;
  long long ldv;
  const int* positions;
  const float* inv_freq;
  const int* slots;
  __nv_bfloat16* q_out;
  long long ldqo;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  long long num_slots;
  int page_size;
  long long page_stride, token_stride, head_stride;
  WsHeader* ws;
};

// Eight components as loaded.  Plain loads: q_out may be q.
template <typename X>
struct Chunk {
  uint4 w[sizeof(X) / 2];
};
template <typename X>
__device__ __forceinline__ Chunk<X> load_chunk(const X* p) {
  Chunk<X> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(X) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void unpack(const Chunk<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void unpack(const Chunk<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// One unit of a token: where it comes from and goes to, and its first angle (-1:
// copied).
template <typename X>
struct Unit {
  Chunk<X> lo, hi;
  __nv_bfloat16 *dlo, *dhi;
  int angle;
};

template <typename X, bool PAIRS>
__device__ __forceinline__ void load_unit(const AppendArgs& p, int t, long long slot_at, int u, int per_head, Unit<X>& r) {
  int head = u / per_head;
  const int c = u - head * per_head;
  const X* src;
  __nv_bfloat16* dst;
  bool turn = c < p.rot / 16;
  if (head < p.H) {
    src = static_cast<const X*>(p.q) + (long long)t * p.ldq + (long long)head * p.Dh;
    dst = p.q_out + (long long)t * p.ldqo + (long long)head * p.Dh;
  } else if ((head -= p.H) < p.Hkv) {
    src = static_cast<const X*>(p.k) + (long long)t * p.ldk + (long long)head * p.Dh;
    dst = p.k_cache + slot_at + head * p.head_stride;
  } else {
    head -= p.Hkv;
    src = static_cast<const X*>(p.v) + (long long)t * p.ldv + (long long)head * p.Dh;
    dst = p.v_cache + slot_at + head * p.head_stride;
    turn = false;
  }
  // WST_ROPE_HALVES turns components 8c.. with rot/2 + 8c..; everything else is 16
  // consecutive components.
  const int lo = turn && !PAIRS ? 8 * c : 16 * c;
  const int hi = turn && !PAIRS ? p.rot / 2 + 8 * c : lo + 8;
  r.lo = load_chunk(src + lo);
  r.hi = load_chunk(src + hi);
  r.dlo = dst + lo;
  r.dhi = dst + hi;
  r.angle = turn ? 8 * c : -1;
}

template <typename X, bool PAIRS>
__device__ __forceinline__ void store_unit(const Unit<X>& r, const float2* cs) {
  float a[8], b[8];
  unpack(r.lo, a);
  unpack(r.hi, b);
  if (r.angle >= 0) {
    const float4* c4 = reinterpret_cast<const float4*>(cs + r.angle);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 z = c4[i];  // cosine and sine of angles 2i and 2i + 1
      if constexpr (PAIRS) {
        // pairs 2i and 2i+1 lie in `a` (i < 2) or `b`
        float* v = i < 2 ? a + 4 * i : b + 4 * (i - 2);
        const float x0 = v[0], y0 = v[1], x1 = v[2], y1 = v[3];
        v[0] = fmaf(x0, z.x, -(y0 * z.y));
        v[1] = fmaf(y0, z.x, x0 * z.y);
        v[2] = fmaf(x1, z.z, -(y1 * z.w));
        v[3] = fmaf(y1, z.z, x1 * z.w);
      } else {
        const float x0 = a[2 * i], y0 = b[2 * i], x1 = a[2 * i + 1], y1 = b[2 * i + 1];
        a[2 * i] = fmaf(x0, z.x, -(y0 * z.y));
        b[2 * i] = fmaf(y0, z.x, x0 * z.y);
        a[2 * i + 1] = fmaf(x1, z.z, -(y1 * z.w));
        b[2 * i + 1] = fmaf(y1, z.z, x1 * z.w);
      }
    }
  }
  store_chunk(r.dlo, a);
  store_chunk(r.dhi, b);
}

template <typename X, bool PAIRS>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks<X>) k_cache_append(const AppendArgs p) {
  __shared__ __align__(16) float2 cs[2][kAppendMaxDh / 2];
  const int tid = (int)threadIdx.x;
  const int half = p.rot / 2;
  const int per_head = p.Dh / 16;
  const int units = (p.H + 2 * p.Hkv) * per_head;
  early_wait();
  unsigned long long turn = 0;  // this thread's angle: turns per position, as a 64-bit fraction
  if (tid < half) {
    double x = (double)__ldg(p.inv_freq + tid) * 0.15915494309189533577;  // 1 / (2 pi)
    x -= floor(x);                                                         // in [0, 1]
    turn = x < 1.0 ? (unsigned long long)(x * 18446744073709551616.0) : 0ull;
  }
  int buf = 0;
  for (int t = (int)blockIdx.x; t < p.T; t += (int)gridDim.x) {
    const int slot = __ldg(p.slots + t);
    if (slot < 0 || slot >= p.num_slots) {
      if (slot >= 0 && tid == 0) latch_error(p.ws, (uint32_t)ST_INVALID_ARG, kRoleProducer << 16);
      continue;
    }
    const int page = slot / p.page_size;
    const long long slot_at = page * p.page_stride + (slot - page * p.page_size) * p.token_stride;
    Unit<X> u0, u1;
    const bool has0 = tid < units, has1 = tid + kAppendThreads < units;
    if (has0) load_unit<X, PAIRS>(p, t, slot_at, tid, per_head, u0);
    if (has1) load_unit<X, PAIRS>(p, t, slot_at, tid + kAppendThreads, per_head, u1);
    if (tid < half) {
      // signed half turns, in [-1, 1)
      const long long at = (long long)(turn * (unsigned long long)(long long)__ldg(p.positions + t));
      float s, c;
      sincospif((float)at * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
      cs[buf][tid] = make_float2(c, s);
    }
    __syncthreads();  // (the other buffer is written next, after every thread has left this one's last use)
    if (has0) store_unit<X, PAIRS>(u0, cs[buf]);
    if (has1) store_unit<X, PAIRS>(u1, cs[buf]);
    for (int u = tid + 2 * kAppendThreads; u < units; u += 2 * kAppendThreads) {
      const bool more = u + kAppendThreads < units;
      load_unit<X, PAIRS>(p, t, slot_at, u, per_head, u0);
      if (more) load_unit<X, PAIRS>(p, t, slot_at, u + kAppendThreads, per_head, u1);
      store_unit<X, PAIRS>(u0, cs[buf]);
      if (more) store_unit<X, PAIRS>(u1, cs[buf]);
    }
    buf ^= 1;
  }
}

// The same for steps of several tokens, two units to a thread.  (One kernel for both takes
// 74 us for the 16,384 tokens above, a token a step, against 71.6.)
template <typename X, bool PAIRS>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks<X>) k_cache_append_several(const AppendArgs p) {
  __shared__ __align__(16) float2 cs[2][kAppendAngles];
  const int tid = (int)threadIdx.x;
  const int half = p.rot / 2;
  const int per_head = p.Dh / 16;
  const int units = (p.H + 2 * p.Hkv) * per_head;
  // A thread's angle is the same for all its tokens; `angles` tokens at a time.
  const int angles = half ? kAppendThreads / half : 0;
  const int k_angle = half ? tid / half : 0, j_angle = tid - k_angle * half;
  early_wait();
  unsigned long long turn = 0;
  if (k_angle < angles) {
    double x = (double)__ldg(p.inv_freq + j_angle) * 0.15915494309189533577;
    x -= floor(x);
    turn = x < 1.0 ? (unsigned long long)(x * 18446744073709551616.0) : 0ull;
  }
  // this thread's two units of a step: token and unit of it
  const int k0 = tid / units, k1 = (tid + kAppendThreads) / units;
  const int u0 = tid - k0 * units, u1 = tid + kAppendThreads - k1 * units;
  const int stride = (int)gridDim.x * p.tokens;
  // (T is below 2^31 - 65536, a stride below 65536)
  auto slot_of = [&](int t, int k) { return k < p.tokens && t + k < p.T ? __ldg(p.slots + t + k) : -1; };
  auto place = [&](int slot) {
    const int page = slot / p.page_size;
    return page * p.page_stride + (slot - page * p.page_size) * p.token_stride;
  };
  int t = (int)blockIdx.x * p.tokens;
  int slot0 = slot_of(t, k0), slot1 = slot_of(t, k1);
  int buf = 0;
  for (; t < p.T; t += stride) {
    const bool has0 = slot0 >= 0 && slot0 < p.num_slots, has1 = slot1 >= 0 && slot1 < p.num_slots;
    if (slot0 >= p.num_slots || slot1 >= p.num_slots) latch_error(p.ws, (uint32_t)ST_INVALID_ARG, kRoleProducer << 16);
    Unit<X> a, b;
    if (has0) load_unit<X, PAIRS>(p, t + k0, place(slot0), u0, per_head, a);
    if (has1) load_unit<X, PAIRS>(p, t + k1, place(slot1), u1, per_head, b);
    slot0 = slot_of(t + stride, k0);  // (the next step's)
    slot1 = slot_of(t + stride, k1);
    if (k_angle < angles)
      for (int k = k_angle; k < min(p.tokens, p.T - t); k += angles) {
        const long long at = (long long)(turn * (unsigned long long)(long long)__ldg(p.positions + t + k));
        float s, c;
        sincospif((float)at * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
        cs[buf][k * half + j_angle] = make_float2(c, s);
      }
    __syncthreads();  // (as above)
    if (has0) store_unit<X, PAIRS>(a, cs[buf] + k0 * half);
    if (has1) store_unit<X, PAIRS>(b, cs[buf] + k1 * half);
    buf ^= 1;
  }
}

template <typename X>
cudaError_t launch_append(AppendArgs a, bool pairs, int num_sms, cudaStream_t stream) {
  // Blocks for all SMs first, then tokens to a step: as many as their units and angles
  // allow, no more than make the steps of a block equally long.  (Eight times the blocks, a
  // step each, take 97 us and 15 us for the two prompts named above.)
  const int blocks = num_sms * kAppendBlocks<X>;
  const int units = (a.H + 2 * a.Hkv) * (a.Dh / 16);
  const int most = std::max(1, std::min(2 * kAppendThreads / units, kAppendAngles / std::max(64, a.rot / 2)));
  const int steps = (int)((a.T + (long long)blocks * most - 1) / ((long long)blocks * most));
  a.tokens = (int)((a.T + (long long)blocks * steps - 1) / ((long long)blocks * steps));
  const int grid = std::min((a.T + a.tokens - 1) / a.tokens, blocks);
  const auto kern = a.tokens > 1 ? (pairs ? k_cache_append_several<X, true> : k_cache_append_several<X, false>)
                                 : (pairs ? k_cache_append<X, true> : k_cache_append<X, false>);
  return launch_early(kern, dim3((unsigned)grid), kAppendThreads, 0, stream, a);
}

}  // namespace

int check_cache(const char* what, const void* k_cache, const void* v_cache, int num_pages, int page_size, long page_stride,
                long token_stride, long head_stride) {
  if (num_pages < 1 || page_size < 1) return reject(ST_INVALID_ARG, "%s: num_pages=%d page_size=%d", what, num_pages, page_size);
  if ((long long)num_pages * page_size > 0x7fffffffll)
    return reject(ST_UNSUPPORTED, "%s: %d pages of %d: slots are below 2^31", what, num_pages, page_size);
  if (!k_cache || !v_cache) return reject(ST_INVALID_ARG, "%s: NULL cache", what);
  if (page_stride < 0 || token_stride < 0 || head_stride < 0) return reject(ST_INVALID_ARG, "%s: negative stride", what);
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || page_stride % 8 || token_stride % 8 || head_stride % 8)
    return reject(ST_ALIGNMENT, "%s: the caches must be 16-byte aligned, their strides multiples of 16 bytes", what);
  return ST_OK;
}

}  // namespace wst

using namespace wst;

#define WST_TRY(expr)                  \
  do {                                 \
    int st__ = (expr);                 \
    if (st__) return (wst_status)st__; \
  } while (0)

extern "C" {

wst_status wst_cache_append_bf16(int T, int H, int Hkv, int Dh, int rot, wst_rope style, const void* q, long ldq,
                                 const void* k, long ldk, const void* v, long ldv, wst_dtype x_type,
                                 const int* positions, const float* inv_freq, const int* slots, void* q_out,
                                 long ldqo, void* k_cache, void* v_cache, int num_pages, int page_size,
                                 long page_stride, long token_stride, long head_stride, void* workspace,
                                 void* stream) {
  set_error("%s", "");
  if (!q) H = 0;
  if (T < 0 || Hkv < 1 || Dh < 1 || rot < 0 || rot > Dh || (q && H < 1))
    return (wst_status)reject(ST_INVALID_ARG, "append: sizes out of range (T=%d H=%d Hkv=%d Dh=%d rot=%d)", T, H, Hkv, Dh, rot);
  if (Dh % 16 || rot % 16 || Dh > kAppendMaxDh)
    return (wst_status)reject(ST_UNSUPPORTED, "append: Dh=%d rot=%d: multiples of 16, Dh up to %d", Dh, rot, kAppendMaxDh);
  if (T > 0x7fffffff - 65536 || (long long)H + 2ll * Hkv > (1ll << 26))
    return (wst_status)reject(ST_UNSUPPORTED, "append: T=%d with %d + 2 x %d heads: too large", T, H, Hkv);
  if ((int)style != WST_ROPE_HALVES && (int)style != WST_ROPE_PAIRS)
    return (wst_status)reject(ST_INVALID_ARG, "append: unknown pairing %d", (int)style);
  if (x_type != WST_F32 && x_type != WST_BF16) return (wst_status)reject(ST_INVALID_ARG, "append: unknown type %d", (int)x_type);
  if (T && (!k || !v || !slots || (q && !q_out) || (rot && (!positions || !inv_freq))))
    return (wst_status)reject(ST_INVALID_ARG, "append: NULL array");
  if (!workspace) return (wst_status)reject(ST_INVALID_ARG, "append: workspace is NULL");
  WST_TRY(check_cache("append", k_cache, v_cache, num_pages, page_size, page_stride, token_stride, head_stride));
  const long es = x_type == WST_F32 ? 4 : 2;
  if (ldk < (long)Hkv * Dh || ldv < (long)Hkv * Dh || (q && (ldq < (long)H * Dh || ldqo < (long)H * Dh)))
    return (wst_status)reject(ST_INVALID_ARG, "append: leading dimensions too small (ldq=%ld ldk=%ld ldv=%ld ldqo=%ld)", ldq, ldk, ldv, ldqo);
  if (head_stride < Dh && Hkv > 1) return (wst_status)reject(ST_INVALID_ARG, "append: head_stride=%ld makes heads overlap", head_stride);
  if (q && q_out == q && (x_type != WST_BF16 || ldqo != ldq))
    return (wst_status)reject(ST_INVALID_ARG, "append: in place q has to be bf16 with ldqo == ldq");
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || ldk * es % 16 || ldv * es % 16 ||
      (q && (!aligned_to(q, 16) || !aligned_to(q_out, 16) || ldq * es % 16 || ldqo % 8)))
    return (wst_status)reject(ST_ALIGNMENT, "append: q, k, v and q_out must be 16-byte aligned, leading dimensions multiples of 16 bytes");
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(slots, 4) || !aligned_to(workspace, 16))
    return (wst_status)reject(ST_ALIGNMENT, "append: positions, inv_freq and slots must be 4-byte, the workspace 16-byte aligned");
  if (T == 0) return WST_OK;
  if (q) {
    WST_TRY(check_operand(q, "q"));
    WST_TRY(check_operand(q_out, "q_out"));
  }
  WST_TRY(check_operand(k, "k"));
  WST_TRY(check_operand(v, "v"));
  if (rot) {
    WST_TRY(check_operand(positions, "positions"));
    WST_TRY(check_operand(inv_freq, "inv_freq"));
  }
  WST_TRY(check_operand(slots, "slots"));
  WST_TRY(check_operand(k_cache, "k_cache"));
  WST_TRY(check_operand(v_cache, "v_cache"));
  WST_TRY(check_operand(workspace, "workspace"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  AppendArgs a{};
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.Dh = Dh;
  a.rot = rot;
  a.q = q;
  a.ldq = ldq;
  a.k = k;
  a.ldk = ldk;
  a.v = v;
  a.ldv = ldv;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.slots = slots;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.ldqo = ldqo;
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.num_slots = (long long)num_pages * page_size;
  a.page_size = page_size;
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.ws = static_cast<WsHeader*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = x_type == WST_F32 ? launch_append<float>(a, style == WST_ROPE_PAIRS, dev.num_sms, s)
                                          : launch_append<__nv_bfloat16>(a, style == WST_ROPE_PAIRS, dev.num_sms, s);
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_cache_append");
}

}  // extern "C"
