// 4-bit KV cache rows: quantising whole rows, appending the rows of one decode
// step, and reading rows back.
//
// A row x of d values (one key or value of one KV head) is held as d codes of
// four bits, two to a byte (element 2i in the low half of byte i), and one
// 32-bit word of two bf16 numbers, a scale s and a zero point z:
//
//   lo = min(0, min x), hi = max(0, max x)
//   s  = the smallest bf16 value >= (hi - lo) / 15
//   z  = rint(-lo / s)                       (an integer, 0..15)
//   c  = min(15, rint(x / s) + z)            (rint: nearest, ties to even)
//
// and stands for s (c - z); it is off by at most s / 2.  Zero is held exactly
// (the range includes it and z is an integer).  An all-zero row has s = 0.  A
// row that holds an infinity or a NaN has s = NaN and stands for NaN.
//
// The decisions are those of exact arithmetic, although everything is fp32:
// * s: subtracting and dividing with rounding up, then rounding up to bf16,
//   gives the smallest bf16 above the exact quotient, because 15 times a bf16
//   value is an fp32 value, so no intermediate rounding crosses one.  The
//   subtraction is of hi/16 and lo/16 (exact), so it cannot overflow.
// * rint(x / s): x and s have 8-bit significands, so x / s is either exactly
//   a half integer or at least 2^-11 away from one (relative to quotients up
//   to 16); the fp32 quotient can only land on a half integer if the exact
//   one does.
//
// All three kernels are bound by HBM: 2 d bytes of bf16 and d/2 + 4 bytes of
// codes and word a row.
#include "plx_internal.cuh"

#include <math_constants.h>

namespace plx {
namespace {

constexpr int kThreads = 256;

// Four packed bf16 pairs of a row: the minimum and maximum of the eight
// values, NaN if one is NaN.
__device__ __forceinline__ void minmax8(const uint4& x, __nv_bfloat162& mn, __nv_bfloat162& mx) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&x);
  mn = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
  mx = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
}

__device__ __forceinline__ __nv_bfloat162 shfl_xor2(__nv_bfloat162 v, int o) {
  uint32_t u = *reinterpret_cast<uint32_t*>(&v);
  u = __shfl_xor_sync(0xffffffffu, u, o);
  return *reinterpret_cast<__nv_bfloat162*>(&u);
}

// Scale (as fp32) and zero point of a row from its extrema.
__device__ __forceinline__ void row_params(float lo, float hi, float& s, float& z) {
  // NaN extrema stay NaN through the sums below; infinities are caught first.
  if (!(fabsf(lo) < CUDART_INF_F) || !(fabsf(hi) < CUDART_INF_F)) {
    s = CUDART_NAN_F;
    z = 0.f;
    return;
  }
  lo = fminf(lo, 0.f);
  hi = fmaxf(hi, 0.f);
  const float s16 = __fdiv_ru(__fsub_ru(hi * 0.0625f, lo * 0.0625f), 15.f) * 16.f;
  s = __uint_as_float((__float_as_uint(s16) + 0xffffu) & 0xffff0000u);  // bf16, rounded up
  z = s > 0.f ? rintf(__fdiv_rn(-lo, s)) : 0.f;
}

// The eight codes of a thread's values as one word.
__device__ __forceinline__ uint32_t pack_codes(const uint4& x, float s, float z) {
  if (!(s > 0.f)) return 0u;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    const float c = fminf(rintf(__fdiv_rn(v, s)) + z, 15.f);
    out |= (uint32_t)(int)c << (4 * i);
  }
  return out;
}

__device__ __forceinline__ uint32_t pack_word(float s, float z) {
  // The canonical bf16 NaN for a NaN scale; both are exact otherwise.
  const uint32_t us = s == s ? __float_as_uint(s) >> 16 : 0x7fffu;
  return us | (__float_as_uint(z) & 0xffff0000u);
}

// bf16 values of eight codes.
__device__ __forceinline__ uint4 unpack_values(uint32_t c, uint32_t word) {
  const float s = __uint_as_float(word << 16), z = __uint_as_float(word & 0xffff0000u);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = s * ((float)((c >> (8 * i)) & 15u) - z);
    const float b = s * ((float)((c >> (8 * i + 4)) & 15u) - z);
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    r[i] = *reinterpret_cast<uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// kLanes = d / 8 neighbouring lanes hold a row, eight values each.
template <int kLanes>
__device__ __forceinline__ void quantise_lane(const uint4& x, uint32_t& codes, uint32_t& word) {
  __nv_bfloat162 mn, mx;
  minmax8(x, mn, mx);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    mn = __hmin2_nan(mn, shfl_xor2(mn, o));
    mx = __hmax2_nan(mx, shfl_xor2(mx, o));
  }
  const float lo = __bfloat162float(__hmin_nan(mn.x, mn.y)), hi = __bfloat162float(__hmax_nan(mx.x, mx.y));
  float s, z;
  row_params(lo, hi, s, z);
  codes = pack_codes(x, s, z);
  word = pack_word(s, z);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_quantize_int4_kernel(const uint4* __restrict__ X,
                                                                      uint32_t* __restrict__ codes,
                                                                      uint32_t* __restrict__ params,
                                                                      long long rows) {
  constexpr int kLanes = D / 8;
  const long long total = rows * kLanes;
  const long long step = (long long)gridDim.x * kThreads;
  // Whole warps stay together for the shuffles; a row never straddles two.
  for (long long base = (long long)blockIdx.x * kThreads + (threadIdx.x & ~31); base < total; base += step) {
    const long long i = base + (threadIdx.x & 31);
    const bool live = i < total;
    const uint4 x = live ? X[i] : make_uint4(0u, 0u, 0u, 0u);
    uint32_t c, w;
    quantise_lane<kLanes>(x, c, w);
    if (live) {
      codes[i] = c;
      if ((threadIdx.x & (kLanes - 1)) == 0) params[i / kLanes] = w;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_dequantize_int4_kernel(const uint32_t* __restrict__ codes,
                                                                        const uint32_t* __restrict__ params,
                                                                        uint4* __restrict__ out, long long rows) {
  constexpr int kLanes = D / 8;
  const long long total = rows * kLanes;
  const long long step = (long long)gridDim.x * kThreads;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += step)
    out[i] = unpack_values(codes[i], params[i / kLanes]);
}

// The new key and value rows of every (b, KV head) go to row seqlens[b] - 1 of
// their caches; optionally the values they now stand for are given back.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_int4_kernel(Int4AppendArgs a) {
  constexpr int kLanes = D / 8;
  const int per = a.B * a.Hkv;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int row = (int)(i / kLanes), lane = (int)(i % kLanes);  // row: K rows, then V rows
  const bool live = row < 2 * per;
  const bool isv = row >= per;
  const int u = live ? (isv ? row - per : row) : 0;
  const int n = a.seqlens[u / a.Hkv];
  const bool ok = n >= 1 && n <= a.L;
  const uint4 x = live ? static_cast<const uint4*>(isv ? a.v : a.k)[(size_t)u * kLanes + lane]
                       : make_uint4(0u, 0u, 0u, 0u);
  uint32_t c, w;
  quantise_lane<kLanes>(x, c, w);
  if (!live) return;
  void* back = isv ? a.v_out : a.k_out;
  if (back)
    static_cast<uint4*>(back)[(size_t)u * kLanes + lane] = ok ? unpack_values(c, w) : make_uint4(0u, 0u, 0u, 0u);
  if (!ok) {
    if (lane == 0) atomicOr(a.status, kStatusBadSeqlen);
    return;
  }
  const size_t at = (size_t)u * a.L + (n - 1);
  static_cast<uint32_t*>(isv ? a.Vcodes : a.Kcodes)[at * kLanes + lane] = c;
  if (lane == 0) static_cast<uint32_t*>(isv ? a.Vparams : a.Kparams)[at] = w;
}

}  // namespace

cudaError_t launch_kv_quantize_int4(const void* X, void* codes, void* params, long long rows, int d,
                                    cudaStream_t st, int num_sms) {
  const long long blocks = (rows * (d / 8) + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)(blocks < 64ll * num_sms ? blocks : 64ll * num_sms);
  auto x = static_cast<const uint4*>(X);
  auto c = static_cast<uint32_t*>(codes);
  auto p = static_cast<uint32_t*>(params);
  if (d == 128) {
    kv_quantize_int4_kernel<128><<<grid, kThreads, 0, st>>>(x, c, p, rows);
  } else if (d == 64) {
    kv_quantize_int4_kernel<64><<<grid, kThreads, 0, st>>>(x, c, p, rows);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_dequantize_int4(const void* codes, const void* params, void* out, long long rows, int d,
                                      cudaStream_t st, int num_sms) {
  const long long blocks = (rows * (d / 8) + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)(blocks < 64ll * num_sms ? blocks : 64ll * num_sms);
  auto c = static_cast<const uint32_t*>(codes);
  auto p = static_cast<const uint32_t*>(params);
  auto o = static_cast<uint4*>(out);
  if (d == 128) {
    kv_dequantize_int4_kernel<128><<<grid, kThreads, 0, st>>>(c, p, o, rows);
  } else if (d == 64) {
    kv_dequantize_int4_kernel<64><<<grid, kThreads, 0, st>>>(c, p, o, rows);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_append_int4(const Int4AppendArgs& a, cudaStream_t st) {
  const long long threads = 2ll * a.B * a.Hkv * (a.d / 8);
  const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
  if (a.d == 128) {
    kv_append_int4_kernel<128><<<grid, kThreads, 0, st>>>(a);
  } else if (a.d == 64) {
    kv_append_int4_kernel<64><<<grid, kThreads, 0, st>>>(a);
  } else {
    return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace plx
