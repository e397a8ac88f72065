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
// * rint(x / s): x and s have 8-bit significands, so x / s (at most 15.5) is a
//   half integer or at least 2^-11 away from one.  x r with r = 1 / s rounded is
//   within 2^-19 of it, and one FMA rounds that to a multiple of 2^-12: ties are
//   ties again, and nothing else is.  Adding 1.5 2^23 then rounds to an integer,
//   ties to even, which sits in the low mantissa bits.
//
// Bound: HBM.  2 d bytes of bf16 and d/2 + 4 bytes of codes and word a row; a
// division an element would cost more than the stream (84 us for 8 x 16 x 4096
// rows of 128, where this takes 29).
#include "launch.cuh"
#include "plx_internal.cuh"

#include <math_constants.h>

namespace plx {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;               // independent loads of a thread (reading back)
constexpr float kGrid = 0x1.8p11f;       // its ulp is 2^-12
constexpr float kWhole = 0x1.8p23f;      // its ulp is 1
constexpr uint32_t kWholeBits = 0x4b400000u;

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// A row is held by kRowLanes neighbouring lanes, lane t with its pieces (of eight
// values) t, t + 4, ...: what is computed once a row costs a fourth of it a lane.
constexpr int kRowLanes = 4;
template <int D>
constexpr int kPieces = D / (8 * kRowLanes);

// (minimum, -maximum) of a row, NaN if one is NaN.
template <int N>
__device__ __forceinline__ __nv_bfloat162 row_range(const uint4 (&x)[N]) {
  __nv_bfloat162 mn = as_bf2(x[0].x), mx = mn;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mn = __hmin2_nan(__hmin2_nan(mn, as_bf2(x[i].x)), __hmin2_nan(as_bf2(x[i].y), __hmin2_nan(as_bf2(x[i].z), as_bf2(x[i].w))));
    mx = __hmax2_nan(__hmax2_nan(mx, as_bf2(x[i].x)), __hmax2_nan(as_bf2(x[i].y), __hmax2_nan(as_bf2(x[i].z), as_bf2(x[i].w))));
  }
  const uint32_t a = as_u32(mn), b = as_u32(mx) ^ 0x80008000u;
  __nv_bfloat162 r = __hmin2_nan(as_bf2(__byte_perm(a, b, 0x5410)), as_bf2(__byte_perm(a, b, 0x7632)));
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) r = __hmin2_nan(r, as_bf2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
  return r;
}

// Integers k = rint(x / s) as kWholeBits + k.
__device__ __forceinline__ float whole(float x, float r) { return fmaf(x, r, kGrid) + (kWhole - kGrid); }

// Codes of a lane's pieces, and the row's word.
template <int N>
__device__ __forceinline__ void quantise_lane(const uint4 (&x)[N], uint32_t (&codes)[N], uint32_t& word) {
  const __nv_bfloat162 range = row_range(x);
  float lo = __bfloat162float(range.x), hi = -__bfloat162float(range.y);
#pragma unroll
  for (int p = 0; p < N; ++p) codes[p] = 0u;
  if (!(fabsf(lo) < CUDART_INF_F) || !(fabsf(hi) < CUDART_INF_F)) {
    word = 0x7fffu;  // NaN, 0
    return;
  }
  lo = fminf(lo, 0.f);
  hi = fmaxf(hi, 0.f);
  const float s16 = __fdiv_ru(__fsub_ru(hi * 0.0625f, lo * 0.0625f), 15.f) * 16.f;
  const uint32_t su = (__float_as_uint(s16) + 0xffffu) & 0xffff0000u;  // bf16, rounded up
  word = su >> 16;
  if (su == 0u) return;
  const float s = __uint_as_float(su);
  if (s < 0x1p-100f) {  // 1 / s may overflow: divide
    const float z = rintf(__fdiv_rn(-lo, s));
#pragma unroll
    for (int p = 0; p < N; ++p) {
      const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
        codes[p] |= (uint32_t)(int)fminf(rintf(__fdiv_rn(v, s)) + z, 15.f) << (4 * i);
      }
    }
    word |= __float_as_uint(z) & 0xffff0000u;
    return;
  }
  const float r = __frcp_rn(s);
  const float z = whole(-lo, r) - kWhole;
  const float top = kWhole + 15.f - z;
  // Sum of (kWholeBits + k_i) 16^i, modulo 2^32; the codes k_i + z lie in 0..15.
  const uint32_t less = ((uint32_t)(int)z - kWholeBits) * 0x11111111u;
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
    codes[p] = less;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
      codes[p] += __float_as_uint(fminf(whole(v, r), top)) << (4 * i);
    }
  }
  word |= __float_as_uint(z) & 0xffff0000u;
}

// bf16 values of eight codes.
__device__ __forceinline__ uint4 unpack_values(uint32_t c, uint32_t word) {
  const float s = __uint_as_float(word << 16), z = __uint_as_float(word & 0xffff0000u) + 0x1p23f;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 2^23 + c, less 2^23 + z
    const float a = s * (__uint_as_float(((c >> (8 * i)) & 15u) | 0x4b000000u) - z);
    const float b = s * (__uint_as_float(((c >> (8 * i + 4)) & 15u) | 0x4b000000u) - z);
    r[i] = as_u32(__floats2bfloat162_rn(a, b));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_quantize_int4_kernel(const uint4* X, uint32_t* codes, uint32_t* params,
                                                                    long long rows) {
  constexpr int N = kPieces<D>, kRows = kThreads / kRowLanes;
  const int t = threadIdx.x % kRowLanes;
  const long long step = (long long)gridDim.x * kRows;
  grid_dep_wait();  // (no __restrict__ here: loads that count as invariant may move above this)
  grid_dep_launch();
  // Whole warps stay together for the shuffles.
  for (long long base = (long long)blockIdx.x * kRows + (threadIdx.x & ~31) / kRowLanes; base < rows; base += step) {
    const long long row = base + (threadIdx.x & 31) / kRowLanes, at = row * (D / 8) + t;
    uint4 x[N];
#pragma unroll
    for (int p = 0; p < N; ++p) x[p] = row < rows ? __ldcs(X + at + kRowLanes * p) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t c[N], w;
    quantise_lane(x, c, w);
    if (row < rows) {
#pragma unroll
      for (int p = 0; p < N; ++p) codes[at + kRowLanes * p] = c[p];
      if (t == 0) params[row] = w;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_dequantize_int4_kernel(const uint32_t* codes, const uint32_t* params,
                                                                      uint4* out, long long total) {
  constexpr int kLanes = D / 8;
  const long long step = (long long)gridDim.x * kThreads * kUnroll;
  grid_dep_wait();
  grid_dep_launch();
  for (long long base = (long long)blockIdx.x * kThreads * kUnroll + threadIdx.x; base < total; base += step) {
    uint32_t c[kUnroll], w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = base + u * kThreads;
      if (i < total) {
        c[u] = codes[i];
        w[u] = params[i / kLanes];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = base + u * kThreads;
      if (i < total) __stcs(out + i, unpack_values(c[u], w[u]));
    }
  }
}

// The new key and value rows of every (b, KV head) go to row seqlens[b] - 1 of
// their caches; optionally the values they now stand for are given back.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_int4_kernel(Int4AppendArgs a) {
  constexpr int N = kPieces<D>, kLanes = D / 8;
  grid_dep_wait();
  grid_dep_launch();
  const int per = a.B * a.Hkv, t = threadIdx.x % kRowLanes;
  const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) / kRowLanes;  // K rows, then V rows
  const bool live = row < 2ll * per, isv = row >= per;
  const int u = live ? (int)(isv ? row - per : row) : 0;
  const int n = a.seqlens[u / a.Hkv];
  const bool ok = n >= 1 && n <= a.L;
  const uint4* from = static_cast<const uint4*>(isv ? a.v : a.k) + (size_t)u * kLanes + t;
  uint4 x[N];
#pragma unroll
  for (int p = 0; p < N; ++p) x[p] = live ? from[kRowLanes * p] : make_uint4(0u, 0u, 0u, 0u);
  uint32_t c[N], w;
  quantise_lane(x, c, w);
  if (!live) return;
  if (void* back = isv ? a.v_out : a.k_out) {
    uint4* to = static_cast<uint4*>(back) + (size_t)u * kLanes + t;
#pragma unroll
    for (int p = 0; p < N; ++p) to[kRowLanes * p] = ok ? unpack_values(c[p], w) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (!ok) {
    if (t == 0) atomicOr(a.status, kStatusBadSeqlen);
    return;
  }
  const size_t at = (size_t)u * a.L + (n - 1);
  uint32_t* to = static_cast<uint32_t*>(isv ? a.Vcodes : a.Kcodes) + at * kLanes + t;
#pragma unroll
  for (int p = 0; p < N; ++p) to[kRowLanes * p] = c[p];
  if (t == 0) static_cast<uint32_t*>(isv ? a.Vparams : a.Kparams)[at] = w;
}

}  // namespace

cudaError_t launch_kv_quantize_int4(const void* X, void* codes, void* params, long long rows, int d,
                                    cudaStream_t st, int num_sms) {
  const long long blocks = (rows + kThreads / kRowLanes - 1) / (kThreads / kRowLanes);
  const unsigned grid = (unsigned)(blocks < 64ll * num_sms ? blocks : 64ll * num_sms);
  if (d != 64 && d != 128) return cudaErrorInvalidValue;
  return launch_dependent(d == 128 ? kv_quantize_int4_kernel<128> : kv_quantize_int4_kernel<64>, grid, kThreads, 0, 1, st,
                          static_cast<const uint4*>(X), static_cast<uint32_t*>(codes), static_cast<uint32_t*>(params),
                          rows);
}

cudaError_t launch_kv_dequantize_int4(const void* codes, const void* params, void* out, long long rows, int d,
                                      cudaStream_t st, int num_sms) {
  const long long total = rows * (d / 8), blocks = (total + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const unsigned grid = (unsigned)(blocks < 64ll * num_sms ? blocks : 64ll * num_sms);
  if (d != 64 && d != 128) return cudaErrorInvalidValue;
  return launch_dependent(d == 128 ? kv_dequantize_int4_kernel<128> : kv_dequantize_int4_kernel<64>, grid, kThreads, 0, 1,
                          st, static_cast<const uint32_t*>(codes), static_cast<const uint32_t*>(params),
                          static_cast<uint4*>(out), total);
}

cudaError_t launch_kv_append_int4(const Int4AppendArgs& a, cudaStream_t st) {
  const long long threads = 2ll * a.B * a.Hkv * kRowLanes;
  const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
  if (a.d != 64 && a.d != 128) return cudaErrorInvalidValue;
  return launch_dependent(a.d == 128 ? kv_append_int4_kernel<128> : kv_append_int4_kernel<64>, grid, kThreads, 0, 1, st,
                          a);
}

}  // namespace plx
