// Decode over a 4-bit KV cache, and decodes (4-bit or bf16 cache) that also
// collect every key's softmax weight.
//
// Per query head h of a group of G that reads KV head g, over the n visible
// rows of its cache:
//
//   s_j = q.k_j / sqrt(d),  p = softmax(s),  t_j = rho.k_j
//   out = sum_j p_j (1 - t_j + tbar) v_j,    tbar = sum_j p_j t_j
//   w_out[j] = w_in[j] + sum over the heads of the group of p_j     (optional)
//
// streamed with one running reference m: omega = sum w, T = sum w t,
// O1 = sum w v, O2 = sum w t v with w = 2^(s log2 e - m), and
// out = ((1 + T/omega) O1 - O2) / omega.  Taking one number off all t_j does not
// change out, so T and O2 are sums over t_j - t0, t0 the mean of t over the first
// tile that a warp weighs: with t far from 0 for all keys (a direction that they
// share and the probe sees) out would else be the small difference of two large
// sums whose weights keep 16 bits.  300 keys with t of 2^15 + N(0, 9): off by up to
// 0.06 in outputs of 0.1 without, by their rounding with t0.
//
// Bound: HBM.  A key costs 2 (d/2 + 4) bytes (4-bit) or 4 d (bf16) and 8 d
// flops per query head; at 4 bits and d = 128 the stream leaves an SM 5.8
// clocks per key, so the arithmetic is arranged to stay well below that:
//
// * Everything is on m16n8k16 MMAs with the keys (scores) or the head dims
//   (values) as the 16 rows and the query rows as the 8 columns: columns 2t and
//   2t+1 of lane t are q and rho of one head, so a lane holds a head's s and t
//   of a key together, and one MMA per key serves groups up to 4 (d = 128).
//   [w s_v, w t s_v] packs into one register, and movmatrix turns the score
//   layout into the value MMA's operand.  Measured rate: one MMA in 2.0 clocks
//   an SM.
// * AND picks two nibbles of a code word, and these bits are bf16 numbers:
//   c 2^-133 (or c 2^-129: bits 4..7 still lie in the linear range of bf16).
//   Key codes go into the MMA as such, against queries scaled by a power of two;
//   z (sum of q) goes off each score.  Value codes become (c - z) 2^-6 in one FMA
//   first, exactly: sums over raw codes would be large, with small differences.
//   The dims are paired as the nibbles fall; the other operand is permuted to match.
//   Value codes come transposed, four keys of a byte in a register (ldmatrix on bytes).
// * Groups of 1 and 2 leave columns free: the weights go in as bf16 hi + lo
//   pairs there; larger groups issue a second MMA for the lo part.  So the
//   weights keep 16 bits.
// * The reference m is raised lazily, when a score passes it: a raise sets it
//   2^8 above the largest score seen, so weights stay in (0, 1].
// * Each warp runs its own ring of key tiles with cp.async (no block barrier in
//   the loop, no wait that could not end) and its own partial state.
//
// Three ways to cut the keys (cache_decode_space chooses): one CTA a (b, KV head);
// a cluster of CTAs, merged through distributed shared memory; or all tiles of the
// batch in equal shares, one a warp, with partial records in the caller's
// workspace that a second kernel merges.  There are no counters and no
// library-owned memory: calls on several streams are independent.
//
// What bounds it now: instructions.  14.6 a key and warp at G = 1, d = 128, 17 at
// G = 4 (issue slots 60 % and 55 % busy, the ALU pipe 59 % and 46 %, the MMA pipe
// 34 % and 38 %; 12 or 20 warps an SM in place of 16 change nothing or lose).  64 x
// 16 sequences of 4096 keys, one row appended to each before: 101 to 104 us on a
// rested GPU, 115 to 118 us at the clock that a long run keeps: 0.87 and 0.75 of a
// copy's rate.
#include "launch.cuh"
#include "plx_internal.cuh"

#include <cooperative_groups.h>
#include <math_constants.h>

#include <atomic>

namespace cg = cooperative_groups;

namespace plx {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kHeadroom = 8.f;   // log2 units a raise leaves above the largest score
constexpr float kNoRef = -3e38f;   // reference before any key (finite: no inf - inf)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zeros.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Two 16 x 16 byte matrices, transposed: lane (g, t) gets bytes of rows 4t .. 4t + 3,
// of column g and of column g + 8, for each.  Lanes 0-15 (16-31) give the first's
// (second's) row addresses.
__device__ __forceinline__ void ldmatrix2_bytes_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// 16- and 4-byte asynchronous copies; in the z forms ok == false fills zeros and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
// How rows stay in L2: as other lines, or first to go.
__device__ __forceinline__ uint64_t l2_policy(bool first) {
  uint64_t normal, early;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(early));
  return first ? early : normal;
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds64(uint32_t& x, uint32_t& y, uint32_t a) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
}
__device__ __forceinline__ void lds128(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Two nibbles of x as bf16: kEven picks bits 0..3 and 16..19, kOdd bits 4..7
// and 20..23; they read as c 2^-133 and c 2^-129.  nib_*: (c - z) 2^-6, with
// mz = (-z 2^-6) of each half's key.
constexpr uint32_t kEven = 0x000f000fu, kOdd = 0x00f000f0u;
constexpr uint32_t kScaleEven = 0x7f007f00u;  // 2^127: c 2^-133 -> c 2^-6
constexpr uint32_t kScaleOdd = 0x7d007d00u;   // 2^123: c 2^-129 -> c 2^-6
__device__ __forceinline__ uint32_t nib_even(uint32_t x, uint32_t mz) {
  return fma_bf16x2(x & kEven, kScaleEven, mz);
}
__device__ __forceinline__ uint32_t nib_odd(uint32_t x, uint32_t mz) {
  return fma_bf16x2(x & kOdd, kScaleOdd, mz);
}
__device__ __forceinline__ uint32_t neg_zero_points(uint32_t z2) {  // (z, z') -> (-z 2^-6, -z' 2^-6)
  return fma_bf16x2(z2, 0xbc80bc80u, 0u);
}

// Sizes of one instantiation.
template <bool I4, int D>
struct Tile {
  static constexpr int kRow = I4 ? D / 2 : 2 * D;         // bytes of a row
  static constexpr int kKeys = I4 ? 32 : 2048 / D;        // keys of a stage
  static constexpr int kStages = 3;
  static constexpr int kChunks = kRow / 16;               // 16-byte pieces of a row
  static constexpr int kVOff = kKeys * kRow;              // a stage: K rows, V rows, (K word, V word) of every key
  static constexpr int kPOff = 2 * kKeys * kRow;
  static constexpr int kBytes = kPOff + (I4 ? 8 * kKeys : 0);
  static constexpr int kWarpBytes = kStages * kBytes;
  static constexpr int kRing = kWarps * kWarpBytes;
};

// Where a V row and its 16-byte pieces sit in a stage: ldmatrix reads one piece of
// 8 rows at a time, so the pieces change places from row to row.
template <bool I4, int D>
__device__ __forceinline__ int v_place(int key, int chunk) {
  if constexpr (I4) {
    return key * Tile<I4, D>::kRow + 16 * (D == 128 ? chunk ^ ((key >> 1) & 3) : chunk ^ ((key >> 2) & 1));
  } else {
    return key * Tile<I4, D>::kRow + 16 * (chunk ^ (key & 7));
  }
}
// K rows.  4-bit: the transposed bytes of V pair keys 4t, 4t + 2 and 4t + 1, 4t + 3 in
// the value MMA, so rows g and g + 8 of a block's score MMA are keys 2g and 2g + 1:
// the even keys of a block first, then the odd ones.  bf16: rows g and g + 8 are
// keys g and g + 8, and the 64-byte halves of odd rows change places (two rows a
// quarter warp).
template <bool I4, int D>
__device__ __forceinline__ int k_place(int key, int chunk) {
  if constexpr (I4) {
    return ((key & ~15) | ((key & 1) << 3) | ((key >> 1) & 7)) * Tile<I4, D>::kRow + 16 * chunk;
  } else {
    return key * Tile<I4, D>::kRow + 16 * (chunk ^ ((key & 1) << 2));
  }
}
template <bool I4>
__device__ __forceinline__ int key_of_row(int g, int r) {  // of row g + 8 r of a block
  return I4 ? 2 * g + r : g + 8 * r;
}

// A lane's part of its warp's tile copies: 32 pieces of 16 bytes a step, so every
// step is 512 bytes further on both sides (4-bit rows; bf16 V pieces move within
// their row with the key).
template <bool I4, int D>
struct Loader {
  using T = Tile<I4, D>;
  static constexpr int kSteps = T::kKeys * T::kChunks / 32;
  int key0, c;
  uint32_t kdst, vdst;
  uint64_t policy;

  __device__ __forceinline__ Loader(int lane, bool once) {
    policy = l2_policy(once);
    key0 = lane / T::kChunks;
    c = lane % T::kChunks;
    kdst = k_place<I4, D>(key0, c);
    vdst = T::kVOff + v_place<I4, D>(key0, c);
  }
  // The tile whose first row is `row` of all cache rows, `left` rows before the sequence's end.
  __device__ __forceinline__ void copy(const CacheDecodeArgs& a, uint32_t stage, int row, int left, int lane) const {
    constexpr int kStep = 32 / T::kChunks;  // keys a step
    const char* K = static_cast<const char*>(a.K) + (size_t)row * T::kRow;
    const char* V = static_cast<const char*>(a.V) + (size_t)row * T::kRow;
    const char* Kp = static_cast<const char*>(a.Kp) + (size_t)row * 4;
    const char* Vp = static_cast<const char*>(a.Vp) + (size_t)row * 4;
    if (left >= T::kKeys) {
      K += lane * 16;
      V += lane * 16;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        // (4-bit, d = 128: eight keys a step, so the even and odd ones of half a block.)
        cp16(stage + kdst + (I4 && D == 128 ? (i >> 1) * 1024 + (i & 1) * 256 : 512 * i), K + 512 * i, policy);
        if constexpr (I4) {
          cp16(stage + vdst + 512 * i, V + 512 * i, policy);
        } else {
          cp16(stage + T::kVOff + v_place<I4, D>(key0 + kStep * i, c), V + 512 * i, policy);
        }
      }
      if constexpr (I4) {
        cp4(stage + T::kPOff + 8 * lane, Kp + 4 * lane);
        cp4(stage + T::kPOff + 8 * lane + 4, Vp + 4 * lane);
      }
    } else {  // the sequence's last tile: rows behind the end are zeros, and are not read
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const bool ok = key0 + kStep * i < left;
        const int off = ok ? 512 * i + 16 * lane : 0;
        cp16z(stage + k_place<I4, D>(key0 + kStep * i, c), K + off, ok);
        cp16z(stage + T::kVOff + v_place<I4, D>(key0 + kStep * i, c), V + off, ok);
      }
      if constexpr (I4) {
        const bool ok = lane < left;
        cp4z(stage + T::kPOff + 8 * lane, Kp + (ok ? 4 * lane : 0), ok);
        cp4z(stage + T::kPOff + 8 * lane + 4, Vp + (ok ? 4 * lane : 0), ok);
      }
    }
  }
};

// Partial state of one warp for NT column tiles (four heads each).
template <int D, int NT>
struct State {
  float O[NT][D / 16][4];  // rows: head dims; columns 2t, 2t+1: O1, O2 of lane t's head
  float m[NT], omega[NT], T[NT];
  float t0[NT];  // T and O2 are sums over t - t0
};

// The query rows as MMA columns: column g is q (even) or rho (odd) of head g/2 of
// the column tile (modulo G).  4-bit: a row x goes in as x 2^(126 - E), E the
// exponent of its largest element, and over 16 for the odd nibbles, so that sums
// over raw codes are (sum of x c) 2^(-7 - E); all of it exact.  sum and scale
// belong to the lane's own columns 2t and 2t + 1.
template <int D, int NT>
struct Query {
  uint32_t b[NT][D / 16][2];
  float sum[NT][2];    // (sum of x) 2^(-7 - E)
  float scale[NT][2];  // 2^(7 + E), with log2(e) / sqrt(d) for q
  float cs;
};

template <int D, int G>
__device__ __forceinline__ void load_query_int4(Query<D, (G + 3) / 4>& q, const __nv_bfloat16* qrow,
                                                const __nv_bfloat16* rrow, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int u = 0; u < (G + 3) / 4; ++u) {
    const int h = (G >= 4) ? 4 * u + (g >> 1) : (g >> 1) % G;
    const uint4* row = reinterpret_cast<const uint4*>(((g & 1) ? rrow : qrow) + h * D) + (D / 32) * t;
    uint4 v[D / 32];  // the eight dims of each code word
    uint32_t top = 0;  // largest magnitude, as bits
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v[i] = row[i];
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // Subnormal rows take the exponent of the smallest normal number.
    const int E = top >= 0x00800000u ? (int)(top >> 23) - 127 : -126;
    // 2^-E in two factors, each a normal number (E in [-126, 128]).
    const float f0 = __uint_as_float((uint32_t)(127 - (E >> 1)) << 23);
    const float f1 = __uint_as_float((uint32_t)(127 - (E - (E >> 1))) << 23);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = bf_lo(x[e]) * f0 * f1;
        y[2 * e + 1] = bf_hi(x[e]) * f0 * f1;
        sum += y[2 * e] + y[2 * e + 1];
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        q.b[u][2 * i + p][0] = pack_bf16(y[2 * p] * 0x1p126f, y[2 * p + 4] * 0x1p126f);
        q.b[u][2 * i + p][1] = pack_bf16(y[2 * p + 1] * 0x1p122f, y[2 * p + 5] * 0x1p122f);
      }
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum *= 0x1p-7f;
    // 2^(7 + E), as 2^7 2^E: E = 121 and above (rows beyond 2^121) overflow to infinity.
    const float up = __uint_as_float((uint32_t)(min(E, 127) + 127) << 23) * 128.f * ((g & 1) ? 1.f : q.cs);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      q.sum[u][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e));
      q.scale[u][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
    }
  }
}

template <int D, int G>
__device__ __forceinline__ void load_query_bf16(Query<D, (G + 3) / 4>& q, const __nv_bfloat16* qrow,
                                                const __nv_bfloat16* rrow, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int u = 0; u < (G + 3) / 4; ++u) {
    const int h = (G >= 4) ? 4 * u + (g >> 1) : (g >> 1) % G;
    const uint4* row = reinterpret_cast<const uint4*>(((g & 1) ? rrow : qrow) + h * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = row[4 * i + t];
      q.b[u][2 * i][0] = v.x;
      q.b[u][2 * i][1] = v.y;
      q.b[u][2 * i + 1][0] = v.z;
      q.b[u][2 * i + 1][1] = v.w;
    }
  }
}

// Rows of (b, KV head) `unit` as q, and an empty state.
template <bool I4, int D, int G>
__device__ __forceinline__ void begin_unit(const CacheDecodeArgs& a, Query<D, (G + 3) / 4>& q,
                                           State<D, (G + 3) / 4>& s, int unit, int lane) {
  const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + (size_t)unit * G * D;
  const __nv_bfloat16* rrow = static_cast<const __nv_bfloat16*>(a.r) + (size_t)unit * G * D;
  if constexpr (I4) {
    load_query_int4<D, G>(q, qrow, rrow, lane);
  } else {
    load_query_bf16<D, G>(q, qrow, rrow, lane);
  }
#pragma unroll
  for (int u = 0; u < (G + 3) / 4; ++u) {
    s.m[u] = kNoRef;
    s.omega[u] = s.T[u] = s.t0[u] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.O[u][i][e] = 0.f;
  }
}

// Score accumulators of a tile: rows = keys g, g + 8 of a block, columns = q, rho
// of the heads.
template <bool I4, int D, int G>
struct Scores {
  static constexpr int NT = (G + 3) / 4, NB = Tile<I4, D>::kKeys / 16;
  float S[NB][NT][4];
};

// Scores of block b of the tile in `stage`.
template <bool I4, int D, int G>
__device__ __forceinline__ void score_block(Scores<I4, D, G>& sc, uint32_t stage, const Query<D, (G + 3) / 4>& q,
                                            int b, int lane) {
  using T = Tile<I4, D>;
  using Sc = Scores<I4, D, G>;
  constexpr int NT = Sc::NT;
  const int g = lane >> 2, t = lane & 3;
  auto mma = [&](int u, int step, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    if (step == 0) {
      mma_bf16_first(sc.S[b][u], a0, a1, a2, a3, q.b[u][step][0], q.b[u][step][1]);
    } else {
      mma_bf16(sc.S[b][u], a0, a1, a2, a3, q.b[u][step][0], q.b[u][step][1]);
    }
  };
  if constexpr (I4) {
    constexpr int WPL = D / 32;  // code words a lane has of a key
    uint32_t w[2][WPL];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t at = stage + (16 * b + g + 8 * r) * T::kRow + 4 * WPL * t;
      if constexpr (WPL == 4) {
        lds128(w[r], at);
      } else {
        lds64(w[r][0], w[r][1], at);
      }
    }
#pragma unroll
    for (int i = 0; i < WPL; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t x0 = p ? w[0][i] >> 8 : w[0][i], x1 = p ? w[1][i] >> 8 : w[1][i];
#pragma unroll
        for (int u = 0; u < NT; ++u)
          mma(u, 2 * i + p, x0 & kEven, x1 & kEven, x0 & kOdd, x1 & kOdd);
      }
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t x[4], y[4];
      lds128(x, stage + k_place<I4, D>(16 * b + g, 4 * i + t));
      lds128(y, stage + k_place<I4, D>(16 * b + g + 8, 4 * i + t));
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int u = 0; u < NT; ++u)
          mma(u, 2 * i + p, x[2 * p], y[2 * p], x[2 * p + 1], y[2 * p + 1]);
    }
  }
}

// Weights of a tile as the value MMAs' operand: bf16 hi + lo of [w s_v, w t s_v].
template <bool I4, int D, int G>
struct Weights {
  uint32_t hi[Tile<I4, D>::kKeys / 16][(G + 3) / 4][2], lo[Tile<I4, D>::kKeys / 16][(G + 3) / 4][2];
};

// With G <= 2 and two blocks a tile, lanes t and t ^ G hold the same scores: the
// one with bit G of t clear weighs block 0, the other block 1.
template <bool I4, int D, int G>
constexpr bool kHalves = G <= 2 && Tile<I4, D>::kKeys == 32;

template <bool I4, int D, int G, bool W>
__device__ __forceinline__ void weigh_tile(State<D, (G + 3) / 4>& s, Weights<I4, D, G>& wt, const Scores<I4, D, G>& sco,
                                           uint32_t stage, const Query<D, (G + 3) / 4>& q,
                                           float* scores, int j0, int n, int lane) {
  using T = Tile<I4, D>;
  using Sc = Scores<I4, D, G>;
  constexpr bool kHalf = kHalves<I4, D, G>;
  constexpr int NT = Sc::NT, KS = D / 16, NB = kHalf ? 1 : Sc::NB;  // blocks this lane weighs
  const int g = lane >> 2, t = lane & 3;
  const bool second = kHalf && (t & G);
  const int block0 = second ? 16 : 0;  // first key of this lane's block
  float sc[NB][NT][2], tt[NB][NT][2], sv[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t kv[4] = {};  // (K word, V word) of both keys
    if constexpr (I4) lds128(kv, stage + T::kPOff + 8 * (block0 + 16 * b + 2 * g));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int key = block0 + 16 * b + key_of_row<I4>(g, r);
      const uint32_t pk = kv[2 * r], pv = kv[2 * r + 1];
      sv[b][r] = I4 ? bf_lo(pv) : 1.f;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float s1 = sco.S[b][u][2 * r], s2 = sco.S[b][u][2 * r + 1];
        if constexpr (kHalf) {
          s1 = second ? sco.S[1][u][2 * r] : s1;
          s2 = second ? sco.S[1][u][2 * r + 1] : s2;
        }
        if constexpr (I4) {  // sums of raw codes: the zero point times the row's sum goes off
          const float z = bf_hi(pk), sk = bf_lo(pk);
          s1 = fmaf(-z, q.sum[u][0], s1) * (q.scale[u][0] * sk);
          // (t's power of two comes in write_records)
          s2 = fmaf(fmaf(-z, q.sum[u][1], s2), sk, -s.t0[u]);
        } else {
          s1 *= q.cs;
          s2 -= s.t0[u];
        }
        sc[b][u][r] = s1;
        tt[b][u][r] = s2;
        if constexpr (W) {
          const bool mine = kHalf ? t < 2 * G : t < G;
          if (j0 + key < n && mine) scores[(size_t)(j0 + key) * G + 4 * u + (kHalf ? t & (G - 1) : t)] = s1;
        }
      }
    }
  }
  if (j0 + T::kKeys > n) {  // keys behind the end
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (j0 + block0 + 16 * b + key_of_row<I4>(g, r) >= n) sc[b][u][r] = -CUDART_INF_F;
  }
  bool raise = false;
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int b = 0; b < NB; ++b) raise |= sc[b][u][0] > s.m[u] || sc[b][u][1] > s.m[u];
  if (__any_sync(0xffffffffu, raise)) {
    const float share = __fdividef(32.f, (float)min(T::kKeys, n - j0));
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float mx = sc[0][u][0], by = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mx = fmaxf(mx, fmaxf(sc[b][u][0], sc[b][u][1]));
        by += (tt[b][u][0] + tt[b][u][1]) * (1.f / 32);  // (a sum of large t would pass fp32's range)
      }
      if constexpr (kHalf) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, G));
        by += __shfl_xor_sync(0xffffffffu, by, G);
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o)), by += __shfl_xor_sync(0xffffffffu, by, o);
      const float m = mx > s.m[u] ? mx + kHeadroom : s.m[u];
      const float f = ex2(s.m[u] - m);
      by = s.m[u] == kNoRef ? by * share : 0.f;  // the first tile of this state (keys behind the end: t is 0)
      s.t0[u] += by;
#pragma unroll
      for (int b = 0; b < NB; ++b) tt[b][u][0] -= by, tt[b][u][1] -= by;
      s.m[u] = m;
      s.omega[u] *= f;
      s.T[u] *= f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.O[u][i][e] *= f;
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const float w = ex2(sc[b][u][r] - s.m[u]);
        const float w_t = w * tt[b][u][r];
        s.omega[u] += w;
        s.T[u] += w_t;
        const float p0 = I4 ? w * sv[b][r] : w, p1 = I4 ? w_t * sv[b][r] : w_t;
        const uint32_t h = pack_bf16(p0, p1);
        const uint32_t l = pack_bf16(p0 - bf_lo(h), p1 - bf_hi(h));
        if constexpr (kHalf) {  // hi in the columns with bit G of t clear, lo in the others
          const uint32_t other = __shfl_xor_sync(0xffffffffu, second ? h : l, G);
          wt.hi[0][u][r] = movmatrix_trans(second ? other : h);
          wt.hi[1][u][r] = movmatrix_trans(second ? l : other);
        } else if constexpr (G <= 2) {
          wt.hi[b][u][r] = movmatrix_trans((t & G) ? l : h);  // columns 4..7 repeat 0..3 for G = 1, unused
        } else {
          wt.hi[b][u][r] = movmatrix_trans(h);
          wt.lo[b][u][r] = movmatrix_trans(l);
        }
      }
    }
}

// Values of block b: rows = head dims, contraction over the 16 keys.
template <bool I4, int D, int G>
__device__ __forceinline__ void value_block(State<D, (G + 3) / 4>& s, const Weights<I4, D, G>& wt, uint32_t stage, int b,
                                            int lane) {
  using T = Tile<I4, D>;
  constexpr int NT = (G + 3) / 4, KS = D / 16;
  const int g = lane >> 2, t = lane & 3;
  auto mma = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      mma_bf16(s.O[u][mt], a0, a1, a2, a3, wt.hi[b][u][0], wt.hi[b][u][1]);
      if constexpr (G >= 4) mma_bf16(s.O[u][mt], a0, a1, a2, a3, wt.lo[b][u][0], wt.lo[b][u][1]);
    }
  };
  if constexpr (I4) {
    // Register r of a 16-byte piece: the bytes 8 r + g of keys 4t .. 4t + 3, so two
    // neighbouring dims; their even keys' codes and (8 bits on) their odd keys'.
    uint32_t kv[2][4], mz[2];  // (K word, V word) of four keys
#pragma unroll
    for (int e = 0; e < 2; ++e) lds128(kv[e], stage + T::kPOff + 8 * (16 * b + 4 * t + 2 * e));
    mz[0] = neg_zero_points(__byte_perm(kv[0][1], kv[1][1], 0x7632));
    mz[1] = neg_zero_points(__byte_perm(kv[0][3], kv[1][3], 0x7632));
    const int key = 16 * b + (lane & 15);
#pragma unroll
    for (int c = 0; c < T::kChunks; c += 2) {
      uint32_t w[4];
      ldmatrix2_bytes_trans(w, stage + T::kVOff + v_place<I4, D>(key, c + (lane >> 4)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = w[e], y = w[e] >> 8;
        mma(2 * c + e, nib_even(x, mz[0]), nib_odd(x, mz[0]), nib_even(y, mz[1]), nib_odd(y, mz[1]));
      }
    }
  } else {
    // Matrices of ldmatrix: (dims 0-7 | 8-15 of the tile) x (keys 0-7 | 8-15).
    const int key = 16 * b + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t x[4];
      ldmatrix4_trans(x, stage + T::kVOff + v_place<I4, D>(key, 2 * mt + half));
      mma(mt, x[0], x[1], x[2], x[3]);
    }
  }
}

// A record: m, omega, T, t0, O1[D], O2[D]; T and O2 of t - t0.
template <int D>
constexpr int kRec = 2 * D + 4;

// The warp's state as G records.
template <bool I4, int D, int G>
__device__ __forceinline__ void write_records(State<D, (G + 3) / 4>& s, const Query<D, (G + 3) / 4>& q, float* recs,
                                              int lane) {
  constexpr int KS = D / 16, R = kRec<D>;
  const int g = lane >> 2, t = lane & 3;
  constexpr float kUnit = I4 ? 64.f : 1.f;  // (c - z) 2^-6
#pragma unroll
  for (int u = 0; u < (G + 3) / 4; ++u) {
    const float f2 = I4 ? q.scale[u][1] : 1.f;  // of what holds t
    s.T[u] *= f2;
    if constexpr (kHalves<I4, D, G>) {
      s.omega[u] += __shfl_xor_sync(0xffffffffu, s.omega[u], G);
      s.T[u] += __shfl_xor_sync(0xffffffffu, s.T[u], G);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      s.omega[u] += __shfl_xor_sync(0xffffffffu, s.omega[u], o);
      s.T[u] += __shfl_xor_sync(0xffffffffu, s.T[u], o);
    }
    if constexpr (G <= 2) {  // hi + lo
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.O[u][i][e] += __shfl_xor_sync(0xffffffffu, s.O[u][i][e], G);
    }
    if (t < G) {
      float* rec = recs + (4 * u + t) * R;
      if (g == 0) *reinterpret_cast<float4*>(rec) = make_float4(s.m[u], s.omega[u], s.T[u], s.t0[u] * f2);
      if constexpr (I4) {  // rows g, g + 8 of tile i: dims 16 i + 2 g, 16 i + 2 g + 1
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const float(&x)[4] = s.O[u][i];
          *reinterpret_cast<float2*>(rec + 4 + 16 * i + 2 * g) = make_float2(x[0] * kUnit, x[2] * kUnit);
          *reinterpret_cast<float2*>(rec + 4 + D + 16 * i + 2 * g) =
              make_float2(x[1] * f2 * kUnit, x[3] * f2 * kUnit);  // (2^6 2^(7 + E) may pass fp32's range)
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const int d0 = 16 * i + g;
          rec[4 + d0] = s.O[u][i][0];
          rec[4 + D + d0] = s.O[u][i][1];
          rec[4 + d0 + 8] = s.O[u][i][2];
          rec[4 + D + d0 + 8] = s.O[u][i][3];
        }
      }
    }
  }
}

__device__ __forceinline__ bool bad_len(int n, int L) { return n < 1 || n > L; }

// Zeros for all heads of a sequence whose length is not in 1..L.
__device__ void zero_sequence(const CacheDecodeArgs& a, int b, int first, int step) {
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)b * a.H * a.d;
  for (int e = first; e < a.H * a.d; e += step) out[e] = __float2bfloat16(0.f);
  if (first == 0) atomicOr(a.status, kStatusBadSeqlen);
}

// The tiles of all (b, KV head) in one row of T, cut into P shares that differ by
// one tile at most, the larger ones first.
struct Shares {
  int size, more;  // shares 0 .. more - 1 have size + 1 tiles
  __device__ __forceinline__ Shares(int T, int P) : size(T / P), more(T % P) {}
  __device__ __forceinline__ int begin(int c) const { return c * size + min(c, more); }
  __device__ __forceinline__ int of(int x) const {  // the share of tile x
    const int y = x - more * (size + 1);
    return y < 0 ? x / (size + 1) : more + y / size;
  }
};

// One warp a share, with no barrier between the warps after the prologue.  The
// part of (b, KV head) u that begins it goes to record slot u, the part that
// share c begins with inside of one to slot B Hkv + c.  A warp's ring runs on
// over the end of a (b, KV head).
template <bool I4, int D, int G, bool W>
__global__ void __launch_bounds__(kThreads, G == 8 ? 3 : 4) cache_decode_flat_kernel(const CacheDecodeArgs a) {
  using T = Tile<I4, D>;
  constexpr int NT = (G + 3) / 4, R = kRec<D>, kKeys = T::kKeys;
  extern __shared__ __align__(128) char smem[];
  __shared__ int s_sum[kWarps], s_b[kWarps], s_begin[kWarps], s_n[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.shares;
  grid_dep_wait();
  grid_dep_launch();
  // ---- T, and the sequences that hold the warps' first tiles.
  int total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int x = 0, n = 0;
      if (b < a.B) {
        n = a.seqlens[b];
        if (!bad_len(n, a.L)) {
          x = (n + kKeys - 1) / kKeys * a.Hkv;
        } else if (pass == 0 && b % gridDim.x == blockIdx.x) {
          zero_sequence(a, b, 0, 1);
        }
      }
      int incl = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      int before = base;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        base += s_sum[w];
      }
      const int excl = before + incl - x;
      if (a.B <= kThreads) total = base;  // one turn: the sum is known already
      if ((pass == 1 || a.B <= kThreads) && b < a.B) {
        const Shares shares(total, P);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const int begin = shares.begin(blockIdx.x * kWarps + w);
          if (excl <= begin && begin < excl + x) {
            s_b[w] = b;
            s_begin[w] = excl;
            s_n[w] = n;
          }
        }
        if (x == 0 && b % gridDim.x == blockIdx.x)
          for (int h = 0; h < a.Hkv; ++h) a.parts[b * a.Hkv + h] = make_int2(-1, -1);
      }
      __syncthreads();
    }
    total = base;
    if (a.B <= kThreads) break;
  }
  const Shares shares(total, P);
  const int c = blockIdx.x * kWarps + warp;
  const int begin = shares.begin(c), end = shares.begin(c + 1);
  if (begin >= end) return;
  // ---- two cursors, the copies' ahead of the MMAs'.
  struct Cursor {
    int b, h, n, tiles, tile;  // sequence, KV head, its length and tiles, the tile
    __device__ __forceinline__ void next_unit(const CacheDecodeArgs& a) {
      tile = 0;
      if (++h == a.Hkv) {
        h = 0;
        do n = a.seqlens[++b];
        while (bad_len(n, a.L));
        tiles = (n + kKeys - 1) / kKeys;
      }
    }
  };
  Cursor at;
  at.b = s_b[warp];
  at.n = s_n[warp];
  at.tiles = (at.n + kKeys - 1) / kKeys;
  at.h = (begin - s_begin[warp]) / at.tiles;
  at.tile = begin - s_begin[warp] - at.h * at.tiles;
  Cursor ld = at;
  const Loader<I4, D> loader(lane, a.once);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * T::kWarpBytes;
  int ahead = begin;  // next tile to copy
  auto copy_next = [&](uint32_t stage) {
    if (ahead < end) {
      if (ld.tile == ld.tiles) ld.next_unit(a);
      loader.copy(a, stage, (ld.b * a.Hkv + ld.h) * a.L + ld.tile * kKeys, ld.n - ld.tile * kKeys,
                  lane);
      ++ld.tile;
      ++ahead;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) copy_next(ring + i * T::kBytes);
  Query<D, NT> q;
  q.cs = kLog2e * rsqrtf((float)D);
  State<D, NT> s;
  int unit = at.b * a.Hkv + at.h;
  begin_unit<I4, D, G>(a, q, s, unit, lane);
  // The first share of a (b, KV head) notes where its records are: shares c to the
  // one of its last tile.  No share between them is empty: with more shares than
  // tiles the first T have one tile each.
  auto note = [&](int x) {
    if (lane == 0) a.parts[unit] = make_int2(c, x + at.tiles <= end ? c : shares.of(x + at.tiles - 1));
  };
  int slot = a.B * a.Hkv + c;
  if (at.tile == 0) {
    slot = unit;
    note(begin);
  }
  Scores<I4, D, G> sc;
  Weights<I4, D, G> wt;
  uint32_t now = ring;
  cp_wait<T::kStages - 2>();
  __syncwarp();
#pragma unroll
  for (int b = 0; b < kKeys / 16; ++b) score_block<I4, D, G>(sc, now, q, b, lane);
  for (int x = begin;;) {
    weigh_tile<I4, D, G, W>(s, wt, sc, now, q, W ? a.scores + (size_t)unit * a.L * G : nullptr, at.tile * kKeys, at.n,
                            lane);
    cp_wait<T::kStages - 3>();
    __syncwarp();  // every lane's copies have landed, and the stage refilled below is no longer read
    const uint32_t after = now == ring + (T::kStages - 1) * T::kBytes ? ring : now + T::kBytes;
    copy_next(now == ring ? ring + (T::kStages - 1) * T::kBytes : now - T::kBytes);
    ++x;
    if (++at.tile < at.tiles && x < end) {
      // The value MMAs beside the next tile's score MMAs.
#pragma unroll
      for (int b = 0; b < kKeys / 16; ++b) {
        score_block<I4, D, G>(sc, after, q, b, lane);
        value_block<I4, D, G>(s, wt, now, b, lane);
      }
    } else {
#pragma unroll
      for (int b = 0; b < kKeys / 16; ++b) value_block<I4, D, G>(s, wt, now, b, lane);
      write_records<I4, D, G>(s, q, a.records + (size_t)slot * G * R, lane);
      if (x == end) break;
      at.next_unit(a);
      slot = unit = at.b * a.Hkv + at.h;
      note(x);
      begin_unit<I4, D, G>(a, q, s, unit, lane);
#pragma unroll
      for (int b = 0; b < kKeys / 16; ++b) score_block<I4, D, G>(sc, after, q, b, lane);
    }
    now = after;
  }
  cp_wait<0>();
}

// Shared memory of a CTA of the next kernel: the rings, and over them at the end
// a record for each warp and head and the merged ones.
template <bool I4, int D, int G>
constexpr int kSmem = Tile<I4, D>::kRing > (kWarps + 1) * G * kRec<D> * 4 ? Tile<I4, D>::kRing
                                                                        : (kWarps + 1) * G * kRec<D> * 4;

// One (b, KV head) a CTA, or a cluster of `splits` CTAs that cut its keys evenly
// and merge through distributed shared memory.  The warps take tiles in turn.
template <bool I4, int D, int G, bool W>
__global__ void __launch_bounds__(kThreads, G == 8 ? 3 : 4) cache_decode_kernel(const CacheDecodeArgs a) {
  using T = Tile<I4, D>;
  constexpr int NT = (G + 3) / 4, R = kRec<D>, kKeys = T::kKeys;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  grid_dep_wait();
  grid_dep_launch();
  const int n = a.seqlens[unit / a.Hkv];
  if (bad_len(n, a.L)) {  // the same for every CTA of the cluster
    if (split == 0 && unit % a.Hkv == 0) zero_sequence(a, unit / a.Hkv, threadIdx.x, kThreads);
    return;
  }
  const int tiles = (n + kKeys - 1) / kKeys;
  const int tile0 = (int)((long long)tiles * split / a.splits) + warp;
  const int tile1 = (int)((long long)tiles * (split + 1) / a.splits);
  const int row0 = unit * a.L;
  const Loader<I4, D> loader(lane, a.once);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * T::kWarpBytes;
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) {
    const int tile = tile0 + i * kWarps;
    if (tile < tile1) loader.copy(a, ring + i * T::kBytes, row0 + tile * kKeys, n - tile * kKeys, lane);
    cp_commit();
  }
  Query<D, NT> q;
  q.cs = kLog2e * rsqrtf((float)D);
  State<D, NT> s;
  begin_unit<I4, D, G>(a, q, s, unit, lane);
  Scores<I4, D, G> sc;
  Weights<I4, D, G> wt;
  float* scores = W ? a.scores + (size_t)unit * a.L * G : nullptr;
  uint32_t now = ring;
  if (tile0 < tile1) {
    cp_wait<T::kStages - 2>();
    __syncwarp();
#pragma unroll
    for (int b = 0; b < kKeys / 16; ++b) score_block<I4, D, G>(sc, now, q, b, lane);
  }
  // Each turn weighs a tile, then runs its value MMAs beside the next tile's
  // score MMAs (of a tile behind the last: of whatever the stage holds, unused).
  for (int tile = tile0; tile < tile1; tile += kWarps) {
    weigh_tile<I4, D, G, W>(s, wt, sc, now, q, scores, tile * kKeys, n, lane);
    cp_wait<T::kStages - 3>();
    __syncwarp();  // every lane's copies have landed, and the stage refilled below is no longer read
    const uint32_t after = now == ring + (T::kStages - 1) * T::kBytes ? ring : now + T::kBytes;
    const uint32_t fill = now == ring ? ring + (T::kStages - 1) * T::kBytes : now - T::kBytes;
    const int next = tile + (T::kStages - 1) * kWarps;
    if (next < tile1) loader.copy(a, fill, row0 + next * kKeys, n - next * kKeys, lane);
    cp_commit();
#pragma unroll
    for (int b = 0; b < kKeys / 16; ++b) {
      score_block<I4, D, G>(sc, after, q, b, lane);
      value_block<I4, D, G>(s, wt, now, b, lane);
    }
    now = after;
  }
  // ---- merge the warps.
  cp_wait<0>();
  __syncthreads();
  float* recs = reinterpret_cast<float*>(smem);  // [warp][G][R], then the merged [G][R]
  float* merged = recs + kWarps * G * R;
  write_records<I4, D, G>(s, q, recs + warp * G * R, lane);
  __syncthreads();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)unit * G * D;
  for (int e = threadIdx.x; e < G * D; e += kThreads) {
    const int h = e / D, dim = e % D;
    float m = recs[h * R];
    const float t0 = recs[h * R + 3];  // (where the first warp has no tile, none has)
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, recs[(w * G + h) * R]);
    float omega = 0.f, tsum = 0.f, o1 = 0.f, o2 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* rec = recs + (w * G + h) * R;
      const float4 x = *reinterpret_cast<const float4*>(rec);
      const float f = ex2(x.x - m), by = x.w - t0;
      omega += f * x.y;
      tsum += f * fmaf(by, x.y, x.z);
      o1 += f * rec[4 + dim];
      o2 += f * fmaf(by, rec[4 + dim], rec[4 + D + dim]);
    }
    if (a.splits == 1) {
      const float inv = 1.f / omega;
      out[e] = __float2bfloat16(((1.f + tsum * inv) * o1 - o2) * inv);
      if (W && dim == 0) a.stats[(size_t)unit * G + h] = make_float2(m, omega);
    } else {
      float* rec = merged + h * R;
      if (dim == 0) {
        rec[0] = m;
        rec[1] = omega;
        rec[2] = tsum;
        rec[3] = t0;
      }
      rec[4 + dim] = o1;
      rec[4 + D + dim] = o2;
    }
  }
  if (a.splits == 1) return;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = split * kThreads + threadIdx.x; e < G * D; e += a.splits * kThreads) {
    const int h = e / D, dim = e % D;
    float m = kNoRef;
    const float t0 = cluster.map_shared_rank(merged, a.splits - 1)[h * R + 3];  // the last CTA always has a tile
    for (int c = 0; c < a.splits; ++c) m = fmaxf(m, cluster.map_shared_rank(merged, c)[h * R]);
    float omega = 0.f, tsum = 0.f, o1 = 0.f, o2 = 0.f;
    for (int c = 0; c < a.splits; ++c) {
      const float* rec = cluster.map_shared_rank(merged, c) + h * R;
      const float4 x = *reinterpret_cast<const float4*>(rec);
      const float f = ex2(x.x - m), by = x.w - t0;
      omega += f * x.y;
      tsum += f * fmaf(by, x.y, x.z);
      o1 += f * rec[4 + dim];
      o2 += f * fmaf(by, rec[4 + dim], rec[4 + D + dim]);
    }
    const float inv = 1.f / omega;
    out[e] = __float2bfloat16(((1.f + tsum * inv) * o1 - o2) * inv);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// The records of (b, KV head) `unit` after a decode in shares: slot `unit` (by
// share c0), then slot `units + c` of the shares c in (c0, c1].
struct Parts {
  int unit, units, c0, c1;
  __device__ __forceinline__ Parts(const CacheDecodeArgs& a, int u) : unit(u), units(a.B * a.Hkv) {
    const int2 x = a.parts[u];  // (-1, -1): a sequence of bad length
    c0 = x.x;
    c1 = x.y;
  }
  __device__ __forceinline__ int slot(int c) const { return c == c0 ? unit : units + c; }
};

// Outputs of HP heads from their records, by all kT threads of a CTA: four dims a
// lane, a head's records over groups of D / 4 lanes, each with its own running m.
template <int D, int G, int kT, int HP>
struct Merge {
  static constexpr int kLanes = D / 4, kGroups = kT / (HP * kLanes);
  float4 o1[kT], o2[kT], head[HP * kGroups];

  __device__ __forceinline__ void run(const CacheDecodeArgs& a, const Parts& p, int h0) {
    constexpr int R = kRec<D>;
    const int dl = threadIdx.x % kLanes, grp = threadIdx.x / kLanes % kGroups, hp = threadIdx.x / (kLanes * kGroups);
    float4 x1 = make_float4(0.f, 0.f, 0.f, 0.f), x2 = x1;
    float m = kNoRef, omega = 0.f, tsum = 0.f;
    // The first record's t0 for all of them.
    const float t0 = a.records[((size_t)p.slot(p.c0) * G + h0 + hp) * R + 3];
#pragma unroll 4
    for (int c = p.c0 + grp; c <= p.c1; c += kGroups) {
      const float4* rec = reinterpret_cast<const float4*>(a.records + ((size_t)p.slot(c) * G + h0 + hp) * R);
      const float4 x = rec[0], y1 = rec[1 + dl], y2 = rec[1 + kLanes + dl];
      const float top = fmaxf(m, x.x), f0 = ex2(m - top), f = ex2(x.x - top), by = x.w - t0;
      m = top;
      omega = f0 * omega + f * x.y;
      tsum = f0 * tsum + f * fmaf(by, x.y, x.z);
      x1.x = f0 * x1.x + f * y1.x, x1.y = f0 * x1.y + f * y1.y;
      x1.z = f0 * x1.z + f * y1.z, x1.w = f0 * x1.w + f * y1.w;
      x2.x = f0 * x2.x + f * fmaf(by, y1.x, y2.x), x2.y = f0 * x2.y + f * fmaf(by, y1.y, y2.y);
      x2.z = f0 * x2.z + f * fmaf(by, y1.z, y2.z), x2.w = f0 * x2.w + f * fmaf(by, y1.w, y2.w);
    }
    o1[threadIdx.x] = x1;
    o2[threadIdx.x] = x2;
    if (dl == 0) head[hp * kGroups + grp] = make_float4(m, omega, tsum, 0.f);
    __syncthreads();
    for (int e = threadIdx.x; e < HP * D; e += kT) {
      const int i = e / D, dim = e % D;
      m = kNoRef;
#pragma unroll
      for (int c = 0; c < kGroups; ++c) m = fmaxf(m, head[i * kGroups + c].x);
      const float* f1 = reinterpret_cast<const float*>(o1) + i * kGroups * D + dim;
      const float* f2 = reinterpret_cast<const float*>(o2) + i * kGroups * D + dim;
      float x = 0.f, y = 0.f;
      omega = tsum = 0.f;
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        const float4 r = head[i * kGroups + c];
        const float f = ex2(r.x - m);
        omega += f * r.y;
        tsum += f * r.z;
        x += f * f1[c * D];
        y += f * f2[c * D];
      }
      const float inv = 1.f / omega;
      static_cast<__nv_bfloat16*>(a.out)[((size_t)p.unit * G + h0 + i) * D + dim] =
          __float2bfloat16(((1.f + tsum * inv) * x - y) * inv);
    }
  }
};

// After a decode in shares: HP heads of a (b, KV head) a CTA.
template <int D, int G, int kT, int HP>
__global__ void __launch_bounds__(kT) cache_merge_kernel(const CacheDecodeArgs a) {
  __shared__ Merge<D, G, kT, HP> merge;
  grid_dep_wait();
  grid_dep_launch();
  const Parts p(a, blockIdx.x / (G / HP));
  if (p.c0 >= 0) merge.run(a, p, blockIdx.x % (G / HP) * HP);
}

constexpr int kFinThreads = 256;
constexpr int kFinKeys = 2048;  // keys of a CTA that makes weights

// Scores to weights: w_out = w_in + sum_h 2^(s_h - m_h) / omega_h, kFinKeys keys of
// a (b, KV head) a CTA.  After a decode in shares the first CTAs merge outputs
// instead, kFinHeads heads each.
template <int D, int G>
constexpr int kFinHeads = G < 128 / (D / 4) ? G : 128 / (D / 4);  // two groups of records a head at least
template <int D, int G>
__global__ void __launch_bounds__(kFinThreads) cache_weights_kernel(const CacheDecodeArgs a, int parts) {
  constexpr int kTurns = kFinKeys / kFinThreads, HP = kFinHeads<D, G>;
  __shared__ float sm[G], sinv[G];
  __shared__ Merge<D, G, kFinThreads, HP> merge;
  int id = blockIdx.x;
  const int merging = a.shares > 0 ? a.B * a.H / HP : 0;
  grid_dep_wait();
  grid_dep_launch();
  if (id < merging) {
    const Parts p(a, id / (G / HP));
    if (p.c0 >= 0) merge.run(a, p, id % (G / HP) * HP);
    return;
  }
  id -= merging;
  const int unit = id / parts, part = id % parts;
  // Scores and totals do not wait for the length and the statistics: what lies
  // behind the length is read (inside of the arrays) and not used.
  const size_t row0 = (size_t)unit * a.L + part * kFinKeys;
  const int room = a.L - part * kFinKeys;
  float x[kTurns][G], w[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int j = min(i * kFinThreads + (int)threadIdx.x, room - 1);
    const float* sc = a.scores + (row0 + j) * G;
    if constexpr (G >= 4) {
#pragma unroll
      for (int h = 0; h < G; h += 4) *reinterpret_cast<float4*>(x[i] + h) = *reinterpret_cast<const float4*>(sc + h);
    } else if constexpr (G == 2) {
      *reinterpret_cast<float2*>(x[i]) = *reinterpret_cast<const float2*>(sc);
    } else {
      x[i][0] = sc[0];
    }
    w[i] = a.w_in[row0 + j];
  }
  const int n = a.seqlens[unit / a.Hkv];
  const int lane = threadIdx.x & 31;
  if (a.shares > 0) {
    const Parts p(a, unit);
    if (p.c0 < 0) return;
    for (int h = threadIdx.x >> 5; h < G; h += kFinThreads / 32) {
      float m = kNoRef, omega = 0.f;
#pragma unroll 4
      for (int c = p.c0 + lane; c <= p.c1; c += 32) {
        const float2 r = *reinterpret_cast<const float2*>(a.records + ((size_t)p.slot(c) * G + h) * kRec<D>);
        const float top = fmaxf(m, r.x);
        omega = omega * ex2(m - top) + r.y * ex2(r.x - top);
        m = top;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), omega2 = __shfl_xor_sync(0xffffffffu, omega, o);
        const float top = fmaxf(m, m2);
        omega = omega * ex2(m - top) + omega2 * ex2(m2 - top);
        m = top;
      }
      if (lane == 0) {
        sm[h] = m;
        sinv[h] = 1.f / omega;
      }
    }
  } else {
    if (bad_len(n, a.L)) return;
    if (threadIdx.x < G) {
      const float2 r = a.stats[(size_t)unit * G + threadIdx.x];
      sm[threadIdx.x] = r.x;
      sinv[threadIdx.x] = 1.f / r.y;
    }
  }
  __syncthreads();
  const int here = n - part * kFinKeys;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int j = i * kFinThreads + threadIdx.x;
    if (j >= here) continue;
    float p = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) p += ex2(x[i][h] - sm[h]) * sinv[h];
    a.w_out[row0 + j] = w[i] + p;
  }
}

template <bool I4, int D, int G, bool W>
cudaError_t run(const CacheDecodeArgs& a, cudaStream_t st) {
  const int smem = a.shares > 0 ? Tile<I4, D>::kRing : kSmem<I4, D, G>;
  const unsigned units = (unsigned)a.B * a.Hkv;
  auto kern = a.shares > 0 ? cache_decode_flat_kernel<I4, D, G, W> : cache_decode_kernel<I4, D, G, W>;
  // Once a device and kernel: which devices this one is set up on.
  static std::atomic<uint64_t> ready[2];
  std::atomic<uint64_t>& set = ready[a.shares > 0];
  cudaError_t e = cudaSuccess;
  if (!(set.load(std::memory_order_acquire) >> a.device & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set.fetch_or(1ull << a.device, std::memory_order_release);
  }
  e = a.shares > 0 ? launch_dependent(kern, a.shares / kWarps, kThreads, smem, 1, st, a)
                   : launch_dependent(kern, units * a.splits, kThreads, smem, a.splits, st, a);
  if (e != cudaSuccess) return e;
  if constexpr (W) {
    const int parts = (a.L + kFinKeys - 1) / kFinKeys;
    return launch_dependent(cache_weights_kernel<D, G>, units * parts + (a.shares > 0 ? units * G / kFinHeads<D, G> : 0),
                            kFinThreads, 0, 1, st, a, parts);
  } else {
    if (a.shares == 0) return cudaSuccess;
    // Few records each: up to four heads a CTA, four groups a head.  Many: a CTA a head.
    constexpr int HP = G < 4 ? G : 4;
    return a.shares <= 8 * (long long)units
               ? launch_dependent(cache_merge_kernel<D, G, HP * D, HP>, units * (G / HP), HP * D, 0, 1, st, a)
               : launch_dependent(cache_merge_kernel<D, G, 512, 1>, units * G, 512, 0, 1, st, a);
  }
}

template <bool I4, bool W>
cudaError_t pick(const CacheDecodeArgs& a, cudaStream_t st) {
  const int G = a.H / a.Hkv;
#define PLX_CACHE_CASE(D_, G_) \
  if (a.d == D_ && G == G_) return run<I4, D_, G_, W>(a, st);
  PLX_CACHE_CASE(128, 1)
  PLX_CACHE_CASE(128, 2)
  PLX_CACHE_CASE(128, 4)
  PLX_CACHE_CASE(128, 8)
  PLX_CACHE_CASE(64, 1)
  PLX_CACHE_CASE(64, 2)
  PLX_CACHE_CASE(64, 4)
  PLX_CACHE_CASE(64, 8)
#undef PLX_CACHE_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

// How the keys are cut, by sizes alone.  Measured on a B200, us a step (4-bit: with
// the append before it) in a row of 20, with shares / one CTA a (b, KV head) / the
// best cluster of 2 to 8; * is what the rule takes:
//   4-bit rows                                               d = 128                  d = 64
//   many (b, KV head) balance      64 x 16 of 4096           108 / 104* / 110         69 / 64* / 67
//   (less so where ragged)         64 x 16 of 2048..4096      81 /  89* /  92         55 / 60* / 59
//   fewer need shares              64 x 8 of 2048..4096, G 4  53* /  59 /  63         35* / 39 / 41
//                                  80 x 8 of 1024..2048, G 8  59* /  63 /  73         36* / 38 / 44
//                                  1 x 8 of 32768, G 4        20* / 175 /  29         14* / 110 / 19
//                                  1 x 2 of 32768             13* / 149 /  24         10* /  97 / 17
//   little work ends soonest       8 x 8 of 1024..2048, G 4   14  /  15 / 12.4* (4: 11.4)   11.5 / 10.5 / 8.8*
//   in one launch                  1 x 2 of 4096, G 4        9.4  /  27 / 9.5*              7.8 / 17.6 / 7.3*
//   the limit of 28 MB             2 x 8 of 8192 (17 MB)     15.2 /  41 / 13.3*
//                                  2 x 8 of 12288 (26 MB)    15.5 /  59 / 16.6*
//                                  2 x 8 of 16384 (34 MB)    17.4* /  77 / 19.8
//                                  8 x 8 of 2048..4096, G 4 (34 MB)  17.2* / 26 / 15.1
// Weights take a second launch in any case, so only many units go without shares:
//   4-bit, shares / one CTA        64 x 8 of 2048..4096, G 4  61* /  73               42* / 49
//                                  110 x 8 of 512..1024       28* /  30               22* / 20
//                                  128 x 8 of 512..1024       32  /  32*              26  / 23*
//   bf16                           64 x 8 of 2048..4096, G 4 138* / 140               75* / 76
//                                  110 x 8 of 512..1024       58* /  57               36* / 33
//                                  128 x 8 of 512..1024       67  /  65*              41  / 39*
//                                  8 x 8 of 1024..2048, G 4  19.5* / 19.1            12.9* / 11.3
// The rule's slots are of the 4-bit kernels: the bf16 ring lets two CTAs an SM run at
// once, so half of the shares wait for the others there.
CacheDecodeSpace cache_decode_space(int B, int H, int Hkv, int L, int d, int num_sms, bool int4, bool weights) {
  CacheDecodeSpace w;
  const long long units = (long long)B * Hkv, slots = (H / Hkv == 8 ? 3ll : 4ll) * num_sms;
  const int keys = int4 ? 32 : 2048 / d;
  const long long tiles = units * ((L + keys - 1) / keys);
  const long long bytes = units * L * (int4 ? d + 8 : 4 * d);
  const bool flat = 2 * units < 3 * slots && (weights || bytes > (28ll << 20) || L > 16384);
  if (!flat && !weights)
    while (w.splits < 8 && units * w.splits * 2 <= slots && (long long)L > 128ll * w.splits &&
           (units * w.splits * 2 <= num_sms || (long long)L > 1024ll * w.splits))
      w.splits *= 2;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  if (flat) {
    // A tile for every warp, and 256 records to merge for a (b, KV head), on average.
    // Shares are dealt by the tiles that there are, so one long sequence among hundreds
    // of short ones gets nearly all of them: 40000 keys beside 511 x 1..3 keys, d = 64,
    // 1250 records and 96 us, 9 us alone.
    const long long warps = tiles < 256 * units ? tiles : 256 * units;
    w.shares = kWarps * (int)((warps + kWarps - 1) / kWarps < slots ? (warps + kWarps - 1) / kWarps : slots);
    w.records = take(sizeof(float) * (size_t)(units + w.shares) * (H / Hkv) * (2 * d + 4));
    w.parts = take(sizeof(int2) * (size_t)units);
  }
  if (weights) {
    w.stats = take(sizeof(float2) * (size_t)B * H);
    w.scores = take(sizeof(float) * (size_t)B * H * L);
  }
  w.bytes = at;
  // Rows that will have left L2 before the next step reads them again need not stay
  // there: scores, records and what others keep stay instead (bf16 batch of 64 x 8 x
  // 2048..4096 keys with weights: 145 -> 133 us).  By the capacity: the lengths are on
  // the device, and a large cache with few rows gives up its stay in L2.
  w.once = bytes > (96ll << 20);
  return w;
}

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t st) {
  const bool i4 = a.Kp != nullptr, w = a.w_out != nullptr;
  if (i4) return w ? pick<true, true>(a, st) : pick<true, false>(a, st);
  return w ? pick<false, true>(a, st) : cudaErrorInvalidValue;
}

}  // namespace plx
