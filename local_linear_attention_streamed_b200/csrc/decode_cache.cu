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
// out = ((1 + T/omega) O1 - O2) / omega.
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
// * Codes become bf16 in two instructions a pair: AND picks two nibbles, which
//   as bf16 bits are c 2^-133 (or c 2^-129: bits 4..7 still lie in the linear
//   range of bf16), and one FMA turns them into (c - z) 2^-6, exactly.  The
//   zero point is thus gone before the sums: summing raw codes and subtracting
//   z omega afterwards would lose the small differences of large sums.  The
//   dims are paired as the nibbles fall; the other operand is permuted to match.
// * Groups of 1 and 2 leave columns free: the weights go in as bf16 hi + lo
//   pairs there; larger groups issue a second MMA for the lo part.  So the
//   weights keep 16 bits.
// * The reference m is raised lazily, when a score passes it: a raise sets it
//   2^8 above the largest score seen, so weights stay in (0, 1].
// * Each warp runs its own ring of key tiles with cp.async (no block barrier in
//   the loop, no wait that could not end) and its own partial state.
//
// The keys of a sequence are cut evenly (by its own length) over `splits` CTAs.
// Up to 8 splits are a cluster and merge through distributed shared memory; a
// larger number, and every decode with weights, writes partial records to the
// caller's workspace, and a second kernel merges them.  There are no counters
// and no library-owned memory: calls on several streams are independent.
#include "plx_internal.cuh"

#include <cooperative_groups.h>
#include <math_constants.h>

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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// 16- or 4-byte asynchronous copy; ok == false fills zeros and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
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
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Two nibbles to (c - z) 2^-6: kEven picks bits 0..3 and 16..19 of x, kOdd bits
// 4..7 and 20..23.  mz = (-z 2^-6) in both halves (or one for each half's key).
constexpr uint32_t kScaleEven = 0x7f007f00u;  // 2^127: c 2^-133 -> c 2^-6
constexpr uint32_t kScaleOdd = 0x7d007d00u;   // 2^123: c 2^-129 -> c 2^-6
__device__ __forceinline__ uint32_t nib_even(uint32_t x, uint32_t mz) {
  return fma_bf16x2(x & 0x000f000fu, kScaleEven, mz);
}
__device__ __forceinline__ uint32_t nib_odd(uint32_t x, uint32_t mz) {
  return fma_bf16x2(x & 0x00f000f0u, kScaleOdd, mz);
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
  static constexpr int kVOff = kKeys * kRow;              // a stage: K rows, V rows, K words, V words
  static constexpr int kPOff = 2 * kKeys * kRow;
  static constexpr int kBytes = kPOff + (I4 ? 8 * kKeys : 0);
  static constexpr int kWarpBytes = kStages * kBytes;
  static constexpr int kSmem = kWarps * kWarpBytes;
};

// Where a V row and its 16-byte pieces sit in a stage.  4-bit: lane t reads
// keys 2t, 2t+1, 2t+8, 2t+9 of a block one after the other, so keys of the same
// turn are neighbours; the pieces of every other row pair are exchanged so that
// four rows of 64 bytes cover all banks.  bf16: ldmatrix reads one piece of 8 rows.
template <bool I4, int D>
__device__ __forceinline__ int v_place(int key, int chunk) {
  if constexpr (I4) {
    const int slot = (key & ~7) | ((key & 1) << 2) | ((key >> 1) & 3);
    const int c = D == 128 ? chunk ^ (slot & 2) : chunk;
    return slot * Tile<I4, D>::kRow + 16 * c;
  } else {
    return key * Tile<I4, D>::kRow + 16 * (chunk ^ (key & 7));
  }
}
// K rows: bf16 swaps the 64-byte halves of odd rows (two rows a quarter warp).
template <bool I4, int D>
__device__ __forceinline__ int k_place(int key, int chunk) {
  if constexpr (I4) {
    return key * Tile<I4, D>::kRow + 16 * chunk;
  } else {
    return key * Tile<I4, D>::kRow + 16 * (chunk ^ ((key & 1) << 2));
  }
}

template <bool I4, int D>
__device__ __forceinline__ void load_tile(uint32_t stage, const CacheDecodeArgs& a, size_t row0, int j0, int n,
                                          int lane) {
  using T = Tile<I4, D>;
  const char* K = static_cast<const char*>(a.K) + (row0 + j0) * T::kRow;
  const char* V = static_cast<const char*>(a.V) + (row0 + j0) * T::kRow;
#pragma unroll
  for (int i = lane; i < T::kKeys * T::kChunks; i += 32) {
    const int key = i / T::kChunks, c = i % T::kChunks;
    const bool ok = j0 + key < n;
    const size_t off = ok ? (size_t)i * 16 : 0;
    cp16(stage + k_place<I4, D>(key, c), K + off, ok);
    cp16(stage + T::kVOff + v_place<I4, D>(key, c), V + off, ok);
  }
  if constexpr (I4) {
    const bool ok = j0 + lane < n;
    const size_t off = (row0 + j0 + (ok ? lane : 0)) * 4;
    cp4(stage + T::kPOff + 4 * lane, static_cast<const char*>(a.Kp) + off, ok);
    cp4(stage + T::kPOff + 4 * T::kKeys + 4 * lane, static_cast<const char*>(a.Vp) + off, ok);
  }
}

// Partial state of one warp for NT column tiles (four heads each).
template <int D, int NT>
struct State {
  float O[NT][D / 16][4];  // rows: head dims; columns 2t, 2t+1: O1, O2 of lane t's head
  float m[NT], omega[NT], T[NT];
};

template <bool I4, int D, int G, bool W>
__device__ __forceinline__ void compute_block(State<D, (G + 3) / 4>& s, uint32_t stage, int blk,
                                              const uint32_t (&qf)[(G + 3) / 4][D / 16][2], float cs,
                                              float* __restrict__ scores, int j0, int n, int lane) {
  using T = Tile<I4, D>;
  constexpr int NT = (G + 3) / 4, KS = D / 16;
  const int g = lane >> 2, t = lane & 3;
  const int kb = 16 * blk;
  // ---- scores: rows = keys g, g + 8; columns = q, rho of the heads.
  float S[NT][2][4];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[u][0][e] = S[u][1][e] = 0.f;
  uint32_t pk[2] = {0u, 0u};
  if constexpr (I4) {
    constexpr int WPL = D / 32;  // code words a lane has of a key
    uint32_t w[2][4], mz[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t at = stage + (kb + g + 8 * r) * T::kRow + 4 * WPL * t;
      if constexpr (WPL == 4) {
        lds128(w[r], at);
      } else {
        lds64(w[r][0], w[r][1], at);
      }
      pk[r] = lds32(stage + T::kPOff + 4 * (kb + g + 8 * r));
      mz[r] = neg_zero_points(__byte_perm(pk[r], 0, 0x3232));
    }
#pragma unroll
    for (int i = 0; i < WPL; ++i) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t x0 = p ? w[0][i] >> 8 : w[0][i], x1 = p ? w[1][i] >> 8 : w[1][i];
        const uint32_t a0 = nib_even(x0, mz[0]), a1 = nib_even(x1, mz[1]);
        const uint32_t a2 = nib_odd(x0, mz[0]), a3 = nib_odd(x1, mz[1]);
#pragma unroll
        for (int u = 0; u < NT; ++u) mma_bf16(S[u][p], a0, a1, a2, a3, qf[u][2 * i + p][0], qf[u][2 * i + p][1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t x[4], y[4];
      lds128(x, stage + k_place<I4, D>(kb + g, 4 * i + t));
      lds128(y, stage + k_place<I4, D>(kb + g + 8, 4 * i + t));
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int u = 0; u < NT; ++u)
          mma_bf16(S[u][p], x[2 * p], y[2 * p], x[2 * p + 1], y[2 * p + 1], qf[u][2 * i + p][0],
                   qf[u][2 * i + p][1]);
    }
  }
  // ---- weights.
  uint32_t hi[NT][2], lo[NT][2];
  float sv[2] = {1.f, 1.f}, ks[2] = {cs, cs}, kt[2] = {1.f, 1.f};
  if constexpr (I4) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sv[r] = bf_lo(lds32(stage + T::kPOff + 4 * (T::kKeys + kb + g + 8 * r)));
      kt[r] = bf_lo(pk[r]) * 64.f;
      ks[r] = kt[r] * cs;
    }
  }
  float sc[NT][2], tt[NT][2];
  bool raise = false;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = j0 + kb + g + 8 * r;
      const bool seen = j < n;
      sc[u][r] = seen ? (S[u][0][2 * r] + S[u][1][2 * r]) * ks[r] : -CUDART_INF_F;
      tt[u][r] = (S[u][0][2 * r + 1] + S[u][1][2 * r + 1]) * kt[r];
      if constexpr (W) {
        if (seen && t < G) scores[(size_t)j * G + 4 * u + t] = sc[u][r];
      }
    }
    raise |= fmaxf(sc[u][0], sc[u][1]) > s.m[u];
  }
  if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float mx = fmaxf(sc[u][0], sc[u][1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m = mx > s.m[u] ? mx + kHeadroom : s.m[u];
      const float f = exp2f(s.m[u] - m);
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
  for (int u = 0; u < NT; ++u) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float w = exp2f(sc[u][r] - s.m[u]);
      const float wt = w * tt[u][r];
      s.omega[u] += w;
      s.T[u] += wt;
      const float p0 = w * sv[r], p1 = wt * sv[r];
      const uint32_t h = pack_bf16(p0, p1);
      const uint32_t l = pack_bf16(p0 - bf_lo(h), p1 - bf_hi(h));
      if constexpr (G == 1) {
        hi[u][r] = movmatrix_trans(t == 0 ? h : (t == 1 ? l : 0u));
      } else if constexpr (G == 2) {
        hi[u][r] = movmatrix_trans(t < 2 ? h : l);
      } else {
        hi[u][r] = movmatrix_trans(h);
        lo[u][r] = movmatrix_trans(l);
      }
    }
  }
  // ---- values: rows = head dims, contraction over the block's 16 keys.
  if constexpr (I4) {
    constexpr int WPG = D / 64;  // code words a lane has of a key
    uint32_t w[4][2], mz[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // Key 2t + (e & 1) + 8 (e >> 1); its slot (v_place) is 8 (e >> 1) + 4 (e & 1) + t.
      const int slot = 8 * (e >> 1) + 4 * (e & 1) + t;
      const uint32_t row = stage + T::kVOff + (kb + slot) * T::kRow;
      if constexpr (WPG == 2) {
        lds64(w[e][0], w[e][1], row + ((8 * g) ^ ((slot & 2) << 4)));
      } else {
        w[e][0] = lds32(row + 4 * g);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t pa, pb;
      lds64(pa, pb, stage + T::kPOff + 4 * (T::kKeys + kb + 2 * t + 8 * e));
      mz[e] = neg_zero_points(__byte_perm(pa, pb, 0x7632));
    }
#pragma unroll
    for (int i = 0; i < WPG; ++i) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7632 : 0x5410;
        const uint32_t x = __byte_perm(w[0][i], w[1][i], sel), y = __byte_perm(w[2][i], w[3][i], sel);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t x8 = p ? x >> 8 : x, y8 = p ? y >> 8 : y;
          const uint32_t a0 = nib_even(x8, mz[0]), a1 = nib_odd(x8, mz[0]);
          const uint32_t a2 = nib_even(y8, mz[1]), a3 = nib_odd(y8, mz[1]);
          const int mt = 4 * i + 2 * half + p;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            mma_bf16(s.O[u][mt], a0, a1, a2, a3, hi[u][0], hi[u][1]);
            if constexpr (G >= 4) mma_bf16(s.O[u][mt], a0, a1, a2, a3, lo[u][0], lo[u][1]);
          }
        }
      }
    }
  } else {
    // Matrices of ldmatrix: (dims 0-7 | 8-15 of the tile) x (keys 0-7 | 8-15).
    const int key = kb + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t x[4];
      ldmatrix4_trans(x, stage + T::kVOff + v_place<I4, D>(key, 2 * mt + half));
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        mma_bf16(s.O[u][mt], x[0], x[1], x[2], x[3], hi[u][0], hi[u][1]);
        if constexpr (G >= 4) mma_bf16(s.O[u][mt], x[0], x[1], x[2], x[3], lo[u][0], lo[u][1]);
      }
    }
  }
}

// A record: m, omega, T, unused, O1[D], O2[D].
template <int D>
constexpr int kRec = 2 * D + 4;

template <bool I4, int D, int G, bool W>
__global__ void __launch_bounds__(kThreads, G == 8 ? 3 : 4) cache_decode_kernel(const CacheDecodeArgs a) {
  using T = Tile<I4, D>;
  constexpr int NT = (G + 3) / 4, KS = D / 16, R = kRec<D>;
  static_assert((kWarps + 1) * G * R * 4 <= T::kSmem, "the merge reuses the ring");
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  grid_dep_wait();
  grid_dep_launch();
  const int n = a.seqlens[unit / a.Hkv];
  const size_t head0 = (size_t)unit * G;  // first query row of the group ([B, H, d] with H = Hkv G)
  if (n < 1 || n > a.L) {                 // the same for every CTA of the unit
    if (split == 0) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + head0 * D;
      for (int e = threadIdx.x; e < G * D; e += kThreads) out[e] = __float2bfloat16(0.f);
      if (threadIdx.x == 0) atomicOr(a.status, kStatusBadSeqlen);
    }
    return;
  }
  const size_t row0 = (size_t)unit * a.L;
  const int tiles = (n + T::kKeys - 1) / T::kKeys;
  const int tile0 = (int)((long long)tiles * split / a.splits) + warp;
  const int tile1 = (int)((long long)tiles * (split + 1) / a.splits);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * T::kWarpBytes;
  // ---- fill the ring.
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) {
    const int tile = tile0 + i * kWarps;
    if (tile < tile1) load_tile<I4, D>(ring + i * T::kBytes, a, row0, tile * T::kKeys, n, lane);
    cp_commit();
  }
  // ---- query rows as MMA columns: column g is q (even) or rho (odd) of head g/2 (modulo G).
  uint32_t qf[NT][KS][2];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int h = (G >= 4) ? 4 * u + (g >> 1) : (g >> 1) % G;
    const uint4* row =
        reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>((g & 1) ? a.r : a.q) + (head0 + h) * D);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if constexpr (I4) {
        const uint4 v = row[(D / 32) * t + i];  // the eight dims of one code word
        qf[u][2 * i][0] = __byte_perm(v.x, v.z, 0x5410);
        qf[u][2 * i][1] = __byte_perm(v.x, v.z, 0x7632);
        qf[u][2 * i + 1][0] = __byte_perm(v.y, v.w, 0x5410);
        qf[u][2 * i + 1][1] = __byte_perm(v.y, v.w, 0x7632);
      } else {
        const uint4 v = row[4 * i + t];
        qf[u][2 * i][0] = v.x;
        qf[u][2 * i][1] = v.y;
        qf[u][2 * i + 1][0] = v.z;
        qf[u][2 * i + 1][1] = v.w;
      }
    }
  }
  const float cs = kLog2e * rsqrtf((float)D);
  State<D, NT> s;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    s.m[u] = kNoRef;
    s.omega[u] = s.T[u] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.O[u][i][e] = 0.f;
  }
  float* scores = W ? a.scores + row0 * G : nullptr;
  int stage = 0;
  for (int tile = tile0; tile < tile1; tile += kWarps) {
    cp_wait<T::kStages - 2>();
    __syncwarp();  // every lane's copies have landed, and the stage refilled below is no longer read
    const int next = tile + (T::kStages - 1) * kWarps;
    const int fill = stage == 0 ? T::kStages - 1 : stage - 1;
    if (next < tile1) load_tile<I4, D>(ring + fill * T::kBytes, a, row0, next * T::kKeys, n, lane);
    cp_commit();
#pragma unroll
    for (int blk = 0; blk < T::kKeys / 16; ++blk)
      compute_block<I4, D, G, W>(s, ring + stage * T::kBytes, blk, qf, cs, scores, tile * T::kKeys, n, lane);
    stage = stage == T::kStages - 1 ? 0 : stage + 1;
  }
  // ---- merge the warps: records in shared memory, over the ring.
  cp_wait<0>();
  __syncthreads();
  float* recs = reinterpret_cast<float*>(smem);        // [warp][G][R]
  float* merged = recs + kWarps * G * R;               // [G][R]
  constexpr float kUnit = I4 ? 64.f : 1.f;             // (c - z) 2^-6
#pragma unroll
  for (int u = 0; u < NT; ++u) {
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
      float* rec = recs + (warp * G + 4 * u + t) * R;
      if (g == 0) {
        rec[0] = s.m[u];
        rec[1] = s.omega[u];
        rec[2] = s.T[u];
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int d0 = I4 ? 8 * ((D / 64) * g + (i >> 2)) + 2 * (i & 3) : 16 * i + g;
        const int d1 = I4 ? d0 + 1 : d0 + 8;
        rec[4 + d0] = s.O[u][i][0] * kUnit;
        rec[4 + D + d0] = s.O[u][i][1] * kUnit;
        rec[4 + d1] = s.O[u][i][2] * kUnit;
        rec[4 + D + d1] = s.O[u][i][3] * kUnit;
      }
    }
  }
  __syncthreads();
  const bool final_here = !W && a.splits == 1;
  float* dst = a.partials ? a.partials + ((size_t)unit * a.splits + split) * G * R : merged;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + head0 * D;
  for (int e = threadIdx.x; e < G * D; e += kThreads) {
    const int h = e / D, dim = e % D;
    float m = recs[h * R];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, recs[(w * G + h) * R]);
    float omega = 0.f, tsum = 0.f, o1 = 0.f, o2 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* rec = recs + (w * G + h) * R;
      const float f = exp2f(rec[0] - m);
      omega += f * rec[1];
      tsum += f * rec[2];
      o1 += f * rec[4 + dim];
      o2 += f * rec[4 + D + dim];
    }
    if (final_here) {
      const float inv = 1.f / omega;
      out[e] = __float2bfloat16(((1.f + tsum * inv) * o1 - o2) * inv);
    } else {
      float* rec = dst + h * R;
      if (dim == 0) {
        rec[0] = m;
        rec[1] = omega;
        rec[2] = tsum;
      }
      rec[4 + dim] = o1;
      rec[4 + D + dim] = o2;
    }
  }
  if (a.partials || final_here) return;
  // ---- merge the cluster's CTAs, a share of the outputs each.
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = split * kThreads + threadIdx.x; e < G * D; e += a.splits * kThreads) {
    const int h = e / D, dim = e % D;
    float m = kNoRef;
    for (int c = 0; c < a.splits; ++c) m = fmaxf(m, cluster.map_shared_rank(merged, c)[h * R]);
    float omega = 0.f, tsum = 0.f, o1 = 0.f, o2 = 0.f;
    for (int c = 0; c < a.splits; ++c) {
      const float* rec = cluster.map_shared_rank(merged, c) + h * R;
      const float f = exp2f(rec[0] - m);
      omega += f * rec[1];
      tsum += f * rec[2];
      o1 += f * rec[4 + dim];
      o2 += f * rec[4 + D + dim];
    }
    const float inv = 1.f / omega;
    out[e] = __float2bfloat16(((1.f + tsum * inv) * o1 - o2) * inv);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

constexpr int kFinThreads = 256;
constexpr int kFinKeys = 1024;  // keys of a CTA of the second kernel

// Merges the records of a unit (the CTA of its first keys writes the output)
// and turns scores into weights: w_out = w_in + sum_h 2^(s_h - m_h) / omega_h.
template <int D, int G, bool W>
__global__ void __launch_bounds__(kFinThreads) cache_finish_kernel(const CacheDecodeArgs a, int parts) {
  constexpr int R = kRec<D>;
  __shared__ float sm[G], sinv[G], stb[G];
  const int unit = blockIdx.x / parts, part = blockIdx.x % parts;
  grid_dep_wait();
  grid_dep_launch();
  const int n = a.seqlens[unit / a.Hkv];
  if (n < 1 || n > a.L || part * kFinKeys >= n) return;
  const float* recs = a.partials + (size_t)unit * a.splits * G * R;
  const int lane = threadIdx.x & 31;
  for (int h = threadIdx.x >> 5; h < G; h += kFinThreads / 32) {
    float m = kNoRef;
    for (int c = lane; c < a.splits; c += 32) m = fmaxf(m, recs[(size_t)(c * G + h) * R]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float omega = 0.f, tsum = 0.f;
    for (int c = lane; c < a.splits; c += 32) {
      const float* rec = recs + (size_t)(c * G + h) * R;
      const float f = exp2f(rec[0] - m);
      omega += f * rec[1];
      tsum += f * rec[2];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      omega += __shfl_xor_sync(0xffffffffu, omega, o);
      tsum += __shfl_xor_sync(0xffffffffu, tsum, o);
    }
    if (lane == 0) {
      sm[h] = m;
      sinv[h] = 1.f / omega;
      stb[h] = tsum / omega;
    }
  }
  __syncthreads();
  if (part == 0) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)unit * G * D;
    for (int e = threadIdx.x; e < G * D; e += kFinThreads) {
      const int h = e / D, dim = e % D;
      float o1 = 0.f, o2 = 0.f;
      for (int c = 0; c < a.splits; ++c) {
        const float* rec = recs + (size_t)(c * G + h) * R;
        const float f = exp2f(rec[0] - sm[h]);
        o1 += f * rec[4 + dim];
        o2 += f * rec[4 + D + dim];
      }
      out[e] = __float2bfloat16(((1.f + stb[h]) * o1 - o2) * sinv[h]);
    }
  }
  if constexpr (W) {
    const size_t row0 = (size_t)unit * a.L;
    const int end = min(n, (part + 1) * kFinKeys);
    for (int j = part * kFinKeys + threadIdx.x; j < end; j += kFinThreads) {
      const float* sc = a.scores + (row0 + j) * G;
      float x[G];
      if constexpr (G >= 4) {
#pragma unroll
        for (int h = 0; h < G; h += 4) *reinterpret_cast<float4*>(x + h) = *reinterpret_cast<const float4*>(sc + h);
      } else {
#pragma unroll
        for (int h = 0; h < G; ++h) x[h] = sc[h];
      }
      float w = 0.f;
#pragma unroll
      for (int h = 0; h < G; ++h) w += exp2f(x[h] - sm[h]) * sinv[h];
      a.w_out[row0 + j] = a.w_in[row0 + j] + w;
    }
  }
}

template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, unsigned grid, unsigned block, size_t smem, int cluster, cudaStream_t st,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  // The kernel may be set up while the one before it in the stream drains; it
  // waits for that one's end before it touches memory.
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool I4, int D, int G, bool W>
cudaError_t run(const CacheDecodeArgs& a, cudaStream_t st) {
  using T = Tile<I4, D>;
  auto kern = cache_decode_kernel<I4, D, G, W>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)a.B * a.Hkv;
  const int cluster = a.partials ? 1 : a.splits;
  e = launch(kern, units * a.splits, kThreads, T::kSmem, cluster, st, a);
  if (e != cudaSuccess || !a.partials) return e;
  const int parts = W ? (a.L + kFinKeys - 1) / kFinKeys : 1;
  return launch(cache_finish_kernel<D, G, W>, units * parts, kFinThreads, 0, 1, st, a, parts);
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

int cache_decode_splits(long long units, int L, int num_sms, bool weights) {
  // Two waves of four CTAs an SM, while a CTA keeps a 32-key tile for each of its warps.
  int s = 1;
  while (s < 64 && units * s < 8ll * num_sms && (long long)L > 128ll * s) s *= 2;
  (void)weights;
  return s;
}

CacheDecodeSpace cache_decode_space(int B, int H, int Hkv, int L, int d, int num_sms, bool weights) {
  CacheDecodeSpace w;
  w.splits = cache_decode_splits((long long)B * Hkv, L, num_sms, weights);
  if (weights || w.splits > 8) w.partials = sizeof(float) * (size_t)B * H * w.splits * (2 * d + 4);
  if (weights) w.scores = sizeof(float) * (size_t)B * H * L;
  w.partials = (w.partials + 255) / 256 * 256;
  return w;
}

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t st) {
  const bool i4 = a.Kp != nullptr, w = a.w_out != nullptr;
  if (i4) return w ? pick<true, true>(a, st) : pick<true, false>(a, st);
  return w ? pick<false, true>(a, st) : cudaErrorInvalidValue;
}

}  // namespace plx
