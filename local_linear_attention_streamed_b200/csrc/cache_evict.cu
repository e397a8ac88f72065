// Eviction from a KV cache by accumulated attention weight.
//
// For every (b, KV head) with n visible rows and n > budget, the rows that stay
// are the first `sinks`, the last `recent` and, between them, the
// budget - sinks - recent rows of largest total weight (ties: the lower index
// stays; a NaN total counts as less than any number).  They move to the front
// of the cache (in place, or of another cache) in the order of their positions.
//
// Two kernels, both bound by HBM (4 n bytes of totals, then each kept row read
// and written once):
// * select: one CTA (or cluster) a (b, KV head), the totals in its registers.  Radix select over
//   them as ordered 32-bit integers (11 + 11 + 10 bits, histograms in shared
//   memory) gives the
//   smallest kept value and how many of its equals stay; ballots then number
//   the kept rows in order.  Integer counts only, so the result does not depend
//   on the order of the atomics.
// * move: CTAs over (b, KV head), kept rows and caches; the totals are one more
//   cache of 4-byte rows, with zeros behind the last.  A row moved within its
//   cache goes to a lower index, so an in-place cache is compacted by one CTA a
//   (b, KV head) and slice of the rows that reads a run, waits, and writes it:
//   rows still to be read always lie behind those written.
#include "launch.cuh"
#include "plx_internal.cuh"

#include <cooperative_groups.h>
#include <type_traits>

namespace cg = cooperative_groups;

namespace plx {
namespace {

constexpr int kBins = 2048;

// Totals as unsigned integers in the same order: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive sum of x over the W warps of the block; *total gets the sum.
template <int W>
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int v = lane < W ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  *total = __shfl_sync(0xffffffffu, v, 31);
  const int base = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
  __syncthreads();
  return (warp ? base : 0) + s - x;
}

// C CTAs (a cluster) of W warps a (b, KV head).  Warp w of them has the rows
// [w 32 K, (w + 1) 32 K), lane l of it every 32nd from l, as K order keys in
// registers: the totals are read once.  K = 0: any length, the totals are read
// (from L2) in every pass.  In a cluster the first CTA adds the histograms up and
// tells the others what it found.
template <int W, int K, int C>
__global__ void __launch_bounds__(W * 32) evict_select_kernel(const EvictArgs a) {
  constexpr int kSelThreads = W * 32;
  constexpr int kCopies = W >= 32 ? 4 : 1;  // histograms, for fewer collisions between warps
  constexpr int kPer = kBins / kSelThreads;
  __shared__ __align__(16) int hist[kCopies][kBins];         // the largest digit first
  __shared__ __align__(16) int all[C > 1 ? kBins : 4];       // the cluster's, in its first CTA
  __shared__ int sums[W], counts[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  grid_dep_wait();
  grid_dep_launch();
  const int room = min(a.budget, a.L);
  int n = a.seqlens[unit / a.Hkv];
  if (n < 1 || n > a.L) {
    if (rank == 0 && tid == 0) atomicOr(a.status, kStatusBadSeqlen);
    n = 0;
  }
  const float* w = a.w + (size_t)unit * a.L;
  int* kept = a.kept + (size_t)unit * room;
  const int nk = min(n, a.budget);
  for (int i = nk + rank * kSelThreads + tid; i < room; i += C * kSelThreads) kept[i] = -1;
  if (n <= a.budget) {  // the same for the whole cluster
    for (int i = rank * kSelThreads + tid; i < n; i += C * kSelThreads) kept[i] = i;
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // rows that compete
  const int turns = K > 0 ? K : (n + C * kSelThreads - 1) / (C * kSelThreads);
  const int j0 = (rank * W + warp) * 32 * turns + lane;
  uint32_t keys[K > 0 ? K : 1];
  if constexpr (K > 0) {
#pragma unroll
    for (int i = 0; i < K; ++i) keys[i] = __float_as_uint(w[min(j0 + 32 * i, n - 1)]);
#pragma unroll
    for (int i = 0; i < K; ++i) keys[i] = order_key(__uint_as_float(keys[i]));
  }
  auto key = [&](int i, int j) { return K > 0 ? keys[K > 0 ? i : 0] : order_key(w[j]); };
  // ---- the value of rank `need` among them, 11, 11 and 10 bits at a time.
  uint32_t prefix = 0;                       // decided high bits of the threshold
  int need = a.budget - a.sinks - a.recent;  // rows to keep among those that match the prefix
  const bool any = need > 0;
  int low = 0;  // bits below the prefix
  if (any) {
    if constexpr (C > 1) {
      if (rank == 0)
        for (int i = tid; i < kBins; i += kSelThreads) all[i] = 0;
      cg::this_cluster().sync();
    }
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kCopies * kBins / 4; i += kSelThreads)
        reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < turns; ++i) {
        const int j = j0 + 32 * i;
        if (j >= lo && j < hi) {
          const uint32_t k = key(i, j);
          const bool in = pass == 0 || (pass == 1 ? k >> 21 : k >> 10) == prefix;
          if (in) atomicAdd(&hist[warp % kCopies][~(k >> shift) & mask], 1);
        }
      }
      __syncthreads();
      const int* from = hist[0];
      if constexpr (C > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        int* sum = cluster.map_shared_rank(all, 0);
        for (int i = tid; i < kBins; i += kSelThreads)
          if (const int x = hist[0][i]) atomicAdd(&sum[i], x);
        cluster.sync();
        from = all;
      }
      if (rank == 0) {
        // Bins, the largest values first, kPer a thread: the one where the running count reaches `need`.
        using Vec = typename std::conditional<kPer >= 4, int4, int2>::type;
        constexpr int kVec = sizeof(Vec) / 4;
        int c[kPer] = {}, mine = 0, total;
#pragma unroll
        for (int copy = 0; copy < kCopies; ++copy)
#pragma unroll
          for (int i = 0; i < kPer; i += kVec) {
            const Vec v = *reinterpret_cast<const Vec*>(from + copy * kBins + kPer * tid + i);
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[i + e] += reinterpret_cast<const int*>(&v)[e];
          }
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += c[i];
        int above = block_scan<W>(mine, sums, &total);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (above < need && need <= above + c[i]) {
            const uint32_t p = (prefix << (pass == 2 ? 10 : 11)) | (mask - (uint32_t)(kPer * tid + i));
#pragma unroll
            for (int o = 0; o < C; ++o) {
              if constexpr (C > 1) {
                *cg::this_cluster().map_shared_rank(&s_prefix, o) = p;
                *cg::this_cluster().map_shared_rank(&s_need, o) = need - above;
                *cg::this_cluster().map_shared_rank(&s_found, o) = c[i];
              } else {
                s_prefix = p;
                s_need = need - above;
                s_found = c[i];
              }
            }
          }
          above += c[i];
          if constexpr (C > 1) all[kPer * tid + i] = 0;
        }
      }
      if constexpr (C > 1) {
        cg::this_cluster().sync();
      } else {
        __syncthreads();
      }
      prefix = s_prefix;
      need = s_need;
      low = shift;
      if (need == s_found) break;  // all that match stay: no need to tell them apart
    }
  }
  // ---- number the kept rows: every competitor above the threshold and the first
  // `need` equal to it, the first and the last rows.
  uint32_t sure_at[K > 0 ? K : 1], tie_at[K > 0 ? K : 1];
  auto vote = [&](int i, uint32_t& gm, uint32_t& em) {
    const int j = j0 + 32 * i;
    bool sure = false, tie = false;
    if (j < n) {
      const bool fixed = j < lo || j >= hi;
      const uint32_t k = fixed ? 0u : key(i, j) >> low;
      sure = fixed || (any && k > prefix);
      tie = !fixed && any && k == prefix;
    }
    gm = __ballot_sync(0xffffffffu, sure);
    em = __ballot_sync(0xffffffffu, tie);
  };
  int gt = 0, eq = 0, gsum, esum;
#pragma unroll
  for (int i = 0; i < turns; ++i) {
    uint32_t gm, em;
    vote(i, gm, em);
    gt += __popc(gm);
    eq += __popc(em);
    if constexpr (K > 0) sure_at[i] = gm, tie_at[i] = em;
  }
  int gbase = block_scan<W>(lane == 0 ? gt : 0, sums, &gsum);
  int ebase = block_scan<W>(lane == 0 ? eq : 0, sums, &esum);
  gbase = __shfl_sync(0xffffffffu, gbase, 0);
  ebase = __shfl_sync(0xffffffffu, ebase, 0);
  if constexpr (C > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (tid == 0) counts[0] = gsum, counts[1] = esum;
    cluster.sync();
    for (int o = 0; o < rank; ++o) {
      const int* before = cluster.map_shared_rank(counts, o);
      gbase += before[0];
      ebase += before[1];
    }
    cluster.sync();  // no CTA leaves while another reads its counts
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < turns; ++i) {
    uint32_t gm, em;
    if constexpr (K > 0) {
      gm = sure_at[i], em = tie_at[i];
    } else {
      vote(i, gm, em);
    }
    const int er = ebase + __popc(em & below);  // equals before this row
    if ((gm >> lane & 1) || ((em >> lane & 1) && er < need))
      kept[gbase + __popc(gm & below) + min(er, need)] = j0 + 32 * i;
    gbase += __popc(gm);
    ebase += __popc(em);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 1024;  // kept rows of a CTA, at most
constexpr int kMoveUnroll = 8;

struct MoveList {
  int vec[kEvictMaxCaches + 1];    // bytes a thread moves at once: 16, 4 or 1
  int shift[kEvictMaxCaches + 1];  // log2 of the pieces of a row; -1: no power of two
  int rows;                        // kept rows of a CTA
  int slices;                      // of an in-place cache's rows, at most
};

template <typename V, bool kShift>
__device__ __forceinline__ void move_rows(const V* src, V* dst, const int* kept, int rows, int per_row, int shift) {
  const int total = rows * per_row;
  for (int base = threadIdx.x; base < total; base += kMoveUnroll * kMoveThreads) {
    V v[kMoveUnroll];
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const int x = base + e * kMoveThreads;
      if (x < total) {
        const int row = kShift ? x >> shift : x / per_row;
        v[e] = __ldcs(src + (size_t)kept[row] * per_row + (x - row * per_row));  // read once
      }
    }
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const int x = base + e * kMoveThreads;
      if (x < total) dst[x] = v[e];
    }
  }
}

// Within one cache, pieces [first, first + width) of its rows: a run is read by all
// threads before any of it is written.
constexpr int kCompactUnroll = 8;
template <typename V>
__device__ __forceinline__ void compact_rows(V* rows, const int* kept, int nk, int per_row, int first, int width) {
  const int shift = (width & (width - 1)) == 0 ? __ffs(width) - 1 : -1;
  const long long total = (long long)nk * width;
  rows += first;
  for (long long base = 0; base < total; base += kCompactUnroll * kMoveThreads) {
    V v[kCompactUnroll];
#pragma unroll
    for (int e = 0; e < kCompactUnroll; ++e) {
      const long long x = base + e * kMoveThreads + threadIdx.x;
      if (x < total) {
        const long long row = shift >= 0 ? x >> shift : x / width;
        v[e] = rows[(long long)kept[row] * per_row + (x - row * width)];
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kCompactUnroll; ++e) {
      const long long x = base + e * kMoveThreads + threadIdx.x;
      if (x < total) {
        const long long row = shift >= 0 ? x >> shift : x / width;
        rows[row * per_row + (x - row * width)] = v[e];
      }
    }
    __syncthreads();
  }
}

// blockIdx.y: the cache, the totals last.  New lengths are written by the CTAs
// of the totals of head 0.  Lengths may be updated in place, while other CTAs read
// them: all that is taken from a length here is min(n, budget), which a new length
// gives as well.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, const MoveList list, int parts) {
  const int unit = blockIdx.x / parts, part = blockIdx.x % parts, c = blockIdx.y;
  grid_dep_wait();
  grid_dep_launch();
  const int room = min(a.budget, a.L);
  const int n = a.seqlens[unit / a.Hkv];
  const int nk = n < 1 || n > a.L ? 0 : min(n, a.budget);
  const int* kept = a.kept + (size_t)unit * room;
  const bool totals = c == a.count;
  const int rb = totals ? 4 : a.row_bytes[c];
  const char* src = static_cast<const char*>(totals ? a.w : a.src[c]) + (size_t)unit * a.L * rb;
  char* dst = static_cast<char*>(totals ? static_cast<void*>(a.w_out) : a.dst[c]) + (size_t)unit * a.Lout * rb;
  const int vec = list.vec[c];
  if (src == dst) {
    // Slices of a row, 64 bytes or more, move on their own.
    const int slices = max(1, min(min(parts, list.slices), rb / 64));
    const bool mine = part < slices && nk > 0 && kept[nk - 1] != nk - 1;  // else every row is in its place
    if (mine) {
      auto run = [&](auto piece) {
        using V = decltype(piece);
        const int pieces = rb / (int)sizeof(V), each = (pieces + slices - 1) / slices;
        const int first = part * each, width = min(each, pieces - first);
        if (width > 0) compact_rows(reinterpret_cast<V*>(dst), kept, nk, pieces, first, width);
      };
      if (vec == 16) {
        run(uint4());
      } else if (vec == 4) {
        run(uint32_t());
      } else {
        run((unsigned char)0);
      }
    }
  } else {
    const int i0 = part * list.rows, rows = min(nk - i0, list.rows);
    if (rows > 0) {
      __shared__ int ids[kMoveRows];
      for (int i = threadIdx.x; i < rows; i += kMoveThreads) ids[i] = kept[i0 + i];
      __syncthreads();
      dst += (size_t)i0 * rb;
      auto run = [&](auto piece) {
        using V = decltype(piece);
        const V* from = reinterpret_cast<const V*>(src);
        V* to = reinterpret_cast<V*>(dst);
        if (list.shift[c] >= 0) {
          move_rows<V, true>(from, to, ids, rows, rb / (int)sizeof(V), list.shift[c]);
        } else {
          move_rows<V, false>(from, to, ids, rows, rb / (int)sizeof(V), 0);
        }
      };
      if (vec == 16) {
        run(uint4());
      } else if (vec == 4) {
        run(uint32_t());
      } else {
        run((unsigned char)0);
      }
      dst -= (size_t)i0 * rb;
    }
  }
  if (totals && part == 0) {
    float* w = reinterpret_cast<float*>(dst);
    for (int i = nk + threadIdx.x; i < a.Lout; i += kMoveThreads) w[i] = 0.f;
    if (unit % a.Hkv == 0 && threadIdx.x == 0) a.seqlens_out[unit / a.Hkv] = nk;
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st, int num_sms) {
  const unsigned units = (unsigned)a.B * a.Hkv;
  // The smallest block whose registers hold the longest sequence's totals; a
  // cluster where long sequences would leave most SMs without work (16 sequences
  // of 32768: 15 us, one CTA each 29 us).
  cudaError_t e;
  if (a.L <= 1024) {
    e = launch_dependent(evict_select_kernel<4, 8, 1>, units, 128, 0, 1, st, a);
  } else if (a.L <= 4096) {
    e = launch_dependent(evict_select_kernel<8, 16, 1>, units, 256, 0, 1, st, a);
  } else if (units < (unsigned)num_sms) {
    e = a.L <= 32768 ? launch_dependent(evict_select_kernel<8, 16, 8>, units * 8, 256, 0, 8, st, a)
                     : launch_dependent(evict_select_kernel<8, 0, 8>, units * 8, 256, 0, 8, st, a);
  } else if (a.L <= 16384) {
    e = launch_dependent(evict_select_kernel<32, 16, 1>, units, 1024, 0, 1, st, a);
  } else if (a.L <= 32768) {
    e = launch_dependent(evict_select_kernel<32, 32, 1>, units, 1024, 0, 1, st, a);
  } else {
    e = launch_dependent(evict_select_kernel<32, 0, 1>, units, 1024, 0, 1, st, a);
  }
  if (e != cudaSuccess) return e;
  MoveList list;
  for (int c = 0; c <= a.count; ++c) {
    const int rb = c == a.count ? 4 : a.row_bytes[c];
    const uintptr_t at = c == a.count
                             ? reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.w_out)
                             : reinterpret_cast<uintptr_t>(a.src[c]) | reinterpret_cast<uintptr_t>(a.dst[c]);
    list.vec[c] = ((at | rb) & 15) == 0 ? 16 : ((at | rb) & 3) == 0 ? 4 : 1;
    const int pieces = rb / list.vec[c];
    list.shift[c] = -1;
    for (int k = 0; k < 17; ++k)
      if (pieces == 1 << k) list.shift[c] = k;
  }
  const int room = a.budget < a.L ? a.budget : a.L;
  // Long runs of rows where they still make four CTAs an SM (64 x 8 batch of 1024
  // rows of 256 bytes: 97 us, with runs of 256 104 us, of 128 109 us).
  const long long runs = (long long)units * ((room + kMoveRows - 1) / kMoveRows) * a.count;
  list.rows = runs >= 4ll * num_sms ? kMoveRows : kMoveRows / 4;
  const int parts = (room + list.rows - 1) / list.rows;
  // In place, slices only where whole rows leave SMs idle (8 x 131072 rows to half:
  // 0.89 ms, whole 2.25 ms; a batch of 64 x 8 x 4096 to a quarter, whole: 0.16 ms).
  list.slices = (long long)units * a.count >= 2ll * num_sms ? 1 : parts;
  return launch_dependent(evict_move_kernel, dim3(units * parts, a.count + 1), kMoveThreads, 0, 1, st, a, list, parts);
}

}  // namespace plx
