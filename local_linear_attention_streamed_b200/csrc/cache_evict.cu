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
// * select: one CTA a (b, KV head).  Radix select over the totals as ordered
//   32-bit integers (11 + 11 + 10 bits, histograms in shared memory) gives the
//   smallest kept value and how many of its equals stay; ballots then number
//   the kept rows in order.  Integer counts only, so the result does not depend
//   on the order of the atomics.
// * move: CTAs over (b, KV head), kept rows and caches; the totals are one more
//   cache of 4-byte rows, with zeros behind the last.  A row moved within its
//   cache goes to a lower index, so an in-place cache is compacted by one CTA a
//   (b, KV head) that reads a run of rows, waits, and writes it: rows still to
//   be read always lie behind those written.
#include "plx_internal.cuh"

namespace plx {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Totals as unsigned integers in the same order: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive sum of x over the block's threads (kSelThreads); *total gets the sum.
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
  int v = warp_sums[lane];
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int sums[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x;
  const int room = min(a.budget, a.L);
  int n = a.seqlens[unit / a.Hkv];
  if (n < 1 || n > a.L) {
    if (tid == 0) atomicOr(a.status, kStatusBadSeqlen);
    n = 0;
  }
  const float* w = a.w + (size_t)unit * a.L;
  int* kept = a.kept + (size_t)unit * room;
  const int nk = min(n, a.budget);
  for (int i = nk + tid; i < room; i += kSelThreads) kept[i] = -1;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // rows that compete
  // ---- the value of rank `need` among them, 11, 11 and 10 bits at a time.
  uint32_t prefix = 0;                        // decided high bits of the threshold
  int need = a.budget - a.sinks - a.recent;   // rows to keep among those that match the prefix
  const int shifts[3] = {21, 10, 0};
  if (need > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = shifts[pass];
      const uint32_t bins = pass == 2 ? 1024u : 2048u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t k = order_key(w[j]);
        const bool in = pass == 0 || (pass == 1 ? k >> 21 : k >> 10) == prefix;
        if (in) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // Bins from the top, two a thread: the bin where the running count reaches `need`.
      const int b1 = kBins - 1 - 2 * tid, c1 = hist[b1], c0 = hist[b1 - 1];
      int total;
      const int above = block_scan(c1 + c0, sums, &total);
      if (above < need && need <= above + c1) {
        s_prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)b1;
        s_need = need - above;
      } else if (above + c1 < need && need <= above + c1 + c0) {
        s_prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)(b1 - 1);
        s_need = need - above - c1;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      __syncthreads();
    }
  }
  // Keep every competitor above the threshold and the first `need` equal to it
  // (need == 0 only where no competitor stays: nothing is above or equal then).
  const bool any = a.budget > a.sinks + a.recent;
  const int seg = ((n + kSelThreads - 1) / kSelThreads) * 32;  // rows of a warp
  const int j0 = warp * seg, j1 = min(n, j0 + seg);
  int gt = 0, eq = 0;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    bool sure = false, tie = false;
    if (j < j1) {
      const bool fixed = j < lo || j >= hi;
      const uint32_t k = order_key(w[j]);
      sure = fixed || (any && k > prefix);
      tie = !fixed && any && k == prefix;
    }
    gt += __popc(__ballot_sync(0xffffffffu, sure));
    eq += __popc(__ballot_sync(0xffffffffu, tie));
  }
  int total;
  int gbase = block_scan(lane == 0 ? gt : 0, sums, &total);
  int ebase = block_scan(lane == 0 ? eq : 0, sums, &total);
  gbase = __shfl_sync(0xffffffffu, gbase, 0);
  ebase = __shfl_sync(0xffffffffu, ebase, 0);
  const uint32_t below = (1u << lane) - 1u;
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    bool sure = false, tie = false;
    if (j < j1) {
      const bool fixed = j < lo || j >= hi;
      const uint32_t k = order_key(w[j]);
      sure = fixed || (any && k > prefix);
      tie = !fixed && any && k == prefix;
    }
    const uint32_t gm = __ballot_sync(0xffffffffu, sure), em = __ballot_sync(0xffffffffu, tie);
    const int er = ebase + __popc(em & below);  // equals before this row
    if (sure || (tie && er < need)) kept[gbase + __popc(gm & below) + min(er, need)] = j;
    gbase += __popc(gm);
    ebase += __popc(em);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 128;  // kept rows of a CTA
constexpr int kMoveUnroll = 4;

struct MoveList {
  int vec[kEvictMaxCaches + 1];  // bytes a thread moves at once: 16, 4 or 1
};

template <typename V>
__device__ __forceinline__ void move_rows(const V* src, V* dst, const int* kept, int i0, int i1, int per_row) {
  const int total = (i1 - i0) * per_row;
  for (int base = threadIdx.x; base < total; base += kMoveUnroll * kMoveThreads) {
    V v[kMoveUnroll];
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const int x = base + e * kMoveThreads;
      if (x < total) v[e] = src[(size_t)kept[i0 + x / per_row] * per_row + x % per_row];
    }
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const int x = base + e * kMoveThreads;
      if (x < total) dst[(size_t)i0 * per_row + x] = v[e];
    }
  }
}

// Within one cache: a run is read by all threads before any of it is written.
template <typename V>
__device__ __forceinline__ void compact_rows(V* rows, const int* kept, int nk, int per_row) {
  const long long total = (long long)nk * per_row;
  for (long long base = 0; base < total; base += kMoveUnroll * kMoveThreads) {
    V v[kMoveUnroll];
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const long long x = base + e * kMoveThreads + threadIdx.x;
      if (x < total) v[e] = rows[(long long)kept[x / per_row] * per_row + x % per_row];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) {
      const long long x = base + e * kMoveThreads + threadIdx.x;
      if (x < total) rows[x] = v[e];
    }
    __syncthreads();
  }
}

// blockIdx.y: the cache, the totals last.  New lengths are written by the CTAs
// of the totals of head 0; min(n, budget) of a new length is itself, so lengths
// may be updated in place.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, const MoveList list, int parts) {
  const int unit = blockIdx.x / parts, part = blockIdx.x % parts, c = blockIdx.y;
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
    if (part != 0) return;
    if (n > a.budget && nk > 0) {
      if (vec == 16) {
        compact_rows(reinterpret_cast<uint4*>(dst), kept, nk, rb / 16);
      } else if (vec == 4) {
        compact_rows(reinterpret_cast<uint32_t*>(dst), kept, nk, rb / 4);
      } else {
        compact_rows(reinterpret_cast<uint8_t*>(dst), kept, nk, rb);
      }
    }
  } else {
    const int i0 = part * kMoveRows, i1 = min(nk, i0 + kMoveRows);
    if (i0 < i1) {
      if (vec == 16) {
        move_rows(reinterpret_cast<const uint4*>(src), reinterpret_cast<uint4*>(dst), kept, i0, i1, rb / 16);
      } else if (vec == 4) {
        move_rows(reinterpret_cast<const uint32_t*>(src), reinterpret_cast<uint32_t*>(dst), kept, i0, i1, rb / 4);
      } else {
        move_rows(reinterpret_cast<const uint8_t*>(src), reinterpret_cast<uint8_t*>(dst), kept, i0, i1, rb);
      }
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
  (void)num_sms;
  const unsigned units = (unsigned)a.B * a.Hkv;
  evict_select_kernel<<<units, kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  MoveList list;
  for (int c = 0; c <= a.count; ++c) {
    const int rb = c == a.count ? 4 : a.row_bytes[c];
    const uintptr_t at = c == a.count
                             ? reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.w_out)
                             : reinterpret_cast<uintptr_t>(a.src[c]) | reinterpret_cast<uintptr_t>(a.dst[c]);
    list.vec[c] = ((at | rb) & 15) == 0 ? 16 : ((at | rb) & 3) == 0 ? 4 : 1;
  }
  const int room = a.budget < a.L ? a.budget : a.L;
  const int parts = (room + kMoveRows - 1) / kMoveRows;
  evict_move_kernel<<<dim3(units * parts, a.count + 1), kMoveThreads, 0, st>>>(a, list, parts);
  return cudaGetLastError();
}

}  // namespace plx
