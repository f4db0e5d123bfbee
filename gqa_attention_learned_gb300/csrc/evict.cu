// Eviction from the paged cache by accumulated attention weight: of each
// (request, KV head) the first tokens, the most recent ones and the heaviest
// of the rest stay, `budget` keys in all, in their order; their K and V rows
// and their mass move to the first slots of the request's pages (in place) or
// of other pages.
//
// Two kernels.  select: one CTA per (request, KV head) finds the weight of the
// last key that stays by a radix select over the weights' bits (exact, four
// passes of 8 bits), takes ties from the lowest index on, and writes the kept
// indices in order.  move: copies rows by that list.  In place is safe because
// the r-th kept key has index >= r: a batch of rows is read whole before any
// of it is written, and a write to slot r can only hit rows of this batch or
// earlier ones.
// Bound by HBM: 4 bytes of mass per key, 512 bytes of K and V per kept one.

#include "kernels.cuh"
#include "ptx.cuh"

#include <cmath>

namespace sa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;             // rows in flight per thread and batch

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Order-preserving bits of a weight: larger weight, larger number; -0 = +0,
// NaN below everything.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of v over the block; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();                                       // the previous scan's sums are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    const int s = warp_sums[w];
    before += w < warp ? s : 0;
    sum += s;
  }
  total = sum;
  return before + x - v;
}

__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelectWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int unit = blockIdx.x, kvh = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  const int n = p.kv_lens[b];
  int *kept = p.kept + static_cast<size_t>(unit) * p.budget;
  const int npages = cdiv(max(n, 0), kPageSize);
  const int count = min(n, p.budget);
  const int dst_pages = cdiv(max(count, 0), kPageSize);
  bool bad = n < 0 || n > p.max_kv_len || n > p.mass_stride || count > p.dst_mass_stride ||
             npages > p.max_pages_per_seq || dst_pages > p.dst_max_pages;
  if (!bad) {
    const int32_t *src = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    const int32_t *dst = p.dst_page_table + static_cast<size_t>(b) * p.dst_max_pages;
    for (int i = tid; i < npages; i += kSelectThreads) bad = bad || src[i] < 0 || src[i] >= p.num_pages;
    for (int i = tid; i < dst_pages; i += kSelectThreads) bad = bad || dst[i] < 0 || dst[i] >= p.num_pages;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && kvh == 0) p.new_kv_lens[b] = bad ? -1 : count;
  for (int i = bad ? tid : count + tid; i < p.budget; i += kSelectThreads) kept[i] = -1;
  if (bad) return;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += kSelectThreads) kept[i] = i;
    return;
  }

  const float *mass = p.mass + static_cast<size_t>(unit) * p.mass_stride;
  const int lo = p.first_tokens, hi = n - p.recent;       // the keys that compete
  int want = p.budget - p.first_tokens - p.recent;        // how many of them stay
  // the want-th largest weight, from the top 8 bits down
  uint32_t prefix = 0;
  int left = want;                                        // to take among those with the prefix
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t high = shift == 24 ? 0u : ~((1u << (shift + 8)) - 1u);
      for (int i = lo + tid; i < hi; i += kSelectThreads) {
        const uint32_t u = order_bits(mass[i]);
        if ((u & high) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int bin = 255, rest = left;
        while (hist[bin] < rest) rest -= hist[bin--];
        s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
        s_left = rest;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
  }
  // ordered compaction: weights above the threshold, and the first `left` equal to it
  int at = 0, equal_before = 0;
  for (int base = 0; base < n; base += kSelectThreads) {
    const int i = base + tid;
    bool keep = false, equal = false;
    if (i < n) {
      if (i < lo || i >= hi) {
        keep = true;
      } else if (want > 0) {
        const uint32_t u = order_bits(mass[i]);
        keep = u > prefix;
        equal = u == prefix;
      }
    }
    int total;
    const int e = block_scan(equal ? 1 : 0, warp_sums, total);
    keep = keep || (equal && equal_before + e < left);
    equal_before += total;
    const int r = block_scan(keep ? 1 : 0, warp_sums, total);
    if (keep) kept[at + r] = i;
    at += total;
  }
}

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictParams p) {
  // CTA: K rows, V rows or mass of one (request, KV head)
  const int unit = blockIdx.x % (p.batch * p.num_kv_heads);
  const int what = blockIdx.x / (p.batch * p.num_kv_heads);
  const int kvh = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
  grid_dependency_wait();
  const int count = p.new_kv_lens[b];
  if (count < 0) return;
  const int n = p.kv_lens[b];
  const int *kept = p.kept + static_cast<size_t>(unit) * p.budget;
  if (what == 2) {
    const float *src = p.mass + static_cast<size_t>(unit) * p.mass_stride;
    float *dst = p.dst_mass + static_cast<size_t>(unit) * p.dst_mass_stride;
    for (int base = 0; base < count; base += kMoveThreads) {
      const int r = base + threadIdx.x;
      const float v = r < count ? src[kept[r]] : 0.f;
      __syncthreads();
      if (r < count) dst[r] = v;
    }
    __syncthreads();
    // evicted places start again from nothing
    for (int i = count + threadIdx.x; i < min(n, p.dst_mass_stride); i += kMoveThreads) dst[i] = 0.f;
    return;
  }
  uint4 *cache = reinterpret_cast<uint4 *>(what == 0 ? p.k_cache : p.v_cache);
  const int32_t *src_table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
  const int32_t *dst_table = p.dst_page_table + static_cast<size_t>(b) * p.dst_max_pages;
  constexpr int kPieces = kHeadDim * 2 / 16;              // 16-byte pieces of a row
  constexpr int kRowsAtOnce = kMoveThreads / kPieces;
  const int piece = threadIdx.x % kPieces, row = threadIdx.x / kPieces;
  auto address = [&](const int32_t *table, int key) {
    return (static_cast<size_t>(table[key / kPageSize]) * p.num_kv_heads + kvh) * kPageSize * kPieces +
           (key % kPageSize) * kPieces + piece;
  };
  for (int base = 0; base < count; base += kRowsAtOnce * kMoveRows) {
    uint4 v[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int r = base + u * kRowsAtOnce + row;
      if (r < count) v[u] = cache[address(src_table, kept[r])];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int r = base + u * kRowsAtOnce + row;
      if (r < count) cache[address(dst_table, r)] = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream) {
  const unsigned long long units = static_cast<unsigned long long>(p.batch) * p.num_kv_heads;
  if (units == 0) return cudaSuccess;
  if (3 * units > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  const cudaError_t err = launch_kernel(evict_select_kernel, static_cast<unsigned>(units),
                                        kSelectThreads, 0, stream, true, p);
  if (err != cudaSuccess) return err;
  return launch_kernel(evict_move_kernel, static_cast<unsigned>(3 * units), kMoveThreads, 0, stream,
                       true, p);
}

}  // namespace sa
