// Eviction from the paged cache by accumulated attention weight: of each
// (request, KV head) the first tokens, the most recent ones and the heaviest
// of the rest stay, `budget` keys in all, in their order; their K and V rows
// and their mass move to the first slots of the request's pages (in place) or
// of other pages.
//
// select: a cluster of CTAs per (request, KV head), each with a contiguous
//   share of the keys, whose weights it keeps in shared memory (what exceeds
//   104 KB is read again, from L2, in each pass).  A radix select over
//   the weights' order-preserving bits (11 + 11 + 10 bits; histograms in shared
//   memory, joined in the first CTA's through distributed shared memory) gives
//   the weight of the last key that stays and how many of its equals stay,
//   lowest index first; ballots and prefix sums over warps and CTAs then place
//   the kept indices in order.  A row is split only while all CTAs are
//   resident at once: its passes are chains of cluster-wide steps, so a second
//   wave of CTAs costs more than longer shares do.
// move: copies rows by that list, whole 128-byte rows.  A row that one CTA
//   selects is moved by it as well, K and V side by side (64 rows of up to 4096
//   keys, 8 heads, cut to 1024: 50 us, 4.8 TB/s, against 60 us with a second
//   kernel); where a cluster shares a row a second kernel, launched under the
//   first one's end, moves K, V and mass in CTAs of their own with 64 KB in
//   flight (8 rows of up to 131072 keys cut to 8192: 91 us, 40% of it the
//   selection's 5 passes over each weight, bound by their instructions).  In
//   place is safe because the r-th kept key has index >= r: a batch of rows is
//   read whole before any of it is written, and a write to slot r can only hit
//   rows of this batch or earlier ones.
// The least it can move: 4 bytes of mass per key, 520 bytes per kept key.

#include "bounded.cuh"
#include "bounded_ptx.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

namespace sa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxSplit = 8;             // CTAs per (request, KV head)
constexpr int kKeysPerCta = 4096;        // keys per CTA at least, where a row has more than one
constexpr int kGroup = 128;              // keys a warp looks at together, four per lane
constexpr int kMaxCached = 1664;         // weights per warp in shared memory: what two CTAs per SM hold
constexpr int kMoveThreads = 1024;
constexpr int kMoveRows = 4;             // rows in flight per thread and batch

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Order-preserving bits of a weight: larger weight, larger number; -0 = +0,
// NaN below everything.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

struct SelectSmem {
  int hist[kBins];
  int warp_sure[kSelectWarps], warp_equal[kSelectWarps];
  int cta_sure[kMaxSplit], cta_equal[kMaxSplit];
  uint32_t prefix;
  int left;
};

// The bin of rank 0's joined histogram that holds the `left`-th largest, and
// what is left to take within it.  Called by the whole CTA.
__device__ void find_bin(SelectSmem &s, int left, int &bin, int &rest) {
  constexpr int kPer = kBins / kSelectThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // thread 0 owns the highest bins
  const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) mine += s.hist[top - k];
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 31) s.warp_sure[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w)
    if (w < warp) upto += s.warp_sure[w];
  int above = upto - mine;
  if (above < left && upto >= left) {                    // exactly one thread
    int b = top;
    while (above + s.hist[b] < left) above += s.hist[b--];
    s.prefix = static_cast<uint32_t>(b);
    s.left = left - above;
  }
  __syncthreads();
  bin = static_cast<int>(s.prefix);
  rest = s.left;
}

// The mass of one (request, KV head), by a whole CTA.
template <int kThreads>
__device__ __forceinline__ void move_mass(const EvictParams &p, int unit, int count) {
  const int tid = static_cast<int>(threadIdx.x);
  const int *kept = p.kept + static_cast<size_t>(unit) * p.budget;
  const float *src = p.mass + static_cast<size_t>(unit) * p.mass_stride;
  float *dst = p.dst_mass + static_cast<size_t>(unit) * p.dst_mass_stride;
  for (int base = 0; base < count; base += kThreads * kMoveRows) {
    float v[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int r = base + u * kThreads + tid;
      if (r < count) v[u] = src[kept[r]];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int r = base + u * kThreads + tid;
      if (r < count) dst[r] = v[u];
    }
  }
  __syncthreads();
  // evicted places start again from nothing
  const int n = p.kv_lens[unit / p.num_kv_heads];
  for (int i = count + tid; i < min(n, p.dst_mass_stride); i += kThreads) dst[i] = 0.f;
}

// The K rows, V rows or both (kPools 2) of one (request, KV head), by a whole
// CTA: K and V rows lie at the same place of their pools.
template <int kThreads, int kPools, int kRows>      // kRows: of each pool in flight per thread
__device__ __forceinline__ void move_rows(const EvictParams &p, int unit, int count, uint16_t *first) {
  const int tid = static_cast<int>(threadIdx.x);
  const int kvh = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
  const int *kept = p.kept + static_cast<size_t>(unit) * p.budget;
  uint4 *pool[2] = {reinterpret_cast<uint4 *>(first), reinterpret_cast<uint4 *>(p.v_cache)};
  const int32_t *src_table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
  const int32_t *dst_table = p.dst_page_table + static_cast<size_t>(b) * p.dst_max_pages;
  const bool in_place = src_table == dst_table;
  constexpr int kPieces = kHeadDim * 2 / 16;              // 16-byte pieces of a row
  constexpr int kAtOnce = kThreads / kPieces, kBatch = kAtOnce * kRows;
  const int row = tid / kPieces, piece = tid % kPieces;
  auto address = [&](const int32_t *table, int key) {
    return (static_cast<size_t>(table[key / kPageSize]) * p.num_kv_heads + kvh) * (kPageSize * kPieces) +
           (key % kPageSize) * kPieces + piece;
  };
  // the indices of a batch are read while the one before is on its way
  int from[kRows];
  auto look_up = [&](int base) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = base + u * kAtOnce + row;
      from[u] = r < count ? kept[r] : -1;
      if (in_place && from[u] == r) from[u] = -1;         // where it belongs already
    }
  };
  look_up(0);
  for (int base = 0; base < count; base += kBatch) {
    uint4 v[kPools][kRows];
    bool moves[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      moves[u] = from[u] >= 0;
      if (!moves[u]) continue;
      const size_t at = address(src_table, from[u]);
#pragma unroll
      for (int q = 0; q < kPools; ++q) v[q][u] = pool[q][at];
    }
    look_up(base + kBatch);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (!moves[u]) continue;
      const size_t at = address(dst_table, base + u * kAtOnce + row);
#pragma unroll
      for (int q = 0; q < kPools; ++q) pool[q][at] = v[q][u];
    }
  }
}

// Sum of a number over the lanes before this one, as ballots of its four bits.
struct Four {
  unsigned b[4];
  __device__ __forceinline__ explicit Four(const bool (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = __ballot_sync(0xffffffffu, v[q]);
  }
  __device__ __forceinline__ int before(unsigned below) const {
    return __popc(b[0] & below) + __popc(b[1] & below) + __popc(b[2] & below) + __popc(b[3] & below);
  }
  __device__ __forceinline__ int total() const {
    return __popc(b[0]) + __popc(b[1]) + __popc(b[2]) + __popc(b[3]);
  }
};

// What a CTA of the first kernel does with its list where it has the row to
// itself.
__device__ __forceinline__ void move_all(const EvictParams &p, int unit, int count) {
  __syncthreads();                                        // the kept indices are written
  move_rows<kSelectThreads, 2, 2>(p, unit, count, p.k_cache);
  move_mass<kSelectThreads>(p, unit, count);
}

template <bool kMoves>        // the row is this CTA's alone: it moves what it keeps, too
__global__ void __launch_bounds__(kSelectThreads, 3)
evict_select_kernel(const EvictParams p) {
  __shared__ SelectSmem s;
  extern __shared__ uint4 kept_bits[];                    // [warps][p.cached / 4]
  cg::cluster_group cluster = cg::this_cluster();
  const int split = p.split;
  const int rank = static_cast<int>(blockIdx.x % split), unit = static_cast<int>(blockIdx.x / split);
  const int kvh = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  const int n = p.kv_lens[b];
  int *kept = p.kept + static_cast<size_t>(unit) * p.budget;
  const int npages = cdiv(min(max(n, 0), p.max_kv_len), kPageSize);
  const int count = min(n, p.budget);
  const int dst_pages = cdiv(max(count, 0), kPageSize);
  bool bad = n < 0 || n > p.max_kv_len || n > p.mass_stride || count > p.dst_mass_stride ||
             npages > p.max_pages_per_seq || dst_pages > p.dst_max_pages;
  if (!bad) {
    const int32_t *src = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
    const int32_t *dst = p.dst_page_table + static_cast<size_t>(b) * p.dst_max_pages;
    // (bitwise, so that the loads do not wait for one another)
#pragma unroll 8
    for (int i = tid; i < npages; i += kSelectThreads) bad |= (src[i] < 0) | (src[i] >= p.num_pages);
#pragma unroll 4
    for (int i = tid; i < dst_pages; i += kSelectThreads) bad |= (dst[i] < 0) | (dst[i] >= p.num_pages);
  }
  bad = __syncthreads_or(bad);                           // the same in every CTA of the cluster
  if (tid == 0 && rank == 0 && kvh == 0) p.new_kv_lens[b] = bad ? -1 : count;
  const int step = split * kSelectThreads;
  // (64 bits, as a budget may be the largest int; nvcc does not unroll the loop over
  // an unsigned index, which cost 5% of the call for 64 rows)
  for (long long i = (bad ? 0 : count) + rank * kSelectThreads + tid; i < p.budget; i += step) kept[i] = -1;
  if (bad) return;
  if (n <= p.budget) {
    for (int i = rank * kSelectThreads + tid; i < n; i += step) kept[i] = i;
    if (kMoves) move_all(p, unit, count);
    return;
  }

  const float *mass = p.mass + static_cast<size_t>(unit) * p.mass_stride;
  const int lo = p.first_tokens, hi = n - p.recent;       // the keys that compete
  const int want = p.budget - p.first_tokens - p.recent;  // how many of them stay
  // This warp's keys: a contiguous run, whole multiples of kGroup, of which a
  // lane takes four neighbours at a time.  Order bits of the first p.cached of
  // them are kept, the others come from global memory in every pass.
  const int run = cdiv(cdiv(n, split * kSelectWarps), kGroup) * kGroup;
  const long long from = static_cast<long long>(rank * kSelectWarps + warp) * run;
  const int begin = static_cast<int>(min(static_cast<long long>(n), from));
  const int end = static_cast<int>(min(static_cast<long long>(n), from + run));
  uint4 *cache = kept_bits + warp * (p.cached / 4);
  const int cached_end = min(begin + min(run, p.cached), cdiv(end - begin, kGroup) * kGroup + begin);
  constexpr int kUnroll = 8;
  for (int i0 = begin; i0 < cached_end; i0 += 32 * kUnroll) {
    float v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + 32 * u + lane;
      v[u] = i < end ? mass[i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i < cached_end) reinterpret_cast<uint32_t *>(cache)[i - begin] = order_bits(v[u]);
    }
  }
  __syncwarp();
  // f(key, order bits of key .. key + 3, whether all 128 keys of the warp
  // compete); keys >= end do not exist
  auto each = [&](auto f) {
    auto plain = [&](int i0) { return i0 >= lo && i0 + kGroup <= min(hi, end); };
#pragma unroll 2
    for (int i0 = begin; i0 < cached_end; i0 += kGroup) {
      const uint4 w = cache[(i0 - begin) / 4 + lane];
      const uint32_t four[4] = {w.x, w.y, w.z, w.w};
      f(i0 + 4 * lane, four, plain(i0));
    }
    for (int i0 = cached_end; i0 < end; i0 += kGroup) {
      uint32_t four[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) four[q] = i0 + 4 * lane + q < end ? order_bits(mass[i0 + 4 * lane + q]) : 0u;
      f(i0 + 4 * lane, four, plain(i0));
    }
  };

  // ---- the want-th largest weight, from the top bits down
  uint32_t prefix = 0;
  int left = want;                                        // to take among those with the prefix
  if (want > 0) {
    uint32_t known = 0;                                   // bits of the prefix found so far
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kSelectThreads) s.hist[i] = 0;
      cluster.sync();
      each([&](int i, const uint32_t (&w)[4], bool plain) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if ((w[q] & known) == prefix && (plain || (i + q >= lo && i + q < min(hi, end))))
            atomicAdd(&s.hist[(w[q] >> shift) & digits], 1);
      });
      if (split > 1) {
        __syncthreads();
        if (rank != 0) {
          int *joined = cluster.map_shared_rank(s.hist, 0);
          for (int i = tid; i < kBins; i += kSelectThreads) {
            const int mine = s.hist[i];
            if (mine) atomicAdd(joined + i, mine);
          }
        }
        cluster.sync();
        if (rank == 0) {
          int bin, rest;
          find_bin(s, left, bin, rest);
          if (tid < split) {
            SelectSmem *peer = cluster.map_shared_rank(&s, tid);
            peer->prefix = static_cast<uint32_t>(bin);
            peer->left = rest;
          }
        }
        cluster.sync();
        prefix |= s.prefix << shift;
        left = s.left;
      } else {
        __syncthreads();
        int bin, rest;
        find_bin(s, left, bin, rest);
        prefix |= static_cast<uint32_t>(bin) << shift;
        left = rest;
      }
      known |= digits << shift;
      __syncthreads();                                    // prefix and hist are read
    }
  }

  // ---- how many stay for sure, and how many equal the threshold, per warp
  // and CTA
  auto kind = [&](int i, uint32_t w, bool &sure, bool &equal) {
    const bool competes = i >= lo && i < hi;
    sure = i < end && (!competes || (want > 0 && w > prefix));
    equal = i < end && competes && want > 0 && w == prefix;
  };
  int n_sure = 0, n_equal = 0;
  each([&](int i, const uint32_t (&w)[4], bool plain) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bool sure = w[q] > prefix, equal = w[q] == prefix;
      if (!plain || want == 0) kind(i + q, w[q], sure, equal);
      n_sure += sure;
      n_equal += equal;
    }
  });
  n_sure = warp_sum(n_sure);
  n_equal = warp_sum(n_equal);
  if (lane == 0) {
    s.warp_sure[warp] = n_sure;
    s.warp_equal[warp] = n_equal;
  }
  __syncthreads();
  int cta_sure = 0, cta_equal = 0, sure_before = 0, equal_before = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    if (w == warp) {
      sure_before = cta_sure;
      equal_before = cta_equal;
    }
    cta_sure += s.warp_sure[w];
    cta_equal += s.warp_equal[w];
  }
  if (split > 1) {
    if (want == 0) cluster.sync();                        // (no pass has met the peers: they may not run yet)
    if (tid < split) {
      SelectSmem *peer = cluster.map_shared_rank(&s, tid);
      peer->cta_sure[rank] = cta_sure;
      peer->cta_equal[rank] = cta_equal;
    }
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      sure_before += s.cta_sure[r];
      equal_before += s.cta_equal[r];
    }
  }

  // ---- the kept indices, in order
  int at = sure_before + min(equal_before, left);         // kept before this warp's keys
  const unsigned below = (1u << lane) - 1u;
  each([&](int i, const uint32_t (&w)[4], bool plain) {
    bool keep[4], equal[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      keep[q] = w[q] > prefix;
      equal[q] = w[q] == prefix;
      if (!plain || want == 0) kind(i + q, w[q], keep[q], equal[q]);
    }
    if (n_equal) {                                        // warp-uniform: ties to number
      const Four eq(equal);
      int e = equal_before + eq.before(below);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (equal[q]) keep[q] = e++ < left;
      equal_before += eq.total();
    }
    const Four all(keep);
    int r = at + all.before(below);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (keep[q]) kept[r++] = i + q;
    at += all.total();
  });
  if (kMoves) move_all(p, unit, count);
  if (split > 1) cluster.sync();                          // peers have written this CTA's counts
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
evict_move_kernel(const EvictParams p) {
  const int units = p.batch * p.num_kv_heads;
  const int role = static_cast<int>(blockIdx.x) / units, unit = static_cast<int>(blockIdx.x) % units;
  grid_dependency_wait();
  const int count = p.new_kv_lens[unit / p.num_kv_heads];
  if (count < 0) return;
  if (role == 2) move_mass<kThreads>(p, unit, count);
  else move_rows<kThreads, 1, kMoveRows>(p, unit, count, role == 0 ? p.k_cache : p.v_cache);
}

}  // namespace

cudaError_t launch_evict(EvictParams &p, int num_sms, cudaStream_t stream) {
  const unsigned long long units = static_cast<unsigned long long>(p.batch) * p.num_kv_heads;
  if (units == 0) return cudaSuccess;
  // CTAs per row: as many as are resident at once (two per SM with 104 KB of
  // weights each), of kKeysPerCta keys at least
  p.split = 1;
  while (p.split < kMaxSplit && p.max_kv_len > kKeysPerCta * p.split &&
         units * 2 * p.split <= 2ull * num_sms)
    p.split *= 2;
  if (3 * units > 0x7fffffffull || p.split * units > 0x7fffffffull)
    return cudaErrorInvalidConfiguration;
  // every weight of a CTA's share where 104 KB hold them
  const long long share = cdiv(p.max_kv_len, p.split * kSelectWarps);
  p.cached = static_cast<int>(std::min<long long>((share + kGroup - 1) / kGroup * kGroup, kMaxCached));
  if (p.split == 1) {
    const cudaError_t err = set_smem_once<evict_select_kernel<true>>(kSelectWarps * kMaxCached * 4);
    if (err != cudaSuccess) return err;
    return launch_clusters(evict_select_kernel<true>, static_cast<unsigned>(units), 1, kSelectThreads,
                           kSelectWarps * p.cached * 4, stream, true, p);
  }
  cudaError_t err = set_smem_once<evict_select_kernel<false>>(kSelectWarps * kMaxCached * 4);
  if (err != cudaSuccess) return err;
  err = launch_clusters(evict_select_kernel<false>, static_cast<unsigned>(p.split * units),
                        static_cast<unsigned>(p.split), kSelectThreads,
                        kSelectWarps * p.cached * 4, stream, true, p);
  if (err != cudaSuccess) return err;
  return launch_kernel(evict_move_kernel<kMoveThreads>, static_cast<unsigned>(3 * units),
                       kMoveThreads, 0, stream, true, p);
}

}  // namespace sa
