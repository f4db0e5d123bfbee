// Attention weight drawn by each cached key ("mass"):
//
//   mass[b][g][j] += sum over the call's rows (token i, head h of KV head g)
//                    that see key j of e^(scale q_ih . k_gj - lse_ih),
//
// the column sums of the attention's own weights: lse is what decode /
// prefill returned for the row, so one pass over K suffices and no softmax
// state is carried.  Exponents, weights and sums are fp32.  Every sum has a
// fixed order (one addition to memory per entry), so equal inputs give equal bits.
//
// decode_mass (one token per request) reads 128 bytes of K per (key, KV head)
// and is bound by HBM.  Each warp takes whole 16-key pages: S^T[16 keys x 8
// heads] = K Q^T by mma.sync.m16n8k16, K straight from global memory into the
// A fragments.  A dot product does not care about the order of its terms, so
// the k index of the MMA is permuted to make each lane's share of a K row two
// 16-byte pieces: no shared memory and no copies to wait for; many resident
// warps with one page each in flight hide the latency better than few warps
// with several (a page's 16 registers per lane cost occupancy, and the loads
// of several pages wait for one another).
//
// prefill_mass (ragged rows at the end of the keys) is bound by its
// exponentials, one per (row, key).  A CTA holds 256 keys of one KV head and
// streams the query rows that see them past the resident K, 128 (token, head)
// rows at a time: S^T[128 keys x 128 rows] by tcgen05 into tensor memory for
// each of two groups of four warps, in which one thread per key adds its row
// of weights in registers -- no sums across threads.  A group has two score
// buffers of 64 columns, so the next scores are made while these are summed, and
// an issuing thread of its own.  With many query tiles a cluster of CTAs shares
// the rows of a key pair and its mirror image, joined in rank order through
// distributed shared memory; with few, each CTA takes an equal share of all key
// pairs, whose K tiles stream as well.
//
// Measured (64 / 8 heads): decode_mass 24 us for 64 requests of up to 4096 keys
// and 106 us for 8 of up to 131072 (6.4 and 6.5 TB/s).  prefill_mass 218 us for 4
// whole prompts of up to 4096 tokens, 80 us for the last 32 tokens of 8 prompts
// of up to 32k: the exponential unit is busy 58% of the time and no single part
// binds (without exponentials 172 us, without reading lse 205, with a quarter of
// the product 203, without all three 126).  Tried: 16 columns at a time with the
// next ones on their way (225 us), 64 at once (285, spills), both key tiles of a
// pair by each thread, lse read once for both (239).

#include "bounded.cuh"
#include "bounded_ptx.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sa {
namespace {

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ bool bad_request(const MassParams &p, int kv_len) {
  return kv_len < 0 || kv_len > p.max_kv_len || kv_len > p.mass_stride ||
         cdiv(kv_len, kPageSize) > p.max_pages_per_seq;
}

// NaN over the whole mass row of a request whose arguments are out of range.
__device__ __forceinline__ void poison_row(const MassParams &p, float *row) {
  for (unsigned j = threadIdx.x; j < static_cast<unsigned>(p.mass_stride); j += blockDim.x) row[j] = NAN;
}

// ------------------------------------------------------------------ decode
constexpr int kDecodeWarps = 8;
constexpr int kDecodeCtas = 4;                   // per SM
constexpr int kPieces = kHeadDim * 2 / 16;       // 16-byte pieces of a row

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Columns 8 nb .. 8 nb + 7 of the query heads: Q as B fragments (column g holds
// pieces t and t + 4 of its head, the k order of K's pieces) and -lse in base 2
// of columns 2t, 2t + 1; -inf marks one that adds nothing, whatever its score (for
// columns past the heads 0 * inf, where a key is infinite).
struct HeadBlock {
  uint4 q0, q1;
  float nl0, nl1;
  __device__ __forceinline__ void load(const MassParams &p, size_t row0, int nb, int g, int t) {
    const int col = nb * 8 + g;
    const uint4 *q = reinterpret_cast<const uint4 *>(p.q) + (row0 + col) * kPieces;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    q0 = col < p.group ? __ldg(q + t) : zero;
    q1 = col < p.group ? __ldg(q + t + 4) : zero;
    auto neg = [&](int c) {
      const float l = c < p.group ? __ldg(p.lse + row0 + c) : -INFINITY;
      return l == INFINITY ? -FLT_MAX : l == -INFINITY ? -INFINITY : -l * kLog2e;
    };
    nl0 = neg(nb * 8 + 2 * t);
    nl1 = neg(nb * 8 + 2 * t + 1);
  }
};

template <bool kOneBlock>             // at most 8 query heads per KV head
__global__ void __launch_bounds__(kDecodeWarps * 32, kOneBlock ? kDecodeCtas : 3)
decode_mass_kernel(const MassParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int chunk = static_cast<int>(blockIdx.x % p.num_chunks);
  const int unit = static_cast<int>(blockIdx.x / p.num_chunks);
  const int kvh = unit % p.num_kv_heads, b = unit / p.num_kv_heads;
  grid_dependency_wait();
  const int kv_len = p.kv_lens[b];
  float *mass = p.mass + static_cast<size_t>(unit) * p.mass_stride;
  if (bad_request(p, kv_len)) {
    if (chunk == 0) poison_row(p, mass);
    return;
  }
  const int end = min(cdiv(kv_len, kPageSize), (chunk + 1) * p.pages_per_chunk);
  int page = chunk * p.pages_per_chunk + warp;
  if (page >= end) return;                               // warp-uniform; no barriers below
  const int32_t *table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;
  const size_t row0 = static_cast<size_t>(b) * p.num_qo_heads + kvh * p.group;
  const uint4 *cache = reinterpret_cast<const uint4 *>(p.k_cache) + g * kPieces + t;
  int id = __ldg(table + page);
  HeadBlock q;
  if constexpr (kOneBlock) q.load(p, row0, 0, g, t);
  for (; page < end; page += kDecodeWarps) {
    const int next = page + kDecodeWarps < end ? __ldg(table + page + kDecodeWarps) : 0;
    const bool bad = id < 0 || id >= p.num_pages;        // never dereferenced
    const uint4 *k =
        cache + (static_cast<size_t>(bad ? 0 : id) * p.num_kv_heads + kvh) * (kPageSize * kPieces);
    // A fragments: key rows g and g + 8, pieces t and t + 4
    const uint4 lo0 = ld_stream(k), lo1 = ld_stream(k + 4);
    const uint4 hi0 = ld_stream(k + 8 * kPieces), hi1 = ld_stream(k + 8 * kPieces + 4);
    // lane 0 of a quad adds to key g of the page, lane 1 to key g + 8
    const int key = page * kPageSize + g + (t == 1 ? 8 : 0);
    const bool writes = t < 2 && key < kv_len;
    const float before = writes ? mass[key] : 0.f;
    float w_lo = 0.f, w_hi = 0.f;
    auto add = [&]() {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t a0[4] = {lo0.x, hi0.x, lo0.y, hi0.y}, a1[4] = {lo0.z, hi0.z, lo0.w, hi0.w};
      const uint32_t a2[4] = {lo1.x, hi1.x, lo1.y, hi1.y}, a3[4] = {lo1.z, hi1.z, lo1.w, hi1.w};
      mma_bf16_16816(s, a0, q.q0.x, q.q0.y);
      mma_bf16_16816(s, a1, q.q0.z, q.q0.w);
      mma_bf16_16816(s, a2, q.q1.x, q.q1.y);
      mma_bf16_16816(s, a3, q.q1.z, q.q1.w);
      auto weight = [&](float score, float nl) {
        return nl == -INFINITY ? 0.f : ex2(fmaf(score, p.scale_log2, nl));
      };
      w_lo += weight(s[0], q.nl0) + weight(s[1], q.nl1);
      w_hi += weight(s[2], q.nl0) + weight(s[3], q.nl1);
    };
    if constexpr (kOneBlock) {
      add();
    } else {
      for (int nb = 0; nb < cdiv(p.group, 8); ++nb) {
        q.load(p, row0, nb, g, t);
        add();
      }
    }
    // sums over the quad; lanes 0 and 1 end up with keys g and g + 8
    w_lo += __shfl_xor_sync(0xffffffffu, w_lo, 1);
    w_hi += __shfl_xor_sync(0xffffffffu, w_hi, 1);
    float w = (t & 1) ? w_hi : w_lo;
    w += __shfl_xor_sync(0xffffffffu, w, 2);
    if (writes) mass[key] = bad ? NAN : before + w;
    id = next;
  }
}

// ----------------------------------------------------------------- prefill
constexpr int kKeys = 128;                       // keys per tile: rows of S^T
constexpr int kRows = 128;                       // query rows per streamed tile: columns of S^T
constexpr int kKStages = 3, kQStages = 3;
constexpr int kMaxSplit = 8;                     // CTAs per cluster (the portable limit)
constexpr int kTileBytes = 128 * kHeadDim * 2;
constexpr int kGroups = 2;                       // groups of four warps, one key tile each
constexpr int kLoadWarp = 4 * kGroups, kMmaWarp = kLoadWarp + 1;   // one issuing warp per group
constexpr int kThreads = (kMmaWarp + kGroups) * 32;
constexpr int kHalf = kRows / 2;                 // columns per score buffer: one is read, one filled
constexpr uint32_t kTmemCols = 2 * kHalf * kGroups;

constexpr int kOffK = 0;
constexpr int kOffQ = kOffK + kKStages * kTileBytes;
constexpr int kOffL = kOffQ + kQStages * kTileBytes;
constexpr int kOffSum = kOffL + kQStages * kRows * 4;
constexpr int kOffBars = kOffSum + 2 * kGroups * kKeys * 4;
constexpr int kSmemBytes = kOffBars + 256 + 1024;
static_assert(kSmemBytes <= 113 * 1024, "two CTAs per SM");

struct Bars {
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t q_full[kQStages], q_empty[kQStages];  // Q and -lse of a tile
  uint64_t s_full[kGroups][2], s_free[kGroups][2];
  uint32_t tmem_base;
  int bad_wait;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

constexpr uint32_t kIdesc = umma_idesc_bf16(128, kHalf, false, false);

// Bits below n (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Sum over 32 columns of 2^(s * scale + nl), s in r, nl in shared memory; on an
// edge over those with a bit in `see`.  Hidden columns are left out behind the
// exponent, not in the score: a row whose lse is NaN would be so in its exponent all
// the same, and spoil keys that it does not see.
template <bool kEdge, int E = 0>
__device__ __forceinline__ void add_chunk(uint32_t (&r)[32], const float4 *nl, uint64_t scale2,
                                          uint32_t see, uint64_t &acc0, uint64_t &acc1) {
  if constexpr (E < 8) {
    const float4 l = nl[E];
    float x0, x1, x2, x3;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[4 * E]), __uint_as_float(r[4 * E + 1])), scale2,
                     f2_pack(l.x, l.y)), x0, x1);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[4 * E + 2]), __uint_as_float(r[4 * E + 3])), scale2,
                     f2_pack(l.z, l.w)), x2, x3);
    if constexpr (kEdge) {
      x0 = (see >> (4 * E)) & 1u ? x0 : -INFINITY;
      x1 = (see >> (4 * E + 1)) & 1u ? x1 : -INFINITY;
      x2 = (see >> (4 * E + 2)) & 1u ? x2 : -INFINITY;
      x3 = (see >> (4 * E + 3)) & 1u ? x3 : -INFINITY;
    }
    acc0 = f2_add(acc0, f2_pack(ex2(x0), ex2(x1)));
    acc1 = f2_add(acc1, f2_pack(ex2(x2), ex2(x3)));
    add_chunk<kEdge, E + 1>(r, nl, scale2, see, acc0, acc1);
  }
}

// The query tiles that a CTA of a cluster takes of one key pair (256 keys, one
// tile of 128 per group of warps): of those with a row that sees the pair,
// every split-th.
struct Steps {
  int key0, i_start, n;               // first key, first token that sees one of the keys, tiles
  int skip[kGroups];                  // first tile that the group takes part in (n: none)
};

// What a CTA works on: key pairs of (request, KV head) units.  Every role walks
// the same sequence.
//   mirror      : pair c of the unit and its mirror image n - 1 - c, which
//                 together are seen by about as many rows whatever c is; the
//                 CTAs of a cluster share the rows.  For many rows per key.
//   not mirror  : an equal share of all pairs of the launch, in order.  For few.
struct Walk {
  int seq, kvh, kp, pairs;            // current pair, pairs of its request
  int left;                           // pairs to go, this one included
  int q_start, q_len, kv_len, shift;  // shift: position of the first row's token
  int tiles;                          // this CTA's query tiles of a pair that every row sees

  // How many of `n` tiles (this rank's, then every split-th) are this CTA's.
  __device__ __forceinline__ static int share(const MassParams &p, int n) {
    const int rank = static_cast<int>(blockIdx.x) & (p.split - 1);    // split: a power of two
    return n > rank ? (n - rank + p.split - 1) >> p.split_log2 : 0;
  }
  // Loads request `seq`; pairs = 0 if there is nothing to add.  True if its
  // arguments are out of range.
  __device__ __forceinline__ bool request(const MassParams &p, int r) {
    seq = r;
    q_start = p.cu_seqlens_q[r];
    const int q_end = p.cu_seqlens_q[r + 1];
    q_len = q_end - q_start;
    kv_len = p.kv_lens[r];
    shift = kv_len - q_len;
    const bool bad = bad_request(p, kv_len) || q_start < 0 || q_len < 0 || q_end > p.total_q ||
                     q_len > p.max_q_len || kv_len < q_len;
    pairs = bad || q_len == 0 ? 0 : cdiv(kv_len, kKeys * kGroups);
    tiles = share(p, cdiv(q_len, p.tile_tokens));
    return bad;
  }
  // Called by whole warps.
  __device__ void begin(const MassParams &p) {
    if (p.mirror) {
      // heaviest requests first (as many as a warp can rank; the others after
      // them in order), so that the last wave holds the light ones
      const int item = static_cast<int>(blockIdx.x) >> p.split_log2;
      const int per_seq = (cdiv(p.max_kv_len, kKeys * kGroups) + 1) / 2 * p.num_kv_heads;
      const int place = item / per_seq, rest = item % per_seq;
      kvh = rest % p.num_kv_heads;
      kp = rest / p.num_kv_heads;
      int r = place;
      if (place < 32) {
        const int lane = threadIdx.x & 31;
        float weight = -1.f;                             // no request: after all that exist
        if (lane < p.num_seqs)
          weight = static_cast<float>(max(0, p.cu_seqlens_q[lane + 1] - p.cu_seqlens_q[lane])) *
                   static_cast<float>(max(0, p.kv_lens[lane]));
        int rank = 0;
#pragma unroll
        for (int l = 0; l < 32; ++l) {
          const float other = __shfl_sync(0xffffffffu, weight, l);
          rank += other > weight || (other == weight && l < lane);
        }
        r = __ffs(__ballot_sync(0xffffffffu, rank == place)) - 1;
      }
      request(p, r);
      left = kp >= (pairs + 1) / 2 ? 0 : kp == pairs - 1 - kp ? 1 : 2;
      return;
    }
    // pairs before each request, 32 requests at a time: first their number,
    // then where this CTA's share begins
    const int lane = threadIdx.x & 31;
    long long total = 0, first = 0;
    for (int pass = 0; pass < 2; ++pass) {
      long long before = 0;
      for (int r0 = 0; r0 < p.num_seqs; r0 += 32) {
        pairs = 0;
        if (r0 + lane < p.num_seqs) request(p, r0 + lane);
        long long upto = static_cast<long long>(pairs) * p.num_kv_heads;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        const unsigned reach = __ballot_sync(0xffffffffu, pass == 1 && before + upto > first);
        if (reach) {                                     // the request of this CTA's first pair
          const int l = __ffs(reach) - 1;
          const long long at =
              first - before - (l ? __shfl_sync(0xffffffffu, upto, max(l - 1, 0)) : 0);
          request(p, r0 + l);
          kvh = static_cast<int>(at / pairs);
          kp = static_cast<int>(at % pairs);
          return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
      total = before;
      first = total * blockIdx.x / gridDim.x;
      left = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x - first);
      if (left == 0) return;
    }
  }
  // The next pair, by a whole warp, for a walk in shared memory: lanes read it
  // while others may be ahead, so one of them moves it, between two barriers.
  __device__ __forceinline__ void next_of_warp(const MassParams &p) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) next(p);
    __syncwarp();
  }
  __device__ __forceinline__ void next(const MassParams &p) {
    if (--left == 0) return;
    if (p.mirror) {
      kp = pairs - 1 - kp;
    } else if (++kp == pairs) {
      kp = 0;
      if (++kvh == p.num_kv_heads) {
        kvh = 0;
        do request(p, seq + 1);
        while (pairs == 0);
      }
    }
  }
  __device__ __forceinline__ Steps steps(const MassParams &p) const {
    Steps s;
    const int rank = static_cast<int>(blockIdx.x) & (p.split - 1);
    s.key0 = kp * kKeys * kGroups;
    const int key1 = s.key0 + kKeys;
    if (key1 + kKeys <= shift) {                         // every row sees every key
      s.i_start = 0;
      s.n = tiles;
      s.skip[0] = s.skip[1] = 0;
    } else {
      s.i_start = max(0, s.key0 - shift);
      s.n = share(p, cdiv(q_len - s.i_start, p.tile_tokens));
      // the second tile's first row is some tiles further on
      s.skip[0] = 0;
      s.skip[1] = key1 >= kv_len
                      ? s.n
                      : min(s.n, share(p, (max(0, key1 - shift) - s.i_start) / p.tile_tokens));
    }
    s.i_start += rank * p.tile_tokens;                   // of this CTA's first tile
    return s;
  }
  __device__ __forceinline__ float *row(const MassParams &p) const {
    return p.mass + (static_cast<size_t>(seq) * p.num_kv_heads + kvh) * p.mass_stride;
  }
};

__global__ void __launch_bounds__(kThreads, 2)
prefill_mass_kernel(const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap, const MassParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // in shared memory, a copy per warp: it is looked at between key pairs, and
  // registers are what the loops run out of
  __shared__ Walk walks[kThreads / 32];
  Walk &walk = walks[warp];
  {
    Walk first;
    first.begin(p);
    if (lane == 0) walk = first;
    __syncwarp();
  }
  const int step_tokens = p.split * p.tile_tokens;       // from one tile of this CTA to its next
  // requests whose arguments are out of range: NaN over their mass rows
  for (int r = static_cast<int>(blockIdx.x); r < p.num_seqs; r += static_cast<int>(gridDim.x)) {
    Walk bad;
    if (bad.request(p, r))
      for (int h = 0; h < p.num_kv_heads; ++h)
        poison_row(p, p.mass + (static_cast<size_t>(r) * p.num_kv_heads + h) * p.mass_stride);
  }
  if (walk.left == 0) return;                            // the whole cluster returns

  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: accesses stay known to be shared memory's)
  uint8_t *smem = smem_raw + (0u - smem_u32(smem_raw)) % 1024;
  Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
  auto sK = [&](int s) { return smem + kOffK + s * kTileBytes; };
  auto sQ = [&](int s) { return smem + kOffQ + s * kTileBytes; };
  auto sL = [&](int s) { return reinterpret_cast<float *>(smem + kOffL) + s * kRows; };
  float *sums = reinterpret_cast<float *>(smem + kOffSum);

  if (warp == kMmaWarp) {
    tmem_alloc(&bar.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
    }
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(&bar.q_full[s], 1 + 32);                 // the copy, and the lanes that write -lse
      mbar_init(&bar.q_empty[s], kGroups + 128 * kGroups);   // the MMAs, and the readers of -lse
    }
    for (int w = 0; w < kGroups; ++w) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bar.s_full[w][h], 1);
        mbar_init(&bar.s_free[w][h], 128);
      }
    }
    bar.bad_wait = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp == kLoadWarp) {
    // ---------------------------------------- key tiles, query tiles and -lse
    bool ok = true;
    int kn = 0, qn = 0;                                  // tiles loaded so far
    // this lane's rows of a query tile, and their lse (read a step ahead:
    // the copies are asynchronous, so these loads are the latency that counts)
    constexpr int kMine = kRows / 32;
    int in_tile[kMine], row_at[kMine];
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int r = lane + 32 * u, tk = r / p.group;
      in_tile[u] = r;
      row_at[u] = tk * p.num_qo_heads + (r - tk * p.group);
    }
    auto load_lse = [&](const Steps &st, int step, float (&l)[kMine]) {
      if (step >= st.n) return;
      const int tok = st.i_start + step * step_tokens;
      const int rows = min(p.tile_tokens, walk.q_len - tok) * p.group;
      const float *from = p.lse + static_cast<size_t>(walk.q_start + tok) * p.num_qo_heads +
                          walk.kvh * p.group;
#pragma unroll
      for (int u = 0; u < kMine; ++u)                    // columns past the rows add nothing
        l[u] = in_tile[u] < rows ? __ldg(from + row_at[u]) : INFINITY;
    };
    for (; ok && walk.left > 0; walk.next_of_warp(p)) {
      const Steps st = walk.steps(p);
      float lse[1][kMine];
      load_lse(st, 0, lse[0]);
      for (int j = 0; ok && j < st.n; ++j, ++qn) {
        for (int w = 0; w < kGroups; ++w) {
          if (j != 0 || st.skip[w] >= st.n) continue;
          // lanes 0..7 each own one 16-key page of the tile
          const int s = kn % kKStages;
          const int pg = (st.key0 + w * kKeys) / kPageSize + lane;
          int id = -1;
          bool bad = false;
          if (lane < kKeys / kPageSize && pg < cdiv(walk.kv_len, kPageSize)) {
            id = p.page_table[static_cast<size_t>(walk.seq) * p.max_pages_per_seq + pg];
            bad = id < 0 || id >= p.num_pages;
          }
          if (kn >= kKStages && !__all_sync(0xffffffffu, mbar_wait(&bar.k_empty[s], ((kn / kKStages) + 1) & 1))) {
            ok = false;
            break;
          }
          // a page outside the pool is never read: its keys are NaN, and so
          // become their scores and sums
          for (unsigned m = __ballot_sync(0xffffffffu, bad); m; m &= m - 1) {
            uint4 *to = reinterpret_cast<uint4 *>(sK(s) + (__ffs(m) - 1) * kPageSize * kHeadDim * 2);
            for (int i = lane; i < kPageSize * kPieces; i += 32)
              to[i] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          const unsigned mask = __ballot_sync(0xffffffffu, id >= 0 && !bad);
          if (lane == 0)
            mbar_arrive_expect_tx(&bar.k_full[s], __popc(mask) * kPageSize * kHeadDim * 2);
          __syncwarp();
          if (id >= 0 && !bad)
            tma_load_3d(sK(s) + lane * kPageSize * kHeadDim * 2, &kmap, &bar.k_full[s], 0,
                        walk.kvh * kPageSize, id);
          __syncwarp();
          ++kn;
        }
        const int s = qn % kQStages;
        if (ok && qn >= kQStages && !__all_sync(0xffffffffu, mbar_wait(&bar.q_empty[s], ((qn / kQStages) + 1) & 1)))
          ok = false;
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.q_full[s], p.tile_tokens * p.group * kHeadDim * 2);
          tma_load_3d(sQ(s), &qmap, &bar.q_full[s], 0, walk.kvh * p.group,
                      walk.q_start + st.i_start + j * step_tokens);
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const float l = lse[0][u];
          sL(s)[in_tile[u]] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        }
        load_lse(st, j + 1, lse[0]);
        mbar_arrive(&bar.q_full[s]);
      }
    }
    if (!ok && lane == 0) atomicOr(&bar.bad_wait, 1);
  } else if (warp >= kMmaWarp) {
    // ------------------------------- S^T = K Q^T of one group (one thread).  A
    // thread each: with one for both, each group waited for the other's turn.
    const int w = warp - kMmaWarp;
    bool ok = true;
    int kn = 0, qn = 0, sn = 0;
    for (; ok && walk.left > 0; walk.next_of_warp(p)) {
      const Steps st = walk.steps(p);
      // number of this group's key tile among those loaded
      const int tile = kn + (w == 1 && st.skip[0] < st.n ? 1 : 0);
      kn += (st.skip[0] < st.n ? 1 : 0) + (st.skip[1] < st.n ? 1 : 0);
      const int my_skip = w == 0 ? st.skip[0] : st.skip[1];
      const int k = tile % kKStages;
      const uint64_t dk = umma_desc_sw128(smem_u32(sK(k)), 16, 1024);
      for (int j = 0; ok && j < st.n; ++j, ++qn) {
        const int s = qn % kQStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.q_full[s], (qn / kQStages) & 1));
        if (ok && j == my_skip) ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_full[k], (tile / kKStages) & 1));
        if (j >= my_skip) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && (sn == 0 || __all_sync(0xffffffffu, mbar_wait(&bar.s_free[w][h], (sn - 1) & 1)));
            if (!ok) continue;
            tc_fence_after();
            if (lane == 0) {
              const uint64_t dq = umma_desc_sw128(smem_u32(sQ(s) + h * (kTileBytes / 2)), 16, 1024);
#pragma unroll
              for (int kk = 0; kk < kHeadDim / 16; ++kk)
                umma_ss(tmem + (2 * w + h) * kHalf, dk + 2 * kk, dq + 2 * kk, kIdesc, kk > 0);
              umma_commit(&bar.s_full[w][h]);
            }
            __syncwarp();
          }
          ++sn;
        }
        if (ok && lane == 0) {
          umma_commit(&bar.q_empty[s]);
          if (j == st.n - 1 && my_skip < st.n) umma_commit(&bar.k_empty[k]);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) atomicOr(&bar.bad_wait, 1);
  } else {
    // ------------------------------------------------ one thread per key
    const int w = warp / 4;                              // group
    const uint32_t trow = tmem + 2 * w * kHalf + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int row = threadIdx.x & 127;
    const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
    bool ok = true;
    int qn = 0, sn = 0;
    for (int item = 0; ok && walk.left > 0; ++item, walk.next_of_warp(p)) {
      const Steps st = walk.steps(p);
      const int my_skip = w == 0 ? st.skip[0] : st.skip[kGroups - 1];
      const int key = st.key0 + w * kKeys + row;
      // tokens from this CTA's current tile to the first one that sees the key
      int ahead = key - walk.shift - st.i_start;
      int tokens_left = walk.q_len - st.i_start;
      uint64_t acc0 = 0, acc1 = 0;                       // (+0.f, +0.f)
      for (int j = 0; j < st.n; ++j, ++qn) {
        const int s = qn % kQStages;
        // -lse of the tile (and, for a group that skips it, its turn)
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.q_full[s], (qn / kQStages) & 1))) {
          ok = false;
          break;
        }
        // columns [from, rows) see this key
        const int rows = min(p.tile_tokens, tokens_left) * p.group, from = max(0, ahead) * p.group;
        ahead -= step_tokens;
        tokens_left -= step_tokens;
        if (j < my_skip) {
          mbar_arrive(&bar.q_empty[s]);
          continue;
        }
        const bool edge = __any_sync(0xffffffffu, from > 0 || rows < kRows);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!__all_sync(0xffffffffu, mbar_wait(&bar.s_full[w][h], sn & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld32(trow + h * kHalf + 32 * c, x);
            tmem_ld_wait32(x);
            if (c == 1) {
              tc_fence_before();
              mbar_arrive(&bar.s_free[w][h]);
            }
            const int c0 = h * kHalf + 32 * c;
            const float4 *nl = reinterpret_cast<const float4 *>(sL(s) + c0);
            if (edge) add_chunk<true>(x, nl, scale2, first_bits(rows - c0) & ~first_bits(from - c0), acc0, acc1);
            else add_chunk<false>(x, nl, scale2, 0u, acc0, acc1);
          }
        }
        if (!ok) break;
        ++sn;
        mbar_arrive(&bar.q_empty[s]);
      }
      float a, b, c, d;
      f2_unpack(acc0, a, b);
      f2_unpack(acc1, c, d);
      const float sum = (a + b) + (c + d);
      if (p.mirror) sums[item * kKeys * kGroups + threadIdx.x] = sum;
      else if (row + w * kKeys + walk.kp * kKeys * kGroups < walk.kv_len) {
        // The key's only sum of the launch, so the order of additions is fixed;
        // added in memory, as a value read before the loop cost its latency
        // (2500 of 8300 cycles per pair) where no register was left for it.
        float *to = walk.row(p) + walk.kp * kKeys * kGroups + w * kKeys + row;
        if (ok) atomicAdd(to, sum);
        else *to = NAN;
      }
    }
    if (!ok) {
      // a wait ran out: none of the sums to come can be made
      atomicOr(&bar.bad_wait, 1);
      for (; !p.mirror && walk.left > 0; walk.next_of_warp(p)) {
        const int key = walk.kp * kKeys * kGroups + w * kKeys + row;
        if (key < walk.kv_len) walk.row(p)[key] = NAN;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (p.mirror) {
    // the shares of the cluster's CTAs, in rank order; a wait that ran out
    // gives NaN
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (bar.bad_wait)
      for (int i = threadIdx.x; i < 2 * kKeys * kGroups; i += kThreads) sums[i] = NAN;
    cluster.sync();
    Walk mine;
    mine.begin(p);
    for (int item = 0; mine.left > 0; ++item, mine.next(p)) {
      // rank r writes keys r, r + split, ... of the pair
      for (int i = static_cast<int>(blockIdx.x % p.split) + p.split * static_cast<int>(threadIdx.x);
           i < kKeys * kGroups; i += p.split * kThreads) {
        const int key = mine.kp * kKeys * kGroups + i;
        if (key >= mine.kv_len) continue;
        float total = mine.row(p)[key];
        float part[kMaxSplit];                           // all on their way before the first is added
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
          part[r] = r < p.split ? *cluster.map_shared_rank(sums + item * kKeys * kGroups + i, r) : 0.f;
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) total += part[r];
        mine.row(p)[key] = total;
      }
    }
    cluster.sync();                                      // peers keep their sums until here
  }
}

}  // namespace

cudaError_t launch_decode_mass(const MassParams &p, cudaStream_t stream) {
  const unsigned long long ctas =
      static_cast<unsigned long long>(p.num_seqs) * p.num_kv_heads * p.num_chunks;
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  return launch_kernel(p.group <= 8 ? decode_mass_kernel<true> : decode_mass_kernel<false>,
                       static_cast<unsigned>(ctas), kDecodeWarps * 32, 0, stream, true, p);
}

int decode_mass_warps() { return kDecodeWarps; }

int prefill_mass_pair_keys() { return kKeys * kGroups; }

cudaError_t launch_prefill_mass(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                const MassParams &p, cudaStream_t stream) {
  // a cluster per (unit, pair and its mirror image), or a share of everything
  // for each CTA that the GPU holds (some, even where no key is in bounds: they
  // flag the requests that have any)
  const unsigned long long units = static_cast<unsigned long long>(p.num_seqs) * p.num_kv_heads;
  const unsigned long long pairs = cdiv(p.max_kv_len, kKeys * kGroups);
  const unsigned long long ctas = p.mirror ? units * ((pairs + 1) / 2) * p.split
                                              : std::min<unsigned long long>(units * std::max(pairs, 1ull), 2 * p.num_sms);
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  cudaError_t err = set_smem_once<prefill_mass_kernel>(kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_clusters(prefill_mass_kernel, static_cast<unsigned>(ctas),
                         static_cast<unsigned>(p.split), kThreads, kSmemBytes, stream, false, qmap,
                         kmap, p);
}

}  // namespace sa
