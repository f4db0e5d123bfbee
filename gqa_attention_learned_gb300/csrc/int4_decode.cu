// Attention of few query rows per KV head over a cache held in 4 bits: one token per
// request, the draft tokens of a verification, or the last few of ragged requests.
//
// Mathematics.  Keys are k_j = s_j (n_j - z_j), n_j in 0..15.  A code under the exponent
// of 16 is the bf16 number 16 + n.  K's codes go into the product as that, V's less 16 + z
// (a bf16 subtraction, exact):
//     scale q.k_j   = (scale s_j) (q.(16 + n_j) - (16 + z_j) sum q)
//     sum_j p_j v_j = sum_j (p_j s_j) (n_j - z_j)
// Scales, and zero points of K, so cost a few operations per (key, head) instead of one
// per element; p_j s_j is rounded to bf16 once, the type that the product takes (outputs
// are 0.0023 of their norm off, with their own rounding alone 0.0017).  Zero points of V
// stay out of the sums: tensor cores cut what they add to a running sum, and 16 + n would
// give that a sign.
//
// What bounds it: latency, over instructions that turn 1088 bytes per page and KV head
// into fragments.  At the copy bandwidth an SM gets 23 bytes a cycle, a page every 47
// cycles, or 188 issue slots and 94 of the integer pipe.  A page takes 185 instructions, 97
// of them integer or logical: a word of eight codes becomes four registers by three shifts
// and four logical operations (V: pairs of keys are put together first, four more
// subtractions), and S^T[16 keys x 8 rows] and O^T[64 x 8] take four mma.sync each.  8
// requests of up to 131072 keys run at 3.7 TB/s, 92.8 us, of which those instructions are
// 49 us of issue (a capture of 16 requests of 16384 keys: slots used 55% of the time, the
// integer pipe 55%).  Four warps per scheduler, with a vote over the warp in every page, do
// not fill the rest.  Of 64 requests of 1..4096 tokens, 32.8 us, they are 11 us; the rest is
// start, first data, latency and joins.
//
// Split: every warp takes an equal, contiguous share of all pages of the call, numbered
// through over (request, KV head, row block), whatever the requests' lengths: no wave
// of short ones at the end, and no plan on the host.  A unit (request, KV head, row
// block) inside one warp's share is finished there; parts join by log-sum-exp in shared
// memory within a CTA, and CTAs that share a unit through the workspace, by the last one
// to get there, in page order.  Every warp runs its own ring of bulk copies, four pages
// (4352 bytes) a stage, across the borders of units.
//
// The running maximum is a reference that moves only when a score exceeds it by 2^8
// (p <= 256 is as good in bf16 and fp32), so a step needs one vote instead of six
// shuffles.
//
// Measured on the way (8 requests of up to 131072 keys): zero points of V as a correction
// to the sums, two pages a stage 138 us; four pages, subtracted from the operands 94; as
// it is 92.8.  Slower: one warp of a CTA making all copies (119), 24 warps per SM,
// two pages of a step in flight at once (96), high halves by multiplication.

#include "int4.cuh"
#include "ptx.cuh"
#include "workspace.cuh"

#include <algorithm>
#include <type_traits>

namespace sa {
namespace {

constexpr int kNW = 8;                        // warps per CTA
constexpr int kThreads = kNW * 32;
constexpr int kStepPages = 4;                 // pages per stage
constexpr int kStageBytes = kStepPages * kInt4Block;
// A unit's share of the work beyond its pages, in pages: reading its queries, the first
// maximum, the end.  (64 requests of 1..4096 tokens, us: 36.1 / 32.6 / 33.8 / 33.3 at
// 0 / 4 / 8 / 12 with one token each, 76.7 / 50.2 / 48.6 / 47.6 with two.)
constexpr int kUnitCost = 8;
constexpr float kRaise = 8.f;                 // log2 by which a score may exceed the reference
constexpr float kUnset = -8e37f;              // reference of a row that has seen no key yet

// Stages in flight per warp, and CTAs per SM: 16 warps with 128 registers (three CTAs of
// fewer registers, or 24 warps, were slower); four blocks of rows keep 255 registers.
template <int NB>
struct Tuning {
  static constexpr int kStages = 2;
  static constexpr int kCtas = NB == 4 ? 1 : 2;
};

// A request's share of the work: `units` (KV head, row block) pairs of `pages` pages
// each; a request without keys, or one that is out of range (`bad`), counts one page
// that nothing of is read.
struct Request {
  int kv_len, row0, tokens, pages, units;
  bool bad;
};

template <int NB>
struct Part {                                 // one warp's share of a unit
  float o[8 * NB][kHeadDim];
  float m[8 * NB], d[8 * NB];
};

template <int NB>
struct __align__(128) Shared {
  uint8_t ring[kNW][Tuning<NB>::kStages][kStageBytes];
  Part<NB> begun[kNW];                        // of a unit begun before the warp's share
  uint64_t bars[kNW][Tuning<NB>::kStages];
  long long prefix[kThreads + 1];
  long long scan[kNW];
  struct {                                    // the unit of a part; pages 0: there is none
    long long from;                           // the number of its first page
    Request r;
    int pages, kvh, rb;
  } unit[2][kNW];
  int last[2];
  // 0: a unit begun before the warp's share; 1: one that goes on after it (in the
  // ring, which is idle by then)
  __device__ __forceinline__ Part<NB> &part(int slot, int warp) {
    static_assert(sizeof(Part<NB>) <= sizeof(ring[0]), "a part fits into a warp's ring");
    return slot == 0 ? begun[warp] : *reinterpret_cast<Part<NB> *>(&ring[warp][0][0]);
  }
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <int NB, int kMode>
__device__ __forceinline__ Request request(const Int4AttnParams &p, int b) {
  Request r;
  r.kv_len = p.kv_lens[b];
  if constexpr (kMode == kInt4Ragged) {
    r.row0 = p.cu_seqlens_q[b];
    const int end = p.cu_seqlens_q[b + 1];
    r.tokens = end - r.row0;
    r.bad = r.row0 < 0 || end < r.row0 || end > p.total_q || r.tokens > p.max_q_len || r.kv_len < r.tokens ||
            (b > 0 && r.row0 < p.cu_seqlens_q[b - 1]);
    if (r.bad)                                 // what lies inside the buffers becomes NaN
      r.tokens = r.row0 < 0 || r.row0 >= p.total_q ? 0 : min(max(end, r.row0), p.total_q) - r.row0;
  } else {
    r.tokens = p.q_len;
    r.row0 = b * p.q_len;
    r.bad = r.kv_len < (kMode == kInt4Verify ? p.q_len : 0);
  }
  r.bad = r.bad || r.kv_len > p.max_kv_len || (r.kv_len + kPageSize - 1) / kPageSize > p.max_pages_per_seq;
  r.pages = r.bad ? 1 : max(1, ceil_div(r.kv_len, kPageSize));
  r.units = r.tokens > 0 ? p.num_kv_heads * ceil_div(r.tokens * p.group, 8 * NB) : 0;
  return r;
}

// A place in the numbering of all pages: page `page` of unit `unit` of request b.
template <int NB, int kMode>
struct Place {
  Request r;
  int b, unit, page;
  __device__ __forceinline__ void next_unit(const Int4AttnParams &p) {
    page = 0;
    if (++unit < r.units) return;
    unit = 0;
    do {
      r.units = 0;
      if (++b >= p.num_seqs) return;
      r = request<NB, kMode>(p, b);
    } while (r.units == 0);
  }
};

// KV head of a place's unit, and its row block (usually there is one, and no division).
template <typename At>
__device__ __forceinline__ int kv_head(const Int4AttnParams &p, const At &at) {
  return at.unit < p.num_kv_heads ? at.unit : at.unit % p.num_kv_heads;
}
template <typename At>
__device__ __forceinline__ int row_block(const Int4AttnParams &p, const At &at) {
  return at.unit < p.num_kv_heads ? 0 : at.unit / p.num_kv_heads;
}

// a / b, mostly of small numbers.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return a <= 0xffffffffll && b <= 0xffffffffll ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Copies `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Field of 4 bits in each half of w, at bits 3..6 of the half, below the exponent of
// 16: the bf16 pair (16 + low code, 16 + high code).
// (One logical operation takes one constant: the other, or both, are kept in registers.)
struct Fields {
  uint32_t mask, sixteen;
  __device__ __forceinline__ Fields() {
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(sixteen));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(sixteen));   // w & mask | sixteen
    return r;
  }
};

__device__ __forceinline__ uint32_t word(const uint4 &x, int w) {
  return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w;
}

// A key's scale, and minus 16 plus its zero point, from the low half of m.
__device__ __forceinline__ float k_scale(uint32_t m) { return __uint_as_float((m << 16) & 0xfff00000u); }
__device__ __forceinline__ float k_zero(uint32_t m) {
  return __uint_as_float(((m << 19) & 0x00780000u) | 0xc1800000u);
}
// A value's scale, from the high half.
__device__ __forceinline__ float v_scale(uint32_t m) { return __uint_as_float(m & 0xfff00000u); }
// 16 plus the zero points of two values, from their words' high halves.
__device__ __forceinline__ uint32_t v_zeros(uint32_t m0, uint32_t m1) {
  return ((__byte_perm(m0, m1, 0x7632) << 3) & 0x00780078u) | 0x41804180u;
}

// (16 + n) - (16 + z) for two codes: exact.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// D += A B and D = A B (m16n8k16, bf16, fp32 sums), free for the compiler to move.
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Row r of the block of a unit -> its [.., Hq] row in q, out and lse (-1 past the last).
template <int NB, int kMode>
__device__ __forceinline__ long long row_of(const Int4AttnParams &p, const Request &q, int kvh, int rb,
                                            int r, int &token, int &head) {
  const int i = rb * 8 * NB + r;
  token = kMode == kInt4Decode ? (i >= p.group ? 1 : 0) : i / p.group;
  head = kvh * p.group + (i - token * p.group);
  return token < q.tokens ? (static_cast<long long>(q.row0) + token) * p.num_qo_heads + head : -1;
}

// out and lse of a row from its unnormalised sums; 4 elements from dim dq on.
__device__ __forceinline__ void write_row(const Int4AttnParams &p, long long row, int dq, float4 o,
                                          float m, float d) {
  const float inv = d == 0.f ? 0.f : 1.f / d;          // (NaN spoils the row)
  *reinterpret_cast<uint2 *>(p.out + row * kHeadDim + dq) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (dq == 0 && p.lse) p.lse[row] = d == 0.f ? -INFINITY : (m + lg2(d)) * kLn2;
}

template <int NB, int kMode>
__global__ void __launch_bounds__(kThreads, Tuning<NB>::kCtas)
int4_decode_kernel(const __grid_constant__ Int4AttnParams p) {
  constexpr int kStages = Tuning<NB>::kStages;
  constexpr int kRows = 8 * NB;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Shared<NB> &sh = *reinterpret_cast<Shared<NB> *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // ---- this warp's share of all pages
  const int per = ceil_div(p.num_seqs, kThreads);      // requests per thread of the scan
  long long mine = 0;
  for (int b = threadIdx.x * per; b < min(p.num_seqs, static_cast<int>(threadIdx.x + 1) * per); ++b) {
    const Request r = request<NB, kMode>(p, b);
    mine += static_cast<long long>(r.pages + kUnitCost) * r.units;
  }
  long long upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.bars[warp][s], 1);
    fence_mbar_init();
    sh.unit[0][warp].pages = sh.unit[1][warp].pages = 0;
  }
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kNW; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  sh.prefix[threadIdx.x] = before + upto - mine;       // pages before this thread's requests
  __syncthreads();

  // an even share, so that only its last step is half empty; whole CTAs' worth of it
  const long long slots = static_cast<long long>(gridDim.x) * kNW;
  long long share = quotient(total + slots - 1, slots);
  share = max(share + (share & 1), static_cast<long long>(p.min_pages));
  if (share > 0x7fffff00ll) return;                    // (the host refuses what lengths allow of this)
  const long long cta_share = share * kNW;
  const long long from = min(total, blockIdx.x * cta_share + warp * share);
  const long long to = min(total, from + share);
  if (blockIdx.x * cta_share >= total) return;         // uniform over the CTA

  using At = Place<NB, kMode>;
  At at;                                               // where the pages are worked on
  at.b = at.unit = at.page = 0;
  if (from < to) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i)
      n += __popc(__ballot_sync(0xffffffffu, sh.prefix[i * 32 + lane] <= from));
    at.b = (n - 1) * per;                              // the last threads' requests that begin by `from`
    long long here = sh.prefix[n - 1];
    while (true) {
      at.r = request<NB, kMode>(p, at.b);
      const long long w = static_cast<long long>(at.r.pages + kUnitCost) * at.r.units;
      if (here + w > from) break;
      here += w;
      ++at.b;
    }
    const int each = at.r.pages + kUnitCost;           // a unit's cost comes before its pages
    at.unit = static_cast<int>(quotient(from - here, each));
    at.page = static_cast<int>((from - here) - static_cast<long long>(at.unit) * each) - kUnitCost;
  }
  // this warp's pages and the costs of the units that begin among them
  const int share_left = max(0, static_cast<int>(to - from) + min(at.page, 0));
  at.page = max(at.page, 0);

  // ---- copies: `to_come` runs ahead of `at` by up to kStages steps
  At to_come = at;
  int unissued = share_left;
  int ids = -1, ids_next = -1, ids_at = 0;             // lane j: id of page ids_at + j; of the next 32
  auto load_ids = [&](int first) -> int {
    const int page = first + lane;
    return !to_come.r.bad && page * kPageSize < to_come.r.kv_len
               ? p.page_table[static_cast<size_t>(to_come.b) * p.max_pages_per_seq + page] : -1;
  };
  auto start_ids = [&]() {
    ids_at = to_come.page;
    ids = load_ids(ids_at);
    ids_next = ids_at + 32 < to_come.r.pages ? load_ids(ids_at + 32) : -1;
  };
  if (share_left > 0) start_ids();

  // Up to here only lengths and the page table were read; everything below may
  // depend on the previous kernel on the stream.
  grid_dependency_wait();
  launch_dependents();

  const uint64_t policy = l2_policy_evict_first();
  const long long page_bytes = static_cast<long long>(p.num_kv_heads) * kInt4Block;
  const uint8_t *src = p.kv_cache + static_cast<size_t>(kv_head(p, to_come)) * kInt4Block;
  uint32_t spoilt = 0;                                 // stages with a page outside of the pool
  auto issue = [&](int st) {                           // all lanes call
    const int n = min(min(kStepPages, unissued), to_come.r.pages - to_come.page);
    if (to_come.page - ids_at >= 32) {
      ids_at += 32;
      ids = ids_next;
      ids_next = ids_at + 32 < to_come.r.pages ? load_ids(ids_at + 32) : -1;
    }
    // (a batch of 32 is a whole number of steps: it begins where a unit's share does)
    const int id = __shfl_sync(0xffffffffu, ids, to_come.page - ids_at + (lane & (kStepPages - 1)));
    const bool ok = lane < n && id >= 0 && id < p.num_pages;
    const unsigned good = __ballot_sync(0xffffffffu, ok);
    const bool empty = to_come.r.kv_len <= 0 || to_come.r.bad;
    const int copies = __popc(good);
    spoilt = (spoilt & ~(1u << st)) | (!empty && copies < n ? 1u << st : 0u);
    uint64_t *bar = &sh.bars[warp][st];
    if (lane == 0) mbar_arrive_expect_tx(bar, copies * kInt4Block);
    __syncwarp();
    if (ok) {
      fence_proxy_async_smem();
      bulk_load(&sh.ring[warp][st][lane * kInt4Block], src + id * page_bytes, kInt4Block, bar, policy);
    }
    unissued -= n;
    to_come.page += n;
    if (to_come.page >= to_come.r.pages && unissued > 0) {
      unissued = max(unissued - kUnitCost, 0);
      if (unissued > 0) {
        to_come.next_unit(p);
        src = p.kv_cache + static_cast<size_t>(kv_head(p, to_come)) * kInt4Block;
        start_ids();
      }
    }
  };
  int issued = 0, done = 0;                            // steps
  while (issued < kStages && unissued > 0) issue(issued++);

  // ---- units of this share, one after another
  bool dead = false;                                   // a copy never landed
  int left = share_left;
  while (left > 0) {
    const int kvh = kv_head(p, at), rb = row_block(p, at);
    const int first_page = at.page;
    const int seg = min(left, at.r.pages - at.page);
    const int seg_end = first_page + seg;
    // keys [0, old) are visible to every row, key old + u to the rows of token u and
    // later ones, or by the mask
    const int old = kMode == kInt4Decode ? at.r.kv_len : at.r.kv_len - at.r.tokens;

    // Q^T as B operand: row g of each block; registers 2k and 2k + 1 hold pairs (dim, dim + 4)
    uint32_t qb[NB][8];
    float qs[NB][2];                                   // sum of q of rows 2t and 2t + 1
    float m[NB][2], d[NB][2];                          // reference (base 2), sum
    int limit[NB][2];                                  // keys that a row sees (causal)
    uint64_t vis[NB][2];                               // and its bits of the mask
    float o[NB][4][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      int token, head;
      const long long row = row_of<NB, kMode>(p, at.r, kvh, rb, 8 * nb + g, token, head);
      uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (row >= 0) {
        const uint4 *q = reinterpret_cast<const uint4 *>(p.q) + row * (kHeadDim / 8);
        x[0] = __ldg(q + t);
        x[1] = __ldg(q + t + 4);
      }
      float sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qb[nb][4 * h + j] = __byte_perm(w[j / 2], w[j / 2 + 2], j & 1 ? 0x7632 : 0x5410);
          sum += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[nb][e] = __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e));
        const long long r = row_of<NB, kMode>(p, at.r, kvh, rb, 8 * nb + 2 * t + e, token, head);
        // a sink that is no logit (NaN, +inf) spoils the sum, not the maximum
        const bool sink = first_page == 0 && r >= 0;
        const float logit = sink ? __ldg(p.sinks + head) * kLog2e : -INFINITY;
        const bool fine = logit < INFINITY;
        m[nb][e] = fine ? fmaxf(logit, kUnset) : kUnset;
        d[nb][e] = sink && g == 0 ? (fine ? (logit < kUnset ? 0.f : 1.f) : NAN) : 0.f;
        limit[nb][e] = kMode == kInt4Decode ? at.r.kv_len : min(at.r.kv_len, old + token + 1);
        vis[nb][e] = 0;
        if constexpr (kMode == kInt4Verify) {
          if (p.tree_mask && r >= 0) {
            vis[nb][e] = p.tree_mask[static_cast<size_t>(at.b) * p.q_len + token];
            limit[nb][e] = old;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
    }
    bool bad = at.r.bad || dead;

    const int tok_end = min(at.r.kv_len, seg_end * kPageSize);

    // One page: its block in shared memory, its first key tok0.
    const Fields field;
    auto work = [&](const uint8_t *at_block, int tok0, auto is_edge) {
      constexpr bool kEdge = decltype(is_edge)::value;
      const uint4 kw = *reinterpret_cast<const uint4 *>(at_block + kInt4K + 16 * lane);
      const uint2 mt = *reinterpret_cast<const uint2 *>(at_block + kInt4Meta + 8 * g);             // keys g and g + 8
      float s[NB][4];                      // key g + 8 (i / 2), row 2t + i % 2
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = word(kw, h), hi = word(kw, 2 + h);         // keys g and g + 8
        const uint32_t a0[4] = {field(lo), field(hi), field(lo >> 4), field(hi >> 4)};
        const uint32_t a1[4] = {field(lo >> 8), field(hi >> 8), field(__funnelshift_r(lo, lo, 12)),
                                field(__funnelshift_r(hi, hi, 12))};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (h == 0)
            mma_first(s[nb], a0, qb[nb][0], qb[nb][1]);
          else
            mma_add(s[nb], a0, qb[nb][4], qb[nb][5]);
          mma_add(s[nb], a1, qb[nb][4 * h + 2], qb[nb][4 * h + 3]);
        }
      }
      const float ks[2] = {k_scale(mt.x) * p.scale_log2, k_scale(mt.y) * p.scale_log2};
      const float kz[2] = {k_zero(mt.x), k_zero(mt.y)};
      float vs[2] = {v_scale(mt.x), v_scale(mt.y)};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nb][i] = ks[i / 2] * fmaf(kz[i / 2], qs[nb][i & 1], s[nb][i]);
      if constexpr (kEdge) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = tok0 + g + 8 * (i / 2), u = tok - old;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const bool drafted = kMode == kInt4Verify && u >= 0 && u < 64 && ((vis[nb][i & 1] >> u) & 1);
            if (tok >= tok_end || (tok >= limit[nb][i & 1] && !drafted)) s[nb][i] = -INFINITY;
          }
          // a slot past the last key may hold anything
          if (tok >= tok_end) vs[i / 2] = 0.f;
        }
      }
      // any score far above its row's reference?
      float top = -INFINITY;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        top = fmax3(top, fmaxf(s[nb][0], s[nb][2]) - m[nb][0], fmaxf(s[nb][1], s[nb][3]) - m[nb][1]);
      if (__any_sync(0xffffffffu, top > kRaise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[nb][e], s[nb][2 + e]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
            if (x > m[nb][e]) {
              const float a = ex2(m[nb][e] - x);
              m[nb][e] = x;
              d[nb][e] *= a;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nb][i][e] *= a;
                o[nb][i][2 + e] *= a;
              }
            }
          }
      }
      uint32_t pb[NB][2];                  // p times the value's scale, as B operand: keys 2t.., row g
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = ex2(s[nb][2 * h] - m[nb][0]), p1 = ex2(s[nb][2 * h + 1] - m[nb][1]);
          d[nb][0] += p0;
          d[nb][1] += p1;
          float w0 = p0 * vs[h], w1 = p1 * vs[h];
          if constexpr (kEdge) {           // a hidden key's scale may be NaN
            if (s[nb][2 * h] == -INFINITY) w0 = 0.f;
            if (s[nb][2 * h + 1] == -INFINITY) w1 = 0.f;
          }
          pb[nb][h] = movmatrix_trans(pack_bf16(w0, w1));
        }
      // word g of keys 2t, 2t + 1, 2t + 8, 2t + 9; and their zero points (2t, 2t + 8, ..)
      const uint4 vw = *reinterpret_cast<const uint4 *>(at_block + kInt4V + 16 * lane);
      const uint4 vm = *reinterpret_cast<const uint4 *>(at_block + kInt4Meta + 16 * t);
      const uint32_t z0 = v_zeros(vm.x, vm.z), z1 = v_zeros(vm.y, vm.w);
#pragma unroll
      for (int c = 0; c < 2; ++c) {                            // dims 8g + 4c ..
        const uint32_t sel = c ? 0x7632 : 0x5410;
        const uint32_t lo = __byte_perm(vw.x, vw.y, sel), hi = __byte_perm(vw.z, vw.w, sel);
        const uint32_t a0[4] = {sub_bf16x2(field(lo << 3), z0), sub_bf16x2(field(lo >> 1), z0),
                                sub_bf16x2(field(hi << 3), z1), sub_bf16x2(field(hi >> 1), z1)};
        const uint32_t a1[4] = {sub_bf16x2(field(lo >> 5), z0), sub_bf16x2(field(lo >> 9), z0),
                                sub_bf16x2(field(hi >> 5), z1), sub_bf16x2(field(hi >> 9), z1)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma_add(o[nb][2 * c], a0, pb[nb][0], pb[nb][1]);
          mma_add(o[nb][2 * c + 1], a1, pb[nb][0], pb[nb][1]);
        }
      }
    };

    for (int page = first_page; page < seg_end; page += kStepPages) {
      const int st = done % kStages;
      // (one answer for all lanes: at the limit some may see the phase and others not)
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&sh.bars[warp][st], (done / kStages) & 1))) {
        // a copy never landed: let the others in flight land (with the same limit)
        // before their stages are used otherwise, and start no more
        dead = bad = true;
        for (int i = done + 1; i < issued; ++i) mbar_wait(&sh.bars[warp][i % kStages], (i / kStages) & 1);
      }
      bad = bad || ((spoilt >> st) & 1);
      ++done;
      if (dead) continue;
      const uint8_t *block = &sh.ring[warp][st][0];
      if ((page + kStepPages) * kPageSize <= min(tok_end, old)) {      // whole, keys that all rows see
#pragma unroll
        for (int i = 0; i < kStepPages; ++i) work(block + i * kInt4Block, 0, std::false_type{});
      } else {
        const int end = min(page + kStepPages, seg_end);
#pragma unroll 1
        for (int i = page; i < end; ++i, block += kInt4Block) work(block, i * kPageSize, std::true_type{});
      }
      __syncwarp();                                    // the stage has been read
      if (unissued > 0) issue(issued++ % kStages);
    }

    // ---- the segment's sums; lane (g, t) has dims 8g .. 8g + 7 of rows 2t, 2t + 1
    const bool begun = first_page > 0, goes_on = seg_end < at.r.pages;
    const int slot = begun ? 0 : 1;
    Part<NB> &part = sh.part(slot, warp);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float dd = d[nb][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) dd += __shfl_xor_sync(0xffffffffu, dd, off);
        if (bad) dd = NAN;
        // o[nb][i][e] and [2 + e]: dims 8g + 2i and 8g + 2i + 1
        const float4 lo = make_float4(o[nb][0][e], o[nb][0][2 + e], o[nb][1][e], o[nb][1][2 + e]);
        const float4 hi = make_float4(o[nb][2][e], o[nb][2][2 + e], o[nb][3][e], o[nb][3][2 + e]);
        const int r = 8 * nb + 2 * t + e;
        if (!begun && !goes_on) {
          int token, head;
          const long long row = row_of<NB, kMode>(p, at.r, kvh, rb, r, token, head);
          if (row >= 0) {
            write_row(p, row, 8 * g, lo, m[nb][e], dd);
            write_row(p, row, 8 * g + 4, hi, m[nb][e], dd);
          }
        } else {
          *reinterpret_cast<float4 *>(&part.o[r][8 * g]) = lo;
          *reinterpret_cast<float4 *>(&part.o[r][8 * g + 4]) = hi;
          if (g == 0) {
            part.m[r] = m[nb][e];
            part.d[r] = dd;
          }
        }
      }
    if (lane == 0 && (begun || goes_on)) {
      auto &u = sh.unit[slot][warp];
      u.from = to - left - first_page;
      u.r = at.r;
      u.pages = at.r.pages;
      u.kvh = kvh;
      u.rb = rb;
    }
    left = max(left - seg - kUnitCost, 0);
    if (left > 0) at.next_unit(p);
  }

  // ---- join the parts.  A unit's parts lie in consecutive warps: slot 1 of the warp
  // that begins it, slot 0 of the others.
  __syncthreads();
  const long long cta_from = blockIdx.x * cta_share, cta_to = min(total, cta_from + cta_share);
  constexpr int kQuads = kHeadDim / 4, kItems = kRows * kQuads;
  // 4 elements of a row over the warps that have parts of the unit which warp w0 has in
  // slot s0, up to warp w1.  All loads at once: the others' are taken from w0, for nothing.
  auto last_warp = [&](int w0, long long u_to) {
    int w1 = w0 + 1;
    while (w1 < kNW && cta_from + w1 * share < min(u_to, total)) ++w1;
    return w1;
  };
  auto join_warps = [&](int s0, int w0, int w1, int item, float &mx, float &den) -> float4 {
    const int row = item / kQuads, dq = item % kQuads * 4;
    float wt[kNW];
    mx = kUnset;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      const bool in = w >= w0 && w < w1;
      const float m = (in && w != w0 ? sh.part(0, w) : sh.part(s0, w0)).m[row];
      wt[w] = in ? m : -INFINITY;
      mx = fmaxf(mx, m);
    }
    den = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      const bool in = w >= w0 && w < w1;
      const Part<NB> &x = in && w != w0 ? sh.part(0, w) : sh.part(s0, w0);
      const float d = x.d[row];
      const float4 v = *reinterpret_cast<const float4 *>(&x.o[row][dq]);
      const float e = ex2(wt[w] - mx);
      if (in) {
        den += e * d;
        a.x += e * v.x;
        a.y += e * v.y;
        a.z += e * v.z;
        a.w += e * v.w;
      }
    }
    return a;
  };
  auto write = [&](const auto &u, int item, float4 a, float mx, float den) {
    int token, head;
    const long long row = row_of<NB, kMode>(p, u.r, u.kvh, u.rb, item / kQuads, token, head);
    if (row >= 0) write_row(p, row, item % kQuads * 4, a, mx, den);
  };

  // units inside the CTA: each by the warp that has its first part
  {
    const auto &u = sh.unit[1][warp];
    if (u.pages > 0 && u.from + u.pages <= cta_to) {
      const int w1 = last_warp(warp, u.from + u.pages);
#pragma unroll 2
      for (int item = lane; item < kItems; item += 32) {
        float mx, den;
        const float4 a = join_warps(1, warp, w1, item, mx, den);
        write(u, item, a, mx, den);
      }
    }
  }
  // and by the whole CTA the unit that began before it (0) and the one that goes on
  // after it (1): its part to the workspace.  The last of the CTAs that share a unit
  // joins their parts, in page order, and leaves the counter at zero for the next call.
  int shared_by[2], first_cta[2], from_warp[2];        // CTAs that share it (1: no such unit)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    shared_by[k] = 1;
    from_warp[k] = 0;
    if (k == 1) {
      int w = kNW - 1;                                 // the last warp with a unit of its own beginning
      while (w >= 0 && !(sh.unit[1][w].pages > 0 && sh.unit[1][w].from + sh.unit[1][w].pages > cta_to)) --w;
      if (w < 0) continue;
      from_warp[k] = w;
    } else if (sh.unit[0][0].pages == 0) {
      continue;
    }
    const auto &u = sh.unit[k][from_warp[k]];
    first_cta[k] = static_cast<int>(quotient(u.from, cta_share));
    shared_by[k] = static_cast<int>(quotient(u.from + u.pages - 1, cta_share)) - first_cta[k] + 1;
    const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + k) * kRows;
    const int w1 = last_warp(from_warp[k], u.from + u.pages);
    for (int item = threadIdx.x; item < kItems; item += kThreads) {
      float mx, den;
      const float4 a = join_warps(k, from_warp[k], w1, item, mx, den);
      *reinterpret_cast<float4 *>(p.ws_o + (at + item / kQuads) * kHeadDim + item % kQuads * 4) = a;
      if (item % kQuads == 0) p.ws_md[at + item / kQuads] = make_float2(mx, den);
    }
  }
  if (shared_by[0] == 1 && shared_by[1] == 1) return;  // uniform over the CTA
  __syncthreads();
  if (threadIdx.x < 2) {
    const int k = threadIdx.x;
    sh.last[k] = shared_by[k] > 1 && atomic_add_acq_rel(&p.counters[first_cta[k]], 1) == shared_by[k] - 1;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!sh.last[k]) continue;
    const auto &u = sh.unit[k][from_warp[k]];
    const int c0 = first_cta[k], c1 = c0 + shared_by[k];
    for (int item = threadIdx.x; item < kItems; item += kThreads) {
      const int row = item / kQuads, dq = item % kQuads * 4;
      auto index = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * kRows + row; };
      float mx = -INFINITY;
#pragma unroll 4
      for (int c = c0; c < c1; ++c) mx = fmaxf(mx, __ldcg(&p.ws_md[index(c)]).x);
      float den = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = c0; c < c1; ++c) {
        const float2 md = __ldcg(&p.ws_md[index(c)]);
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + index(c) * kHeadDim + dq));
        const float wt = ex2(md.x - mx);
        den += wt * md.y;
        a.x += wt * v.x;
        a.y += wt * v.y;
        a.z += wt * v.z;
        a.w += wt * v.w;
      }
      write(u, item, a, mx, den);
    }
    if (threadIdx.x == 0) p.counters[c0] = 0;
  }
}

template <int NB, int kMode>
cudaError_t launch_variant(const Int4AttnParams &p, int ctas, cudaStream_t stream, bool programmatic) {
  constexpr int kBytes = static_cast<int>(sizeof(Shared<NB>));
  static_assert(kBytes <= 227 * 1024, "shared memory");
  cudaError_t err = set_smem_once<int4_decode_kernel<NB, kMode>>(kBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(int4_decode_kernel<NB, kMode>, static_cast<unsigned>(ctas), kThreads, kBytes, stream,
                       programmatic, p);
}

template <int NB>
cudaError_t launch_mode(const Int4AttnParams &p, Int4Mode mode, int ctas, cudaStream_t stream,
                        bool programmatic) {
  if (mode == kInt4Decode) return launch_variant<NB, kInt4Decode>(p, ctas, stream, programmatic);
  if (mode == kInt4Verify) return launch_variant<NB, kInt4Verify>(p, ctas, stream, programmatic);
  return launch_variant<NB, kInt4Ragged>(p, ctas, stream, programmatic);
}

template <int NB>
int ctas_per_sm() {
  return std::min(Tuning<NB>::kCtas, 228 * 1024 / static_cast<int>(sizeof(Shared<NB>) + 1024));
}

}  // namespace

int int4_decode_ctas_per_sm(int row_blocks) {
  return row_blocks == 1 ? ctas_per_sm<1>() : row_blocks == 2 ? ctas_per_sm<2>() : ctas_per_sm<4>();
}

size_t int4_decode_results_bytes(int row_blocks, int ctas) {
  return static_cast<size_t>(ctas) * 2 * 8 * row_blocks * (kHeadDim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_int4_decode(const Int4AttnParams &p, Int4Mode mode, int row_blocks, int ctas,
                               cudaStream_t stream, bool programmatic) {
  if (row_blocks == 1) return launch_mode<1>(p, mode, ctas, stream, programmatic);
  if (row_blocks == 2) return launch_mode<2>(p, mode, ctas, stream, programmatic);
  return launch_mode<4>(p, mode, ctas, stream, programmatic);
}

}  // namespace sa
