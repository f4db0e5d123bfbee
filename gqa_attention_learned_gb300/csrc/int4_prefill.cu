// Many query rows per KV head over a paged cache held in 4 bits (chunked prefill, draft
// trees), learned sinks, on the 5th-generation tensor cores.
//
// Mathematics: row (token i, head h) of a request with kv_len keys of which the last
// q_len are its new tokens sees keys j <= kv_len - q_len + i (or the draft keys that its
// mask names); softmax with the sink as one more term, as in plain prefill.  The keys'
// and values' codes become bf16 numbers s (n - z) on the way into shared memory, which
// is exact; P is rounded to bf16, the type that the product with V takes, out once (outputs
// are 0.0023 of their norm off, with their own rounding alone 0.0017).
//
// One CTA per SM = the rows of 2 * (128 / group) tokens of one KV head, ordered (token,
// head), as two 128-row tiles that share every K and V tile of 128 keys: turning a tile
// of codes into bf16 costs half of what it would for one, and one tile's products run
// during the other's softmax.
//   warps 0..7    softmax, one thread per row.  Scores come 32 at a time and are not
//                 compared: P = 2^(s - m) with the row's reference m, and only if a
//                 tile's sum shows that m has become too small (or is not set) the
//                 row's maximum is taken and the tile done once more.  Scores beyond
//                 the causal limit are left out by index.
//   warps 8..15   a page of every key tile each: codes to bf16 (shift, mask under the
//                 exponent of 16, subtract 16 + z, multiply by s), stores into the K and
//                 V rings in the swizzled layout.  A word of codes gives dims (0 4 1 5 2
//                 6 3 7) of a group of eight in that order: Q is permuted likewise, O's
//                 columns are put right at the end.
//   warp 16       S = Q K^T into one of three score buffers of tensor memory as soon as
//                 its last P has been used
//   warp 17       O += P V, P in place of its scores
//   warp 18       packed pages into a ring of four key tiles, by bulk copies
//
// Where there are few such CTAs, a request's keys are cut into parts with a CTA each: as
// many as make the least time (plan_parts()), each at least 512 keys long.  Parts join by
// log-sum-exp through the workspace, by the last one to get there, in the keys' order.
//
// What bounds it, for 4 x 2048 tokens on up to 14336 keys (1351 us, 1017 TFLOP/s, where
// the kernel of the bf16 cache does 1046): the chain score - exponentials - P V of the two
// tiles in turn.  P V of 128 x 64 x 128 from tensor memory takes about twice its
// arithmetic's time, and start and end of a CTA some 5 us.  Measured on the way: one tile
// per CTA 1839 us; eight unpacking warps, two score buffers 1692; three buffers and a ring
// of packed pages 1555; softmax warps with 168 registers, sleeping waits 1537; products
// started by polling warps 1485; a row's mask as bits 1376; fewer spills 1351.  Slower or
// no better: 16 softmax warps with half a row each; products started by one thread that
// walks the tiles alone (1558 against 1482); persistent CTAs (1720: spills); four stages
// of K and V; both halves of a CTA on one query tile where there is one only (64 rows 1%
// faster, full tiles 3% slower).
//
// A value row that is not finite must spoil the rows that see it and no others, but
// 0 * NaN in P V would spoil the whole tile: such a value is stored as zero and its key
// as NaN, so the rows that see it get there by their score (and their lse is NaN, too).

#include "int4.cuh"
#include "ptx.cuh"
#include "workspace.cuh"

#include <cmath>

namespace sa {
namespace {

constexpr int kBM = 128;                       // rows per tile
constexpr int kBN = 128;                       // keys per K / V tile
constexpr int kPages = kBN / kPageSize;        // pages per key tile
constexpr int kStages = 3;                     // of the ring of K and V tiles
constexpr int kTileBytes = kBN * kHeadDim * 2; // 16 KB
constexpr int kThreads = 640;                  // five warpgroups
constexpr int kUnpackWarp = 8, kUnpackWarps = kPages, kQkWarp = 16, kPvWarp = 17, kLoadWarp = 18;
// Registers per thread: the launch has 96 for all; softmax warps take from the others.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 168, kOtherRegs = 48;
static_assert(2 * kSoftmaxRegs + 3 * kOtherRegs <= 5 * kLaunchRegs, "the split fits the launch's registers");
constexpr int kBuffers = 3;                    // of scores in tensor memory
// Requests up to which every warp counts through them by itself, 32 at a time, instead of
// the CTA at once (us of either, prompts of 40..80 tokens: 100 requests 129 and 133, 200
// 278 and 258, 1000 2416 and 1303).
constexpr int kFewRequests = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = kBuffers * kBN;      // behind the scores: 64 columns per tile
constexpr int kPartTiles = kInt4PartKeys / kBN;        // that a part has at least
// What a part costs beyond its tiles, in tiles (4 x 128 tokens on 4000..16000 keys: 183 us
// at 8, 170 at 14, 189 at 20, when an edge still cost three times as much).
constexpr float kPartCost = 14.f;
constexpr float kUnset = -8e37f;               // reference of a row that has seen no key yet
constexpr float kMostSum = 1024.f;             // sum of a tile's P from which the reference is moved

constexpr int kOffQ = 0;                       // two tiles
constexpr int kOffK = 2 * kTileBytes;
constexpr int kOffV = kOffK + kStages * kTileBytes;
constexpr int kRaw = 4;                        // key tiles of packed pages on their way or waiting
constexpr int kOffRaw = kOffV + kStages * kTileBytes;
constexpr int kOffBars = kOffRaw + kRaw * kPages * kInt4Block;

// Products are numbered through: key tile 0 of query tile 0, of query tile 1, key tile 1
// of query tile 0, ..; product n uses scores buffer n % 3.  A parity tells two phases
// apart, no more, so a wait has to be sure of the phase before (S of product n says that
// P of product n - 3 has been used) and that the one after cannot have passed (P V are
// done in order: none after product n before its P is there; and a query tile's last
// product has at most two behind it).
struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[kBuffers];   // S is in the buffer
  uint64_t p_full[kBuffers];   // P is, in its place
  uint64_t p_used[kBuffers];   // P V has finished: the buffer is free
  uint32_t tmem_base;
  int bad, last;
  int part_tiles, numbers;     // as plan_parts says
  int seq, number;             // this CTA's request and its place in that
  long long scan[kThreads / 32];
  uint64_t vis[2 * kBM];       // mask of a row
  int shared_by, part, first;  // of the CTAs that share these rows (kept here: registers are short)
};
constexpr int kSmemBytes = kOffBars + static_cast<int>(sizeof(Bars)) + 1024;

constexpr uint32_t kIdescQK = umma_idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescPV = umma_idesc_bf16(128, 64, false, true);

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// A request's rows and keys, and whether its arguments are in range.
struct Request {
  int q_start, q_len, kv_len;
  bool bad;
};
__device__ __forceinline__ Request request(const Int4AttnParams &p, int seq) {
  Request r;
  r.kv_len = __ldg(p.kv_lens + seq);
  if (p.cu_seqlens_q) {
    r.q_start = __ldg(p.cu_seqlens_q + seq);
    r.q_len = __ldg(p.cu_seqlens_q + seq + 1) - r.q_start;
    r.bad = r.q_start < 0 || r.q_len < 0 || r.q_len > p.total_q - r.q_start || r.q_len > p.max_q_len ||
            (seq > 0 && r.q_start < __ldg(p.cu_seqlens_q + seq - 1));
  } else {
    r.q_start = seq * p.q_len;
    r.q_len = p.q_len;
    r.bad = false;
  }
  r.bad = r.bad || r.kv_len < r.q_len || r.kv_len > p.max_kv_len ||
          (r.kv_len + kPageSize - 1) / kPageSize > p.max_pages_per_seq;
  return r;
}

// CTAs of a request and KV head: one for a request out of range (it makes its rows NaN).
__device__ __forceinline__ int request_ctas(const Request &r, int tokens) {
  return r.bad ? 1 : cdiv(r.q_len, tokens);
}

// Rows of `tokens` tokens from `token` on become NaN, as far as they lie inside the
// buffers (the whole CTA calls).
__device__ __forceinline__ void spoil_rows(const Int4AttnParams &p, int kvh, int token, int tokens) {
  if (token < 0 || token >= p.total_q) return;
  const int rows = min(max(tokens, 0), p.total_q - token) * p.group;
  for (int i = threadIdx.x; i < rows; i += kThreads) {
    const size_t row = static_cast<size_t>(token + i / p.group) * p.num_qo_heads + kvh * p.group + i % p.group;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kHeadDim);
#pragma unroll
    for (int c = 0; c < kHeadDim / 8; ++c) dst[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    if (p.lse) p.lse[row] = NAN;
  }
}

// A row's keys [0, limit), and the draft keys from `draft` on by the bits of *vis (in
// shared memory, registers are short; null: none).
struct Seen {
  int limit, draft;
  const uint64_t *vis;
  // Bit i: whether the row sees key + i, i < 32.
  __device__ __forceinline__ uint32_t operator()(int key) const {
    const int n = limit - key;
    uint32_t w = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    if (vis) {
      const int u = key - draft;
      if (u > -32 && u < 64) w |= static_cast<uint32_t>(u >= 0 ? *vis >> u : *vis << -u);
    }
    return w;
  }
};

// P = 2^(s * scale - m) for 32 scores x as bf16 pairs in y, of the keys of bits `seen`
// alone; their sums in acc.  (Bits made once for 32 keys: a comparison per key, and a
// shift of 64 bits, took 11000 cycles of a tile with an edge.)
template <bool kMask>
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], uint32_t (&y)[16], uint64_t scale2, uint64_t negm2,
                                      uint32_t seen, uint64_t &acc0, uint64_t &acc1) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, negm2), a, b);
    if constexpr (kMask) {
      if (!(seen >> (2 * e) & 1)) a = -INFINITY;
      if (!(seen >> (2 * e + 1) & 1)) b = -INFINITY;
    }
    const float pa = ex2(a), pb = ex2(b);
    if (e & 1) acc1 = f2_add(acc1, f2_pack(pa, pb));
    else acc0 = f2_add(acc0, f2_pack(pa, pb));
    y[e] = pack_bf16(pa, pb);
  }
}

// All 128 scores of this thread's row (at `ts` in tensor memory) against its reference m.
// P stays in registers: the scores have to be there still if m turns out too small.
// Returns the row's sum.
template <bool kMask>
__device__ __forceinline__ float weigh_tile(uint32_t ts, float sl2, float m, const Seen &seen, int key0,
                                            uint32_t (&y)[4][16]) {
  const uint64_t scale2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m, -m);
  uint64_t acc0 = 0, acc1 = 0;
  uint32_t x[2][32];
  tmem_ld32(ts, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld_wait32(x[c & 1]);
    if (c < 3) tmem_ld32(ts + 32 * (c + 1), x[(c + 1) & 1]);
    weigh<kMask>(x[c & 1], y[c], scale2, negm2, kMask ? seen(key0 + 32 * c) : 0u, acc0, acc1);
  }
  float a, b;
  f2_unpack(f2_add(acc0, acc1), a, b);
  return a + b;
}

// Largest scaled score of this thread's row among the keys that it sees.
__device__ __forceinline__ float row_max(uint32_t ts, float sl2, const Seen &seen, int key0) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_ld32(ts + 32 * c, x);
    const uint32_t bits = seen(key0 + 32 * c);
    tmem_ld_wait32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) mx = fmaxf(mx, bits >> e & 1 ? __uint_as_float(x[e]) * sl2 : -INFINITY);
  }
  return mx;
}

__device__ __forceinline__ void scale_o(uint32_t to, float alpha) {
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t x[32];
    tmem_ld32(to + 32 * h, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
    tmem_st16(to + 32 * h, *reinterpret_cast<uint32_t(*)[16]>(&x[0]));
    tmem_st16(to + 32 * h + 16, *reinterpret_cast<uint32_t(*)[16]>(&x[16]));
  }
  tmem_st_wait();
}

// ------------------------------------------------------------ codes to bf16
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t field(uint32_t w, uint32_t mask, uint32_t sixteen) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(sixteen));   // w & mask | sixteen
  return r;
}
// Eight codes (the word rotated left by 3) as s (n - z), in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 values(uint32_t w, uint32_t s2, uint32_t z2, uint32_t mask, uint32_t sixteen) {
  auto value = [&](uint32_t x) { return mul_bf16x2(sub_bf16x2(field(x, mask, sixteen), z2), s2); };
  return make_uint4(value(w), value(w >> 4), value(w >> 8), value(__funnelshift_r(w, w, 12)));
}
// The pair (s, s) and the pair (16 + z, 16 + z) of K (from the low half of m) or of V.
__device__ __forceinline__ uint32_t pair_scale(uint32_t m, bool v) { return __byte_perm(m, 0, v ? 0x3232 : 0x1010) & 0xfff0fff0u; }
__device__ __forceinline__ uint32_t pair_zero(uint32_t m, bool v) {
  return ((__byte_perm(m, 0, v ? 0x3232 : 0x1010) << 3) & 0x00780078u) | 0x41804180u;
}

// mbar_wait that sleeps: most warps wait for a good part of the time, and what a polling
// one issues is taken from those that work.  The two warps that start the products poll:
// their waits are on the chain (1485 us instead of 1537).
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
  constexpr uint32_t kNap = 100000;                    // ns that one attempt may take
  for (uint64_t i = 0; i <= kWaitLimitNs / kNap; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kNap)
        : "memory");
    if (ok) return true;
  }
  return false;
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
// Pages are read by many CTAs.
__device__ __forceinline__ uint64_t l2_policy_evict_last() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}

constexpr int kSoftmaxThreads = 2 * kBM;
__device__ __forceinline__ void softmax_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}

template <int kRegs, bool kMore>
__device__ __forceinline__ void set_registers() {
  if constexpr (kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Key tiles that a part of the keys has about, and the parts of all token blocks (one
// warp calls).  Every lane thinks one length of parts through, and the least time is
// taken: that of whole waves of equal parts, or of the longest.  There are then no more
// parts than CTAs: the host launched one for each of split_from blocks, and split_parts
// more (or what the shortest parts allow).  (More blocks than that, in sequences that
// overlap: no parts, so nobody waits for one that is not there.)
__device__ __forceinline__ int2 plan_parts(const Int4AttnParams &p, int tokens, int lane) {
  constexpr int kWhole = 1 << 30;
  long long work = 0, ctas = 0;
  for (int s = lane; s < p.num_seqs; s += 32) {
    const Request r = request(p, s);
    const int n = request_ctas(r, tokens);
    ctas += n;
    if (!r.bad) work += static_cast<long long>(n) * cdiv(r.kv_len, kBN);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, off);
    ctas += __shfl_xor_sync(0xffffffffu, ctas, off);
  }
  if (ctas > p.split_from || work == 0) return make_int2(kWhole, kWhole);
  const long long aim = p.split_parts * static_cast<long long>(lane + 2);        // of 32
  const int mine = lane == 31 ? kWhole
                              : max(kPartTiles, static_cast<int>(min((32 * work + aim - 1) / aim,
                                                                     static_cast<long long>(kWhole))));
  int n = 0, longest = 0, bad = 0;
  for (int s = 0; s < p.num_seqs; ++s) {
    const Request r = request(p, s);
    if (r.bad) {
      ++bad;
      continue;
    }
    // (the keys of a request without new tokens are nobody's work)
    const int tiles = r.q_len > 0 ? cdiv(r.kv_len, kBN) : 0, cut = max(1, cdiv(tiles, mine));
    n += request_ctas(r, tokens) * cut;
    longest = max(longest, cdiv(tiles, cut));
  }
  const float waves = ceilf(static_cast<float>(n) * p.num_kv_heads / p.sms);
  const float cost = mine == kWhole ? 0.f : kPartCost;
  const float time = fmaxf(waves * (static_cast<float>(work) / n + cost), longest + cost);
  const unsigned best = __reduce_min_sync(0xffffffffu, __float_as_uint(time));   // (positive: ordered as integers)
  const int at = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(time) == best)) - 1;
  return make_int2(__shfl_sync(0xffffffffu, mine, at), bad + __shfl_sync(0xffffffffu, n, at));
}

// A number that is the same in all lanes, known to be so: addresses and branches made of
// the warp's number then take no registers of the lanes (100 bytes spilled
// without; 490 us to 478 for 2 x 2048 tokens on 6000).
__device__ __forceinline__ int uniform(int x) {
  return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(x)));
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
int4_prefill_kernel(const __grid_constant__ Int4AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int tile_tokens = kBM / p.group, tokens = 2 * tile_tokens;

  // ---- this CTA's request, tokens and part of the keys.  CTAs are numbered through
  // request by request; the last ones, whose rows see the most keys, are launched first.
  const int kvh = static_cast<int>(blockIdx.x % p.num_kv_heads);
  int numbers = static_cast<int>(gridDim.x / p.num_kv_heads);
  int part_tiles = 0;                                  // key tiles that a part has about
  bool leftover = p.cu_seqlens_q != nullptr;           // whether there may be more blocks than CTAs
  if constexpr (kSplit) {
    if (warp == 0) {
      const int2 plan = plan_parts(p, tokens, lane);
      if (lane == 0) {
        bar.part_tiles = plan.x;
        bar.numbers = plan.y;
      }
    }
    __syncthreads();
    part_tiles = bar.part_tiles;
    leftover = leftover && bar.numbers > numbers;      // (a plan has counted them)
    numbers = min(bar.numbers, numbers);
  }
  // parts of a request's every token block
  auto request_parts = [&](const Request &r) { return kSplit && !r.bad ? max(1, cdiv(cdiv(r.kv_len, kBN), part_tiles)) : 1; };
  const int global = numbers - 1 - static_cast<int>(blockIdx.x / p.num_kv_heads);
  if (global < 0) return;
  int number = global, seq = -1;
  if (p.num_seqs <= kFewRequests) {                    // every warp by itself
    for (int s0 = 0; s0 < p.num_seqs && seq < 0; s0 += 32) {
      const int s = s0 + lane;
      int mine = 0;
      if (s < p.num_seqs) {
        const Request r = request(p, s);
        mine = request_ctas(r, tokens) * request_parts(r);
      }
      int upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, upto > number);
      if (hit) {
        const int at = __ffs(hit) - 1;
        seq = s0 + at;
        number -= __shfl_sync(0xffffffffu, upto - mine, at);
      } else {
        number -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  } else {
    // every thread counts the CTAs of a few requests in a row; the one in whose requests
    // this CTA falls finds the very one
    const int per = cdiv(p.num_seqs, kThreads), s0 = threadIdx.x * per, s1 = min(s0 + per, p.num_seqs);
    auto ctas = [&](int s) {
      const Request r = request(p, s);
      return request_ctas(r, tokens) * request_parts(r);
    };
    long long mine = 0;
    for (int s = s0; s < s1; ++s) mine += ctas(s);
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) bar.scan[warp] = upto;
    if (threadIdx.x == 0) bar.seq = -1;
    __syncthreads();
    long long left = global - (upto - mine);           // CTAs from this thread's first on
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
      if (w < warp) left -= bar.scan[w];
    if (left >= 0 && left < mine) {
      int s = s0;
      while (true) {
        const int n = ctas(s);
        if (left < n) break;
        left -= n;
        ++s;
      }
      bar.seq = s;
      bar.number = static_cast<int>(left);
    }
    __syncthreads();
    seq = bar.seq;
    number = bar.number;
  }
  if (seq < 0) return;                                 // fewer than the host allowed for
  const Request rq = request(p, seq);
  const int parts = request_parts(rq);
  if (leftover && global == numbers - 1) {
    // Sequences that fall back and overlap can hold more rows than the launch has CTAs
    // for: nobody comes to those behind this CTA's, and they become NaN.  (Of prefix sums
    // there are none: a CTA with this number then has the last rows of all, if it has any.)
    const int done = rq.bad ? rq.q_len : (number / parts + 1) * tokens;
    if (done < rq.q_len) spoil_rows(p, kvh, rq.q_start + done, rq.q_len - done);
    for (int s = seq + 1; s < p.num_seqs; ++s) {
      const Request r = request(p, s);
      spoil_rows(p, kvh, r.q_start, r.q_len);
    }
  }
  if (rq.bad) {
    spoil_rows(p, kvh, rq.q_start, rq.q_len);
    return;
  }
  const int part = kSplit ? number % parts : 0;
  const int tok0 = (kSplit ? number / parts : number) * tokens;      // first token of this CTA
  const int shift = rq.kv_len - rq.q_len;              // keys before the new tokens
  // rows and key tiles of either tile (tile 1 may have none)
  int rows[2], ntiles[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int n = min(max(rq.q_len - tok0 - x * tile_tokens, 0), tile_tokens);
    rows[x] = n * p.group;
    const int keys = p.tree_mask ? rq.kv_len : shift + tok0 + x * tile_tokens + n;
    ntiles[x] = n > 0 ? cdiv(keys, kBN) : 0;
  }
  // keys before this CTA's part (keys, pages and key tiles are counted from there on); CTAs
  // that share its rows
  int first_key = 0, shared_by = 1;
  if constexpr (kSplit) {
    const int all = max(ntiles[0], ntiles[1]), each = cdiv(all, parts);
    const int first_tile = part * each;
    first_key = first_tile * kBN;
    shared_by = cdiv(all, each);
    if (part >= shared_by) return;                     // uniform over the CTA
#pragma unroll
    for (int x = 0; x < 2; ++x) ntiles[x] = min(max(ntiles[x] - first_tile, 0), each);
  }
  const int n_tiles = max(ntiles[0], ntiles[1]), both = min(ntiles[0], ntiles[1]);
  // number of the product of key tile j and query tile x
  auto product = [&](int j, int x) { return j < both ? 2 * j + x : both + j; };
  auto sK = [&](int s) { return smem + kOffK + s * kTileBytes; };
  auto sV = [&](int s) { return smem + kOffV + s * kTileBytes; };

  if (warp == kPvWarp) {
    tmem_alloc(&bar.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // Packed pages of key tile j into their ring, once its slot has been unpacked (all
  // lanes of the loading warp call; lanes 0..7 copy a page each).
  const int npages = cdiv(rq.kv_len - first_key, kPageSize);
  const int32_t *table = p.page_table + static_cast<size_t>(seq) * p.max_pages_per_seq + first_key / kPageSize;
  auto page_id = [&](int j) {
    const int page = j * kPages + lane;
    return lane < kPages && page < npages ? __ldg(table + page) : -1;
  };
  const uint64_t policy = l2_policy_evict_last();
  auto load_raw = [&](int j, int id) -> bool {
    const int s = j % kRaw;
    if (j >= kRaw && !__all_sync(0xffffffffu, wait(&bar.raw_empty[s], (j / kRaw + 1) & 1))) return false;
    const bool ok = id >= 0 && id < p.num_pages;
    if (lane < kPages && j * kPages + lane < npages && !ok) atomicOr(&bar.bad, 1);
    const unsigned good = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) mbar_arrive_expect_tx(&bar.raw_full[s], __popc(good) * kInt4Block);
    __syncwarp();
    if (ok) {
      bulk_load(smem + kOffRaw + (s * kPages + lane) * kInt4Block,
                p.kv_cache + (static_cast<size_t>(id) * p.num_kv_heads + kvh) * kInt4Block, kInt4Block,
                &bar.raw_full[s], policy);
    }
    return true;
  };
  if (warp == kLoadWarp) {
   if (lane == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&bar.raw_full[s], 1);
      mbar_init(&bar.raw_empty[s], kPages);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.kv_full[s], kPages);
      mbar_init(&bar.kv_empty[s], 1);
    }
    for (int b = 0; b < kBuffers; ++b) {
      mbar_init(&bar.s_full[b], 1);
      mbar_init(&bar.p_full[b], kBM);
      mbar_init(&bar.p_used[b], 1);
    }
    bar.bad = 0;
    if constexpr (kSplit) {
      bar.shared_by = shared_by;
      bar.part = part;
      bar.first = global - part;
    }
    fence_mbar_init();
   }
   __syncwarp();
   for (int j = 0; j < min(kRaw, n_tiles); ++j) load_raw(j, page_id(j));      // fresh slots: no waits
  }
  // Q, its dims permuted as the codes' are; rows of nobody are zero
  {
    constexpr int kChunks = 2 * kBM * (kHeadDim / 8), kEach = (kChunks + kThreads - 1) / kThreads;
    uint4 q[kEach];                                    // (all loads at once)
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      const int i = threadIdx.x + n * kThreads, r = i / (kHeadDim / 8), c = i % (kHeadDim / 8);
      const int x = r / kBM, rr = r % kBM;
      q[n] = make_uint4(0, 0, 0, 0);
      if (i < kChunks && rr < (x ? rows[1] : rows[0])) {
        const int token = rq.q_start + tok0 + x * tile_tokens + rr / p.group;
        q[n] = __ldg(reinterpret_cast<const uint4 *>(p.q) +
                     (static_cast<size_t>(token) * p.num_qo_heads + kvh * p.group + rr % p.group) * (kHeadDim / 8) + c);
      }
    }
#pragma unroll
    for (int n = 0; n < kEach; ++n) {
      const int i = threadIdx.x + n * kThreads, r = i / (kHeadDim / 8), c = i % (kHeadDim / 8);
      if (i < kChunks)
        *reinterpret_cast<uint4 *>(smem + kOffQ + r * 128 + ((c ^ (r & 7)) << 4)) =
            make_uint4(__byte_perm(q[n].x, q[n].z, 0x5410), __byte_perm(q[n].x, q[n].z, 0x7632),
                       __byte_perm(q[n].y, q[n].w, 0x5410), __byte_perm(q[n].y, q[n].w, 0x7632));
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp >= kUnpackWarp && warp < kUnpackWarp + kUnpackWarps) {
    // --------------------------------------------------- packed pages to tiles
    set_registers<kOtherRegs, false>();
    const int uw = warp - kUnpackWarp;                 // this warp's page of every tile
    const int g = lane >> 2, t = lane & 3;
    const int keys = rq.kv_len - first_key - uw * kPageSize;
    uint32_t mask, sixteen;
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(sixteen));
    // Stores of eight lanes fall into different banks: every other row of K has its
    // second chunk first.
    const int odd_row = g & 1;
    const uint32_t k_first = g * 128 + (((t + 4 * odd_row) ^ g) << 4), k_second = g * 128 + (((t + 4 - 4 * odd_row) ^ g) << 4);
    const uint32_t v_even = 2 * t * 128 + ((g ^ (2 * t)) << 4), v_odd = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4);

    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int s = j % kStages, raw = j % kRaw;
      if (!__all_sync(0xffffffffu, wait(&bar.raw_full[raw], (j / kRaw) & 1))) {
        ok = false;
        break;
      }
      const uint8_t *block = smem + kOffRaw + (raw * kPages + uw) * kInt4Block;
      const uint4 kw = *(reinterpret_cast<const uint4 *>(block + kInt4K) + lane);
      const uint4 vw = *(reinterpret_cast<const uint4 *>(block + kInt4V) + lane);
      uint2 km = *(reinterpret_cast<const uint2 *>(block + kInt4Meta) + g);      // keys g, g + 8
      uint4 vm = *(reinterpret_cast<const uint4 *>(block + kInt4Meta) + t);      // keys 2t, 2t + 8, 2t + 1, 2t + 9
      const uint32_t own = *reinterpret_cast<const uint32_t *>(block + kInt4Meta + 8 * (lane & 7) + 4 * ((lane >> 3) & 1));
      // Odd keys of the page (`own` is that of lanes 0..15): those past the last one
      // become zeros, and a value that is not finite zeros with a key that is not finite.
      const unsigned odd = __ballot_sync(0xffffffffu, (own & 0x7f800000u) == 0x7f800000u) & 0xffffu;
      const int live = keys - j * kBN;
      if (odd != 0 || live < kPageSize) {
        const unsigned gone = live >= kPageSize ? 0u : live <= 0 ? 0xffffu : 0xffffu & (0xffffu << live);
        auto k = [&](uint32_t &m, int key) {
          if (odd >> key & 1) m |= 0x7fc0u;
          if (gone >> key & 1) m = 0;
        };
        auto v = [&](uint32_t &m, int key) {
          if ((odd | gone) >> key & 1) m = 0;
        };
        k(km.x, g);
        k(km.y, g + 8);
        v(vm.x, 2 * t);
        v(vm.y, 2 * t + 8);
        v(vm.z, 2 * t + 1);
        v(vm.w, 2 * t + 9);
      }
      if (j >= kStages && !__all_sync(0xffffffffu, wait(&bar.kv_empty[s], (j / kStages + 1) & 1))) {
        ok = false;
        break;
      }
      uint8_t *ka = sK(s) + uw * (kPageSize * 128), *va = sV(s) + uw * (kPageSize * 128);
#pragma unroll
      for (int h = 0; h < 2; ++h) {                    // keys g, g + 8
        const uint32_t m = h ? km.y : km.x;
        const uint32_t s2 = pair_scale(m, false), z2 = pair_zero(m, false);
        const uint32_t w0 = h ? kw.z : kw.x, w1 = h ? kw.w : kw.y;
        *reinterpret_cast<uint4 *>(ka + h * 1024 + k_first) = values(odd_row ? w1 : w0, s2, z2, mask, sixteen);
        *reinterpret_cast<uint4 *>(ka + h * 1024 + k_second) = values(odd_row ? w0 : w1, s2, z2, mask, sixteen);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {                    // keys 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t m = i == 0 ? vm.x : i == 1 ? vm.z : i == 2 ? vm.y : vm.w;
        const uint32_t w = i == 0 ? vw.x : i == 1 ? vw.y : i == 2 ? vw.z : vw.w;
        *reinterpret_cast<uint4 *>(va + (i >> 1) * 1024 + (i & 1 ? v_odd : v_even)) =
            values(__funnelshift_l(w, w, 3), pair_scale(m, true), pair_zero(m, true), mask, sixteen);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.kv_full[s]);
        mbar_arrive(&bar.raw_empty[raw]);
      }
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------------ Q K^T
    set_registers<kOtherRegs, false>();
    bool ok = true;
    int made = 0;                                      // products
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.kv_full[s], (j / kStages) & 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || j >= ntiles[x]) continue;
        const int n = product(j, x), b = n % kBuffers;
        if (n >= kBuffers) ok = __all_sync(0xffffffffu, mbar_wait(&bar.p_used[b], (n / kBuffers + 1) & 1));
        if (!ok) continue;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dq = umma_desc_sw128(smem_u32(smem + kOffQ + x * kTileBytes), 16, 1024);
          const uint64_t dk = umma_desc_sw128(smem_u32(sK(s)), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)
            umma_ss(tmem + b * kBN, dq + 2 * kk, dk + 2 * kk, kIdescQK, kk > 0);
          umma_commit(&bar.s_full[b]);
        }
        made = n + 1;
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(&bar.bad, 1);
      if (made > 0) mbar_wait(&bar.s_full[(made - 1) % kBuffers], ((made - 1) / kBuffers) & 1);
    }
  } else if (warp == kPvWarp) {
    // -------------------------------------------------------------------- P V
    // (its V is there when P is: S was made after K and V of the key tile had come)
    set_registers<kOtherRegs, false>();
    bool ok = true;
    int made = 0;
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kStages;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || j >= ntiles[x]) continue;
        const int n = product(j, x), b = n % kBuffers;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.p_full[b], (n / kBuffers) & 1));
        if (!ok) continue;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dv = umma_desc_sw128(smem_u32(sV(s)), kTileBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)        // 16 keys = 2 KB
            umma_ts(tmem + kColO + x * kHeadDim, tmem + b * kBN + 8 * kk, dv + (2048 >> 4) * kk, kIdescPV,
                    (j > 0) || (kk > 0));
          umma_commit(&bar.p_used[b]);
        }
        made = n + 1;
        __syncwarp();
      }
      if (ok && lane == 0) umma_commit(&bar.kv_empty[s]);
      __syncwarp();
    }
    if (!ok) {
      if (lane == 0) atomicOr(&bar.bad, 1);
      if (made > 0) mbar_wait(&bar.p_used[(made - 1) % kBuffers], ((made - 1) / kBuffers) & 1);
    }
  } else if (warp < kUnpackWarp) {
    // ---------------------------------------------------------------- softmax
    set_registers<kSoftmaxRegs, true>();
    const int x = warp >> 2;
    const int r = threadIdx.x & (kBM - 1);             // row = tensor-memory lane
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t to = trow + kColO + x * kHeadDim;
    const int i = tok0 + x * tile_tokens + r / p.group;       // token within the request
    const int head = kvh * p.group + r % p.group;
    const bool live = r < rows[x];
    Seen seen;
    seen.limit = min(shift + i + 1, rq.kv_len) - first_key;
    seen.draft = shift - first_key;
    seen.vis = nullptr;
    if (p.tree_mask) {
      seen.limit = shift - first_key;
      seen.vis = &bar.vis[threadIdx.x];
      bar.vis[threadIdx.x] = live ? p.tree_mask[static_cast<size_t>(seq) * p.q_len + i] & (~0ull >> (64 - p.q_len)) : 0;
    }
    const float sl2 = p.scale_log2;
    // a sink that is no logit (NaN, +inf) spoils the sum, not the reference
    float m = kUnset, d = 0.f;
    if (live && first_key == 0) {
      const float logit = __ldg(p.sinks + head) * kLog2e;
      if (logit < INFINITY) {
        m = fmaxf(logit, kUnset);
        d = logit < kUnset ? 0.f : 1.f;
      } else {
        d = NAN;
      }
    }
    bool ok = true;
    const int mine = ntiles[x];
    for (int j = 0; j < mine; ++j) {
      const int n = product(j, x), b = n % kBuffers;
      if (!__all_sync(0xffffffffu, wait(&bar.s_full[b], (n / kBuffers) & 1))) { ok = false; break; }
      tc_fence_after();
      const int key0 = j * kBN;
      const uint32_t ts = trow + b * kBN;
      const bool edge = __any_sync(0xffffffffu, key0 + kBN > seen.limit);
      uint32_t y[4][16];
      // a reference that is not set at all needs no try
      const bool unset = j == 0 && __any_sync(0xffffffffu, m == kUnset);
      float sum = unset ? INFINITY : edge ? weigh_tile<true>(ts, sl2, m, seen, key0, y) : weigh_tile<false>(ts, sl2, m, seen, key0, y);
      if (__any_sync(0xffffffffu, !(sum <= kMostSum))) {
        // some reference is too small: the rows' maxima, and the tile again
        const float mx = row_max(ts, sl2, seen, key0);
        const float now = fmaxf(m, mx);
        const float alpha = ex2(m - now);
        m = now;
        d *= alpha;
        if (j > 0) {
          const int before = product(j - 1, x);
          if (!__all_sync(0xffffffffu, wait(&bar.p_used[before % kBuffers], (before / kBuffers) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          scale_o(to, alpha);
        }
        sum = weigh_tile<true>(ts, sl2, m, seen, key0, y);
      }
      d += sum;
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_st16(ts + 16 * c, y[c]);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bar.p_full[b]);
    }
    if (mine > 0 && ok) {
      const int last = product(mine - 1, x);
      ok = __all_sync(0xffffffffu, wait(&bar.p_used[last % kBuffers], (last / kBuffers) & 1));
    }
    tc_fence_after();
    if (!ok) atomicOr(&bar.bad, 1);
    uint32_t o[2][32];
    if (mine > 0 && ok) {
      tmem_ld32(to, o[0]);
      tmem_ld32(to + 32, o[1]);
      tmem_ld_wait32(o[0]);
      reg_tie32(o[1]);
    }
    tc_fence_before();
    __syncthreads();
    const bool failed = bar.bad != 0;
    if constexpr (kSplit) {
      const int shared_by = bar.shared_by, part = bar.part, first = bar.first;
      if (shared_by > 1) {
        // This part's sums to the workspace; the last of the CTAs that share the rows
        // joins them, in the keys' order, and leaves the counter at zero.  Sums of a
        // row: 16 vectors of four, rows next to each other.
        constexpr int kVectors = kHeadDim / 4;
        const int row = threadIdx.x;
        auto slot = [&](int c) { return static_cast<size_t>(first + c) * p.num_kv_heads + kvh; };
        float4 *ws_o = reinterpret_cast<float4 *>(p.ws_o);
        if (live) {
          const bool any = mine > 0 && ok;
          float4 *dst = ws_o + slot(part) * kVectors * kSoftmaxThreads + row;
#pragma unroll
          for (int c = 0; c < kVectors; ++c) {
            auto sum = [&](int e) { return any ? __uint_as_float(o[(4 * c + e) >> 5][(4 * c + e) & 31]) : 0.f; };
            dst[c * kSoftmaxThreads] = make_float4(sum(0), sum(1), sum(2), sum(3));
          }
          p.ws_md[slot(part) * kSoftmaxThreads + row] = make_float2(m, failed ? NAN : d);
        }
        softmax_barrier();
        int *counter = p.counters + slot(0);
        if (threadIdx.x == 0) bar.last = atomic_add_acq_rel(counter, 1) == shared_by - 1;
        softmax_barrier();
        if (!bar.last) return;
        if (threadIdx.x == 0) *counter = 0;
        if (live) {
          m = kUnset;
          for (int c = 0; c < shared_by; ++c) m = fmaxf(m, __ldcg(&p.ws_md[slot(c) * kSoftmaxThreads + row]).x);
          d = 0.f;
#pragma unroll
          for (int i = 0; i < kHeadDim; ++i) o[i >> 5][i & 31] = 0;
#pragma unroll 1
          for (int c = 0; c < shared_by; ++c) {
            const float2 md = __ldcg(&p.ws_md[slot(c) * kSoftmaxThreads + row]);
            const float4 *src = ws_o + slot(c) * kVectors * kSoftmaxThreads + row;
            const float w = ex2(md.x - m);
            d = fmaf(w, md.y, d);
#pragma unroll
            for (int v = 0; v < kVectors; ++v) {
              const float4 a = __ldcg(src + v * kSoftmaxThreads);
              const float f[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t &to_sum = o[(4 * v + e) >> 5][(4 * v + e) & 31];
                to_sum = __float_as_uint(fmaf(w, f[e], __uint_as_float(to_sum)));
              }
            }
          }
        }
      }
    }
    // rows through shared memory (Q's place), so that a warp stores whole lines
    const float inv = failed ? NAN : d == 0.f ? 0.f : 1.f / d;           // (a part that failed made d NaN)
    uint8_t *mine_out = smem + kOffQ + threadIdx.x * 128;
#pragma unroll
    for (int c = 0; c < kHeadDim / 8; ++c) {
      // column 8c + 2j holds dim 8c + j, column 8c + 2j + 1 dim 8c + 4 + j
      auto dim = [&](int e) {
        const int col = 8 * c + 2 * (e & 3) + (e >> 2);
        return failed ? NAN : __uint_as_float(o[col >> 5][col & 31]) * inv;
      };
      *reinterpret_cast<uint4 *>(mine_out + ((c ^ (r & 7)) << 4)) =
          make_uint4(pack_bf16(dim(0), dim(1)), pack_bf16(dim(2), dim(3)), pack_bf16(dim(4), dim(5)),
                     pack_bf16(dim(6), dim(7)));
    }
    if (live && p.lse)
      p.lse[static_cast<size_t>(rq.q_start + i) * p.num_qo_heads + head] =
          failed ? NAN : d == 0.f ? -INFINITY : (m + lg2(d)) * kLn2;
    __syncwarp();
#pragma unroll 4
    for (int n = 0; n < 8; ++n) {
      const int rr = (warp & 3) * 32 + 4 * n + (lane >> 3), c = lane & 7;       // row of the tile
      if (rr < rows[x]) {
        const size_t row = static_cast<size_t>(rq.q_start + tok0 + x * tile_tokens + rr / p.group) * p.num_qo_heads +
                           kvh * p.group + rr % p.group;
        *reinterpret_cast<uint4 *>(p.out + row * kHeadDim + 8 * c) =
            *reinterpret_cast<const uint4 *>(smem + kOffQ + (x * kBM + rr) * 128 + ((c ^ (rr & 7)) << 4));
      }
    }
    return;
  } else {
    set_registers<kOtherRegs, false>();                // the last warpgroup's other two warps
    if (warp == kLoadWarp) {
      bool ok = true;
      int id = page_id(kRaw), asked = min(kRaw, n_tiles);
      for (int j = kRaw; ok && j < n_tiles; ++j) {
        const int next = page_id(j + 1);
        ok = load_raw(j, id);
        if (ok) asked = j + 1;
        id = next;
      }
      if (!ok && lane == 0) atomicOr(&bar.bad, 1);
      // no copy is in flight when the CTA ends, whoever gave up
      for (int j = max(asked - kRaw, 0); j < asked; ++j) wait(&bar.raw_full[j % kRaw], (j / kRaw) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();          // the softmax warps have read O: tensor memory is free
  if (warp == kPvWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int int4_prefill_tokens(int group) { return 2 * (kBM / group); }

size_t int4_prefill_results_bytes(int ctas) {
  return static_cast<size_t>(ctas) * kSoftmaxThreads * (kHeadDim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_int4_prefill(const Int4AttnParams &p, long long ctas, cudaStream_t stream) {
  static_assert(kSmemBytes > 114 * 1024 && kSmemBytes <= 227 * 1024, "one CTA per SM");
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto kernel = p.split_parts > 0 ? int4_prefill_kernel<true> : int4_prefill_kernel<false>;
  cudaError_t err = p.split_parts > 0 ? set_smem_once<int4_prefill_kernel<true>>(kSmemBytes)
                                      : set_smem_once<int4_prefill_kernel<false>>(kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, static_cast<unsigned>(ctas), kThreads, kSmemBytes, stream, false, p);
}

}  // namespace sa
