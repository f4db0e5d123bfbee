// Many query rows per KV head over a paged cache held in 4 bits (chunked prefill, draft
// trees), learned sinks, on the 5th-generation tensor cores.
//
// Mathematics: row (token i, head h) of a request with kv_len keys of which the last
// q_len are its new tokens sees keys j <= kv_len - q_len + i (or the draft keys that its
// mask names); softmax with the sink as one more term, as in plain prefill.  The keys'
// and values' codes become bf16 numbers s (n - z) on the way into shared memory, which
// is exact; P is rounded to bf16 for the product with V, out once.
//
// One CTA per SM = the rows of 2 * (128 / group) tokens of one KV head, ordered (token,
// head), as two 128-row tiles that share every K and V tile of 128 keys: turning a tile
// of codes into bf16 costs half of what it would for one, and one tile's products run
// during the other's softmax.
//   warps 8..15   packed pages from global memory into registers, a tile ahead; codes
//                 to bf16 (shift, mask under the exponent of 16, subtract 16 + z,
//                 multiply by s); stores into K and V rings in the swizzled layout.
//                 A word of codes gives dims (0 4 1 5 2 6 3 7) of a group of eight in
//                 that order: Q is permuted likewise, O's columns are put right at the end.
//   warp 16       S = Q K^T for either tile as soon as its last S has been used
//   warp 17       O += P V for either tile
//   warps 0..7    softmax, one thread per row.  Scores come 32 at a time and are not
//                 compared: P = 2^(s - m) with the row's reference m, and only if a
//                 tile's sum shows that m has become too small (or is not set) the
//                 row's maximum is taken and the tile done once more.  Scores beyond
//                 the causal limit are left out by index.
// A value row that is not finite must spoil the rows that see it and no others, but
// 0 * NaN in P V would spoil the whole tile: such a value is stored as zero and its key
// as NaN, so the rows that see it get there by their score (and their lse is NaN, too).

#include "int4.cuh"
#include "ptx.cuh"

#include <cmath>

namespace sa {
namespace {

constexpr int kBM = 128;                       // rows per tile
constexpr int kBN = 128;                       // keys per K / V tile
constexpr int kStages = 3;                     // of the K ring and of the V ring
constexpr int kTileBytes = kBN * kHeadDim * 2; // 16 KB
constexpr int kThreads = 640;                  // five warpgroups
constexpr int kUnpackWarp = 8, kUnpackWarps = 8, kQkWarp = 16, kPvWarp = 17;
// Registers per thread: the launch has 96 for all; softmax warps take from the others.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 144, kOtherRegs = 64;
static_assert(2 * kSoftmaxRegs + 3 * kOtherRegs <= 5 * kLaunchRegs, "the split fits the launch's registers");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192, kColTile = 256;   // of tile 0; tile 1 kColTile on
constexpr float kUnset = -8e37f;               // reference of a row that has seen no key yet
constexpr float kMostSum = 1024.f;             // sum of a tile's P from which the reference is moved

constexpr int kOffQ = 0;                       // two tiles
constexpr int kOffK = 2 * kTileBytes;
constexpr int kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffBars = kOffV + kStages * kTileBytes;

struct Bars {
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t s_full[2];      // S of the tile's current keys is in tensor memory
  uint64_t p_full[2];      // P is, and S has been used
  uint64_t pv_done[2];     // P has been used and O holds the keys so far
  uint32_t tmem_base;
  int bad;
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

// A row's keys [0, limit), and the draft keys from `draft` on by the bits of `vis`.
struct Seen {
  int limit, draft;
  uint64_t vis;
  __device__ __forceinline__ bool operator()(int key) const {
    if (key < limit) return true;
    const unsigned u = static_cast<unsigned>(key - draft);
    return u < 64u && ((vis >> u) & 1);
  }
};

// P = 2^(s * scale - m) for 32 scores as bf16 pairs in x[0..15]; their sums in acc.
template <bool kMask>
__device__ __forceinline__ void weigh(uint32_t (&x)[32], uint64_t scale2, uint64_t negm2, const Seen &seen,
                                      int key0, uint64_t &acc0, uint64_t &acc1) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale2, negm2), a, b);
    if constexpr (kMask) {
      if (!seen(key0 + 2 * e)) a = -INFINITY;
      if (!seen(key0 + 2 * e + 1)) b = -INFINITY;
    }
    const float pa = ex2(a), pb = ex2(b);
    if (e & 1) acc1 = f2_add(acc1, f2_pack(pa, pb));
    else acc0 = f2_add(acc0, f2_pack(pa, pb));
    x[e] = pack_bf16(pa, pb);
  }
}

__device__ __forceinline__ void store_p(uint32_t taddr, const uint32_t (&x)[32]) {
  tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(&x[0]));
}

// All 128 scores of this thread's row against its reference m: P into tensor memory once
// the previous P has been used.  Returns the row's sum, or a negative number if a wait
// timed out.
template <bool kMask>
__device__ __forceinline__ float weigh_tile(uint32_t trow, float sl2, float m, const Seen &seen, int key0,
                                            uint64_t *pv_done, int parity) {
  const uint64_t scale2 = f2_pack(sl2, sl2), negm2 = f2_pack(-m, -m);
  uint64_t acc0 = 0, acc1 = 0;
  uint32_t x0[32], x1[32], x2[32];
  tmem_ld32(trow + kColS, x0);
  tmem_ld_wait32(x0);
  tmem_ld32(trow + kColS + 32, x1);
  weigh<kMask>(x0, scale2, negm2, seen, key0, acc0, acc1);
  tmem_ld_wait32(x1);
  tmem_ld32(trow + kColS + 64, x2);
  weigh<kMask>(x1, scale2, negm2, seen, key0 + 32, acc0, acc1);
  bool ok = true;
  if (parity >= 0) ok = __all_sync(0xffffffffu, mbar_wait(pv_done, parity));
  tc_fence_after();
  store_p(trow + kColP, x0);
  store_p(trow + kColP + 16, x1);
  tmem_ld_wait32(x2);
  tmem_ld32(trow + kColS + 96, x0);
  weigh<kMask>(x2, scale2, negm2, seen, key0 + 64, acc0, acc1);
  store_p(trow + kColP + 32, x2);
  tmem_ld_wait32(x0);
  weigh<kMask>(x0, scale2, negm2, seen, key0 + 96, acc0, acc1);
  store_p(trow + kColP + 48, x0);
  tmem_st_wait();
  float a, b;
  f2_unpack(f2_add(acc0, acc1), a, b);
  return ok ? a + b : -1.f;
}

// Largest scaled score of this thread's row among the keys that it sees.
__device__ __forceinline__ float row_max(uint32_t trow, float sl2, Seen seen, int key0) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_ld32(trow + kColS + 32 * c, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      mx = fmaxf(mx, seen(key0 + 32 * c + e) ? __uint_as_float(x[e]) * sl2 : -INFINITY);
  }
  return mx;
}

__device__ __forceinline__ void scale_o(uint32_t trow, float alpha) {
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t x[32];
    tmem_ld32(trow + kColO + 32 * h, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
    tmem_st16(trow + kColO + 32 * h, *reinterpret_cast<uint32_t(*)[16]>(&x[0]));
    tmem_st16(trow + kColO + 32 * h + 16, *reinterpret_cast<uint32_t(*)[16]>(&x[16]));
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

// One page's share of a lane: unit (g, t) of K and of V, and the scales it needs.
struct Packed {
  uint4 k, v, vm;        // vm: keys 2t, 2t + 8, 2t + 1, 2t + 9
  uint2 km;              // keys g, g + 8
  uint32_t own;          // key `lane` (of lanes 0..15), to be looked at for odd values
};

template <int kRegs, bool kMore>
__device__ __forceinline__ void set_registers() {
  if constexpr (kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__global__ void __launch_bounds__(kThreads, 1)
int4_prefill_kernel(const __grid_constant__ Int4AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_tokens = kBM / p.group, tokens = 2 * tile_tokens;

  // ---- this CTA's request and tokens.  CTAs are numbered through request by request;
  // the last ones, whose rows see the most keys, are launched first.
  const int kvh = static_cast<int>(blockIdx.x % p.num_kv_heads);
  int number = static_cast<int>(gridDim.x / p.num_kv_heads) - 1 - static_cast<int>(blockIdx.x / p.num_kv_heads);
  int seq = -1;
  Request rq;
  for (int s0 = 0; s0 < p.num_seqs && seq < 0; s0 += 32) {
    const int s = s0 + lane;
    const int mine = s < p.num_seqs ? request_ctas(request(p, s), tokens) : 0;
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
  if (seq < 0) return;                                 // fewer than the host allowed for
  rq = request(p, seq);
  if (rq.bad) {
    // this request's rows, as far as they lie inside the buffers
    if (rq.q_start < 0 || rq.q_start >= p.total_q) return;
    const int rows = min(max(rq.q_len, 0), p.total_q - rq.q_start) * p.group;
    for (int i = threadIdx.x; i < rows; i += kThreads) {
      const size_t row = static_cast<size_t>(rq.q_start + i / p.group) * p.num_qo_heads + kvh * p.group + i % p.group;
      uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kHeadDim);
#pragma unroll
      for (int c = 0; c < kHeadDim / 8; ++c) dst[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
      if (p.lse) p.lse[row] = NAN;
    }
    return;
  }
  const int tok0 = number * tokens;                    // first token of this CTA
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
  const int n_tiles = max(ntiles[0], ntiles[1]);
  auto sK = [&](int s) { return smem + kOffK + s * kTileBytes; };
  auto sV = [&](int s) { return smem + kOffV + s * kTileBytes; };

  if (warp == kPvWarp) {
    tmem_alloc(&bar.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kQkWarp && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.k_full[s], 32 * kUnpackWarps);
      mbar_init(&bar.k_empty[s], 1);
      mbar_init(&bar.v_full[s], 32 * kUnpackWarps);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar.s_full[x], 1);
      mbar_init(&bar.p_full[x], kBM);
      mbar_init(&bar.pv_done[x], 1);
    }
    bar.bad = 0;
    fence_mbar_init();
  }
  // Q, its dims permuted as the codes' are; rows of nobody are zero
  for (int i = threadIdx.x; i < 2 * kBM * (kHeadDim / 8); i += kThreads) {
    const int r = i / (kHeadDim / 8), c = i % (kHeadDim / 8);
    const int x = r / kBM, rr = r % kBM;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (rr < rows[x]) {
      const int token = rq.q_start + tok0 + x * tile_tokens + rr / p.group;
      const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p.q) +
                            (static_cast<size_t>(token) * p.num_qo_heads + kvh * p.group + rr % p.group) * (kHeadDim / 8) + c);
      w = make_uint4(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632), __byte_perm(q.y, q.w, 0x5410),
                     __byte_perm(q.y, q.w, 0x7632));
    }
    *reinterpret_cast<uint4 *>(smem + kOffQ + r * 128 + ((c ^ (r & 7)) << 4)) = w;
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
    const int npages = cdiv(rq.kv_len, kPageSize);
    const int32_t *table = p.page_table + static_cast<size_t>(seq) * p.max_pages_per_seq;
    uint32_t mask, sixteen;
    asm volatile("mov.b32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(sixteen));
    auto page_id = [&](int j) { return 8 * j + uw < npages ? __ldg(table + 8 * j + uw) : 0; };
    auto fetch = [&](int id, int j, Packed &f) {
      if (id < 0 || id >= p.num_pages) {
        id = 0;                                        // never dereferenced as it is
        if (lane == 0) atomicOr(&bar.bad, 1);
      }
      const uint8_t *block = p.kv_cache + (static_cast<size_t>(id) * p.num_kv_heads + kvh) * kInt4Block;
      f.k = __ldg(reinterpret_cast<const uint4 *>(block + kInt4K) + lane);
      f.v = __ldg(reinterpret_cast<const uint4 *>(block + kInt4V) + lane);
      f.km = __ldg(reinterpret_cast<const uint2 *>(block + kInt4Meta) + g);
      f.vm = __ldg(reinterpret_cast<const uint4 *>(block + kInt4Meta) + t);
      f.own = __ldg(reinterpret_cast<const uint32_t *>(block + kInt4Meta + 8 * (lane & 7) + 4 * ((lane >> 3) & 1)));
    };
    // Odd keys of the page: those past the last one become zeros, and a value that is not
    // finite zeros with a key that is not finite.  Rare but for the last tile.
    auto mend = [&](int j, Packed &f) {
      const int key0 = (8 * j + uw) * kPageSize;
      const unsigned odd = __ballot_sync(0xffffffffu, (f.own & 0x7f800000u) == 0x7f800000u) & 0xffffu;
      const int live = rq.kv_len - key0;
      if (odd == 0 && live >= kPageSize) return;
      const unsigned gone = live >= kPageSize ? 0u : live <= 0 ? 0xffffu : 0xffffu & (0xffffu << live);
      auto k = [&](uint32_t &m, int key) {
        if (odd >> key & 1) m |= 0x7fc0u;
        if (gone >> key & 1) m = 0;
      };
      auto v = [&](uint32_t &m, int key) {
        if ((odd | gone) >> key & 1) m = 0;
      };
      k(f.km.x, g);
      k(f.km.y, g + 8);
      v(f.vm.x, 2 * t);
      v(f.vm.y, 2 * t + 8);
      v(f.vm.z, 2 * t + 1);
      v(f.vm.w, 2 * t + 9);
    };
    // Stores of eight lanes fall into different banks: every other row has its second
    // chunk first.
    const int odd_row = g & 1;
    const uint32_t k_at = 16 * uw * 128 + g * 128;     // row g of the page
    const uint32_t k_first = (((t + 4 * odd_row) ^ g) << 4), k_second = (((t + 4 - 4 * odd_row) ^ g) << 4);
    const uint32_t v_at = (16 * uw + 2 * t) * 128;     // row 2t
    const uint32_t v_even = (g ^ (2 * t)) << 4, v_odd = 128 + ((g ^ (2 * t + 1)) << 4);

    bool ok = true;
    Packed f, next;
    int id = page_id(1);
    if (n_tiles > 0) fetch(page_id(0), 0, next);
    for (int j = 0; j < n_tiles; ++j) {
      const int s = j % kStages;
      f = next;
      if (j + 1 < n_tiles) {                           // its latency runs under this tile's work
        fetch(id, j + 1, next);
        id = page_id(j + 2);
      }
      mend(j, f);
      if (j >= kStages && !__all_sync(0xffffffffu, mbar_wait(&bar.k_empty[s], (j / kStages + 1) & 1))) {
        ok = false;
        break;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t m = h ? f.km.y : f.km.x;
        const uint32_t s2 = pair_scale(m, false), z2 = pair_zero(m, false);
        const uint32_t w0 = h ? f.k.z : f.k.x, w1 = h ? f.k.w : f.k.y;
        uint8_t *row = sK(s) + k_at + h * 1024;
        *reinterpret_cast<uint4 *>(row + k_first) = values(odd_row ? w1 : w0, s2, z2, mask, sixteen);
        *reinterpret_cast<uint4 *>(row + k_second) = values(odd_row ? w0 : w1, s2, z2, mask, sixteen);
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar.k_full[s]);
      if (j >= kStages && !__all_sync(0xffffffffu, mbar_wait(&bar.v_empty[s], (j / kStages + 1) & 1))) {
        ok = false;
        break;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {                    // keys 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t m = i == 0 ? f.vm.x : i == 1 ? f.vm.z : i == 2 ? f.vm.y : f.vm.w;
        const uint32_t w = i == 0 ? f.v.x : i == 1 ? f.v.y : i == 2 ? f.v.z : f.v.w;
        *reinterpret_cast<uint4 *>(sV(s) + v_at + (i >> 1) * 1024 + (i & 1 ? v_odd : v_even)) =
            values(__funnelshift_l(w, w, 3), pair_scale(m, true), pair_zero(m, true), mask, sixteen);
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar.v_full[s]);
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------------ Q K^T
    set_registers<kOtherRegs, false>();
    bool ok = true;
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.k_full[s], (j / kStages) & 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || j >= ntiles[x]) continue;
        if (j > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bar.p_full[x], (j - 1) & 1));
        if (!ok) continue;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dq = umma_desc_sw128(smem_u32(smem + kOffQ + x * kTileBytes), 16, 1024);
          const uint64_t dk = umma_desc_sw128(smem_u32(sK(s)), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)
            umma_ss(tmem + x * kColTile + kColS, dq + 2 * kk, dk + 2 * kk, kIdescQK, kk > 0);
          umma_commit(&bar.s_full[x]);
        }
        __syncwarp();
      }
      if (ok && lane == 0) umma_commit(&bar.k_empty[s]);
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
  } else if (warp == kPvWarp) {
    // -------------------------------------------------------------------- P V
    set_registers<kOtherRegs, false>();
    bool ok = true;
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar.v_full[s], (j / kStages) & 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || j >= ntiles[x]) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.p_full[x], j & 1));
        if (!ok) continue;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dv = umma_desc_sw128(smem_u32(sV(s)), kTileBytes, 1024);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)        // 16 keys = 2 KB
            umma_ts(tmem + x * kColTile + kColO, tmem + x * kColTile + kColP + 8 * kk, dv + (2048 >> 4) * kk,
                    kIdescPV, (j > 0) || (kk > 0));
          umma_commit(&bar.pv_done[x]);
        }
        __syncwarp();
      }
      if (ok && lane == 0) umma_commit(&bar.v_empty[s]);
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
  } else if (warp < kUnpackWarp) {
    // ---------------------------------------------------------------- softmax
    set_registers<kSoftmaxRegs, true>();
    const int x = warp >> 2;
    const int r = threadIdx.x & (kBM - 1);             // row = tensor-memory lane
    const uint32_t trow = tmem + x * kColTile + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int i = tok0 + x * tile_tokens + r / p.group;       // token within the request
    const int head = kvh * p.group + r % p.group;
    const bool live = r < rows[x];
    Seen seen;
    seen.limit = min(shift + i + 1, rq.kv_len);
    seen.draft = shift;
    seen.vis = 0;
    if (p.tree_mask) {
      seen.limit = shift;
      if (live) seen.vis = p.tree_mask[static_cast<size_t>(seq) * p.q_len + i];
    }
    const float sl2 = p.scale_log2;
    // a sink that is no logit (NaN, +inf) spoils the sum, not the reference
    float m = kUnset, d = 0.f;
    if (live) {
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
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.s_full[x], j & 1))) { ok = false; break; }
      tc_fence_after();
      const int key0 = j * kBN;
      const int parity = j > 0 ? (j - 1) & 1 : -1;
      const bool edge = __any_sync(0xffffffffu, key0 + kBN > seen.limit);
      float sum = edge ? weigh_tile<true>(trow, sl2, m, seen, key0, &bar.pv_done[x], parity)
                       : weigh_tile<false>(trow, sl2, m, seen, key0, &bar.pv_done[x], parity);
      if (__any_sync(0xffffffffu, sum < 0.f)) { ok = false; break; }
      if (__any_sync(0xffffffffu, !(sum <= kMostSum))) {
        // some reference is too small: the rows' maxima, and the tile again
        const float mx = row_max(trow, sl2, seen, key0);
        const float now = fmaxf(m, mx);
        const float alpha = ex2(m - now);
        m = now;
        d *= alpha;
        if (j > 0) scale_o(trow, alpha);
        sum = weigh_tile<true>(trow, sl2, m, seen, key0, &bar.pv_done[x], -1);
      }
      d += sum;
      tc_fence_before();
      mbar_arrive(&bar.p_full[x]);
    }
    if (mine > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&bar.pv_done[x], (mine - 1) & 1));
    tc_fence_after();
    if (!ok) atomicOr(&bar.bad, 1);
    uint32_t o[2][32];
    if (mine > 0 && ok) {
      tmem_ld32(trow + kColO, o[0]);
      tmem_ld32(trow + kColO + 32, o[1]);
      tmem_ld_wait32(o[0]);
      reg_tie32(o[1]);
    }
    tc_fence_before();
    __syncthreads();
    const bool failed = bar.bad != 0;
    if (live) {
      const float inv = failed ? NAN : d == 0.f ? 0.f : 1.f / d;
      const size_t row = static_cast<size_t>(rq.q_start + i) * p.num_qo_heads + head;
      uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kHeadDim);
#pragma unroll
      for (int c = 0; c < kHeadDim / 8; ++c) {
        // column 8c + 2j holds dim 8c + j, column 8c + 2j + 1 dim 8c + 4 + j
        auto dim = [&](int e) {
          const int col = 8 * c + 2 * (e & 3) + (e >> 2);
          return failed ? NAN : __uint_as_float(o[col >> 5][col & 31]) * inv;
        };
        dst[c] = make_uint4(pack_bf16(dim(0), dim(1)), pack_bf16(dim(2), dim(3)), pack_bf16(dim(4), dim(5)),
                            pack_bf16(dim(6), dim(7)));
      }
      if (p.lse) p.lse[row] = failed ? NAN : d == 0.f ? -INFINITY : (m + lg2(d)) * kLn2;
    }
    return;
  } else {
    set_registers<kOtherRegs, false>();                // the rest of the last warpgroup
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

cudaError_t launch_int4_prefill(const Int4AttnParams &p, long long ctas, cudaStream_t stream) {
  static_assert(kSmemBytes > 114 * 1024 && kSmemBytes <= 227 * 1024, "one CTA per SM");
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t err = set_smem_once<int4_prefill_kernel>(kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(int4_prefill_kernel, static_cast<unsigned>(ctas), kThreads, kSmemBytes, stream, false, p);
}

}  // namespace sa
