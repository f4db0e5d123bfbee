// Pieces shared by the windowed prefill kernels: the keys that a query tile
// needs, the slots that a row sees, and the arithmetic on chunks of scores.
#pragma once

#include "bounded.cuh"
#include "bounded_ptx.cuh"

#include <cmath>

namespace sa {
namespace window {

constexpr int kBM = 128;                       // query rows per tile
constexpr int kBox = 16;                       // keys per copied box
constexpr int kBoxBytes = kBox * kHeadDim * 2;
constexpr uint32_t kIdescPV = umma_idesc_bf16(128, 64, false, true);

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Bits e of a 32-slot chunk starting at v0 with v0 + e < x.
__device__ __forceinline__ uint32_t bits_below(int x, int v0) {
  const int n = x - v0;
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// P = 2^(s * sl2 - mu) for 32 scores, packed as bf16 pairs into r[0..15];
// the pair sums accumulate in `acc` (fp32x2).
template <int E = 0>
__device__ __forceinline__ void pack_chunk(uint32_t (&r)[32], uint64_t scale2, uint64_t negmu2,
                                           uint64_t &acc) {
  if constexpr (E < 16) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * E]), __uint_as_float(r[2 * E + 1])), scale2,
                     negmu2),
              x0, x1);
    const float p0 = ex2(x0);
    const float p1 = ex2(x1);
    acc = f2_add(acc, f2_pack(p0, p1));
    r[E] = pack_bf16(p0, p1);
    pack_chunk<E + 1>(r, scale2, negmu2, acc);
  }
}

// Slot ranges a row sees: [0, a) and [b, c).
struct RowSlots {
  int a, b, c;
  __device__ __forceinline__ uint32_t mask(int v0) const {
    return bits_below(c, v0) & (bits_below(a, v0) | ~bits_below(b, v0));
  }
};

// Masked scores are replaced (by index, so NaN keys cannot leak).  The scale is
// positive -- a negative one negates Q in the product -- so -inf it is.
constexpr uint32_t kMasked = 0xff800000u;

// Masks one chunk of raw scores; their maximum.
__device__ __forceinline__ void mask_chunk(uint32_t (&x)[32], uint32_t mask) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!((mask >> e) & 1u)) x[e] = kMasked;
}
__device__ __forceinline__ float max_chunk(const uint32_t (&x)[32]) {
  float r = __uint_as_float(x[0]);
#pragma unroll
  for (int e = 1; e < 31; e += 2) r = fmax3(r, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
  return fmaxf(r, __uint_as_float(x[31]));
}

// Bits below n (n <= 0: none).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The 16-slot pieces that a row sees whole, as bits.
__device__ __forceinline__ uint32_t full_pieces(const RowSlots &r) {
  return low_bits(r.a / 16) | (low_bits(r.c / 16) & ~low_bits((r.b + 15) / 16));
}

// 16 raw scores: masked by the low bits of `mask`, their maximum, and their
// weights P = 2^(s * sl2 - mu) as bf16 pairs in x[0..7], summed into two
// accumulators.
__device__ __forceinline__ void mask_piece(uint32_t (&x)[16], uint32_t mask) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (!((mask >> e) & 1u)) x[e] = kMasked;
}
__device__ __forceinline__ float max_piece(const uint32_t (&x)[16]) {
  auto f = [&](int e) { return __uint_as_float(x[e]); };
  const float a = fmax3(f(0), f(1), f(2)), b = fmax3(f(3), f(4), f(5)), c = fmax3(f(6), f(7), f(8));
  const float d = fmax3(f(9), f(10), f(11)), e = fmax3(f(12), f(13), f(14));
  return fmaxf(fmax3(a, b, c), fmax3(d, e, f(15)));
}
template <int I = 0>
__device__ __forceinline__ void pack_piece(uint32_t (&x)[16], uint64_t scale2, uint64_t negmu2,
                                           uint64_t &acc0, uint64_t &acc1) {
  if constexpr (I < 8) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * I]), __uint_as_float(x[2 * I + 1])), scale2, negmu2),
              x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    if constexpr (I & 1) acc1 = f2_add(acc1, f2_pack(p0, p1));
    else acc0 = f2_add(acc0, f2_pack(p0, p1));
    x[I] = pack_bf16(p0, p1);
    pack_piece<I + 1>(x, scale2, negmu2, acc0, acc1);
  }
}

// One request's share of the call, and whether its arguments are in range.
struct Request {
  int seq, q_start, q_len, kv_len;
  bool bad;
  // kOrder: a start that falls back spoils this request, too, and not only the one
  // before it.
  template <bool kPaged, bool kOrder = true>
  __device__ __forceinline__ static Request load(const WindowPrefillParams &p, int seq) {
    Request r;
    r.seq = seq;
    r.q_start = p.cu_seqlens_q[seq];
    const int q_end = p.cu_seqlens_q[seq + 1];
    const int before = kOrder ? p.cu_seqlens_q[max(seq - 1, 0)] : r.q_start;
    r.q_len = q_end - r.q_start;
    r.kv_len = kPaged ? p.kv_lens[seq] : r.q_len;
    r.bad = r.q_start < 0 || r.q_start < before || r.q_len < 0 || q_end > p.total_q || r.q_len > p.max_q_len ||
            r.kv_len < r.q_len || r.kv_len > p.max_kv_len ||
            (kPaged && cdiv(r.kv_len, kPageSize) > p.max_pages_per_seq);
    return r;
  }
};

// The query tiles of a launch numbered through request by request; a request
// whose arguments are out of range counts as one tile (its rows become NaN), and
// so does one that starts before any earlier one, so there are never more than
// num_tiles.  Numbering the tiles that exist matters: with an empty CTA for
// every tile that a shorter request lacks, an SM's second slot stayed free while
// CTAs waited (237 of 304 slots taken at a third of empty ones).
// A warp holds 32 requests at a time, one per lane.
template <bool kPaged>
struct Walk {
  Request r;
  int from, tiles;             // this lane's tiles: [from, from + tiles)
  int seq0 = -32, next = 0;    // first request held; tiles up to the last one held
  int top = 0;                 // the largest start so far
  __device__ __forceinline__ bool advance(const WindowPrefillParams &p) {
    if (seq0 + 32 >= p.num_seqs) return false;
    seq0 += 32;
    const int lane = threadIdx.x & 31, seq = seq0 + lane;
    const bool have = seq < p.num_seqs;
    r = have ? Request::load<kPaged, false>(p, seq) : Request{};
    int most = have ? r.q_start : top;
    if (__any_sync(0xffffffffu, have && (r.q_start < top || r.q_len < 0))) {
      most = max(most, top);
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, most, d);
        if (lane >= d) most = max(most, x);
      }
      r.bad = r.bad || r.q_start < most;
    }
    top = __shfl_sync(0xffffffffu, most, min(31, p.num_seqs - 1 - seq0));
    tiles = !have ? 0 : r.bad ? 1 : cdiv(r.q_len, p.tile_tokens);
    int end = tiles;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += x;
    }
    from = next + end - tiles;
    next += __shfl_sync(0xffffffffu, end, 31);
    return true;
  }
  // Goes on until tile `i` is among those held; i the same for all lanes and never
  // less than before.  False: there are not so many.
  __device__ __forceinline__ bool reach(const WindowPrefillParams &p, int i) {
    while (next <= i)
      if (!advance(p)) return false;
    return true;
  }
  // The request with tile `i` of those held, and its first tile's number; i the
  // same for all lanes.  (The last lane with from <= i, as lanes without tiles start
  // where the next one does.)
  __device__ __forceinline__ Request request(int i, int &first) const {
    const int lane = 31 - __clz(__ballot_sync(0xffffffffu, from <= i));
    Request x;
    x.seq = seq0 + lane;
    x.q_start = __shfl_sync(0xffffffffu, r.q_start, lane);
    x.q_len = __shfl_sync(0xffffffffu, r.q_len, lane);
    x.kv_len = __shfl_sync(0xffffffffu, r.kv_len, lane);
    x.bad = __shfl_sync(0xffffffffu, static_cast<int>(r.bad), lane) != 0;
    first = __shfl_sync(0xffffffffu, from, lane);
    return x;
  }
};

// NaN over `tokens` tokens from `token` on (within the buffers) of one KV
// head's query heads, by `threads` threads of which this is number `thread`.
__device__ inline void poison(const WindowPrefillParams &p, int kvh, int token, int tokens,
                              int thread, int threads) {
  if (token < 0 || token >= p.total_q) return;
  const uint4 nan4 = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
  const long long rows = static_cast<long long>(min(tokens, p.total_q - token)) * p.group;
  for (long long idx = thread; idx < rows; idx += threads) {
    const size_t row = static_cast<size_t>(token + idx / p.group) * p.num_qo_heads +
                       kvh * p.group + idx % p.group;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kHeadDim);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = nan4;
    if (p.lse) p.lse[row] = NAN;
  }
}

// A query tile and the boxes of keys that some row of it sees: the first
// tokens' boxes, then the run [run, hi) that ends at the tile's last position.
struct Tile {
  int i0, tokens;              // first token within the request, tokens
  int pos0, lo, hi;            // first position; keys [lo, hi) and [0, first) are seen
  int first_boxes, run, gap;   // gap: keys left out between the two parts
  int n_boxes;
  template <bool kPaged>
  __device__ __forceinline__ static Tile make(const WindowPrefillParams &p, const Request &r, int qt) {
    Tile t;
    t.i0 = qt * p.tile_tokens;
    t.tokens = min(p.tile_tokens, r.q_len - t.i0);
    t.pos0 = r.kv_len - r.q_len + t.i0;
    t.hi = t.pos0 + t.tokens;
    t.lo = max(0, t.pos0 - p.window + 1);
    t.first_boxes = cdiv(min(p.first_tokens, t.lo), kBox);
    t.run = max(kPaged ? t.lo - t.lo % kBox : t.lo, t.first_boxes * kBox);
    t.gap = t.run - t.first_boxes * kBox;
    t.n_boxes = t.first_boxes + cdiv(max(t.hi - t.run, 0), kBox);
    return t;
  }
  __device__ __forceinline__ int slot_of(int key) const {
    const int first = first_boxes * kBox;
    return key <= first ? key : max(key - gap, first);
  }
  // the slot ranges that the row at position pos sees
  __device__ __forceinline__ RowSlots row(const WindowPrefillParams &p, int pos) const {
    return RowSlots{slot_of(min(p.first_tokens, pos + 1)), slot_of(max(0, pos - p.window + 1)),
                    slot_of(pos + 1)};
  }
  // Where box bx comes from: a page id, or the first row of the box in the
  // ragged K/V; -1 for a page outside the pool.
  template <bool kPaged>
  __device__ __forceinline__ int source(const WindowPrefillParams &p, const Request &r, int bx) const {
    const int key = bx < first_boxes ? bx * kBox : run + (bx - first_boxes) * kBox;
    if constexpr (kPaged) {
      const int id = p.page_table[static_cast<size_t>(r.seq) * p.max_pages_per_seq + key / kPageSize];
      return id >= 0 && id < p.num_pages ? id : -1;
    } else {
      return r.q_start + key;
    }
  }
  // Zeroes the value rows of slots [v0, v1), held from `v` on, that no row
  // sees (0 * NaN would poison whole rows); whole 128-byte rows, so the swizzle
  // is irrelevant.  Called by a warp; true if anything was written.
  __device__ __forceinline__ bool clear_unseen(const WindowPrefillParams &p, uint8_t *v, int v0, int v1) const {
    const int dead_from = slot_of(min(p.first_tokens, hi)), dead_to = slot_of(lo), end = slot_of(hi);
    if (!((dead_from < dead_to && dead_from < v1 && dead_to > v0) || end < v1)) return false;
    uint4 *row = reinterpret_cast<uint4 *>(v);
    auto clear = [&](int from, int to) {
      for (int i = (max(from, v0) - v0) * 8 + static_cast<int>(threadIdx.x & 31); i < (min(to, v1) - v0) * 8; i += 32)
        row[i] = make_uint4(0, 0, 0, 0);
    };
    clear(dead_from, dead_to);
    clear(end, v1);
    return true;
  }
};

// Writes a warp's 32 finished rows (one per lane, x: 64 fp32, times inv) as
// whole 128-byte lines, through 4 KB of shared memory: 8 lanes cover one row.
// row_of(i) is the row index of the warp's i-th row, < 0: none.
template <int N, typename RowOf>
__device__ __forceinline__ void store_rows(const WindowPrefillParams &p, uint4 *stage,
                                           const uint32_t (&x)[kHeadDim / N][N], float inv, RowOf row_of) {
  const int lane = threadIdx.x & 31;
  const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
  for (int c = 0; c < kHeadDim / 8; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = 8 * c + 2 * e;
      float lo, hi;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(x[at / N][at % N]), __uint_as_float(x[at / N][at % N + 1])), inv2),
                lo, hi);
      w[e] = pack_bf16(lo, hi);
    }
    stage[lane * 8 + (c ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const int cc = lane & 7;
  uint4 line[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = 4 * k + (lane >> 3);
    line[k] = stage[i * 8 + (cc ^ (i & 7))];
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const long long row = row_of(4 * k + (lane >> 3));
    if (row >= 0) reinterpret_cast<uint4 *>(p.out + row * kHeadDim)[cc] = line[k];
  }
}

}  // namespace window
}  // namespace sa
