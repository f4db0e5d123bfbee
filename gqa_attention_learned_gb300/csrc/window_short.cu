// Windowed prefill when the keys of a whole query tile fit at once (up to 192
// slots: window 128 with groups of 4 and more, and short prompts).
//
// Such a tile is little work -- two matrix products of 128 x 144 x 64 and 18k
// exponentials for window 128 -- so a CTA per tile spends most of its life
// waiting for its first loads, its few score tiles, its P V and its stores.
// Here one persistent CTA per SM keeps several tiles in work and up to three
// in flight.  Each tile in work has a lane of its own ("slot"): a part of
// tensor memory, a warp that issues its products and four warps of softmax.
//   last warp   walks the CTA's tiles, copies Q and K of each into one ring of
//               stages (free again after S) and V into another, and leaves the
//               tile's geometry beside them;
//   MMA warps   one per slot: S = Q K^T over all of the tile's boxes, later
//               O = P V;
//   softmax     one thread per row: all scores are there before it starts, so
//               it takes the max in one pass over tensor memory and writes P
//               over S in a second, with no running state; O then goes where
//               the last scores were, and out by way of the tile's V stage.
// Tiles go round the slots, so one slot's softmax runs under the others'
// products, loads and stores.  Three slots of 160 columns serve tiles of up to
// 10 boxes of 16 keys (window 128, group 8, without first tokens), two of 256
// columns up to 12.  Rounding is that of the other prefill kernels: P to bf16
// for the product with V, the output once to bf16; max, sum and O in fp32.
//
// Measured (window 128, 4 sequences of 20.9k tokens, 64 / 8 heads; 57 us at the
// copy bandwidth): 90 us, against 299 us with a CTA per tile (window_prefill.cu as
// it was then).  Issue slots are 56% busy, the tensor pipe 38%: the steps of a tile
// follow one another, and three tiles hide part of that.  Tried: two threads per
// row (194 us, registers spill where shared memory leaves no L1), pieces behind
// per-piece branches (111 us), masks in both passes (139 us).

#include "window_tile.cuh"

#include <algorithm>
#include <type_traits>

namespace sa {
namespace {

using namespace window;

constexpr int kQBytes = kBM * kHeadDim * 2;
constexpr uint32_t kTmemCols = 512;

// Sizes of a variant: tiles in work, boxes of 16 keys per tile at most, stages
// of Q and K, stages of V (a tile in work holds one).
template <int S, int B, int NK, int NV>
struct Shape {
  static constexpr int kKStages = NK, kVStages = NV;
  static constexpr int kSlots = S, kBoxes = B;
  static constexpr int kKBytes = B * kBoxBytes;
  static constexpr int kKStageBytes = kQBytes + kKBytes;
  static constexpr int kMmaWarp = 4 * S, kLoadWarp = 5 * S;
  static constexpr int kThreads = (5 * S + 1) * 32;
  // tensor memory of a slot: S from column 0, P over it, O over the last scores
  static constexpr uint32_t kSlotCols = S == 3 ? 160 : 256;
  static constexpr uint32_t kColO = kSlotCols - kHeadDim;
  static constexpr int kOffV = NK * kKStageBytes;
  static constexpr int kOffBars = kOffV + NV * kKBytes;
  static constexpr int kSmemBytes = kOffBars + 1024 + 1024;   // barriers + alignment slack
  static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
  static_assert(S * kSlotCols <= kTmemCols && 16 * B <= static_cast<int>(kSlotCols), "tensor memory");
  static_assert(kKBytes >= kQBytes, "the output rows pass through the V stage");
  static_assert(8 * B <= static_cast<int>(kColO), "P ends before O");
};
constexpr int kMaxSlots = 3, kMaxStages = 5;

struct Work {
  Request req;
  Tile tile;
  int kvh;
  int stop;                    // no more tiles for this slot
  int bad;                     // a page outside the pool
};

struct Bars {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];   // Q, K and the geometry
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t info[kMaxStages];   // the geometry that goes with a stage of V may be read
  uint64_t s_full[kMaxSlots], p_full[kMaxSlots], o_full[kMaxSlots];
  uint64_t free[kMaxSlots];    // O has been read
  uint32_t tmem_base;
  int dead;                    // a wait ran out
  Work work[kMaxStages];       // by V stage
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

template <bool kPaged, bool kNumbered, typename Sh>     // kNumbered: p.tiles_each == 0
__global__ void __launch_bounds__(Sh::kThreads, 1)
window_short_kernel(const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const WindowPrefillParams p) {
  constexpr int kSlots = Sh::kSlots, kMmaWarp = Sh::kMmaWarp, kLoadWarp = Sh::kLoadWarp;
  constexpr int kThreads = Sh::kThreads, kNK = Sh::kKStages, kNV = Sh::kVStages;
  constexpr int kKBytes = Sh::kKBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item i: query tile i / num_kv_heads of KV head i % num_kv_heads
  const int items = p.num_tiles * p.num_kv_heads;
  const int stride = static_cast<int>(gridDim.x);

  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: accesses stay known to be shared memory's)
  uint8_t *smem = smem_raw + (0u - smem_u32(smem_raw)) % 1024;
  Bars &bar = *reinterpret_cast<Bars *>(smem + Sh::kOffBars);
  auto sQ = [&](int n) { return smem + n % kNK * Sh::kKStageBytes; };     // of tile n
  auto sK = [&](int n) { return sQ(n) + kQBytes; };
  auto sV = [&](int n) { return smem + Sh::kOffV + n % kNV * kKBytes; };
  // a bounded wait of the whole warp; once one has run out, all fail at once
  auto wait = [&](uint64_t *b, int uses) -> bool {
    if (__all_sync(0xffffffffu, mbar_wait(b, uses & 1))) return true;
    atomicOr(&bar.dead, 1);
    return false;
  };

  if (warp == kMmaWarp) {
    tmem_alloc(&bar.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    for (int s = 0; s < kNK; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 128);
      mbar_init(&bar.info[s], 1);
    }
    for (int l = 0; l < kSlots; ++l) {
      mbar_init(&bar.s_full[l], 1);
      mbar_init(&bar.p_full[l], 128);
      mbar_init(&bar.o_full[l], 1);
      mbar_init(&bar.free[l], 128);
    }
    bar.dead = 0;
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp == kLoadWarp) {
    // -------------------------------------------------------------- loads
    int n = 0;                                           // tiles handed out
    // tile qt of a request and a KV head into the next stages; false: a wait ran out
    auto hand_out = [&](const Request &r, int qt, int kvh) -> bool {
      Work w;
      w.req = r;
      w.kvh = kvh;
      w.tile = Tile::make<kPaged>(p, r, qt);
      w.stop = 0;
      const bool have = lane < w.tile.n_boxes;
      const int src = have ? w.tile.source<kPaged>(p, r, lane) : -1;
      const unsigned boxes = __ballot_sync(0xffffffffu, src >= 0);
      w.bad = __popc(boxes) != w.tile.n_boxes;
      uint64_t *k_full = &bar.k_full[n % kNK], *v_full = &bar.v_full[n % kNV];
      // the geometry goes by V stage, so that one has to be free first
      if ((n >= kNV && !wait(&bar.v_empty[n % kNV], n / kNV + 1)) ||
          (n >= kNK && !wait(&bar.k_empty[n % kNK], n / kNK + 1)))
        return false;
      if (lane == 0) {
        // for the softmax warps by the arrival on info, for the products' by
        // k_full's.  (Not for both by k_full: its stage may be filled twice more
        // while the softmax warps are behind.  info goes by V stage: its next
        // arrival there needs v_empty, where all of them arrive after they have
        // seen this one, so no phase is passed over unseen.)
        bar.work[n % kNV] = w;
        mbar_arrive(&bar.info[n % kNV]);
        const uint32_t bytes = __popc(boxes) * kBoxBytes;
        mbar_arrive_expect_tx(k_full, p.tile_tokens * p.group * kHeadDim * 2 + bytes);
        mbar_arrive_expect_tx(v_full, bytes);
        // box {64, group, tile_tokens}: rows (token, head)
        tma_load_3d(sQ(n), &qmap, k_full, 0, kvh * p.group, r.q_start + w.tile.i0);
      }
      __syncwarp();
      if (src >= 0) {
        const int y = kPaged ? kvh * kPageSize : kvh;
        tma_load_3d(sK(n) + lane * kBoxBytes, &kmap, k_full, 0, y, src);
        tma_load_3d(sV(n) + lane * kBoxBytes, &vmap, v_full, 0, y, src);
      }
      __syncwarp();
      ++n;
      return true;
    };
    bool ok = true;
    if constexpr (kNumbered) {
      Walk<kPaged> walk;
      for (long long item = blockIdx.x; ok && item < items; item += stride) {
        const int tile_no = static_cast<int>(item) / p.num_kv_heads;
        const int kvh = static_cast<int>(item) - tile_no * p.num_kv_heads;
        if (!walk.reach(p, tile_no)) break;
        int first;
        const Request r = walk.request(tile_no, first);
        if (r.bad) poison(p, kvh, r.q_start, max(r.q_len, 0), lane, 32);
        else ok = hand_out(r, tile_no - first, kvh);
      }
    } else {
      for (int base = static_cast<int>(blockIdx.x); ok && base < items;) {
        // 32 items at a time, one per lane: most ragged batches have empty ones
        const long long mine = base + static_cast<long long>(lane) * stride;
        const int tile_no = mine < items ? static_cast<int>(mine) / p.num_kv_heads : -1;
        const int kvh = static_cast<int>(mine) - tile_no * p.num_kv_heads;
        bool valid = false, poisoned = false;
        int qt = 0;
        Request r{};
        if (tile_no >= 0) {
          const int seq = tile_no / p.tiles_each;
          r = Request::load<kPaged>(p, seq);
          qt = tile_no - seq * p.tiles_each;
          valid = !r.bad && qt * p.tile_tokens < r.q_len;
          poisoned = r.bad && qt == 0;
        }
        for (unsigned m = __ballot_sync(0xffffffffu, poisoned); m; m &= m - 1) {
          const int l = __ffs(m) - 1;
          poison(p, __shfl_sync(0xffffffffu, kvh, l), __shfl_sync(0xffffffffu, r.q_start, l),
                 max(__shfl_sync(0xffffffffu, r.q_len, l), 0), lane, 32);
        }
        for (unsigned m = __ballot_sync(0xffffffffu, valid); ok && m; m &= m - 1) {
          const int l = __ffs(m) - 1;
          Request x;
          x.seq = __shfl_sync(0xffffffffu, r.seq, l);
          x.q_start = __shfl_sync(0xffffffffu, r.q_start, l);
          x.q_len = __shfl_sync(0xffffffffu, r.q_len, l);
          x.kv_len = __shfl_sync(0xffffffffu, r.kv_len, l);
          x.bad = false;
          ok = hand_out(x, __shfl_sync(0xffffffffu, qt, l), __shfl_sync(0xffffffffu, kvh, l));
        }
        if (items - base <= 32ll * stride) break;
        base += 32 * stride;
      }
    }
    // one last entry per slot
    for (int l = 0; ok && l < kSlots; ++l, ++n) {
      if ((n >= kNV && !wait(&bar.v_empty[n % kNV], n / kNV + 1)) ||
          (n >= kNK && !wait(&bar.k_empty[n % kNK], n / kNK + 1)))
        break;
      if (lane == 0) {
        bar.work[n % kNV].stop = 1;
        mbar_arrive(&bar.info[n % kNV]);
        mbar_arrive(&bar.k_full[n % kNK]);
      }
      __syncwarp();
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------- the products of one slot (one thread)
    const int slot = warp - kMmaWarp;
    const uint32_t tS = tmem + slot * Sh::kSlotCols;
    for (int n = slot, k = 0;; n += kSlots, ++k) {
      if (!wait(&bar.k_full[n % kNK], n / kNK)) break;
      if (bar.work[n % kNV].stop) break;
      const Tile tile = bar.work[n % kNV].tile;
      if (k > 0 && !wait(&bar.free[slot], k - 1)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dq = umma_desc_sw128(smem_u32(sQ(n)), 16, 1024);
        const uint64_t dk = umma_desc_sw128(smem_u32(sK(n)), 16, 1024);
        const uint32_t idesc = umma_idesc_bf16(128, kBox * tile.n_boxes, false, false) | p.negate_q;
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          umma_ss(tS, dq + 2 * kk, dk + 2 * kk, idesc, kk > 0);   // +32 bytes per k-step
        umma_commit(&bar.s_full[slot]);
        umma_commit(&bar.k_empty[n % kNK]);
      }
      __syncwarp();
      if (!wait(&bar.v_full[n % kNV], n / kNV)) break;
      if (tile.clear_unseen(p, sV(n), 0, tile.n_boxes * kBox)) fence_proxy_async_smem();
      __syncwarp();
      if (!wait(&bar.p_full[slot], k)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dv = umma_desc_sw128(smem_u32(sV(n)), kKBytes, 1024);
        for (int kk = 0; kk < tile.n_boxes; ++kk)
          umma_ts(tS + Sh::kColO, tS + 8 * kk, dv + (kBoxBytes >> 4) * kk, kIdescPV, kk > 0);
        umma_commit(&bar.o_full[slot]);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------- softmax, output
    const int slot = warp / 4;
    const int r = threadIdx.x & 127;                     // row = tensor-memory lane
    const uint32_t trow = tmem + slot * Sh::kSlotCols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // token of row i of a tile: i / group, exact for i < 128 and group <= 128
    auto token_of = [&](int i) { return static_cast<int>((static_cast<uint32_t>(i) * p.inv_group) >> 16); };
    const int token = token_of(r), in_group = r - token * p.group;
    const int row_skip = p.num_qo_heads - p.group;       // from a token's last row to the next one's first
    const float sl2 = p.scale_log2;
    const uint64_t scale2 = f2_pack(sl2, sl2);
    // What a tile's softmax needs to know; false: no further tile, or a wait ran out.
    struct Geometry {
      RowSlots see;
      int pieces, lead, edges;
      float sink;
    };
    auto look = [&](int n, Geometry &geo) -> bool {
      if (!wait(&bar.info[n % kNV], n / kNV)) return false;
      const Work &w = bar.work[n % kNV];
      if (w.stop) return false;
      const Tile &tile = w.tile;
      // lanes past the rows repeat the last token
      geo.see = tile.row(p, tile.pos0 + min(token, tile.tokens - 1));
      geo.sink = r < tile.tokens * p.group ? __ldg(p.sinks + w.kvh * p.group + in_group) * kLog2e : -INFINITY;
      // Pieces of 16 slots.  Away from a request's ends only the first one or two
      // of the run, the last one or two, and the first tokens' can hold slots
      // that some row does not see; elsewhere all are taken as such edges.
      geo.pieces = tile.n_boxes;
      const uint32_t full = __reduce_and_sync(0xffffffffu, full_pieces(geo.see));
      geo.lead = tile.first_boxes + ((full >> (tile.first_boxes + 1)) & 1u ? 1 : 2);
      geo.edges = geo.lead + ((full >> max(geo.pieces - 2, 0)) & 1u ? 1 : 2);
      const uint32_t inner = low_bits(geo.pieces - (geo.edges - geo.lead)) & ~low_bits(geo.lead);
      if (geo.edges > geo.pieces || (full & inner) != inner) geo.lead = geo.edges = geo.pieces;
      return true;
    };
    Geometry geo;
    bool more = look(slot, geo);
    for (int n = slot, k = 0; more; n += kSlots, ++k) {
      const int pieces = geo.pieces, lead = geo.lead, edges = geo.edges;
      const RowSlots see = geo.see;
      const float sink = geo.sink;
      if (!wait(&bar.s_full[slot], k)) break;
      tc_fence_after();
      // several pieces at a time, straight-line code: `at(u)` is the u-th piece
      uint32_t x[4][16];
      auto fetch = [&](auto count, auto at) {
#pragma unroll
        for (int u = 0; u < count.value; ++u) tmem_ld16(trow + 16 * at(u), x[u]);
        tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < count.value; ++u) reg_tie16(x[u]);
      };
      const std::integral_constant<int, 2> two;
      const std::integral_constant<int, 4> four;
      auto largest = [&]() {
        return fmaxf(fmax3(max_piece(x[0]), max_piece(x[1]), max_piece(x[2])), max_piece(x[3]));
      };
      // pass 1: the row's max; edges are masked for both passes.  (A piece may
      // come twice at the end of a run of pieces, which changes nothing.)
      float mx = -INFINITY;
#pragma unroll 1
      for (int e0 = 0; e0 < edges; e0 += 2) {
        auto at = [&](int u) {
          const int e = min(e0 + u, edges - 1);
          return e < lead ? e : pieces - edges + e;
        };
        fetch(two, at);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mask_piece(x[u], see.mask(16 * at(u)));
          tmem_st16(trow + 16 * at(u), x[u]);
          mx = fmaxf(mx, max_piece(x[u]));
        }
      }
      const int inner_end = pieces - (edges - lead);
#pragma unroll 1
      for (int i0 = lead; i0 < inner_end; i0 += 4) {
        fetch(four, [&](int u) { return min(i0 + u, inner_end - 1); });
        mx = fmaxf(mx, largest());
      }
      tmem_st_wait();
      const float m = fmaxf(sink, mx * sl2);
      const float mu = m == -INFINITY ? 0.f : m;
      const uint64_t negmu2 = f2_pack(-mu, -mu);
      uint64_t acc = 0, acc1 = 0;                        // (+0.f, +0.f)
      // pass 2: P over S: piece i goes to columns 8 i .., whose scores (piece
      // i / 2) are in registers or used up by then
      int i0 = 0;
#pragma unroll 1
      for (; i0 + 4 <= pieces; i0 += 4) {
        fetch(four, [&](int u) { return i0 + u; });
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          pack_piece(x[u], scale2, negmu2, acc, acc1);
          tmem_st8(trow + 8 * (i0 + u), x[u]);
        }
      }
      if (i0 < pieces) {
        fetch(four, [&](int u) { return min(i0 + u, pieces - 1); });
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          if (i0 + u >= pieces) continue;
          pack_piece(x[u], scale2, negmu2, acc, acc1);
          tmem_st8(trow + 8 * (i0 + u), x[u]);
        }
      }
      float s0, s1;
      f2_unpack(f2_add(acc, acc1), s0, s1);
      const float d = ex2(sink - mu) + s0 + s1;          // the sink's term; nothing where it is -inf
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bar.p_full[slot]);
      // while P V is made: lse, and the next tile's geometry (its K takes this
      // tile's place, so it is known by now)
      const Work &w = bar.work[n % kNV];
      const bool bad = w.bad != 0;
      const int rows = w.tile.tokens * p.group;
      const size_t first_row =
          static_cast<size_t>(w.req.q_start + w.tile.i0) * p.num_qo_heads + w.kvh * p.group;
      auto row_index = [&](int i) -> long long {         // row i of the tile
        return i < rows ? static_cast<long long>(first_row + static_cast<size_t>(token_of(i)) * row_skip + i) : -1;
      };
      if (r < rows && p.lse) p.lse[row_index(r)] = bad ? NAN : d == 0.f ? -INFINITY : (mu + lg2(d)) * kLn2;
      const float inv = bad ? NAN : d == 0.f ? 0.f : 1.f / d;
      more = look(n + kSlots, geo);
      if (!wait(&bar.o_full[slot], k)) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld16(trow + Sh::kColO + 16 * i, x[i]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) reg_tie16(x[i]);
      tc_fence_before();
      mbar_arrive(&bar.free[slot]);
      // P V has read V: the stage takes the rows on their way out, then the next
      // copy (written by the asynchronous proxy)
      store_rows(p, reinterpret_cast<uint4 *>(sV(n)) + (r - lane) * 8, x, inv,
                 [&](int i) { return row_index(r - lane + i); });
      fence_proxy_async_smem();
      mbar_arrive(&bar.v_empty[n % kNV]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (bar.dead) {
    // a wait ran out: none of this CTA's tiles can be trusted
    Walk<kPaged> walk;
    for (long long item = blockIdx.x; item < items; item += stride) {
      const int tile_no = static_cast<int>(item) / p.num_kv_heads;
      Request r;
      int first = tile_no;
      if constexpr (kNumbered) {
        if (!walk.reach(p, tile_no)) break;
        r = walk.request(tile_no, first);
      } else {
        r = Request::load<kPaged>(p, tile_no / p.tiles_each);
        first -= tile_no % p.tiles_each;
      }
      const int i0 = (tile_no - first) * p.tile_tokens;
      if (!r.bad && i0 < r.q_len)
        poison(p, static_cast<int>(item) - tile_no * p.num_kv_heads, r.q_start + i0,
               min(p.tile_tokens, r.q_len - i0), threadIdx.x, kThreads);
    }
  }
}

template <bool kPaged, bool kNumbered, typename Sh>
cudaError_t launch_variant(const CUtensorMap &qmap, const CUtensorMap &kmap,
                           const CUtensorMap &vmap, const WindowPrefillParams &p, int num_sms,
                           cudaStream_t stream) {
  cudaError_t err = set_smem_once<window_short_kernel<kPaged, kNumbered, Sh>>(Sh::kSmemBytes);
  if (err != cudaSuccess) return err;
  const int items = p.num_tiles * p.num_kv_heads;
  return launch_kernel(window_short_kernel<kPaged, kNumbered, Sh>,
                       static_cast<unsigned>(std::min(items, num_sms)), Sh::kThreads,
                       Sh::kSmemBytes, stream, false, qmap, kmap, vmap, p);
}

template <typename Sh>
cudaError_t launch_shape(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                         const WindowPrefillParams &p, int num_sms, cudaStream_t stream) {
  const bool numbered = p.tiles_each == 0;
  if (p.page_table)
    return numbered ? launch_variant<true, true, Sh>(qmap, kmap, vmap, p, num_sms, stream)
                    : launch_variant<true, false, Sh>(qmap, kmap, vmap, p, num_sms, stream);
  return numbered ? launch_variant<false, true, Sh>(qmap, kmap, vmap, p, num_sms, stream)
                  : launch_variant<false, false, Sh>(qmap, kmap, vmap, p, num_sms, stream);
}

using Three = Shape<3, 10, 3, 5>;
using Two = Shape<2, 12, 3, 4>;

// Boxes that a tile can need: the first tokens', and those of the run, which
// may start anywhere in its first page; no more than the longest request has.
int most_boxes(const WindowPrefillParams &p) {
  const long long seen = cdiv(p.first_tokens, kBox) +
                         (static_cast<long long>(p.window) + p.tile_tokens - 1 +
                          (p.page_table ? kPageSize - 1 : 0) + kBox - 1) / kBox;
  return static_cast<int>(std::min<long long>(seen, cdiv(p.max_kv_len, kBox)));
}

}  // namespace

bool window_prefill_is_short(const WindowPrefillParams &p) { return most_boxes(p) <= Two::kBoxes; }

cudaError_t launch_window_short(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                const CUtensorMap &vmap, const WindowPrefillParams &p, int num_sms,
                                cudaStream_t stream) {
  return most_boxes(p) <= Three::kBoxes ? launch_shape<Three>(qmap, kmap, vmap, p, num_sms, stream)
                                        : launch_shape<Two>(qmap, kmap, vmap, p, num_sms, stream);
}

}  // namespace sa
