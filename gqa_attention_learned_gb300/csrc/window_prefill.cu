// Prefill with a sliding window and first tokens that stay visible (ragged, or
// appended to a paged KV prefix), learned sinks, on the 5th-generation tensor
// cores (tcgen05 + tensor memory).
//
// Mathematics: the row of the token at position i sees the keys
//   { j <= i : j < first_tokens or j > i - window },
// and its softmax starts at the head's sink (running max = sink, running sum
// = 1) as in plain prefill.
//
// Tile: the 128 rows of a CTA are 128 / group tokens times the query heads of
// one KV head, ordered (token, head).  With the heads in one tile its rows
// span few positions, so a window of W needs W + 128 / group - 1 keys instead
// of the W + 127 that 128 tokens of one head would (window 128, group 8: 143
// keys against 255).
// Keys: the keys that some row of the tile sees are the first tokens and one
// run that ends at the tile's last position.  They are numbered through
// ("slots"): boxes of 16 keys (a page, or 16 rows of ragged K/V) holding the
// first tokens, then boxes from the run's start on; tiles take 8 boxes = 128
// slots each, so the two parts share tiles and nothing between them is
// copied or looked up.  The last tile's MMAs cover its own boxes only.
// Rows see at most two slot ranges.  Most tiles of a long window are seen whole
// by all rows of a warp; on the others the warp first masks the chunks of 32 slots
// that some row does not see, in tensor memory, and then goes the same way.
// Warp roles, barriers and the softmax are those of plain prefill: warp 4
// loads Q and K and issues S = Q K^T, warp 5 loads V and issues O += P V,
// warps 0..3 run the online softmax, one thread per row, between them.
//
// Measured (64 / 8 heads): 563 us for 4 chunks of 2048 new tokens on up to 14336
// cached ones with window 4096, 910 TFLOP/s of the pairs that are seen: tensor pipe
// 52%, exponential unit 40%, issue slots 50% busy; as in plain prefill the tile's
// chain of S, softmax, P V binds.  Few tiles per CTA cost more: 57 us for 7.6k
// tokens of 16 / 2 heads with window 1023 (16.5 us by the tensor peak), where a CTA
// lasts 30k cycles, 2.4k for each of its 9 tiles and the rest for its start and end.

#include "window_tile.cuh"

namespace sa {
namespace {

using namespace window;

constexpr int kBN = 128;                       // key slots per tile
constexpr int kBoxes = kBN / 16;               // copied boxes per tile
constexpr int kKStages = 3, kVStages = 2;
constexpr int kTileBytes = kBN * kHeadDim * 2;
constexpr int kThreads = 192;
constexpr int kQkWarp = 4, kPvWarp = 5;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192;
constexpr float kRescaleLog2 = 8.f;     // lazy O rescale threshold (P < 256)

constexpr int kOffQ = 0;
constexpr int kOffK = kTileBytes;
constexpr int kOffV = kOffK + kKStages * kTileBytes;
constexpr int kOffBars = kOffV + kVStages * kTileBytes;
constexpr int kSmemBytes = kOffBars + 2048 + 1024;          // barriers + alignment slack
static_assert(kSmemBytes <= 113 * 1024, "two CTAs per SM");

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full;     // S of the current tile is in tensor memory
  uint64_t s_free;     // the softmax has read S
  uint64_t p_full;     // P of the current tile is in tensor memory
  uint64_t pv_done;    // the P V of the previous tile has finished
  uint64_t o_final;
  uint32_t tmem_base;
  int bad;
  // what the softmax needs only on edge tiles and at its end: registers are
  // what its loop runs out of
  Tile tile;
  int q_start, kvh;
  RowSlots see[kBM];
};
static_assert(sizeof(Bars) <= 2048, "barrier block");

// Running softmax of a row: reference max m (base 2) that P and the
// tensor-memory O are relative to, sum d.  m starts at the sink and moves only
// when a row max exceeds it by more than kRescaleLog2.
struct RowState {
  float m, d;
  // Takes in the max of a tile; returns the factor that O has to be scaled by.
  __device__ __forceinline__ float advance(float mx, bool first_tile) {
    const float m_new = fmaxf(m, mx);
    if (first_tile) {                  // O holds nothing yet: just re-base d
      if (m_new != -INFINITY) {
        d *= ex2(m - m_new);
        m = m_new;
      }
      return 1.f;
    }
    if (!(m_new > m + kRescaleLog2)) return 1.f;
    const float alpha = ex2(m - m_new);
    d *= alpha;
    m = m_new;
    return alpha;
  }
  __device__ __forceinline__ float reference() const { return m == -INFINITY ? 0.f : m; }
};

// Scales this row's O (rare: the previous P V has finished, the next one is
// issued only after p_full).
__device__ __forceinline__ void rescale_o(uint32_t trow, float alpha) {
  uint32_t x[32];
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    tmem_ld32(trow + kColO + 32 * h, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
    tmem_st16(trow + kColO + 32 * h, *reinterpret_cast<uint32_t(*)[16]>(&x[0]));
    tmem_st16(trow + kColO + 32 * h + 16, *reinterpret_cast<uint32_t(*)[16]>(&x[16]));
  }
  tmem_st_wait();
}

// One 128-slot tile of the online softmax for this thread's row.  `whole`:
// every row of the warp sees all of it.  Returns false when a wait timed out.
__device__ __forceinline__ bool softmax_tile(Bars &bar, uint32_t trow, int j, bool whole, float sl2,
                                             RowState &row) {
  if (!__all_sync(0xffffffffu, mbar_wait(&bar.s_full, j & 1))) return false;
  tc_fence_after();
  const uint64_t scale2 = f2_pack(sl2, sl2);
  uint32_t x[4][32];
  if (!whole) {
    // an edge tile: the chunks with unseen slots are masked in tensor memory
    const RowSlots see = bar.see[threadIdx.x];
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const uint32_t mask = see.mask(j * kBN + 32 * c);
      if (__all_sync(0xffffffffu, mask == 0xffffffffu)) continue;
      tmem_ld32(trow + kColS + 32 * c, x[0]);
      tmem_ld_wait32(x[0]);
      mask_chunk(x[0], mask);
      tmem_st16(trow + kColS + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[0][0]));
      tmem_st16(trow + kColS + 32 * c + 16, *reinterpret_cast<uint32_t(*)[16]>(&x[0][16]));
    }
    tmem_st_wait();
  }
  // S is read once and held in registers
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(trow + kColS + 32 * c, x[c]);
  tmem_ld_wait32(x[0]);
#pragma unroll
  for (int c = 1; c < 4; ++c) reg_tie32(x[c]);
  tc_fence_before();
  mbar_arrive(&bar.s_free);
  const float alpha = row.advance(
      fmaxf(fmax3(max_chunk(x[0]), max_chunk(x[1]), max_chunk(x[2])), max_chunk(x[3])) * sl2, j == 0);
  const float mu = row.reference();
  const uint64_t negmu2 = f2_pack(-mu, -mu);
  uint64_t acc[4] = {0, 0, 0, 0};                    // (+0.f, +0.f)
#pragma unroll
  for (int c = 0; c < 4; ++c) pack_chunk(x[c], scale2, negmu2, acc[c]);
  float s0, s1;
  f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
  // the previous tile's P V reads P and accumulates O: wait for it
  if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(&bar.pv_done, (j - 1) & 1))) return false;
  tc_fence_after();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    tmem_st16(trow + kColP + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[c][0]));
  row.d += s0 + s1;
  tmem_st_wait();
  if (__any_sync(0xffffffffu, alpha != 1.f)) rescale_o(trow, alpha);
  tc_fence_before();
  mbar_arrive(&bar.p_full);
  return true;
}

template <bool kPaged>
__global__ void __launch_bounds__(kThreads, 2)
window_prefill_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const WindowPrefillParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item: (query tile, KV head), a request's last tiles (whose
  // windows are full) first
  const int item = static_cast<int>(blockIdx.x) / p.num_kv_heads;
  const int kvh = static_cast<int>(blockIdx.x) - item * p.num_kv_heads;
  Request req;
  int qt;
  if (p.tiles_each > 0) {
    const int seq = item / p.tiles_each;
    req = Request::load<kPaged>(p, seq);
    qt = p.tiles_each - 1 - (item - seq * p.tiles_each);
    if (req.bad ? qt != 0 : qt * p.tile_tokens >= req.q_len) return;
  } else {
    Walk<kPaged> walk;
    if (!walk.reach(p, item)) return;
    int first;
    req = walk.request(item, first);
    qt = cdiv(req.q_len, p.tile_tokens) - 1 - (item - first);
  }
  if (req.bad) {
    poison(p, kvh, req.q_start, max(req.q_len, 0), threadIdx.x, kThreads);
    return;
  }
  const Tile tile = Tile::make<kPaged>(p, req, qt);
  const int rows = tile.tokens * p.group;
  const int n_tiles = cdiv(tile.n_boxes, kBoxes);
  const int live_threads = min(kBM, 32 * cdiv(rows, 32));

  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: accesses stay known to be shared memory's)
  uint8_t *smem = smem_raw + (0u - smem_u32(smem_raw)) % 1024;
  Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
  uint8_t *sQ = smem + kOffQ;
  auto sK = [&](int s) { return smem + kOffK + s * kTileBytes; };
  auto sV = [&](int s) { return smem + kOffV + s * kTileBytes; };

  if (warp == kPvWarp) {
    tmem_alloc(&bar.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // source of this lane's box of tile j (lanes 0..7), -1 past the last box
  auto source_of = [&](int j) -> int {
    const int bx = j * kBoxes + lane;
    if (lane >= kBoxes || bx >= tile.n_boxes) return -1;
    const int src = tile.source<kPaged>(p, req, bx);
    if (src < 0) atomicOr(&bar.bad, 1);
    return src;
  };
  // K (t = 0) or V (t = 1) of tile j into its ring slot, once the slot is free
  auto load = [&](int j, int t, int src) -> bool {
    const int ns = t == 0 ? kKStages : kVStages;
    const int s = j % ns;
    uint64_t *full = t == 0 ? &bar.k_full[s] : &bar.v_full[s];
    uint64_t *empty = t == 0 ? &bar.k_empty[s] : &bar.v_empty[s];
    uint8_t *dst = (t == 0 ? sK(s) : sV(s)) + lane * kBoxBytes;
    const CUtensorMap *map = t == 0 ? &kmap : &vmap;
    if (j >= ns && !__all_sync(0xffffffffu, mbar_wait(empty, ((j / ns) + 1) & 1))) return false;
    const unsigned mask = __ballot_sync(0xffffffffu, src >= 0);
    if (lane == 0) mbar_arrive_expect_tx(full, __popc(mask) * kBoxBytes);
    __syncwarp();
    if (src >= 0) {
      if constexpr (kPaged) tma_load_3d(dst, map, full, 0, kvh * kPageSize, src);
      else tma_load_3d(dst, map, full, 0, kvh, src);
    }
    __syncwarp();
    return true;
  };

  if (warp == kQkWarp) {
    if (lane == 0) {
      mbar_init(&bar.q_full, 1);
      for (int s = 0; s < kKStages; ++s) {
        mbar_init(&bar.k_full[s], 1);
        mbar_init(&bar.k_empty[s], 1);
      }
      for (int s = 0; s < kVStages; ++s) {
        mbar_init(&bar.v_full[s], 1);
        mbar_init(&bar.v_empty[s], 1);
      }
      mbar_init(&bar.s_full, 1);
      mbar_init(&bar.s_free, live_threads);
      mbar_init(&bar.p_full, live_threads);
      mbar_init(&bar.pv_done, 1);
      mbar_init(&bar.o_final, 1);
      bar.bad = 0;
      bar.tile = tile;
      bar.q_start = req.q_start;
      bar.kvh = kvh;
      fence_mbar_init();
      mbar_arrive_expect_tx(&bar.q_full, p.tile_tokens * p.group * kHeadDim * 2);
      // box {64, group, tile_tokens}: rows (token, head)
      tma_load_3d(sQ, &qmap, &bar.q_full, 0, kvh * p.group, req.q_start + tile.i0);
    }
    __syncwarp();
    load(0, 0, source_of(0));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp == kQkWarp) {
    // ------------------------------------------- loads and QK^T (one thread)
    const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
    auto issue_qk = [&](int j) -> bool {
      const int s = j % kKStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.k_full[s], (j / kKStages) & 1))) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dk = umma_desc_sw128(smem_u32(sK(s)), 16, 1024);
        const uint32_t idesc =
            umma_idesc_bf16(128, kBox * min(kBoxes, tile.n_boxes - j * kBoxes), false, false) | p.negate_q;
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          umma_ss(tmem + kColS, dq + 2 * kk, dk + 2 * kk, idesc, kk > 0);   // +32 bytes per k-step
        umma_commit(&bar.s_full);
        umma_commit(&bar.k_empty[s]);
      }
      __syncwarp();
      return true;
    };
    // A load costs its warp about 100 cycles a box: the second tile's are issued
    // while the first's are on their way, the third's under the first product.
    bool ok = n_tiles < 2 || load(1, 0, source_of(1));
    int src = source_of(2);
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bar.q_full, 0)) && issue_qk(0);
    if (ok && n_tiles > 2) ok = load(2, 0, src);
    src = source_of(kKStages);
    for (int j = 0; ok && j + 1 < n_tiles; ++j) {
      // S of tile j has been read: compute S of tile j+1 during this softmax
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.s_free, j & 1))) { ok = false; break; }
      tc_fence_after();
      ok = issue_qk(j + 1);
      if (ok && j + kKStages < n_tiles) {             // K slot freed by QK^T of tile j
        ok = load(j + kKStages, 0, src);
        src = source_of(j + kKStages + 1);
      }
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
  } else if (warp == kPvWarp) {
    // ---------------------------------------------------- P V (one thread)
    const uint32_t tP = tmem + kColP, tO = tmem + kColO;
    bool ok = true;
    for (int j = 0; ok && j < min(n_tiles, kVStages); ++j) ok = load(j, 1, source_of(j));
    int src = source_of(kVStages);
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kVStages;
      const int boxes = min(kBoxes, tile.n_boxes - j * kBoxes);
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.p_full, j & 1)) ||
          !__all_sync(0xffffffffu, mbar_wait(&bar.v_full[s], (j / kVStages) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (tile.clear_unseen(p, sV(s), j * kBN, j * kBN + boxes * kBox)) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const uint64_t dv = umma_desc_sw128(smem_u32(sV(s)), kTileBytes, 1024);
        for (int kk = 0; kk < boxes; ++kk)
          umma_ts(tO, tP + 8 * kk, dv + (kBoxBytes >> 4) * kk, kIdescPV, (j > 0) || (kk > 0));
        umma_commit(&bar.v_empty[s]);
        umma_commit(&bar.pv_done);
      }
      __syncwarp();
      if (j + kVStages < n_tiles) {
        if (!load(j + kVStages, 1, src)) { ok = false; break; }
        src = source_of(j + kVStages + 1);
      }
    }
    if (!ok && lane == 0) atomicOr(&bar.bad, 1);
    if (lane == 0) umma_commit(&bar.o_final);
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int r = threadIdx.x;                          // row = TMEM lane
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float sl2 = p.scale_log2;
    // token of row i of a tile: i / group, exact for i < 128 and group <= 128
    auto token_of = [&](int i) { return static_cast<int>((static_cast<uint32_t>(i) * p.inv_group) >> 16); };
    RowState state;
    int tiles, whole_b, whole_c;
    {
      const int token = token_of(r);
      const int tile_rows = bar.tile.tokens * p.group;
      tiles = warp * 32 < tile_rows ? cdiv(bar.tile.n_boxes, kBoxes) : 0;   // none without rows
      // lanes past the rows repeat the last token
      const RowSlots see = bar.tile.row(p, bar.tile.pos0 + min(token, bar.tile.tokens - 1));
      bar.see[r] = see;
      // tiles of the run that every row of the warp sees whole: [whole_b, whole_c)
      whole_b = (__reduce_max_sync(0xffffffffu, see.b) + kBN - 1) / kBN;
      whole_c = __reduce_min_sync(0xffffffffu, see.c) / kBN;
      state.m = r < tile_rows ? p.sinks[bar.kvh * p.group + (r - token * p.group)] * kLog2e : -INFINITY;
      state.d = 1.f;                                    // started at the sink
    }
    bool ok = true;
    for (int j = 0; j < tiles; ++j) {
      if (!softmax_tile(bar, trow, j, j >= whole_b && j < whole_c, sl2, state)) {
        ok = false;
        break;
      }
    }
    const bool live = tiles > 0;                        // warp-uniform
    uint32_t x[2][32];
    if (live) {
      if (__all_sync(0xffffffffu, mbar_wait(&bar.o_final, 0))) {
        tc_fence_after();
        if (ok) {
          tmem_ld32(trow + kColO, x[0]);
          tmem_ld32(trow + kColO + 32, x[1]);
          tmem_ld_wait32(x[0]);
          reg_tie32(x[1]);
        }
      } else {
        ok = false;
      }
    }
    if (!ok) atomicOr(&bar.bad, 1);
    // Outputs are written after the CTA-wide barrier below.  Tensor memory is
    // read no more: the P V warp frees it meanwhile.
    tc_fence_before();
    __syncthreads();
    if (!live) return;
    const bool failed = bar.bad != 0;
    const float m = state.m, d = state.d;
    const int rows = bar.tile.tokens * p.group;
    const size_t first_row =
        static_cast<size_t>(bar.q_start + bar.tile.i0) * p.num_qo_heads + bar.kvh * p.group;
    auto row_index = [&](int i) -> long long {           // row i of the tile
      const int tok = token_of(i);
      return i < rows ? static_cast<long long>(first_row + static_cast<size_t>(tok) * p.num_qo_heads + (i - tok * p.group)) : -1;
    };
    // the query buffer is free since the last QK^T completed
    store_rows(p, reinterpret_cast<uint4 *>(sQ) + (r - lane) * 8, x,
               failed ? NAN : d == 0.f ? 0.f : 1.f / d, [&](int i) { return row_index(r - lane + i); });
    if (r < rows && p.lse)
      p.lse[row_index(r)] = failed ? NAN : (d == 0.f ? -INFINITY : (m + lg2(d)) * kLn2);
    return;
  }
  tc_fence_before();
  __syncthreads();          // the softmax warps have read O: tensor memory is free
  if (warp == kPvWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool kPaged>
cudaError_t launch_variant(const CUtensorMap &qmap, const CUtensorMap &kmap,
                           const CUtensorMap &vmap, const WindowPrefillParams &p, unsigned ctas,
                           cudaStream_t stream) {
  cudaError_t err = set_smem_once<window_prefill_kernel<kPaged>>(kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(window_prefill_kernel<kPaged>, ctas, kThreads, kSmemBytes, stream, false,
                       qmap, kmap, vmap, p);
}

}  // namespace

uint32_t window_negate_q(bool negative) { return negative ? kIdescNegateA : 0u; }

cudaError_t launch_window_prefill(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                  const CUtensorMap &vmap, const WindowPrefillParams &p,
                                  cudaStream_t stream) {
  const unsigned ctas = static_cast<unsigned>(p.num_tiles) * p.num_kv_heads;
  return p.page_table ? launch_variant<true>(qmap, kmap, vmap, p, ctas, stream)
                      : launch_variant<false>(qmap, kmap, vmap, p, ctas, stream);
}

}  // namespace sa
