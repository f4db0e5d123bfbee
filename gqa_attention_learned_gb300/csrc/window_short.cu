// Windowed prefill when the keys of a whole query tile fit at once (up to 192
// slots: window 128 with groups of 4 and more, and short prompts).
//
// Such a tile is little work -- two matrix products of 128 x 192 x 64 and 24k
// exponentials -- so a CTA per tile spends most of its life waiting for its
// first loads, its one score tile, its one P V and its stores (window 128, 20.9k
// tokens, 64 / 8 heads: 299 us).  Here one persistent CTA per SM keeps two
// tiles in work and up to three more loads in flight:
//   warp 10     walks the CTA's tiles, copies Q, K and V of each into a ring of
//               three stages and leaves the tile's geometry beside them;
//   warps 8, 9  one per lane of work ("slot", 256 tensor-memory columns): S =
//               Q K^T over all of the tile's boxes, later O = P V;
//   warps 0..7  four per slot, one thread per row: the softmax has all scores
//               before it, so it takes the max in one pass over tensor memory
//               and writes P over S in a second; no running state.
// Tiles alternate between the slots, so one slot's softmax runs under the
// other's products, loads and stores.  Rounding is that of the other prefill
// kernels: P to bf16 for the product with V, the output once to bf16; max, sum
// and O in fp32.

#include "window_tile.cuh"

#include <algorithm>

namespace sa {
namespace {

using namespace window;

constexpr int kMaxBoxes = 12;                  // 192 slots
constexpr int kMaxChunks = kMaxBoxes / 2;
constexpr int kStages = 3, kSlots = 2;
constexpr int kQBytes = kBM * kHeadDim * 2;
constexpr int kKBytes = kMaxBoxes * kBoxBytes;
constexpr int kStageBytes = kQBytes + 2 * kKBytes;
constexpr int kThreads = (4 * kSlots + kSlots + 1) * 32;
constexpr int kMmaWarp = 4 * kSlots, kLoadWarp = kMmaWarp + kSlots;
constexpr uint32_t kTmemCols = 512, kSlotCols = 256;
constexpr uint32_t kColO = 192;                // S (and P over it) from column 0 of the slot

constexpr int kOffOut = kStages * kStageBytes;
constexpr int kOffBars = kOffOut + kSlots * kQBytes;
constexpr int kSmemBytes = kOffBars + 1024 + 1024;          // barriers + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");

struct Work {
  Request req;
  Tile tile;
  int kvh;
  int stop;                    // no more tiles for this slot
  int bad;                     // a page outside the pool
};

struct Bars {
  uint64_t full[kStages];      // Q, K and the geometry
  uint64_t v_full[kStages];
  uint64_t empty[kStages];     // the stage's P V has completed
  uint64_t s_full[kSlots], p_full[kSlots], o_full[kSlots];
  uint64_t free[kSlots];       // O has been read
  uint32_t tmem_base;
  int dead;                    // a wait ran out
  Work work[kStages];
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// The i-th work item of the launch.
template <bool kPaged>
__device__ __forceinline__ void locate(const WindowPrefillParams &p, int item, int &qt, int &seq, int &kvh) {
  kvh = item % p.num_kv_heads;
  const int rest = item / p.num_kv_heads;
  qt = rest % p.num_q_tiles;
  seq = rest / p.num_q_tiles;
}

template <bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
window_short_kernel(const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const WindowPrefillParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = p.num_q_tiles * p.num_seqs * p.num_kv_heads;
  const int stride = static_cast<int>(gridDim.x);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  Bars &bar = *reinterpret_cast<Bars *>(smem + kOffBars);
  auto sQ = [&](int s) { return smem + s * kStageBytes; };
  auto sK = [&](int s) { return smem + s * kStageBytes + kQBytes; };
  auto sV = [&](int s) { return smem + s * kStageBytes + kQBytes + kKBytes; };
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
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.empty[s], 1);
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
    bool ok = true;
    for (int base = static_cast<int>(blockIdx.x); ok && base < items;) {
      // 32 items at a time, one per lane: most ragged batches have empty ones
      const long long mine = base + static_cast<long long>(lane) * stride;
      bool valid = false, poisoned = false;
      int qt = 0, seq = 0, kvh = 0;
      Request r{};
      if (mine < items) {
        locate<kPaged>(p, static_cast<int>(mine), qt, seq, kvh);
        r = Request::load<kPaged>(p, seq);
        valid = !r.bad && qt * p.tile_tokens < r.q_len;
        poisoned = r.bad && qt == 0;
      }
      for (unsigned m = __ballot_sync(0xffffffffu, poisoned); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        poison(p, __shfl_sync(0xffffffffu, kvh, l), __shfl_sync(0xffffffffu, r.q_start, l),
               max(__shfl_sync(0xffffffffu, r.q_len, l), 0), lane, 32);
      }
      for (unsigned m = __ballot_sync(0xffffffffu, valid); ok && m; m &= m - 1, ++n) {
        const int l = __ffs(m) - 1, s = n % kStages;
        Work w;
        w.req.seq = __shfl_sync(0xffffffffu, r.seq, l);
        w.req.q_start = __shfl_sync(0xffffffffu, r.q_start, l);
        w.req.q_len = __shfl_sync(0xffffffffu, r.q_len, l);
        w.req.kv_len = __shfl_sync(0xffffffffu, r.kv_len, l);
        w.req.bad = false;
        w.kvh = __shfl_sync(0xffffffffu, kvh, l);
        w.tile = Tile::make<kPaged>(p, w.req, __shfl_sync(0xffffffffu, qt, l));
        w.stop = 0;
        const bool have = lane < w.tile.n_boxes;
        const int src = have ? w.tile.source<kPaged>(p, w.req, lane) : -1;
        const unsigned boxes = __ballot_sync(0xffffffffu, src >= 0);
        w.bad = __popc(boxes) != w.tile.n_boxes;
        if (n >= kStages && !wait(&bar.empty[s], n / kStages + 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          bar.work[s] = w;                               // published by the arrival below
          const uint32_t bytes = __popc(boxes) * kBoxBytes;
          mbar_arrive_expect_tx(&bar.full[s], p.tile_tokens * p.group * kHeadDim * 2 + bytes);
          mbar_arrive_expect_tx(&bar.v_full[s], bytes);
          // box {64, group, tile_tokens}: rows (token, head)
          tma_load_3d(sQ(s), &qmap, &bar.full[s], 0, w.kvh * p.group, w.req.q_start + w.tile.i0);
        }
        __syncwarp();
        if (src >= 0) {
          const int y = kPaged ? w.kvh * kPageSize : w.kvh;
          tma_load_3d(sK(s) + lane * kBoxBytes, &kmap, &bar.full[s], 0, y, src);
          tma_load_3d(sV(s) + lane * kBoxBytes, &vmap, &bar.v_full[s], 0, y, src);
        }
        __syncwarp();
      }
      if (items - base <= 32ll * stride) break;
      base += 32 * stride;
    }
    // one last entry per slot
    for (int l = 0; ok && l < kSlots; ++l, ++n) {
      const int s = n % kStages;
      if (n >= kStages && !wait(&bar.empty[s], n / kStages + 1)) break;
      if (lane == 0) {
        bar.work[s].stop = 1;
        mbar_arrive(&bar.full[s]);
      }
      __syncwarp();
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------- the products of one slot (one thread)
    const int slot = warp - kMmaWarp;
    const uint32_t tS = tmem + slot * kSlotCols;
    for (int n = slot, k = 0;; n += kSlots, ++k) {
      const int s = n % kStages;
      if (!wait(&bar.full[s], n / kStages)) break;
      if (bar.work[s].stop) break;
      const Tile tile = bar.work[s].tile;
      if (k > 0 && !wait(&bar.free[slot], k - 1)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dq = umma_desc_sw128(smem_u32(sQ(s)), 16, 1024);
        const uint64_t dk = umma_desc_sw128(smem_u32(sK(s)), 16, 1024);
        const uint32_t idesc = umma_idesc_bf16(128, kBox * tile.n_boxes, false, false);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          umma_ss(tS, dq + 2 * kk, dk + 2 * kk, idesc, kk > 0);   // +32 bytes per k-step
        umma_commit(&bar.s_full[slot]);
      }
      __syncwarp();
      if (!wait(&bar.v_full[s], n / kStages)) break;
      if (tile.clear_unseen(p, sV(s), 0, tile.n_boxes * kBox)) fence_proxy_async_smem();
      __syncwarp();
      if (!wait(&bar.p_full[slot], k)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dv = umma_desc_sw128(smem_u32(sV(s)), kKBytes, 1024);
        for (int kk = 0; kk < tile.n_boxes; ++kk)
          umma_ts(tS + kColO, tS + 8 * kk, dv + (kBoxBytes >> 4) * kk, kIdescPV, kk > 0);
        umma_commit(&bar.o_full[slot]);
        umma_commit(&bar.empty[s]);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------- softmax, output
    const int slot = warp / 4;
    const int r = threadIdx.x & 127;                     // row = tensor-memory lane
    const uint32_t trow = tmem + slot * kSlotCols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int token = r / p.group, in_group = r - token * p.group;
    const float sl2 = p.scale_log2;
    const uint64_t scale2 = f2_pack(sl2, sl2);
    const uint32_t masked_raw = sl2 >= 0.f ? 0xff800000u : 0x7f800000u;
    uint4 *stage = reinterpret_cast<uint4 *>(smem + kOffOut + slot * kQBytes) + (r - lane) * 8;
    for (int n = slot, k = 0;; n += kSlots, ++k) {
      const int s = n % kStages;
      if (!wait(&bar.full[s], n / kStages)) break;       // the geometry
      const Work &w = bar.work[s];
      if (w.stop) break;
      const Tile tile = w.tile;
      const bool bad = w.bad != 0;
      const int rows = tile.tokens * p.group;
      const int head = w.kvh * p.group + in_group;
      const size_t first_row =
          static_cast<size_t>(w.req.q_start + tile.i0) * p.num_qo_heads + w.kvh * p.group;
      const int chunks = (tile.n_boxes + 1) / 2;
      // lanes past the rows repeat the last token
      const RowSlots see = tile.row(p, tile.pos0 + min(token, tile.tokens - 1));
      const float sink = r < rows ? __ldg(p.sinks + head) * kLog2e : -INFINITY;
      uint32_t mask[kMaxChunks];
      unsigned live = 0, edge = 0;                       // warp-uniform bits per chunk
#pragma unroll
      for (int c = 0; c < kMaxChunks; ++c) {
        mask[c] = see.mask(32 * c);
        live |= __any_sync(0xffffffffu, mask[c] != 0u) ? 1u << c : 0u;
        edge |= __any_sync(0xffffffffu, mask[c] != 0xffffffffu) ? 1u << c : 0u;
      }
      if (!wait(&bar.s_full[slot], k)) break;
      tc_fence_after();
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < kMaxChunks; ++c) {
        if (!((live >> c) & 1u)) continue;
        uint32_t x[32];
        tmem_ld32(trow + 32 * c, x);
        tmem_ld_wait32(x);
        if ((edge >> c) & 1u) mask_chunk(x, mask[c], masked_raw);
        mx = fmaxf(mx, max_chunk(x, sl2));
      }
      const float m = fmaxf(sink, mx);
      const float mu = m == -INFINITY ? 0.f : m;
      const uint64_t negmu2 = f2_pack(-mu, -mu);
      uint64_t acc = 0;                                  // (+0.f, +0.f)
      // P over S: chunk c goes to columns 16 c .., whose scores (chunk c / 2)
      // are in registers or used up by then
#pragma unroll
      for (int c = 0; c < kMaxChunks; ++c) {
        if (c >= chunks) continue;
        uint32_t x[32];
        if ((live >> c) & 1u) {
          tmem_ld32(trow + 32 * c, x);
          tmem_ld_wait32(x);
          if ((edge >> c) & 1u) mask_chunk(x, mask[c], masked_raw);
          pack_chunk(x, scale2, negmu2, acc);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0u;
        }
        tmem_st16(trow + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&x[0]));
      }
      float s0, s1;
      f2_unpack(acc, s0, s1);
      const float d = ex2(sink - mu) + s0 + s1;          // the sink's term; nothing where it is -inf
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bar.p_full[slot]);
      if (!wait(&bar.o_full[slot], k)) break;
      tc_fence_after();
      uint32_t o[2][32];
      tmem_ld32(trow + kColO, o[0]);
      tmem_ld32(trow + kColO + 32, o[1]);
      tmem_ld_wait32(o[0]);
      reg_tie32(o[1]);
      tc_fence_before();
      mbar_arrive(&bar.free[slot]);
      auto row_index = [&](int i) -> long long {         // row i of the tile
        const int tok = i / p.group;
        return i < rows ? static_cast<long long>(first_row + static_cast<size_t>(tok) * p.num_qo_heads +
                                                 (i - tok * p.group))
                        : -1;
      };
      __syncwarp();                                      // the previous tile's rows are out
      store_rows(p, stage, o, bad ? NAN : d > 0.f ? 1.f / d : 0.f,
                 [&](int i) { return row_index(r - lane + i); });
      if (r < rows && p.lse) p.lse[row_index(r)] = bad ? NAN : d > 0.f ? (mu + lg2(d)) * kLn2 : -INFINITY;
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
    for (long long item = blockIdx.x; item < items; item += stride) {
      int qt, seq, kvh;
      locate<kPaged>(p, static_cast<int>(item), qt, seq, kvh);
      const Request r = Request::load<kPaged>(p, seq);
      const int i0 = qt * p.tile_tokens;
      if (!r.bad && i0 < r.q_len)
        poison(p, kvh, r.q_start + i0, min(p.tile_tokens, r.q_len - i0), threadIdx.x, kThreads);
    }
  }
}

template <bool kPaged>
cudaError_t launch_variant(const CUtensorMap &qmap, const CUtensorMap &kmap,
                           const CUtensorMap &vmap, const WindowPrefillParams &p, int num_sms,
                           cudaStream_t stream) {
  cudaError_t err = set_smem_once<window_short_kernel<kPaged>>(kSmemBytes);
  if (err != cudaSuccess) return err;
  const long long items = static_cast<long long>(p.num_q_tiles) * p.num_seqs * p.num_kv_heads;
  return launch_kernel(window_short_kernel<kPaged>, static_cast<unsigned>(std::min<long long>(items, num_sms)),
                       kThreads, kSmemBytes, stream, false, qmap, kmap, vmap, p);
}

}  // namespace

bool window_prefill_is_short(const WindowPrefillParams &p) {
  // boxes of the first tokens, and of the run, which may start anywhere in its
  // first page; or every box of the longest request
  const long long seen = cdiv(p.first_tokens, kBox) +
                         (static_cast<long long>(p.window) + p.tile_tokens - 1 +
                          (p.page_table ? kPageSize - 1 : 0) + kBox - 1) / kBox;
  return std::min<long long>(seen, cdiv(p.max_kv_len, kBox)) <= kMaxBoxes;
}

cudaError_t launch_window_short(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                const CUtensorMap &vmap, const WindowPrefillParams &p, int num_sms,
                                cudaStream_t stream) {
  const long long items = static_cast<long long>(p.num_q_tiles) * p.num_seqs * p.num_kv_heads;
  if (items == 0) return cudaSuccess;
  if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return p.page_table ? launch_variant<true>(qmap, kmap, vmap, p, num_sms, stream)
                      : launch_variant<false>(qmap, kmap, vmap, p, num_sms, stream);
}

}  // namespace sa
