// Parameters and launchers of the operators that bound a long context: windowed
// attention, attention mass, eviction.
#pragma once

#include "kernels.cuh"

namespace sa {

// launch_kernel with clusters of `cluster` CTAs (`grid` counts CTAs, a multiple).
template <typename... Params, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(Params...), unsigned grid, unsigned cluster,
                                   unsigned block, int smem, cudaStream_t stream,
                                   bool programmatic, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---------------------------------------------------------- windowed decode
// One token per request that sees the keys j >= kv_len - window and j <
// first_tokens.  Chunks and CTAs count pages with a visible key.
struct WindowDecodeParams {
  const uint16_t *q;               // bf16 [B][Hq][64]
  const uint16_t *k_cache, *v_cache;   // bf16 [num_pages][Hkv][16][64]
  const int32_t *page_table;       // [B][max_pages_per_seq]
  const int32_t *kv_lens;          // [B]
  const float *sinks;              // [Hq]
  uint16_t *out;                   // bf16 [B][Hq][64]
  float *lse;                      // [B][Hq] or null
  int *counters;                   // [B][Hkv * head_blocks], zero between calls (splits > 1)
  float *ws_o;                     // fp32 [splits][B][Hq][64] (splits > 1)
  float *ws_lse;                   // fp32 [splits][B][Hq] (base-2 lse)
  float scale_log2;
  int max_pages_per_seq, batch, num_qo_heads, num_kv_heads, group;
  int col_blocks;                  // 8-head blocks per CTA (1 or 2)
  int head_blocks;                 // CTAs per (request, KV head, chunk)
  int num_pages, num_splits, pages_per_chunk;
  int window, first_tokens, max_kv_len;   // window and first_tokens <= max_kv_len
  int num_sms;
};

int window_decode_ctas_per_sm();
cudaError_t launch_window_decode(const WindowDecodeParams &p, cudaStream_t stream,
                                 bool programmatic);

// --------------------------------------------------------- windowed prefill
struct WindowPrefillParams {
  const int32_t *cu_seqlens_q;   // [n+1]; ragged K/V share it
  const int32_t *page_table;     // paged K/V: [n][max_pages_per_seq], null: ragged K/V [Tq][Hkv][64]
  const int32_t *kv_lens;        // paged K/V: [n]
  const float *sinks;            // [Hq]
  uint16_t *out;                 // bf16 [Tq][Hq][64]
  float *lse;                    // [Tq][Hq] or null
  float scale_log2;              // |scale|, not 0: masked scores are -inf, and stay so
  uint32_t negate_q;             // the scale's sign: 0 or the descriptor bit that negates Q
  int num_seqs, total_q, max_q_len, max_kv_len;
  int num_qo_heads, num_kv_heads, group;
  int max_pages_per_seq, num_pages;
  int window, first_tokens;      // both <= max_kv_len, window >= 1
  int tile_tokens;               // tokens per query tile = 128 / group
  unsigned inv_group;            // ceil(2^16 / group): i / group for i < 128
  int num_tiles;                 // query tiles per KV head, at most
  int tiles_each;                // > 0: request r has tiles r * tiles_each ..; 0: numbered through
};

cudaError_t launch_window_prefill(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                  const CUtensorMap &vmap, const WindowPrefillParams &p,
                                  cudaStream_t stream);

uint32_t window_negate_q(bool negative);   // WindowPrefillParams::negate_q

// Whether the keys of every query tile fit the kernel that holds them all at
// once, and that kernel (one persistent CTA per SM).
bool window_prefill_is_short(const WindowPrefillParams &p);
cudaError_t launch_window_short(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                const CUtensorMap &vmap, const WindowPrefillParams &p, int num_sms,
                                cudaStream_t stream);

// ---------------------------------------------------------- attention weight
struct MassParams {
  const uint16_t *q;             // bf16 [Tq][Hq][64]
  const int32_t *cu_seqlens_q;   // [n+1] (prefill form)
  const uint16_t *k_cache;       // bf16 [num_pages][Hkv][16][64]
  const int32_t *page_table;     // [n][max_pages_per_seq]
  const int32_t *kv_lens;        // [n]
  const float *lse;              // [Tq][Hq]
  float *mass;                   // [n][Hkv][mass_stride]
  float scale_log2;
  int num_seqs, total_q, max_q_len, max_kv_len, mass_stride;
  int num_qo_heads, num_kv_heads, group;
  int max_pages_per_seq, num_pages;
  int num_chunks, pages_per_chunk;   // decode form: CTAs per (request, KV head)
  int tile_tokens;                   // prefill form: tokens per query tile = 128 / group
  int mirror;                        // prefill form: many query tiles per key pair
  int split, split_log2;             // then: CTAs that share them (a power of two), else 1
  int num_sms;
};

int prefill_mass_pair_keys();        // keys that a CTA holds at a time
int decode_mass_warps();         // pages a CTA of the decode form works on at a time
cudaError_t launch_decode_mass(const MassParams &p, cudaStream_t stream);
cudaError_t launch_prefill_mass(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                const MassParams &p, cudaStream_t stream);

// ----------------------------------------------------------------- eviction
struct EvictParams {
  uint16_t *k_cache, *v_cache;   // bf16 [num_pages][Hkv][16][64]
  const int32_t *page_table;     // [B][max_pages_per_seq]
  const int32_t *kv_lens;        // [B]
  const float *mass;             // [B][Hkv][mass_stride]
  const int32_t *dst_page_table; // [B][dst_max_pages] (page_table itself: in place)
  float *dst_mass;               // [B][Hkv][dst_mass_stride] (mass itself: in place)
  int32_t *new_kv_lens;          // [B]
  int32_t *kept;                 // [B][Hkv][budget]
  int batch, num_kv_heads, num_pages, max_kv_len;
  int max_pages_per_seq, dst_max_pages, mass_stride, dst_mass_stride;
  int budget, first_tokens, recent;
  int split;                     // CTAs per (request, KV head) that select
  int cached;                    // weights per warp that they keep in shared memory
};

cudaError_t launch_evict(EvictParams &p, int num_sms, cudaStream_t stream);   // sets p.split, p.cached

}  // namespace sa
