// Cache held in 4 bits: layout, parameters and launchers of the operators on it.
//
// A row of 64 keys' or values' elements is 64 codes n of 4 bits, a scale s of 4
// significant bits and a zero point z in 0..15, and stands for s * (n - z): at
// most 4 x 4 significant bits, so each value is a bf16 number exactly and the
// cache equals a bf16 cache of these values.  s and z share 16 bits: s is a bf16
// number whose last four mantissa bits are zero, and z lies in them.
//
// A page holds, for each KV head, one block of 1088 bytes (34 whole 32-byte
// sectors), K and V together, so that one copy brings both.  Every token owns
// whole bytes, in the order in which the matrix fragments want them: lane (g, t)
// of a warp reads its share of 16 keys with one 16-byte load each for K and V.
//   bytes    0..511   K: slot j, t = 0..3: 8 bytes at 64 (j % 8) + 16 t + 8 (j / 8),
//                     two words: dims 8t + e and 32 + 8t + e (e = 0..7) at bits 4e,
//                     the word rotated left by 3 (see field())
//   bytes  512..1023  V: slot j, g = 0..7: the word at 512 + 64 g + 16 (j % 8 / 2) +
//                     8 (j / 8) + 4 (j % 2): dims 8g + e at bits 4e
//   bytes 1024..1087  slot j: the word at 1024 + 8 (j % 8) + 4 (j / 8): K's s and z
//                     in the low half, V's in the high half
#pragma once

#include "kernels.cuh"

namespace sa {

constexpr int kInt4Block = 1088;          // bytes of one KV head's share of a page
constexpr int kInt4K = 0, kInt4V = 512, kInt4Meta = 1024;

// ---------------------------------------------------------------- prologue
struct Int4PrologueParams {
  const uint16_t *qkv;           // bf16 [T][(Hq + 2 Hkv) * 64], q heads, then k, then v
  const uint16_t *bias;          // bf16 [(Hq + 2 Hkv) * 64] or null
  const int32_t *positions;      // [T]: rows of rope; outside of it: NaN
  const int32_t *slot_mapping;   // [T]: page * 16 + slot; < 0 or past the pool: no write
  const float *rope;             // [rope_positions][32 cos, 32 sin]
  uint16_t *q_out;               // bf16 [T][Hq][64]
  uint8_t *kv_cache;             // [num_pages][Hkv][1088]
  int rope_positions;
  int num_tokens, num_qo_heads, num_kv_heads, num_pages;
  int interleaved;               // 0: pairs (i, i + 32); 1: pairs (2i, 2i + 1)
};

cudaError_t launch_int4_prologue(const Int4PrologueParams &p, cudaStream_t stream);

// ------------------------------------------------------------------ gather
struct Int4GatherParams {
  const uint8_t *kv_cache;       // [num_pages][Hkv][1088]
  const int32_t *slots;          // [T]: page * 16 + slot; outside of the pool: NaN rows
  uint16_t *k, *v;               // bf16 [T][Hkv][64]
  int num_rows, num_kv_heads, num_pages;
};

cudaError_t launch_int4_gather(const Int4GatherParams &p, cudaStream_t stream);

// --------------------------------------------------------------- attention
// The query rows of one KV head of a request are ordered (token, head in group).
struct Int4AttnParams {
  const uint16_t *q;             // bf16 [rows][Hq][64]
  const uint8_t *kv_cache;       // [num_pages][Hkv][1088]
  const int32_t *page_table;     // [n][max_pages_per_seq]
  const int32_t *kv_lens;        // [n]
  const int32_t *cu_seqlens_q;   // [n + 1], or null: q_len tokens each
  const uint64_t *tree_mask;     // [n][q_len] or null (causal)
  const float *sinks;            // [Hq]
  uint16_t *out;                 // bf16 [rows][Hq][64]
  float *lse;                    // [rows][Hq] or null
  int *counters;                 // one per CTA, zero between calls
  float *ws_o;                   // fp32 [2 ctas][block rows][64] (tensor cores: [ctas][16][256][4])
  float2 *ws_md;                 // [2 ctas][block rows] (tensor cores: [ctas][256]): maximum (base 2), sum
  float scale_log2;              // scale * log2(e)
  int max_pages_per_seq, num_seqs, q_len, total_q, max_q_len, max_kv_len;
  int num_qo_heads, num_kv_heads, group, num_pages;
  int min_pages;                 // pages that a warp takes at least
  int sms;
  int split_parts, split_from;   // tensor-core form: parts of the keys beyond one for each of split_from
                                 // blocks of a KV head's rows; 0: none
};

enum Int4Mode { kInt4Decode, kInt4Verify, kInt4Ragged };

// 8-row blocks that a CTA works on (1, 2 or 4) for `rows` query rows per KV head.
inline int int4_row_blocks(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }
int int4_decode_ctas_per_sm(int row_blocks);
size_t int4_decode_results_bytes(int row_blocks, int ctas);   // of ws_o and ws_md

cudaError_t launch_int4_decode(const Int4AttnParams &p, Int4Mode mode, int row_blocks, int ctas,
                               cudaStream_t stream, bool programmatic);

// Tensor-core form: for groups of at most 128 heads.  Tokens of a CTA; CTAs for one
// KV head are at most total_q / tokens + num_seqs.
int int4_prefill_tokens(int group);
// Keys that a part has at least (8 tokens on 4000 keys: 32.6 us at 256, 31.4 at 512, 32.9
// at 1024, 37.9 at 2048).
constexpr int kInt4PartKeys = 512;
size_t int4_prefill_results_bytes(int ctas);     // of ws_o and ws_md
cudaError_t launch_int4_prefill(const Int4AttnParams &p, long long ctas, cudaStream_t stream);

}  // namespace sa
