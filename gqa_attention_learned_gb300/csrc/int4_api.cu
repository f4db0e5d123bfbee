// Entry points of the operators on a cache held in 4 bits: argument checks, plans and
// launches.  The operations are specified in include/sinkattn.h.  Nothing here
// allocates device memory or synchronises.

#include "sinkattn.h"
#include "api.cuh"
#include "int4.cuh"
#include "workspace.cuh"

#include <algorithm>
#include <cmath>

namespace {

using sa::kHeadDim;
using sa::kPageSize;

// Pages that a warp takes at least: more warps and parts to join against longer chains.
// us at 2 / 4 / 8 / 16: one token of one request of 2000 keys 9.2 / 10.5 / 12.5 / 15.2,
// four tokens on 4000 keys 18.0 / 19.4 / 21.2 / 27.9; calls that fill the GPU do not care
// (64 requests 32.8 / 32.8 / 32.8 / 32.7).  So 2 is no slower anywhere measured; 8 is what
// everything else here was measured with.
constexpr int kMinPages = 8;

// Query rows per KV head up to which the kernel of few rows is taken.  us of that and of
// the other, 16 requests of 4096..32768 keys: 32 rows 115 and 146, 64 rows 206 and 146;
// 64 requests of up to 4096 keys: 32 rows 71 and 85, 64 rows 122 and 86; one of 4000:
// 20.7 and 17.7, 21.2 and 17.9 (the rule does not look at how few requests there are, and
// loses those 3 us).
constexpr int kFewRows = 32;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// A bound on lengths as the kernels take it: they round it up to whole pages.
int longest(int bound) { return std::min(bound, 0x7fff0000); }

bool known_flags(int flags) {
  return flags == SINKATTN_LAUNCH_DEFAULT || flags == SINKATTN_LAUNCH_PLAIN ||
         flags == SINKATTN_LAUNCH_PROGRAMMATIC;
}

// The kernel of many rows shares a request's keys out among CTAs where there are at most
// kSplitCtas of them per SM without, with up to kSplitParts more per SM: 64 tokens on
// 120000 keys 1028 us without, 172 with; two short turns on 20000 and 30000 keys 268 and
// 196.  What it costs where nothing is gained is 5%: two prompts' chunks of 500 tokens,
// 256 CTAs, 212 us without, 222 with.
constexpr int kSplitCtas = 2, kSplitParts = 3;
int most_split_ctas(int sms) {
  return std::min<long long>((kSplitCtas + kSplitParts) * static_cast<long long>(sms), sa::kCounterSpan / sizeof(int));
}

size_t workspace_for(int sms) {
  size_t most = 0;
  for (int blocks : {1, 2, 4})
    most = std::max(most, sa::int4_decode_results_bytes(blocks, sms * sa::int4_decode_ctas_per_sm(blocks)));
  most = std::max(most, sa::int4_prefill_results_bytes(most_split_ctas(sms)));
  return sa::kCounterSpan + ((most + 255) & ~size_t(255));
}

// Attention of all three forms; cu_seqlens_q null: q_len tokens per request.
int attention_entry(sa::Int4Mode mode, const void *q, const int32_t *cu_seqlens_q, int num_seqs,
                    int total_q, int max_q_len, const void *kv_cache, const int32_t *page_table,
                    int max_pages_per_seq, const int32_t *kv_lens, const uint64_t *tree_mask,
                    int num_pages, int max_kv_len, const float *sinks, float scale, void *out,
                    float *lse, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                    void *workspace, size_t workspace_bytes, int launch_flags, void *stream) {
  if (!known_flags(launch_flags)) return SINKATTN_INVALID_ARGUMENT;
  if (head_dim != kHeadDim || page_size != kPageSize) return SINKATTN_UNSUPPORTED;
  if (num_seqs < 0 || total_q < 0 || max_q_len < 0 || max_kv_len < 0 || num_qo_heads <= 0 ||
      num_kv_heads <= 0 || num_qo_heads % num_kv_heads || num_pages <= 0 || max_pages_per_seq <= 0 ||
      !std::isfinite(scale))
    return SINKATTN_INVALID_ARGUMENT;
  if (num_seqs == 0 || total_q == 0) return SINKATTN_OK;
  if (!q || !kv_cache || !page_table || !kv_lens || !sinks || !out ||
      (mode == sa::kInt4Ragged && !cu_seqlens_q))
    return SINKATTN_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(page_table, 4) ||
      !aligned(kv_lens, 4) || !aligned(sinks, 4) || !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(tree_mask, 8))
    return SINKATTN_INVALID_ARGUMENT;
  // rows and units are counted in ints
  if (static_cast<long long>(num_qo_heads) * std::max(total_q, num_seqs) > 0x7fffff00ll)
    return SINKATTN_UNSUPPORTED;
  max_q_len = std::min(max_q_len, total_q);            // bounds may be loose
  const int sms = sa::api_sm_count();
  if (sms == 0) return sa::api_failure("no CUDA device (SM count query failed)");
  if (!workspace || workspace_bytes < workspace_for(sms)) return SINKATTN_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 256)) return SINKATTN_INVALID_ARGUMENT;

  sa::Int4AttnParams p{};
  p.q = static_cast<const uint16_t *>(q);
  p.kv_cache = static_cast<const uint8_t *>(kv_cache);
  p.page_table = page_table;
  p.kv_lens = kv_lens;
  p.cu_seqlens_q = cu_seqlens_q;
  p.tree_mask = tree_mask;
  p.sinks = sinks;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.scale_log2 = scale * sa::kLog2e;
  p.max_pages_per_seq = max_pages_per_seq;
  p.num_seqs = num_seqs;
  p.q_len = mode == sa::kInt4Ragged ? 0 : max_q_len;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.max_kv_len = longest(max_kv_len);
  p.num_qo_heads = num_qo_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_qo_heads / num_kv_heads;
  p.num_pages = num_pages;
  p.min_pages = kMinPages;
  p.sms = sms;

  const int rows = static_cast<int>(std::min<long long>(static_cast<long long>(max_q_len) * p.group, 1 << 20));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t *const ws = static_cast<uint8_t *>(workspace);
  if (mode != sa::kInt4Decode && p.group <= 128 && rows > kFewRows) {
    const int tokens = sa::int4_prefill_tokens(p.group);
    long long tiles = mode == sa::kInt4Verify ? num_seqs * ceil_div(max_q_len, tokens)
                                              : total_q / tokens + static_cast<long long>(num_seqs);
    if (tiles * num_kv_heads > 0x7fffffffll) return SINKATTN_UNSUPPORTED;
    if (tiles * num_kv_heads <= static_cast<long long>(kSplitCtas) * sms) {
      const int keys = std::min<long long>(p.max_kv_len, static_cast<long long>(max_pages_per_seq) * kPageSize);
      p.split_parts = kSplitParts * sms / num_kv_heads;
      p.split_from = static_cast<int>(tiles);
      const long long more = std::min<long long>(p.split_parts, tiles * (ceil_div(keys, sa::kInt4PartKeys) - 1));
      if (more <= 0 || (tiles + more) * num_kv_heads > most_split_ctas(sms)) p.split_parts = 0;
      else tiles += more;
    }
    if (p.split_parts > 0) {
      p.counters = reinterpret_cast<int *>(ws);
      p.ws_o = reinterpret_cast<float *>(ws + sa::kCounterSpan);
      p.ws_md = reinterpret_cast<float2 *>(p.ws_o + static_cast<size_t>(tiles) * num_kv_heads * 256 * kHeadDim);
    }
    return sa::api_status(sa::launch_int4_prefill(p, tiles * num_kv_heads, st), "int4 attention launch");
  }
  const int blocks = sa::int4_row_blocks(rows);
  const int slots = sms * sa::int4_decode_ctas_per_sm(blocks);
  const long long pages = std::max(1ll, std::min<long long>(ceil_div(p.max_kv_len, kPageSize), max_pages_per_seq));
  // Row blocks of a KV head: of the longest requests, or of all tokens, which leave each
  // request a block that is not full.  (As a double: the product of loose bounds need not
  // fit an integer.)
  const double row_blocks =
      std::min(static_cast<double>(num_seqs) * ceil_div(static_cast<long long>(max_q_len) * p.group, 8 * blocks),
               static_cast<double>(total_q) * p.group / (8 * blocks) + num_seqs);
  const double work = row_blocks * num_kv_heads * static_cast<double>(pages);
  const int ctas = static_cast<int>(std::max(1.0, std::min<double>(slots, std::ceil(work / (8.0 * kMinPages)))));
  // a warp counts its share of the pages, and a unit's start as 8, in ints
  if (work * (1 + 8.0) / (8.0 * ctas) > 0x7f000000) return SINKATTN_UNSUPPORTED;
  p.counters = reinterpret_cast<int *>(ws);
  p.ws_o = reinterpret_cast<float *>(ws + sa::kCounterSpan);
  p.ws_md = reinterpret_cast<float2 *>(p.ws_o + static_cast<size_t>(ctas) * 2 * 8 * blocks * kHeadDim);
  return sa::api_status(sa::launch_int4_decode(p, mode, blocks, ctas, st,
                                               mode != sa::kInt4Ragged && sa::programmatic_for(launch_flags)),
                        "int4 attention launch");
}

}  // namespace

extern "C" {

int sinkattn_int4_workspace_bytes(int num_sms, size_t *workspace_bytes) {
  if (!workspace_bytes || num_sms < 0) return SINKATTN_INVALID_ARGUMENT;
  if (num_sms == 0) {
    num_sms = sa::api_sm_count();
    if (num_sms == 0) return sa::api_failure("no CUDA device to plan for");
  }
  *workspace_bytes = workspace_for(num_sms);
  return SINKATTN_OK;
}

int sinkattn_qkv_prologue_int4(const void *qkv, const void *bias, const int32_t *positions,
                               const int32_t *slot_mapping, const float *rope, int rope_positions,
                               int rope_style, void *q_out, void *kv_cache, int num_tokens,
                               int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                               int num_pages, void *stream) {
  if (head_dim != kHeadDim || page_size != kPageSize) return SINKATTN_UNSUPPORTED;
  if (num_tokens < 0 || num_qo_heads <= 0 || num_kv_heads <= 0 || num_pages <= 0 || rope_positions <= 0 ||
      (rope_style != SINKATTN_ROPE_HALF && rope_style != SINKATTN_ROPE_INTERLEAVED))
    return SINKATTN_INVALID_ARGUMENT;
  if (num_tokens == 0) return SINKATTN_OK;
  if (!qkv || !positions || !slot_mapping || !rope || !q_out || !kv_cache) return SINKATTN_INVALID_ARGUMENT;
  if (!aligned(qkv, 16) || !aligned(bias, 16) || !aligned(q_out, 16) || !aligned(kv_cache, 16) ||
      !aligned(positions, 4) || !aligned(slot_mapping, 4) || !aligned(rope, 4))
    return SINKATTN_INVALID_ARGUMENT;
  if (num_qo_heads + 2ll * num_kv_heads > std::min(0x7ffff000ll / 4 / num_tokens, 0x7fffffffll / kHeadDim))
    return SINKATTN_UNSUPPORTED;
  sa::Int4PrologueParams p{};
  p.qkv = static_cast<const uint16_t *>(qkv);
  p.bias = static_cast<const uint16_t *>(bias);
  p.positions = positions;
  p.slot_mapping = slot_mapping;
  p.rope = rope;
  p.q_out = static_cast<uint16_t *>(q_out);
  p.kv_cache = static_cast<uint8_t *>(kv_cache);
  p.rope_positions = rope_positions;
  p.num_tokens = num_tokens;
  p.num_qo_heads = num_qo_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_pages = num_pages;
  p.interleaved = rope_style == SINKATTN_ROPE_INTERLEAVED;
  return sa::api_status(sa::launch_int4_prologue(p, static_cast<cudaStream_t>(stream)), "int4 prologue launch");
}

int sinkattn_gather_int4(const void *kv_cache, const int32_t *slots, int num_rows, void *k, void *v,
                         int num_kv_heads, int head_dim, int page_size, int num_pages, void *stream) {
  if (head_dim != kHeadDim || page_size != kPageSize) return SINKATTN_UNSUPPORTED;
  if (num_rows < 0 || num_kv_heads <= 0 || num_pages <= 0) return SINKATTN_INVALID_ARGUMENT;
  if (num_rows == 0) return SINKATTN_OK;
  if (!kv_cache || !slots || !k || !v) return SINKATTN_INVALID_ARGUMENT;
  if (!aligned(kv_cache, 16) || !aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16))
    return SINKATTN_INVALID_ARGUMENT;
  // 16 rows of a KV head to a CTA
  if (static_cast<long long>(num_rows) * num_kv_heads > 16ll * 0x7fffffffll) return SINKATTN_UNSUPPORTED;
  sa::Int4GatherParams p{};
  p.kv_cache = static_cast<const uint8_t *>(kv_cache);
  p.slots = slots;
  p.k = static_cast<uint16_t *>(k);
  p.v = static_cast<uint16_t *>(v);
  p.num_rows = num_rows;
  p.num_kv_heads = num_kv_heads;
  p.num_pages = num_pages;
  return sa::api_status(sa::launch_int4_gather(p, static_cast<cudaStream_t>(stream)), "int4 gather launch");
}

int sinkattn_decode_int4(const void *q, const void *kv_cache, const int32_t *page_table,
                         int max_pages_per_seq, const int32_t *kv_lens, const float *sinks, float scale,
                         void *out, float *lse, int batch, int num_qo_heads, int num_kv_heads,
                         int head_dim, int page_size, int num_pages, int max_kv_len, void *workspace,
                         size_t workspace_bytes, int launch_flags, void *stream) {
  return attention_entry(sa::kInt4Decode, q, nullptr, batch, batch, 1, kv_cache, page_table, max_pages_per_seq,
                         kv_lens, nullptr, num_pages, max_kv_len, sinks, scale, out, lse, num_qo_heads,
                         num_kv_heads, head_dim, page_size, workspace, workspace_bytes, launch_flags, stream);
}

int sinkattn_verify_int4(const void *q, const void *kv_cache, const int32_t *page_table,
                         int max_pages_per_seq, const int32_t *kv_lens, const uint64_t *tree_mask,
                         const float *sinks, float scale, void *out, float *lse, int batch, int q_len,
                         int num_qo_heads, int num_kv_heads, int head_dim, int page_size, int num_pages,
                         int max_kv_len, void *workspace, size_t workspace_bytes, int launch_flags,
                         void *stream) {
  if (q_len < 1 || q_len > SINKATTN_MAX_VERIFY_TOKENS || batch < 0) return SINKATTN_INVALID_ARGUMENT;
  const long long rows = static_cast<long long>(batch) * q_len;
  if (rows > 0x7fffffffll) return SINKATTN_UNSUPPORTED;
  return attention_entry(sa::kInt4Verify, q, nullptr, batch, static_cast<int>(rows), q_len, kv_cache,
                         page_table, max_pages_per_seq, kv_lens, tree_mask, num_pages, max_kv_len, sinks,
                         scale, out, lse, num_qo_heads, num_kv_heads, head_dim, page_size, workspace,
                         workspace_bytes, launch_flags, stream);
}

int sinkattn_prefill_paged_int4(const void *q, const int32_t *cu_seqlens_q, int num_seqs, int total_q,
                                int max_q_len, const void *kv_cache, const int32_t *page_table,
                                int max_pages_per_seq, const int32_t *kv_lens, int num_pages,
                                int max_kv_len, const float *sinks, float scale, void *out, float *lse,
                                int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                                void *workspace, size_t workspace_bytes, void *stream) {
  return attention_entry(sa::kInt4Ragged, q, cu_seqlens_q, num_seqs, total_q, max_q_len, kv_cache,
                         page_table, max_pages_per_seq, kv_lens, nullptr, num_pages, max_kv_len, sinks,
                         scale, out, lse, num_qo_heads, num_kv_heads, head_dim, page_size, workspace,
                         workspace_bytes, SINKATTN_LAUNCH_PLAIN, stream);
}

}  // extern "C"
