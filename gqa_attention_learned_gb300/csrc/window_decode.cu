// One new token per request with a sliding window and first tokens that stay
// visible, learned sinks, over the paged cache.
//
// Mathematics: the token (position kv_len - 1) sees keys [0, first) and
// [kv_len - window, kv_len); online softmax in base 2 started at the sink in
// the first chunk's first warp, at -inf elsewhere, joined by log-sum-exp.
//
// A windowed layer reads few pages per request (window 128: nine or ten), so
// the call is bound by latency, not by HBM: what counts is how soon the last
// load is issued and how few steps follow it.  Hence no shared-memory staging
// and no copy engine (nor tensor maps to encode on the host): K and V go from
// global memory straight into mma.sync fragments.  Both products have a free
// permutation that makes every load a whole 16-byte piece:
//   S[heads x keys] = Q K^T   the order of the 64 products of a dot product
//     is free: lane (g, t) of a warp loads pieces t and t + 4 of key row g and
//     takes them as its share of the k index; Q is loaded with the same order.
//   O[heads x dims] = P V     the accumulators of S are the A fragments of P;
//     lane (g, t) loads piece g (dims 8g .. 8g+7) of its four keys 2t, 2t+1,
//     2t+8, 2t+9, pairs the keys by byte permutes, and n-tile i holds dims
//     8n + i: each lane ends up with 16 consecutive dims of its row.
// One CTA = one (request, KV head, block of 8 or 16 query heads, chunk of
// visited pages), 4 warps taking pages round-robin with two pages in flight
// each.  Warps join through shared memory; chunks through the workspace, by the
// last CTA of a request to finish, in chunk order (as in plain decode).
//
// Measured (64 / 8 heads, replayed from a graph): one request of window 128
// 6.3 us, 64 requests 10.4 us (2.6 us at the copy bandwidth: two waves of loads
// that depend on one another), 8 requests of window 16384 50 us (5.4 TB/s; 52.7
// with one page in flight and 4 CTAs per SM).  Three pages in flight and 2 CTAs
// per SM, 2 warps per CTA, or more CTAs with fewer registers are slower.

#include "bounded.cuh"
#include "bounded_ptx.cuh"
#include "workspace.cuh"

#include <algorithm>
#include <cmath>

namespace sa {
namespace {

constexpr int kNW = 4;                       // warps per CTA
constexpr int kCtasPerSm = 3;                // with two pages in flight per warp; four with one
constexpr int kFewPages = 8 * kNW;           // pages per CTA that count as few
constexpr int kPieces = kHeadDim * 2 / 16;   // 16-byte pieces of a row
constexpr int kStride = kHeadDim + 4;        // floats per joined row

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Pages that hold a visible key, numbered through: the first tokens', then the
// window's.  page(v) is the request's page behind number v.
struct VisiblePages {
  int count, skip_from, skip, start;
  __device__ __forceinline__ VisiblePages(const WindowDecodeParams &p, int kv_len) {
    start = max(0, kv_len - p.window);
    skip_from = min(ceil_div(p.first_tokens, kPageSize), start / kPageSize);
    skip = start / kPageSize - skip_from;
    count = ceil_div(max(kv_len, 0), kPageSize) - skip;
  }
  __device__ __forceinline__ int page(int v) const { return v >= skip_from ? v + skip : v; }
};

// One page's K and V as fragments.
struct Page {
  uint4 k[2][2];      // key 8n + g, pieces t and t + 4
  uint4 v[4];         // keys 2t, 2t + 1, 2t + 8, 2t + 9, piece g
};

template <int NB, int kAhead>       // 8-head blocks per CTA, pages in flight per warp: 1 or 2
__global__ void __launch_bounds__(kNW * 32, kCtasPerSm + 2 - kAhead)
window_decode_kernel(const WindowDecodeParams p) {
  constexpr int kRows = 8 * NB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int units = p.num_kv_heads * p.head_blocks;
  const int unit_y = static_cast<int>(blockIdx.x % units);
  const int hb = unit_y % p.head_blocks, kvh = unit_y / p.head_blocks;
  const int slot = static_cast<int>(blockIdx.x / units);
  const int b = slot / p.num_splits, chunk = slot % p.num_splits;
  const int row0 = hb * kRows;                         // first head of this CTA within the group
  const int rows = min(kRows, p.group - row0);
  const size_t head0 = static_cast<size_t>(b) * p.num_qo_heads + kvh * p.group + row0;

  const int kv_len = p.kv_lens[b];
  bool bad = kv_len < 0 || kv_len > p.max_kv_len || ceil_div(kv_len, kPageSize) > p.max_pages_per_seq;
  const VisiblePages visible(p, bad ? 0 : kv_len);
  bad = bad || visible.count > p.num_splits * p.pages_per_chunk;
  const int nchunks = bad ? 1 : max(1, ceil_div(visible.count, p.pages_per_chunk));
  if (chunk >= nchunks) return;                        // uniform over the CTA
  const int p_end = bad ? 0 : min(visible.count, (chunk + 1) * p.pages_per_chunk);
  const int first = chunk * p.pages_per_chunk + warp;
  const int n_my = p_end > first ? ceil_div(p_end - first, kNW) : 0;
  const int32_t *table = p.page_table + static_cast<size_t>(b) * p.max_pages_per_seq;

  // ids of this warp's pages, 32 at a time (lane j holds page j of the batch)
  auto load_ids = [&](int base) -> int {
    const int j = base + lane;
    return j < n_my ? table[visible.page(first + j * kNW)] : -1;
  };
  int ids = load_ids(0), ids_next = load_ids(32);

  // Up to here only kv_lens and page_table were read; everything below may
  // depend on the previous kernel on the stream.
  grid_dependency_wait();
  launch_dependents();

  const uint4 zero4 = make_uint4(0, 0, 0, 0);
  const uint4 *kbase = reinterpret_cast<const uint4 *>(p.k_cache);
  const uint4 *vbase = reinterpret_cast<const uint4 *>(p.v_cache);
  auto fetch = [&](int i, Page &f) {                   // all lanes call, i warp-uniform
    if (i >= n_my) return;
    if ((i & 31) == 0 && i > 0) {
      ids = ids_next;
      ids_next = load_ids(i + 32);
    }
    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
    if (id < 0 || id >= p.num_pages) {
      bad = true;                                      // never dereferenced
      f.k[0][0] = f.k[0][1] = f.k[1][0] = f.k[1][1] = zero4;
      f.v[0] = f.v[1] = f.v[2] = f.v[3] = zero4;
      return;
    }
    const size_t at = (static_cast<size_t>(id) * p.num_kv_heads + kvh) * (kPageSize * kPieces);
    const uint4 *k = kbase + at + g * kPieces + t;
    f.k[0][0] = ld_stream(k);
    f.k[0][1] = ld_stream(k + 4);
    f.k[1][0] = ld_stream(k + 8 * kPieces);
    f.k[1][1] = ld_stream(k + 8 * kPieces + 4);
    const uint4 *v = vbase + at + 2 * t * kPieces + g;
    f.v[0] = ld_stream(v);
    f.v[1] = ld_stream(v + kPieces);
    f.v[2] = ld_stream(v + 8 * kPieces);
    f.v[3] = ld_stream(v + 9 * kPieces);
  };
  Page f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fetch(u, f[u]);

  // Q as A fragments: rows g and g + 8, k index in the order of K's pieces
  uint4 qa[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = g + 8 * nb;
    const uint4 *q = reinterpret_cast<const uint4 *>(p.q) + (head0 + r) * kPieces;
    qa[nb][0] = r < rows ? __ldg(q + t) : zero4;
    qa[nb][1] = r < rows ? __ldg(q + t + 4) : zero4;
  }
  // softmax state of rows g + 8 nb (d: this lane's keys only).  A sink that is no
  // logit (NaN, +inf) is kept out of the running maximum, where a comparison may
  // not see it, and spoils the sum, which spoils the row and its lse.
  float m[NB], d[NB];
  float o[8][2 * NB];                 // n-tile i: row g dims 16t + i, 16t + 8 + i; then row g + 8
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = g + 8 * nb;
    const bool sink = chunk == 0 && warp == 0 && r < rows;
    const float logit = sink ? __ldg(p.sinks + kvh * p.group + row0 + r) * kLog2e : -INFINITY;
    const bool fine = logit < INFINITY;
    m[nb] = fine ? logit : -INFINITY;
    d[nb] = sink && t == 0 ? (fine ? 1.f : NAN) : 0.f;  // e^(sink - m) = 1, counted once
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 2 * NB; ++e) o[i][e] = 0.f;

  auto step = [&](int i, Page &f) {
    const int tok0 = visible.page(first + i * kNW) * kPageSize;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo[4] = {qa[0][h].x, NB > 1 ? qa[NB - 1][h].x : 0u, qa[0][h].y,
                                NB > 1 ? qa[NB - 1][h].y : 0u};
        const uint32_t hi[4] = {qa[0][h].z, NB > 1 ? qa[NB - 1][h].z : 0u, qa[0][h].w,
                                NB > 1 ? qa[NB - 1][h].w : 0u};
        mma_bf16_16816(s[n], lo, f.k[n][h].x, f.k[n][h].y);
        mma_bf16_16816(s[n], hi, f.k[n][h].z, f.k[n][h].w);
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2 * NB; ++e) s[n][e] *= p.scale_log2;
    if (tok0 + kPageSize > kv_len || (tok0 < visible.start && tok0 + kPageSize > p.first_tokens)) {
      // keys 8n + 2t + e of the page outside the visible ranges (they may hold
      // anything, even NaN)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = tok0 + 8 * n + 2 * t + e;
          if (tok < kv_len && (tok >= visible.start || tok < p.first_tokens)) continue;
          s[n][e] = -INFINITY;
          if constexpr (NB > 1) s[n][2 + e] = -INFINITY;
          f.v[2 * n + e] = zero4;
        }
    }
    uint32_t a[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x = fmaxf(fmaxf(s[0][2 * nb], s[0][2 * nb + 1]), fmaxf(s[1][2 * nb], s[1][2 * nb + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const float n = fmaxf(m[nb], x);
      const float u = n == -INFINITY ? 0.f : n;
      // o and d only need rescaling when a running max grew
      if (__any_sync(0xffffffffu, n > m[nb])) {
        const float w = ex2(m[nb] - u);
        d[nb] *= w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i][2 * nb] *= w;
          o[i][2 * nb + 1] *= w;
        }
      }
      m[nb] = n;
      const float p0 = ex2(s[0][2 * nb] - u), p1 = ex2(s[0][2 * nb + 1] - u);
      const float p2 = ex2(s[1][2 * nb] - u), p3 = ex2(s[1][2 * nb + 1] - u);
      d[nb] += (p0 + p1) + (p2 + p3);
      a[nb] = pack_bf16(p0, p1);                       // keys 2t, 2t + 1
      a[2 + nb] = pack_bf16(p2, p3);                   // keys 2t + 8, 2t + 9
    }
    auto word = [](const uint4 &x, int w) { return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // dim 8g + i of the four keys, two keys to a register
      const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
      const uint32_t b0 = __byte_perm(word(f.v[0], i / 2), word(f.v[1], i / 2), sel);
      const uint32_t b1 = __byte_perm(word(f.v[2], i / 2), word(f.v[3], i / 2), sel);
      float c[4] = {o[i][0], o[i][1], NB > 1 ? o[i][2 * NB - 2] : 0.f, NB > 1 ? o[i][2 * NB - 1] : 0.f};
      mma_bf16_16816(c, a, b0, b1);
      o[i][0] = c[0];
      o[i][1] = c[1];
      if constexpr (NB > 1) {
        o[i][2] = c[2];
        o[i][3] = c[3];
      }
    }
  };
  for (int i0 = 0; i0 < n_my; i0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u >= n_my) break;                       // warp-uniform
      step(i0 + u, f[u]);
      fetch(i0 + u + kAhead, f[u]);
    }
  }

  // ---- join the warps
  __shared__ __align__(16) float so[kNW][kRows][kStride];
  __shared__ float sm[kNW][kRows], sd[kNW][kRows];
  __shared__ int is_last;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    d[nb] += __shfl_xor_sync(0xffffffffu, d[nb], 1);
    d[nb] += __shfl_xor_sync(0xffffffffu, d[nb], 2);
    const int r = g + 8 * nb;
    if (t == 0) {
      sm[warp][r] = m[nb];
      sd[warp][r] = d[nb];
    }
    float4 *dst = reinterpret_cast<float4 *>(&so[warp][r][16 * t]);
    dst[0] = make_float4(o[0][2 * nb], o[1][2 * nb], o[2][2 * nb], o[3][2 * nb]);
    dst[1] = make_float4(o[4][2 * nb], o[5][2 * nb], o[6][2 * nb], o[7][2 * nb]);
    dst[2] = make_float4(o[0][2 * nb + 1], o[1][2 * nb + 1], o[2][2 * nb + 1], o[3][2 * nb + 1]);
    dst[3] = make_float4(o[4][2 * nb + 1], o[5][2 * nb + 1], o[6][2 * nb + 1], o[7][2 * nb + 1]);
  }
  const bool failed = __syncthreads_or(bad);
  const size_t stride = static_cast<size_t>(p.batch) * p.num_qo_heads;
  for (int item = threadIdx.x; item < rows * (kHeadDim / 4); item += kNW * 32) {
    const int r = item / (kHeadDim / 4), dq = (item % (kHeadDim / 4)) * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kNW; ++w) mx = fmaxf(mx, sm[w][r]);
    float den = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      const float wt = sm[w][r] == -INFINITY ? 0.f : ex2(sm[w][r] - mx);
      den += wt * sd[w][r];
      const float4 ov = *reinterpret_cast<const float4 *>(&so[w][r][dq]);
      acc[0] += wt * ov.x;
      acc[1] += wt * ov.y;
      acc[2] += wt * ov.z;
      acc[3] += wt * ov.w;
    }
    // (a NaN score leaves den NaN, and so the row and its lse)
    const float inv = failed ? NAN : den == 0.f ? 0.f : 1.f / den;
    const float lse2 = failed ? NAN : den == 0.f ? -INFINITY : mx + lg2(den);
    const size_t row = head0 + r;
    if (nchunks == 1) {
      uint2 packed;
      packed.x = pack_bf16(acc[0] * inv, acc[1] * inv);
      packed.y = pack_bf16(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2 *>(p.out + row * kHeadDim + dq) = packed;
      if (dq == 0 && p.lse) p.lse[row] = lse2 * kLn2;
    } else {
      const size_t wrow = static_cast<size_t>(chunk) * stride + row;
      *reinterpret_cast<float4 *>(p.ws_o + wrow * kHeadDim + dq) =
          make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (dq == 0) p.ws_lse[wrow] = lse2;
    }
  }
  if (nchunks == 1) return;

  // ---- join the chunks: the last CTA of the request to get here (it leaves
  // the counter at zero for the next call)
  __threadfence();
  __syncthreads();
  int *counter = p.counters + static_cast<size_t>(b) * units + unit_y;
  if (threadIdx.x == 0) is_last = atomicAdd(counter, 1) == nchunks - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  for (int item = threadIdx.x; item < rows * (kHeadDim / 4); item += kNW * 32) {
    const int r = item / (kHeadDim / 4), dq = (item % (kHeadDim / 4)) * 4;
    const size_t row = head0 + r;
    float mx = -INFINITY, den = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool poisoned = false;       // a chunk met a page outside the pool, or a NaN score
    for (int c = 0; c < nchunks; ++c) {
      const float lc = __ldcg(p.ws_lse + c * stride + row);
      poisoned = poisoned || lc != lc;
      if (!(lc > -INFINITY)) continue;
      const float4 ov = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + (c * stride + row) * kHeadDim + dq));
      const float nm = fmaxf(mx, lc);
      const float a = mx == -INFINITY ? 0.f : ex2(mx - nm);
      const float wt = ex2(lc - nm);
      den = den * a + wt;
      acc[0] = acc[0] * a + wt * ov.x;
      acc[1] = acc[1] * a + wt * ov.y;
      acc[2] = acc[2] * a + wt * ov.z;
      acc[3] = acc[3] * a + wt * ov.w;
      mx = nm;
    }
    const float inv = poisoned ? NAN : den == 0.f ? 0.f : 1.f / den;
    uint2 packed;
    packed.x = pack_bf16(acc[0] * inv, acc[1] * inv);
    packed.y = pack_bf16(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2 *>(p.out + row * kHeadDim + dq) = packed;
    if (dq == 0 && p.lse) p.lse[row] = poisoned ? NAN : (den == 0.f ? -INFINITY : (mx + lg2(den)) * kLn2);
  }
  if (threadIdx.x == 0) *counter = 0;
  // zero again, too: results where another plan has its counters
  const float *end = counter_span_end(p.counters);
  __syncthreads();                                     // they have been read
  for (int c = 0; c < nchunks && p.ws_o + c * stride * kHeadDim < end; ++c)
    for (int item = threadIdx.x; item < rows * (kHeadDim / 4); item += kNW * 32) {
      float *at = p.ws_o + (c * stride + head0) * kHeadDim + item * 4;
      if (at < end) *reinterpret_cast<float4 *>(at) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  if (p.ws_lse < end)
    for (int item = threadIdx.x; item < nchunks * rows; item += kNW * 32) {
      float *at = p.ws_lse + (item / rows) * stride + head0 + item % rows;
      if (at < end) *at = 0.f;
    }
}

template <int NB, int kAhead>
cudaError_t launch_variant(const WindowDecodeParams &p, cudaStream_t stream, bool programmatic) {
  const unsigned long long ctas =
      static_cast<unsigned long long>(p.num_splits) * p.batch * p.num_kv_heads * p.head_blocks;
  if (ctas > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  return launch_kernel(window_decode_kernel<NB, kAhead>, static_cast<unsigned>(ctas), kNW * 32, 0, stream,
                       programmatic, p);
}

}  // namespace

int window_decode_ctas_per_sm() { return kCtasPerSm; }

cudaError_t launch_window_decode(const WindowDecodeParams &p, cudaStream_t stream, bool programmatic) {
  // More CTAs of few pages than three per SM hold: four fit with one page in
  // flight per warp (64 / 8 heads: 64 requests of window 128 10.4 us instead of
  // 12.6, of window 512 17.8 instead of 19.2; of window 2048 45.2 instead of
  // 40.8, and 8 of window 256 9.7 instead of 8.9).
  const long long units = static_cast<long long>(p.batch) * p.num_kv_heads * p.head_blocks;
  const bool many = p.num_splits == 1 && units > kCtasPerSm * static_cast<long long>(p.num_sms) &&
                    p.pages_per_chunk <= kFewPages + 1;
  if (p.col_blocks == 1)
    return many ? launch_variant<1, 1>(p, stream, programmatic) : launch_variant<1, 2>(p, stream, programmatic);
  return many ? launch_variant<2, 1>(p, stream, programmatic) : launch_variant<2, 2>(p, stream, programmatic);
}

}  // namespace sa
