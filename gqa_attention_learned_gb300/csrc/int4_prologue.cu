// Attention prologue into a cache held in 4 bits, and the way back: bias, rotary
// encoding of q and k, quantisation of k and v rows and their write into the paged
// cache in one pass; and rows of that cache as bf16 values.
//
// A row x of 64 values is quantised as
//     lo = min(0, min x), hi = max(0, max x)
//     s  = (hi - lo) / 15, rounded up to 4 significant bits, at least 2^-126
//     z  = rint(-lo / s),  n = clamp(rint(x / s) + z, 0, 15)
// and stands for s (n - z).  Zero is always a value; the error is at most s / 2,
// but at the ends of the range s, where both lo / s and hi / s round outwards (the
// range then has 16 steps and the last is cut).  Rounding s up costs up to an
// eighth of the step and makes every value a bf16 number.  x is taken in fp32: bias
// added, products and sum of the rotation rounded one by one, with no contraction,
// so that the codes follow from the inputs alone.  A row whose range is not finite
// has s = NaN.  cos and sin come from a table that all layers share: codes next to
// a border would otherwise depend on the sine of this machine.
//
// Bound by HBM: a token's (Hq + 2 Hkv) rows are read, Hq written in bf16 and Hkv
// written in 68 bytes for K and V together.  Every thread takes one (row, dims
// 8c..8c+7 and 32+8c..) item as in the prologue of the bf16 cache; four neighbours
// share a row, so its range takes two shuffles, and each writes 8 bytes of codes.

#include "int4.cuh"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kGatherThreads = 128;            // 20.4 us for 39k rows of 8 heads; 256: 21.0
constexpr int kPairs = kHeadDim / 2;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// A pair rotated, each operation rounded on its own.
__device__ __forceinline__ void turn(float &x1, float &x2, float c, float s) {
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1;
}

// Scale and zero point of the row that four neighbouring lanes share.
__device__ __forceinline__ uint32_t row_scale(const float (&a)[8], const float (&b)[8], float &s,
                                              float &z) {
  float lo = 0.f, hi = 0.f;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, fminf(a[e], b[e]));
    hi = fmaxf(hi, fmaxf(a[e], b[e]));
    finite = finite && a[e] == a[e] && b[e] == b[e];   // fminf and fmaxf pass over NaN
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    finite = __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, off) != 0 && finite;
  }
  const float range = __fsub_rn(hi, lo);
  if (!finite || !(range < INFINITY)) {
    s = NAN;
    z = 0.f;
    return 0x7fc0u;
  }
  const uint32_t bits = max((__float_as_uint(__fdiv_rn(range, 15.f)) + 0xfffffu) & ~0xfffffu, 1u << 23);
  s = __uint_as_float(bits);
  z = rintf(__fdiv_rn(-lo, s));
  return (bits >> 16) + static_cast<uint32_t>(z);
}

// Eight codes of a row as a word; 0 where s is NaN.
__device__ __forceinline__ uint32_t codes(const float (&x)[8], float s, float z) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float n = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(x[e], s)), z), 0.f), 15.f);
    w |= static_cast<uint32_t>(n) << (4 * e);
  }
  return s == s ? w : 0u;
}

template <int kTok, int kThreads>      // tokens per CTA
__global__ void __launch_bounds__(kThreads)
int4_prologue_kernel(const __grid_constant__ Int4PrologueParams p) {
  __shared__ float cs[kTok][2 * kPairs];       // cos, then sin
  launch_dependents();
  // Nothing is read or written before the previous kernel on the stream has
  // finished: only the launch and set-up overlap it.
  grid_dependency_wait();
  const int tok0 = blockIdx.x * kTok;
  for (int j = threadIdx.x; j < kTok * 2 * kPairs; j += kThreads) {
    const int t = tok0 + j / (2 * kPairs);
    if (t >= p.num_tokens) break;
    const int pos = p.positions[t];
    cs[j / (2 * kPairs)][j % (2 * kPairs)] =
        pos >= 0 && pos < p.rope_positions
            ? __ldg(p.rope + static_cast<size_t>(pos) * (2 * kPairs) + j % (2 * kPairs)) : NAN;
  }
  __syncthreads();

  const int rows = p.num_qo_heads + 2 * p.num_kv_heads;
  const int per_tok = rows * 4;
  const int row_elems = rows * kHeadDim;
  const int items = min(kTok, p.num_tokens - tok0) * per_tok;
  // whole warps stay together for the shuffles: items past the last are left out
  // of the loads and stores only
  for (int item0 = threadIdx.x & ~31; item0 < items; item0 += kThreads) {
    const int item = min(item0 + static_cast<int>(threadIdx.x & 31), items - 1);
    const bool live = item0 + static_cast<int>(threadIdx.x & 31) < items;
    const int tt = item / per_tok;
    const int t = tok0 + tt;
    const int r = item % per_tok;
    const int h = r >> 2, c = r & 3;
    const size_t base = static_cast<size_t>(t) * row_elems + h * kHeadDim;
    float a[8], b[8];                          // dims 8c.. and 8c+32..
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p.qkv + base + 8 * c)), a);
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p.qkv + base + 8 * c + 32)), b);
    if (p.bias) {
      float ba[8], bb[8];
      unpack8(__ldg(reinterpret_cast<const uint4 *>(p.bias + h * kHeadDim + 8 * c)), ba);
      unpack8(__ldg(reinterpret_cast<const uint4 *>(p.bias + h * kHeadDim + 8 * c + 32)), bb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = __fadd_rn(a[e], ba[e]);
        b[e] = __fadd_rn(b[e], bb[e]);
      }
    }
    const bool is_v = h >= p.num_qo_heads + p.num_kv_heads;
    if (!is_v) {
      const float *cos = cs[tt], *sin = cs[tt] + kPairs;
      if (!p.interleaved) {
        // pair 8c+e is (a[e], b[e])
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(a[e], b[e], cos[8 * c + e], sin[8 * c + e]);
      } else {
        // pairs 4c+u are (a[2u], a[2u+1]); pairs 16+4c+u are (b[2u], b[2u+1])
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          turn(a[2 * u], a[2 * u + 1], cos[4 * c + u], sin[4 * c + u]);
          turn(b[2 * u], b[2 * u + 1], cos[16 + 4 * c + u], sin[16 + 4 * c + u]);
        }
      }
    }
    // (all lanes take part, unless all have rows of q)
    float s = 0.f, z = 0.f;
    uint32_t sz = 0;
    if (__any_sync(0xffffffffu, h >= p.num_qo_heads)) sz = row_scale(a, b, s, z);
    if (!live) continue;
    if (h < p.num_qo_heads) {
      uint16_t *dst = p.q_out + (static_cast<size_t>(t) * p.num_qo_heads + h) * kHeadDim;
      *reinterpret_cast<uint4 *>(dst + 8 * c) = pack8(a);
      *reinterpret_cast<uint4 *>(dst + 8 * c + 32) = pack8(b);
      continue;
    }
    const int slot = p.slot_mapping[t];
    if (slot < 0 || slot / kPageSize >= p.num_pages) continue;   // no write
    const int kvh = is_v ? h - p.num_qo_heads - p.num_kv_heads : h - p.num_qo_heads;
    const int j = slot % kPageSize;
    uint8_t *block = p.kv_cache +
                     (static_cast<size_t>(slot / kPageSize) * p.num_kv_heads + kvh) * kInt4Block;
    const uint32_t w0 = codes(a, s, z), w1 = codes(b, s, z);
    if (is_v) {
      uint8_t *dst = block + kInt4V + 16 * (j % 8 / 2) + 8 * (j / 8) + 4 * (j % 2);
      *reinterpret_cast<uint32_t *>(dst + 64 * c) = w0;
      *reinterpret_cast<uint32_t *>(dst + 64 * (c + 4)) = w1;
    } else {
      *reinterpret_cast<uint2 *>(block + kInt4K + 64 * (j % 8) + 16 * c + 8 * (j / 8)) =
          make_uint2(__funnelshift_l(w0, w0, 3), __funnelshift_l(w1, w1, 3));
    }
    if (c == 0)
      *reinterpret_cast<uint16_t *>(block + kInt4Meta + 8 * (j % 8) + 4 * (j / 8) + (is_v ? 2 : 0)) =
          static_cast<uint16_t>(sz);
  }
}

// s (n - z) of eight codes, a bf16 number each.
__device__ __forceinline__ uint4 values8(uint32_t w, float s, float z) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = s * (static_cast<float>((w >> (4 * e)) & 15u) - z);
  return pack8(f);
}

// A thread writes 16 bytes each of K and V: dims 8c..8c+7 of one (row, KV head).
__global__ void __launch_bounds__(kGatherThreads)
int4_gather_kernel(const __grid_constant__ Int4GatherParams p) {
  grid_dependency_wait();
  const long long i = static_cast<long long>(blockIdx.x) * kGatherThreads + threadIdx.x;
  const int c = static_cast<int>(i & 7);
  const long long r = i >> 3;
  if (r >= static_cast<long long>(p.num_rows) * p.num_kv_heads) return;
  const int kvh = static_cast<int>(r % p.num_kv_heads);
  const int slot = p.slots[r / p.num_kv_heads];
  uint4 k = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u), v = k;
  if (slot >= 0 && slot / kPageSize < p.num_pages) {
    const int j = slot % kPageSize;
    const uint8_t *block = p.kv_cache +
                           (static_cast<size_t>(slot / kPageSize) * p.num_kv_heads + kvh) * kInt4Block;
    auto word = [&](int at) { return __ldg(reinterpret_cast<const uint32_t *>(block + at)); };
    const uint32_t m = word(kInt4Meta + 8 * (j % 8) + 4 * (j / 8));
    const uint32_t kw = word(kInt4K + 64 * (j % 8) + 16 * (c % 4) + 8 * (j / 8) + 4 * (c / 4));
    const uint32_t vw = word(kInt4V + 64 * c + 16 * (j % 8 / 2) + 8 * (j / 8) + 4 * (j % 2));
    k = values8(__funnelshift_r(kw, kw, 3), __uint_as_float((m << 16) & 0xfff00000u),
                static_cast<float>(m & 15u));
    v = values8(vw, __uint_as_float(m & 0xfff00000u), static_cast<float>((m >> 16) & 15u));
  }
  reinterpret_cast<uint4 *>(p.k)[i] = k;
  reinterpret_cast<uint4 *>(p.v)[i] = v;
}

}  // namespace

cudaError_t launch_int4_prologue(const Int4PrologueParams &p, cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  // Small batches: one token per CTA of 256 threads, more SMs busy (64 tokens of 64 / 8
  // heads 4.0 us; 128 threads 4.6).  Large ones: four tokens per CTA of 128 (20.9k tokens
  // 72 us, 5.5 TB/s; 256 threads 77).
  if (p.num_tokens <= 4096)
    return launch_kernel(int4_prologue_kernel<1, 256>, static_cast<unsigned>(p.num_tokens), 256, 0, stream, true, p);
  return launch_kernel(int4_prologue_kernel<4, 128>, static_cast<unsigned>((p.num_tokens + 3) / 4), 128, 0, stream,
                       true, p);
}

cudaError_t launch_int4_gather(const Int4GatherParams &p, cudaStream_t stream) {
  const long long threads = 8ll * p.num_rows * p.num_kv_heads;
  if (threads == 0) return cudaSuccess;
  const long long ctas = (threads + kGatherThreads - 1) / kGatherThreads;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_kernel(int4_gather_kernel, static_cast<unsigned>(ctas), kGatherThreads, 0, stream, true, p);
}

}  // namespace sa
