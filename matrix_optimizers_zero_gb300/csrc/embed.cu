// Embedding lookup, its gradient by sorted tokens, and dropout.
//
//   lookup   out[t] = drop(scale E[tok_t] + P[t mod rows(P)])
//   gradient dE[v] (+)= scale sum over t with tok_t = v of drop'(dout[t])
//   dropout  y = drop(x) (+ residual)
//
// drop(x)_i = x_i 65536 / (65536 - T) where element i's 16-bit number is at
// least T, and 0 (whatever x_i is) elsewhere; element i is the flat index of
// the [tokens, dim] (or [n]) tensor. The backward pass draws the same numbers
// again: no mask is stored. All of it is bound by memory; arithmetic is fp32.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "philox.cuh"
#include "train_kernels.h"

namespace mo {
namespace {

// Eight consecutive elements of a bf16 or fp32 tensor as raw words.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {   // bf16 bits; 16-byte aligned
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Vec8<float> {   // 16-byte aligned
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Zeroes the dropped ones of a group's eight values and scales the others.
__device__ __forceinline__ void drop8(float (&v)[8], const uint4& g, uint32_t threshold, float factor) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = philox_half(g, i) >= threshold ? v[i] * factor : 0.0f;
}

__device__ __forceinline__ int64_t token_at(const TokenArgs& t, int64_t i) {
  return t.wide ? static_cast<const int64_t*>(t.ids)[i] : int64_t(static_cast<const int32_t*>(t.ids)[i]);
}

// ------------------------------------------------------------------ dropout
// A thread takes kDropGroups groups of eight elements, kDropThreads groups
// apart, and issues all their loads before the first use.
constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropoutParams p) {
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  T* y = static_cast<T*>(p.y);
  const Philox rng(p.drop.rnd);
  const int64_t full = p.n >> 3;
  const int64_t g0 = int64_t(blockIdx.x) * (kDropThreads * kDropGroups) + threadIdx.x;
  Vec8<T> a[kDropGroups], r[kDropGroups];
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    const int64_t g = g0 + u * kDropThreads;
    if (g < full) {
      a[u].load(x + 8 * g);
      if (RES) r[u].load(res + 8 * g);
    }
  }
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    const int64_t g = g0 + u * kDropThreads;
    if (g < full) {
      float v[8];
      a[u].unpack(v);
      drop8(v, rng.group(uint64_t(g)), p.drop.threshold, p.drop.factor);
      if (RES) {
        float w[8];
        r[u].unpack(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
      }
      store8(y + 8 * g, v);
    } else if (g == full) {   // the last, partial group
      const uint4 q = rng.group(uint64_t(g));
      for (int64_t i = 8 * g; i < p.n; ++i) {
        float v = philox_half(q, int(i & 7)) >= p.drop.threshold ? to_float(x[i]) * p.drop.factor : 0.0f;
        if (RES) v += to_float(res[i]);
        store1(y + i, v);
      }
    }
  }
}

// ------------------------------------------------------------------ lookup
// dim % 8 == 0: blockDim.x threads cover a row in groups of eight columns,
// blockDim.y tokens a block.
template <typename T, typename O>
__global__ void __launch_bounds__(256) embed_lookup_kernel(const LookupParams p) {
  const int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.tokens.n) return;
  const Philox rng(p.drop.rnd);
  const int64_t tok = token_at(p.tokens, t);
  const bool valid = tok >= 0 && tok < p.vocab;
  if (!valid && threadIdx.x == 0) atomicExch(p.status, MO_ERR_BAD_TOKEN);
  const int64_t groups = p.dim >> 3;
  const T* row = static_cast<const T*>(p.table) + (valid ? tok : 0) * p.dim;
  const T* add = p.add != nullptr ? static_cast<const T*>(p.add) + (t % p.add_rows) * p.dim : nullptr;
  O* out = static_cast<O*>(p.out) + t * p.dim;
  constexpr int U = 2;
  for (int64_t g0 = threadIdx.x; g0 < groups; g0 += int64_t(U) * blockDim.x) {
    Vec8<T> a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * int64_t(blockDim.x);
      a[u].zero();
      if (g < groups) {
        if (valid) a[u].load(row + 8 * g);
        if (add != nullptr) b[u].load(add + 8 * g);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * int64_t(blockDim.x);
      if (g < groups) {
        float v[8];
        a[u].unpack(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= p.scale;
        if (add != nullptr) {
          float w[8];
          b[u].unpack(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += w[i];
        }
        if (p.drop.threshold != 0) drop8(v, rng.group(uint64_t(t * groups + g)), p.drop.threshold, p.drop.factor);
        store8(out + 8 * g, v);
      }
    }
  }
}

// Any dim: a thread takes eight consecutive elements of the flat output, which
// may cross rows (one random call and one vector store still serve them all).
template <typename T, typename O>
__global__ void __launch_bounds__(256) embed_lookup_flat_kernel(const LookupParams p) {
  const int64_t total = p.tokens.n * p.dim;
  const int64_t g = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (8 * g >= total) return;
  const Philox rng(p.drop.rnd);
  int64_t t = 8 * g / p.dim, c = 8 * g - t * p.dim;
  const int count = int(min(int64_t(8), total - 8 * g));
  int64_t tok = 0;
  bool valid = false, fresh = true;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (i < count) {
      if (fresh) {
        tok = token_at(p.tokens, t);
        valid = tok >= 0 && tok < p.vocab;
        if (!valid) atomicExch(p.status, MO_ERR_BAD_TOKEN);
        fresh = false;
      }
      if (valid) v[i] = to_float(static_cast<const T*>(p.table)[tok * p.dim + c]) * p.scale;
      if (p.add != nullptr) v[i] += to_float(static_cast<const T*>(p.add)[(t % p.add_rows) * p.dim + c]);
      if (++c == p.dim) {
        c = 0;
        ++t;
        fresh = true;
      }
    }
  }
  if (p.drop.threshold != 0) drop8(v, rng.group(uint64_t(g)), p.drop.threshold, p.drop.factor);
  O* out = static_cast<O*>(p.out) + 8 * g;
  if (count == 8) {
    store8(out, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) store1(out + i, v[i]);
  }
}

// ------------------------------------------------------------------ gradient: sort
//
// Launch 1 of the gradient. Cluster 0 (eight CTAs) sorts the tokens with their
// positions by a stable radix sort, 9 bits a pass (two passes for vocabularies
// up to 2^18); the other clusters meanwhile write the zeros of the rows that
// no token names. Every warp owns a contiguous part of the positions, so its
// histogram, its offsets and its scatter need no atomics and keep the order:
// the sums of launch 2 have one order whatever the scheduling. The CTAs'
// histograms meet through distributed shared memory; keys ping-pong through
// the workspace, which L2 holds.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr uint32_t kMaskWords = 8192;   // rows a zeroing CTA marks at a time: 32 a word
constexpr size_t kSortSmem = sizeof(uint32_t) * (size_t(kSortWarps) * kBins + kBins + kSortWarps);
static_assert(sizeof(uint32_t) * kMaskWords <= kSortSmem, "the row mask shares the histograms' memory");

// The sort key of a token: itself, or `vocab` (sorted last, ignored) for the
// padding index and for an index outside the table.
__device__ __forceinline__ uint32_t sort_key(const GradParams& p, int64_t i, bool report) {
  const int64_t tok = token_at(p.tokens, i);
  const bool valid = tok >= 0 && tok < p.vocab;
  if (report && !valid) atomicExch(p.status, MO_ERR_BAD_TOKEN);
  return valid && tok != p.tokens.padding ? uint32_t(tok) : uint32_t(p.vocab);
}

__device__ void sort_tokens(const GradParams& p, uint32_t* sm, uint32_t rank) {
  uint32_t* hist = sm;                                 // [warp][bin]
  uint32_t* total = sm + size_t(kSortWarps) * kBins;   // this CTA's bin counts, read by the cluster
  uint32_t* wsum = total + kBins;
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t n = p.tokens.n;
  // positions a warp: a multiple of 32
  const int64_t per_warp = (n + int64_t(kSortCtas) * kSortThreads - 1) / (int64_t(kSortCtas) * kSortThreads) * 32;
  const int64_t begin = (int64_t(rank) * kSortWarps + warp) * per_warp;
  const int64_t end = min(n, begin + per_warp);
  uint32_t* my = hist + size_t(warp) * kBins;

  // the join's arrival counters, for launch 2
  for (int64_t i = int64_t(rank) * kSortThreads + tid; i < p.counters; i += int64_t(kSortCtas) * kSortThreads)
    p.counter[i] = 0u;

  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * kDigitBits;
    const uint32_t* src_key = p.key[(pass + 1) & 1];   // pass k writes buffer k & 1
    const uint32_t* src_pos = p.pos[(pass + 1) & 1];
    uint32_t* dst_key = p.key[pass & 1];
    uint32_t* dst_pos = p.pos[pass & 1];
    for (int i = tid; i < kSortWarps * kBins; i += kSortThreads) hist[i] = 0u;
    __syncthreads();
    for (int64_t i = begin + lane; i < end; i += 32) {
      const uint32_t k = pass == 0 ? sort_key(p, i, true) : __ldcg(src_key + i);
      atomicAdd(my + ((k >> shift) & (kBins - 1)), 1u);
    }
    __syncthreads();
    // exclusive offsets over (bin, CTA, warp)
    uint32_t sum = 0;
    if (tid < kBins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[size_t(w) * kBins + tid];
        hist[size_t(w) * kBins + tid] = sum;
        sum += c;
      }
      total[tid] = sum;
    }
    ptx::cluster_sync();
    uint32_t before = 0, all = 0;
    if (tid < kBins) {
#pragma unroll
      for (uint32_t c = 0; c < uint32_t(kSortCtas); ++c) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(v)
                     : "r"(ptx::mapa_shared(ptx::smem_addr(total + tid), c))
                     : "memory");
        before += c < rank ? v : 0u;
        all += v;
      }
      uint32_t inc = all;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += v;
      }
      if (lane == 31) wsum[warp] = inc;
      before += inc - all;   // plus the bins before this one in the warp
    }
    __syncthreads();
    if (tid < kBins) {
      for (int w = 0; w < warp; ++w) before += wsum[w];
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) hist[size_t(w) * kBins + tid] += before;
    }
    __syncthreads();
    for (int64_t base = begin; base < end; base += 32) {
      const int64_t i = base + lane;
      const bool live = i < end;
      uint32_t k = 0, at = 0;
      if (live) {
        k = pass == 0 ? sort_key(p, i, false) : __ldcg(src_key + i);
        at = pass == 0 ? uint32_t(i) : __ldcg(src_pos + i);
      }
      const uint32_t bin = live ? (k >> shift) & (kBins - 1) : uint32_t(kBins);
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, bin);
      const uint32_t below = peers & ((1u << lane) - 1u);
      const uint32_t off = live ? my[bin] : 0u;
      __syncwarp();
      if (live && below == 0u) my[bin] = off + uint32_t(__popc(peers));
      __syncwarp();
      if (live) {
        const uint32_t to = off + uint32_t(__popc(below));
        dst_key[to] = k;
        dst_pos[to] = at;
      }
    }
    ptx::cluster_sync();   // the pass is complete and visible to the cluster
  }
}

// CTA z of `ctas` zeroes the untouched ones of the rows z, z + ctas, ...
__device__ void zero_rows(const GradParams& p, uint32_t* mask, uint32_t z, uint32_t ctas) {
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int64_t mine = z < p.vocab ? (p.vocab - z + ctas - 1) / ctas : 0;
  for (int64_t r0 = 0; r0 < mine; r0 += int64_t(kMaskWords) * 32) {
    const int64_t rows = min(mine - r0, int64_t(kMaskWords) * 32);
    for (int i = tid; i < (rows + 31) / 32; i += kSortThreads) mask[i] = 0u;
    __syncthreads();
    for (int64_t i = tid; i < p.tokens.n; i += kSortThreads) {
      const uint32_t k = sort_key(p, i, false);
      const uint32_t q = k / ctas;
      if (k < uint32_t(p.vocab) && k - q * ctas == z && q >= r0 && q < r0 + rows)
        atomicOr(mask + ((q - r0) >> 5), 1u << ((q - r0) & 31));
    }
    __syncthreads();
    for (int64_t r = warp; r < rows; r += kSortWarps) {
      if ((mask[r >> 5] >> (r & 31)) & 1u) continue;
      float* row = p.grad + (int64_t(z) + (r0 + r) * ctas) * p.dim;
      if ((p.dim & 3) == 0) {
        for (int64_t c = lane * 4; c < p.dim; c += 128)
          *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int64_t c = lane; c < p.dim; c += 32) row[c] = 0.0f;
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ GradParams p) {
  extern __shared__ uint32_t sort_smem[];
  const uint32_t cluster = ptx::cluster_id_x();
  if (cluster == 0)
    sort_tokens(p, sort_smem, ptx::cluster_ctarank());
  else
    zero_rows(p, sort_smem, blockIdx.x - kSortCtas, gridDim.x - kSortCtas);
}

// ------------------------------------------------------------------ gradient: sums
//
// Launch 2. A block takes a chunk of consecutive sorted positions and a block
// of columns, V of them a thread, and adds the rows of each token in order. A
// token whose positions lie in one chunk is written at once; the sums of one
// that crosses chunks go to the workspace (slot 2 c for a token that began
// before chunk c, 2 c + 1 for one that begins in it and goes on) and are
// joined, in chunk order, by whichever block arrives last: first within
// aligned groups of kJoin chunks, then over the groups, so that a token that
// fills the batch is not summed by one block alone.
constexpr int kJoin = 32;
constexpr int kMaxChunk = 64;

// First index in [lo, hi) of the sorted keys whose key is at least k, hi if
// none: each step of the warp cuts the range by 32.
__device__ int64_t lower_bound_warp(const uint32_t* key, int64_t lo, int64_t hi, uint32_t k) {
  const int lane = int(threadIdx.x & 31);
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + lane * step;
    const bool less = at < hi && __ldcg(key + at) < k;
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, less);   // a run of ones from lane 0
    const int ones = __popc(votes);
    if (ones == 0) return lo;
    const int64_t next = lo + int64_t(ones - 1) * step + 1;
    hi = min(hi, lo + int64_t(ones) * step);
    lo = next;
  }
  return lo;
}

template <int V>
struct Acc {
  float v[V];
};

template <int V>
__device__ __forceinline__ void write_row(const GradParams& p, uint32_t token, int64_t col, const Acc<V>& a) {
  float* o = p.grad + int64_t(token) * p.dim + col;
  float w[V];
  if (p.accumulate) {
    if (V == 8) {
      const float4 x = reinterpret_cast<const float4*>(o)[0], y = reinterpret_cast<const float4*>(o)[V == 8 ? 1 : 0];
      const float t[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = fmaf(p.factor, a.v[i], t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = fmaf(p.factor, a.v[i], o[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = p.factor * a.v[i];
  }
  if constexpr (V == 8) {
    store8(o, w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = w[i];
  }
}

template <int V>
__device__ __forceinline__ float* slot_at(const GradParams& p, int64_t slot, int64_t col) {
  return p.partial + slot * p.dim_pad + col;
}

template <int V>
__device__ __forceinline__ void add_slot(const GradParams& p, int64_t slot, int64_t col, Acc<V>& a) {
  const float* s = slot_at<V>(p, slot, col);
  if constexpr (V == 8) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(s)), y = __ldcg(reinterpret_cast<const float4*>(s) + 1);
    const float t[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] += t[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] += __ldcg(s + i);
  }
}

template <int V>
__device__ __forceinline__ void put_slot(const GradParams& p, int64_t slot, int64_t col, const Acc<V>& a) {
  float* s = slot_at<V>(p, slot, col);
  if constexpr (V == 8) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = a.v[i];
    store8(s, w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = a.v[i];
  }
}

// This block's sums of a token that crosses chunks c0..c1 are in their slot:
// joins what can be joined now. Called by the whole block.
template <int V>
__device__ void join(const GradParams& p, uint32_t token, int64_t chunk, int64_t c0, int64_t c1, int64_t col, bool live) {
  __shared__ int last;
  const int64_t cb = blockIdx.x;
  auto slot_of = [&](int64_t c) { return 2 * c + (c == c0 ? 1 : 0); };
  auto arrive = [&](int64_t counter, int64_t count) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.counter + counter * gridDim.x + cb, 1u) == uint32_t(count - 1);
    __syncthreads();
    const bool mine = last != 0;
    __syncthreads();   // `last` may be set again
    __threadfence();
    return mine;
  };
  const int64_t g = chunk / kJoin, g0 = c0 / kJoin, g1 = c1 / kJoin;
  const int64_t lo = max(c0, g * kJoin), hi = min(c1, g * kJoin + kJoin - 1);
  if (!arrive(2 * slot_of(lo), hi - lo + 1)) return;
  Acc<V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = 0.0f;
  if (live)
#pragma unroll 4
    for (int64_t c = lo; c <= hi; ++c) add_slot<V>(p, slot_of(c), col, a);
  if (g0 == g1) {
    if (live) write_row<V>(p, token, col, a);
    return;
  }
  if (live) put_slot<V>(p, slot_of(lo), col, a);   // each thread reads and writes its own columns only
  if (!arrive(2 * slot_of(c0) + 1, g1 - g0 + 1)) return;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = 0.0f;
  if (live) {
#pragma unroll 4
    for (int64_t h = g0; h <= g1; ++h) add_slot<V>(p, slot_of(max(c0, h * kJoin)), col, a);
    write_row<V>(p, token, col, a);
  }
}

template <typename T, int V, bool DROP>
__global__ void __launch_bounds__(256) embed_sum_kernel(const __grid_constant__ GradParams p) {
  __shared__ uint32_t s_key[kMaxChunk + 2];   // the chunk's keys between its neighbours'
  __shared__ uint32_t s_pos[kMaxChunk];
  __shared__ int64_t s_bound[3];
  const uint32_t* key = p.key[(p.passes + 1) & 1];
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  const int64_t n = p.tokens.n;
  const int64_t chunk = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  const int64_t s = chunk * p.chunk, e = min(n, s + p.chunk);
  if (s >= n) return;
  const uint32_t none = uint32_t(p.vocab);
  for (int i = int(threadIdx.x); i < int(e - s) + 2; i += int(blockDim.x)) {
    const int64_t at = s - 1 + i;
    s_key[i] = at < 0 || at >= n ? none : __ldcg(key + at);
    if (i >= 1 && i <= int(e - s)) s_pos[i - 1] = __ldcg(pos + at);
  }
  __syncthreads();
  if (s_key[1] == none) return;   // ignored positions only
  const int64_t col = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * V;
  const bool live = col < p.dim;
  const Philox rng(p.drop.rnd);
  const T* dout = static_cast<const T*>(p.dout);
  int count = int(e - s);
  while (s_key[count] == none) --count;   // a block that ends in ignored positions
  const bool from_before = s > 0 && s_key[0] == s_key[1];
  const bool goes_on = count == int(e - s) && s_key[count + 1] == s_key[count];   // the key after the last is `none`

  Acc<V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = 0.0f;
  uint32_t cur = s_key[1];
  bool first = true;
  constexpr int U = V == 8 ? 8 : 8;
  for (int i0 = 0; i0 < count; i0 += U) {
    Vec8<T> q[V == 8 ? U : 1];
    float sc[V == 8 ? 1 : U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < count && live) {
        const T* x = dout + int64_t(s_pos[i0 + u]) * p.dim + col;
        if constexpr (V == 8)
          q[u].load(x);
        else
          sc[u] = to_float(__ldg(x));
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= count) break;
      const uint32_t k = s_key[i0 + u + 1];
      if (k != cur) {   // the same for the whole block
        if (live) {
          if (first && from_before)
            put_slot<V>(p, 2 * chunk, col, a);
          else
            write_row<V>(p, cur, col, a);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) a.v[i] = 0.0f;
        cur = k;
        first = false;
      }
      if (live) {
        const uint64_t at = uint64_t(s_pos[i0 + u]) * uint64_t(p.dim) + uint64_t(col);
        if constexpr (V == 8) {
          float v[8];
          q[u].unpack(v);
          if (DROP) drop8(v, rng.group(at >> 3), p.drop.threshold, 1.0f);
#pragma unroll
          for (int i = 0; i < 8; ++i) a.v[i] += v[i];
        } else {
          a.v[0] += !DROP || rng.element(at) >= p.drop.threshold ? sc[u] : 0.0f;
        }
      }
    }
  }
  // the last token of the chunk
  const bool head = first && from_before;
  if (live) {
    if (head)
      put_slot<V>(p, 2 * chunk, col, a);
    else if (goes_on)
      put_slot<V>(p, 2 * chunk + 1, col, a);
    else
      write_row<V>(p, cur, col, a);
  }
  if (!from_before && !goes_on) return;
  // the positions of the tokens that cross this chunk's ends
  const uint32_t head_key = s_key[1], tail_key = s_key[count];
  if (threadIdx.x < 32) {
    int64_t b0 = 0, b1 = e, b2 = e;
    if (from_before) b0 = lower_bound_warp(key, 0, s, head_key);
    if (from_before && head && goes_on) b1 = lower_bound_warp(key, e, n, head_key + 1u);
    if (goes_on && !head) b2 = lower_bound_warp(key, e, n, tail_key + 1u);
    if (threadIdx.x == 0) {
      s_bound[0] = b0;
      s_bound[1] = b1;
      s_bound[2] = b2;
    }
  }
  __syncthreads();
  if (from_before) join<V>(p, head_key, chunk, s_bound[0] / p.chunk, head && goes_on ? (s_bound[1] - 1) / p.chunk : chunk, col, live);
  if (goes_on && !head) join<V>(p, tail_key, chunk, chunk, (s_bound[2] - 1) / p.chunk, col, live);
}

template <typename T>
cudaError_t dropout_as(const DropoutParams& p, cudaStream_t stream) {
  const int64_t groups = (p.n + 7) / 8;
  const int64_t per = int64_t(kDropThreads) * kDropGroups;
  const unsigned grid = unsigned((groups + per - 1) / per);
  if (p.residual != nullptr)
    dropout_kernel<T, true><<<grid, kDropThreads, 0, stream>>>(p);
  else
    dropout_kernel<T, false><<<grid, kDropThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t lookup_as(const LookupParams& p, cudaStream_t stream) {
  if ((p.dim & 7) == 0) {
    const int64_t groups = p.dim / 8;
    unsigned x = 32;
    while (x < 256 && x < groups) x <<= 1;
    const unsigned y = 256 / x;
    embed_lookup_kernel<T, O><<<unsigned((p.tokens.n + y - 1) / y), dim3(x, y), 0, stream>>>(p);
  } else {
    const int64_t groups = (p.tokens.n * p.dim + 7) / 8;
    embed_lookup_flat_kernel<T, O><<<unsigned((groups + 255) / 256), 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t sum_as(const GradParams& p, cudaStream_t stream) {
  const GradGrid g = grad_grid(p.tokens.n, p.dim);
  const int64_t y = g.chunks < 32768 ? g.chunks : 32768;
  const dim3 grid(unsigned(g.col_blocks), unsigned(y), unsigned((g.chunks + y - 1) / y));
  if (p.drop.threshold != 0)
    embed_sum_kernel<T, V, true><<<grid, unsigned(g.threads), 0, stream>>>(p);
  else
    embed_sum_kernel<T, V, false><<<grid, unsigned(g.threads), 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? dropout_as<uint16_t>(p, stream) : dropout_as<float>(p, stream);
}

cudaError_t launch_embed_lookup(const LookupParams& p, bool table_bf16, bool out_bf16, cudaStream_t stream) {
  if (table_bf16) return out_bf16 ? lookup_as<uint16_t, uint16_t>(p, stream) : lookup_as<uint16_t, float>(p, stream);
  return out_bf16 ? lookup_as<float, uint16_t>(p, stream) : lookup_as<float, float>(p, stream);
}

cudaError_t launch_embed_grad(const GradParams& p, bool dout_bf16, int sms, cudaStream_t stream) {
  static_assert(kSortSmem <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSortSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // one cluster sorts; with zeros to write, one CTA an SM for them
  const int clusters = 1 + (p.accumulate ? 0 : (sms > 2 * kSortCtas ? sms / kSortCtas - 1 : 1));
  cfg.gridDim = dim3(unsigned(kSortCtas * clusters), 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = kSortSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, p)) != cudaSuccess) return e;
  const bool vec = (p.dim & 7) == 0;
  if (dout_bf16) return vec ? sum_as<uint16_t, 8>(p, stream) : sum_as<uint16_t, 1>(p, stream);
  return vec ? sum_as<float, 8>(p, stream) : sum_as<float, 1>(p, stream);
}

}  // namespace mo
