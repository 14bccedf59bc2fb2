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
#include "launch.cuh"
#include "philox.cuh"
#include "ptx_train.cuh"
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
// Halves compare in the upper half of a word: at least T << 16, or above
// (T << 16) - 1, which for T = 65536 is the largest word and drops all.
__device__ __forceinline__ void drop8(float (&v)[8], const uint4& g, uint32_t threshold, float factor) {
  const uint32_t w[4] = {g.x, g.y, g.z, g.w};
  const uint32_t below = (threshold << 16) - 1u;   // threshold >= 1
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] << 16) > below ? v[2 * i] * factor : 0.0f;
    v[2 * i + 1] = w[i] > below ? v[2 * i + 1] * factor : 0.0f;
  }
}

__device__ __forceinline__ int64_t token_at(const TokenArgs& t, int64_t i) {
  return t.wide ? static_cast<const int64_t*>(t.ids)[i] : int64_t(static_cast<const int32_t*>(t.ids)[i]);
}

// The status word is shared with the bounded waits: an expired one, after which a
// result is incomplete, is not replaced.
__device__ __forceinline__ void report_bad_token(int* status) { atomicCAS(status, MO_OK, MO_ERR_BAD_TOKEN); }

// ------------------------------------------------------------------ dropout
// A thread takes kDropGroups groups of eight elements, kDropThreads groups
// apart, and issues all their loads before the first use. Bound by memory
// with a residual (16384 x 4096 bf16: 59 us, 6.8 TB/s), nearly so without
// (44 us, 6.2 TB/s): the random numbers' 20 wide products a group take about
// 18 us of the SMs' time there.
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
  // The numbers are drawn while the loads are on their way: the empty statement keeps the compiler
  // from drawing them only where the loaded values are used (bf16 without a residual 52 -> 46 us).
  uint4 rnd[kDropGroups];
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    rnd[u] = rng.group(uint64_t(g0 + u * kDropThreads));
    asm volatile("" : "+r"(rnd[u].x), "+r"(rnd[u].y), "+r"(rnd[u].z), "+r"(rnd[u].w));
  }
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    const int64_t g = g0 + u * kDropThreads;
    if (g < full) {
      float v[8];
      a[u].unpack(v);
      if (p.drop.threshold != 0) drop8(v, rnd[u], p.drop.threshold, p.drop.factor);
      if (RES) {
        float w[8];
        r[u].unpack(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
      }
      store8(y + 8 * g, v);
    } else if (g == full) {   // the last, partial group
      for (int64_t i = 8 * g; i < p.n; ++i) {
        float v = philox_half(rnd[u], int(i & 7)) >= p.drop.threshold ? to_float(x[i]) * p.drop.factor : 0.0f;
        if (RES) v += to_float(res[i]);
        store1(y + i, v);
      }
    }
  }
}

// ------------------------------------------------------------------ lookup
// dim % 8 == 0: blockDim.x threads cover a row in groups of eight columns,
// blockDim.y tokens at a time; the next token's index is loaded before this
// one's row is used, so the row's address is known when its turn comes.
// 16384 tokens of 128256 x 4096 fp32, to bf16: 63 us with distinct rows (402
// MB, 6.4 TB/s), 46 us with the frequencies of text (254 MB), 58 us with
// dropout, whose numbers are drawn where the loaded row is used. (The next row's
// loads a step ahead in registers: 70 us, for the occupancy they cost.) Rows of
// less than 32 groups share a warp: 2^20 tokens of 64 columns 72 us (distinct
// rows, 398 MB, 5.5 TB/s; 155 with a warp a row), of 8 columns 17 us (112).
template <typename T, typename O, bool ADD, bool DROP>
__global__ void __launch_bounds__(256, ADD ? 4 : 5) embed_lookup_kernel(const LookupParams p) {
  const Philox rng(p.drop.rnd);
  const int groups = int(p.dim >> 3);
  const float scale = ADD ? p.scale : p.scale * p.drop.factor;
  const int64_t stride = int64_t(gridDim.x) * blockDim.y;
  int64_t t = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.tokens.n) return;
  int64_t next = token_at(p.tokens, t);
  for (; t < p.tokens.n; t += stride) {
    const int64_t tok = next;
    if (t + stride < p.tokens.n) next = token_at(p.tokens, t + stride);
    const bool valid = tok >= 0 && tok < p.vocab;
    if (!valid && threadIdx.x == 0) report_bad_token(p.status);
    const T* row = static_cast<const T*>(p.table) + (valid ? tok : 0) * p.dim;
    const T* add = ADD ? static_cast<const T*>(p.add) + (t % p.add_rows) * p.dim : nullptr;
    O* out = static_cast<O*>(p.out) + t * p.dim;
    constexpr int U = 2;
    for (int g0 = int(threadIdx.x); g0 < groups; g0 += U * int(blockDim.x)) {
      Vec8<T> a[U], b[ADD ? U : 1];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = g0 + u * int(blockDim.x);
        a[u].zero();
        if (g < groups) {
          if (valid) a[u].load(row + 8 * g);
          if (ADD) b[ADD ? u : 0].load(add + 8 * g);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = g0 + u * int(blockDim.x);
        if (g < groups) {
          float v[8];
          a[u].unpack(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= scale;
          if (ADD) {
            float w[8];
            b[ADD ? u : 0].unpack(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += w[i];
          }
          if (DROP) drop8(v, rng.group(uint64_t(t) * uint64_t(groups) + uint64_t(g)), p.drop.threshold, ADD ? p.drop.factor : 1.0f);
          store8(out + 8 * g, v);
        }
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
        if (!valid) report_bad_token(p.status);
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
// Launch 1 of the gradient, below 65536 tokens. Cluster 0 (eight CTAs; one for few) sorts
// the tokens with their positions by a stable radix sort, up to 9 bits a pass
// (two passes for vocabularies up to 2^18). The other clusters meanwhile write
// zeros to the first rows of the table, as many as the sort takes the time for;
// the rest are launch 2's. They write every row, since the rows that tokens
// name are not known yet. Writing front to back by many short-lived CTAs is
// what reaches the memory's write rate (2.1 GB: 7.4 TB/s; row by row from
// resident CTAs 4.4).
//
// The sort is bound by latencies: 14 us for 8192 tokens in two passes, 10 us for
// 1024 on one CTA.
//
// Every warp owns a contiguous part of the positions, so its histogram, its
// offsets and its scatter keep the order: the sums of launch 2 have one order
// whatever the scheduling. The CTAs' histograms meet through distributed
// shared memory; keys ping-pong through the workspace, which L2 holds.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kBatch = 4;
constexpr int64_t kOneCtaTokens = 1024;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr size_t kSortSmem = sizeof(uint32_t) * (size_t(kSortWarps) * (kMaxBins + 1) + 2 * kMaxBins + kSortWarps);
constexpr int64_t kZeroBytes = int64_t(kSortThreads) * 16 * 16;   // a zeroing CTA's share: 256 KB
constexpr int kZeroMaskWords = kZeroRowsMost / 32;

// The sort key of a token: itself, or `vocab` (sorted last, ignored) for the
// padding index and for an index outside the table.
__device__ __forceinline__ uint32_t sort_key(const GradParams& p, int64_t i, bool report) {
  const int64_t tok = token_at(p.tokens, i);
  const bool valid = tok >= 0 && tok < p.vocab;
  if (report && !valid) report_bad_token(p.status);
  return valid && tok != p.tokens.padding ? uint32_t(tok) : uint32_t(p.vocab);
}

// The parts of a pass. A warp's positions are [begin, end), per_warp a warp; hist
// is [warp][bin] with a stride of bins + 1 words, so that a bin's counts lie in
// 32 banks.
struct Pass {
  int index, shift, bins, stride;
  const uint32_t* src_key;   // pass k writes buffer k & 1
  const uint32_t* src_pos;
  uint32_t* dst_key;
  uint32_t* dst_pos;
  __device__ __forceinline__ Pass(const GradParams& p, int pass)
      : index(pass), shift(pass * p.digit_bits), bins(1 << p.digit_bits), stride(bins + 1), src_key(p.key[(pass + 1) & 1]),
        src_pos(p.pos[(pass + 1) & 1]), dst_key(p.key[pass & 1]), dst_pos(p.pos[pass & 1]) {}
  __device__ __forceinline__ uint32_t bin(uint32_t key) const { return (key >> shift) & uint32_t(bins - 1); }
  // kBatch loads at a time
  __device__ __forceinline__ void load(const GradParams& p, int64_t base, int64_t end, bool report, uint32_t (&k)[kBatch],
                                       uint32_t (&at)[kBatch]) const {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = base + 32 * u + (threadIdx.x & 31);
      if (i < end) {
        k[u] = index == 0 ? sort_key(p, i, report) : __ldcg(src_key + i);
        at[u] = index == 0 ? uint32_t(i) : __ldcg(src_pos + i);
      }
    }
  }
};

// Counts the digits of a warp's positions into `my`; the last batch stays in k and at.
__device__ __forceinline__ void count_digits(const GradParams& p, const Pass& q, int64_t begin, int64_t end, uint32_t* my,
                                             bool report, uint32_t (&k)[kBatch], uint32_t (&at)[kBatch]) {
  for (int64_t base = begin; base < end; base += 32 * kBatch) {
    q.load(p, base, end, report, k, at);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (base + 32 * u + (threadIdx.x & 31) < end) atomicAdd(my + q.bin(k[u]), 1u);
  }
}

// Turns the warps' counts of each bin into offsets, and writes the bins' totals: a warp
// scans a bin, one count a lane.
__device__ __forceinline__ void scan_warps(const Pass& q, uint32_t* hist, uint32_t* total) {
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  for (int b = warp; b < q.bins; b += kSortWarps) {
    const uint32_t c = hist[size_t(lane) * q.stride + b];
    uint32_t inc = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += v;
    }
    hist[size_t(lane) * q.stride + b] = inc - c;
    if (lane == 31) total[b] = inc;
  }
}

// Sum of `value` over the threads before this one (those with a value come first).
__device__ __forceinline__ uint32_t scan_block(uint32_t value, uint32_t* wsum) {
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  uint32_t inc = value;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  return inc - value + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wsum[lane] : 0u);
}

// Writes a warp's keys and positions where start[bin] and its offsets `my` say, in order.
__device__ __forceinline__ void scatter(const GradParams& p, const Pass& q, int64_t begin, int64_t end, int64_t per_warp,
                                        uint32_t* my, const uint32_t* start, uint32_t (&k)[kBatch], uint32_t (&at)[kBatch]) {
  const int lane = int(threadIdx.x & 31);
  for (int64_t base = begin; base < end; base += 32 * kBatch) {
    if (per_warp > 32 * kBatch) q.load(p, base, end, false, k, at);   // one batch is still there
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (base + 32 * u >= end) break;   // the same for the whole warp
      const bool live = base + 32 * u + lane < end;
      const uint32_t bin = live ? q.bin(k[u]) : uint32_t(q.bins);
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, bin);
      const uint32_t below = peers & ((1u << lane) - 1u);
      const uint32_t off = live ? my[bin] : 0u;
      __syncwarp();
      if (live && below == 0u) my[bin] = off + uint32_t(__popc(peers));
      __syncwarp();
      if (live) {
        const uint32_t to = start[bin] + off + uint32_t(__popc(below));
        q.dst_key[to] = k[u];
        q.dst_pos[to] = at[u];
      }
    }
  }
}

// The join's arrival counters, for the sums' launch.
__device__ __forceinline__ void clear_counters(const GradParams& p, int64_t cta, int64_t ctas) {
  for (int64_t i = cta * kSortThreads + threadIdx.x; i < p.counters; i += ctas * kSortThreads) p.counter[i] = 0u;
}

__device__ void sort_tokens(const GradParams& p, uint32_t* sm, uint32_t rank, uint32_t ctas) {
  const int tid = int(threadIdx.x), warp = tid >> 5;
  const int64_t n = p.tokens.n;
  // positions a warp: a multiple of 32
  const int64_t per_warp = (n + int64_t(ctas) * kSortThreads - 1) / (int64_t(ctas) * kSortThreads) * 32;
  const int64_t begin = (int64_t(rank) * kSortWarps + warp) * per_warp;
  const int64_t end = min(n, begin + per_warp);
  clear_counters(p, rank, ctas);
  for (int pass = 0; pass < p.passes; ++pass) {
    const Pass q(p, pass);
    uint32_t* hist = sm;
    uint32_t* total = sm + size_t(kSortWarps) * q.stride;   // this CTA's bin counts, read by the cluster
    uint32_t* start = total + q.bins;                       // where this CTA's part of each bin begins
    uint32_t* wsum = start + q.bins;
    uint32_t* my = hist + size_t(warp) * q.stride;
    for (int i = tid; i < kSortWarps * q.stride; i += kSortThreads) hist[i] = 0u;
    __syncthreads();
    uint32_t k[kBatch], at[kBatch];
    count_digits(p, q, begin, end, my, true, k, at);
    __syncthreads();
    scan_warps(q, hist, total);
    ptx::cluster_sync();
    uint32_t before = 0, all = 0;   // this bin in the CTAs before, and in all
    if (tid < q.bins)
      for (uint32_t c = 0; c < ctas; ++c) {
        const uint32_t v = ptx::ld_shared_cluster_u32(ptx::mapa_shared(ptx::smem_addr(total + tid), c));
        before += c < rank ? v : 0u;
        all += v;
      }
    before += scan_block(all, wsum);
    if (tid < q.bins) start[tid] = before;
    __syncthreads();
    scatter(p, q, begin, end, per_warp, my, start, k, at);
    ptx::cluster_sync();   // the pass is complete and visible to the cluster
  }
}

// Many tokens: three launches a pass on all SMs instead. A block counts its
// part's digits, a block a bin scans the parts' counts, and the blocks scatter,
// in the same order as the cluster would. Launch 2 then writes all the zeros.
// (The gradient of 2^20 x 64 fp32, 1000000 rows, three passes: 572 us with one
// cluster's sort, 196 so; 2^20 x 1024 bf16, 128256 rows, two passes: 821 and 504,
// of which the sort takes 63.)
__global__ void __launch_bounds__(kSortThreads) radix_count_kernel(const __grid_constant__ GradParams p, int pass) {
  __shared__ uint32_t count[kMaxBins];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const Pass q(p, pass);
  for (int i = int(threadIdx.x); i < q.bins; i += kSortThreads) count[i] = 0u;
  if (pass == 0) clear_counters(p, blockIdx.x, gridDim.x);
  __syncthreads();
  const int64_t begin = (int64_t(blockIdx.x) * kSortWarps + (threadIdx.x >> 5)) * p.per_warp;
  uint32_t k[kBatch], at[kBatch];
  count_digits(p, q, begin, min(p.tokens.n, begin + p.per_warp), count, true, k, at);
  __syncthreads();
  for (int i = int(threadIdx.x); i < q.bins; i += kSortThreads) p.part_count[size_t(i) * gridDim.x + blockIdx.x] = count[i];
}

__global__ void __launch_bounds__(kSortThreads) radix_scan_kernel(const __grid_constant__ GradParams p, int parts) {
  __shared__ uint32_t wsum[kSortWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  uint32_t* c = p.part_count + size_t(blockIdx.x) * parts;   // at most kSortThreads parts
  const uint32_t v = int(threadIdx.x) < parts ? c[threadIdx.x] : 0u, before = scan_block(v, wsum);
  if (int(threadIdx.x) < parts) c[threadIdx.x] = before;
  if (int(threadIdx.x) == parts - 1) p.bin_count[blockIdx.x] = before + v;
}

__global__ void __launch_bounds__(kSortThreads) radix_scatter_kernel(const __grid_constant__ GradParams p, int pass) {
  extern __shared__ uint32_t sort_smem[];
  ptx::griddep_launch_dependents();
  const Pass q(p, pass);
  const int tid = int(threadIdx.x), warp = tid >> 5;
  uint32_t* hist = sort_smem;
  uint32_t* total = hist + size_t(kSortWarps) * q.stride;
  uint32_t* start = total + q.bins;
  uint32_t* wsum = start + q.bins;
  uint32_t* my = hist + size_t(warp) * q.stride;
  for (int i = tid; i < kSortWarps * q.stride; i += kSortThreads) hist[i] = 0u;
  ptx::griddep_wait();
  __syncthreads();
  const int64_t begin = (int64_t(blockIdx.x) * kSortWarps + warp) * p.per_warp, end = min(p.tokens.n, begin + p.per_warp);
  uint32_t k[kBatch], at[kBatch];
  count_digits(p, q, begin, end, my, false, k, at);
  __syncthreads();
  scan_warps(q, hist, total);
  const uint32_t base = scan_block(tid < q.bins ? p.bin_count[tid] : 0u, wsum);
  if (tid < q.bins) start[tid] = base + p.part_count[size_t(tid) * gridDim.x + blockIdx.x];
  __syncthreads();
  scatter(p, q, begin, end, p.per_warp, my, start, k, at);
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ GradParams p) {
  extern __shared__ uint32_t sort_smem[];
  ptx::griddep_launch_dependents();   // launch 2 waits for this grid's end by itself
  const uint32_t ctas = ptx::cluster_nctarank();
  if (ptx::cluster_id_x() == 0) {
    sort_tokens(p, sort_smem, ptx::cluster_ctarank(), ctas);
    return;
  }
  const int64_t floats = p.zero_first * p.dim, begin = int64_t(blockIdx.x - ctas) * (kZeroBytes / 4);
  float* g = p.grad + begin;
  const int64_t mine = min(floats - begin, kZeroBytes / 4);
#pragma unroll 4
  for (int64_t i = int64_t(threadIdx.x) * 4; i + 4 <= mine; i += kSortThreads * 4)
    *reinterpret_cast<float4*>(g + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (int64_t(threadIdx.x) < (mine > 0 ? (mine & 3) : 0)) g[(mine & ~int64_t(3)) + threadIdx.x] = 0.0f;
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
// fills the batch is not summed by one block alone. With the zeros beside them
// the sums are bound by memory at 8B size (both launches: 316 us for 2.24 GB,
// 7.1 TB/s); alone they take 14 us for 8192 x 1280, most of it the chain of
// loading positions, rows and partial sums.
constexpr int kJoin = 32;

// First and last chunk of a token that crosses chunks. A chunk after this one
// holds it if its first key is the token's, one before if its last key is;
// `near` is that key of the 32 chunks next to this one, a lane each, loaded
// before the token was known. Farther ones are searched for, 32 at a time.
__device__ __forceinline__ int64_t reach(const GradParams& p, const uint32_t* key, uint32_t token, int64_t chunk,
                                         uint32_t near, int dir) {
  const uint32_t votes = __ballot_sync(0xFFFFFFFFu, near == token);   // a run of ones from lane 0
  if (votes != 0xFFFFFFFFu) return chunk + dir * int64_t(__ffs(int(~votes)) - 1);
  const int lane = int(threadIdx.x & 31);
  // chunk + dir lo holds the token, chunk + dir hi does not (or is none)
  int64_t lo = 32, hi = dir > 0 ? (p.tokens.n - 1) / p.chunk - chunk + 1 : chunk + 1;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, d = lo + (lane + 1) * step;
    bool holds = false;
    if (d < hi) {
      const int64_t c = chunk + dir * d;
      holds = __ldcg(key + (dir > 0 ? c * p.chunk : c * p.chunk + p.chunk - 1)) == token;
    }
    const int ones = __popc(__ballot_sync(0xFFFFFFFFu, holds));
    hi = min(hi, lo + (ones + 1) * step);
    lo += ones * step;
  }
  return chunk + dir * lo;
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
    __syncthreads();   // the block's sums are written; thread 0 releases them
    if (threadIdx.x == 0) last = ptx::atomic_add_acq_rel(p.counter + counter * gridDim.x + cb, 1u) == uint32_t(count - 1);
    __syncthreads();
    const bool mine = last != 0;
    __syncthreads();   // `last` may be set again
    return mine;
  };
  const int64_t g = chunk / kJoin, g0 = c0 / kJoin, g1 = c1 / kJoin;
  const int64_t lo = max(c0, g * kJoin), hi = min(c1, g * kJoin + kJoin - 1);
  if (!arrive(2 * slot_of(lo), hi - lo + 1)) return;
  Acc<V> a;
#pragma unroll
  for (int i = 0; i < V; ++i) a.v[i] = 0.0f;
  if (live)
#pragma unroll 8
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
#pragma unroll 8
    for (int64_t h = g0; h <= g1; ++h) add_slot<V>(p, slot_of(max(c0, h * kJoin)), col, a);
    write_row<V>(p, token, col, a);
  }
}

// First index in [0, n) of the sorted keys whose key is at least k, n if none:
// each step of the warp cuts the range by 32.
__device__ int64_t lower_bound_warp(const uint32_t* key, int64_t n, uint32_t k) {
  const int lane = int(threadIdx.x & 31);
  int64_t lo = 0, hi = n;
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const int ones = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && __ldcg(key + at) < k));   // a run from lane 0
    if (ones == 0) return lo;
    hi = min(hi, lo + int64_t(ones) * step);
    lo += int64_t(ones - 1) * step + 1;
  }
  return lo;
}

// Zeroes the rows of [r0, r1) that no token names (launch 2's share of the
// zeros, written while the sums wait for their rows).
__device__ void zero_untouched(const GradParams& p, const uint32_t* key, int64_t r0, int64_t r1, uint32_t* mask) {
  __shared__ int64_t bound[2];
  if (threadIdx.x < 32) {
    const int64_t lo = lower_bound_warp(key, p.tokens.n, uint32_t(r0)), hi = lower_bound_warp(key, p.tokens.n, uint32_t(r1));
    if (threadIdx.x == 0) {
      bound[0] = lo;
      bound[1] = hi;
    }
  }
  const int rows = int(r1 - r0);
  for (int i = int(threadIdx.x); i < (rows + 31) / 32; i += int(blockDim.x)) mask[i] = 0u;
  __syncthreads();
  if (bound[1] - bound[0] <= 16 * int64_t(max(rows, int(blockDim.x)))) {
    for (int64_t i = bound[0] + threadIdx.x; i < bound[1]; i += blockDim.x) {
      const uint32_t r = __ldcg(key + i) - uint32_t(r0);
      atomicOr(mask + (r >> 5), 1u << (r & 31u));
    }
  } else {   // a frequent token among them: look the rows up instead of walking its keys
             // (16384 x 768, all the last of 50257 rows: 69 -> 46 us)
    for (int r = int(threadIdx.x); r < rows; r += int(blockDim.x)) {
      int64_t lo = bound[0], hi = bound[1];
      while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (__ldcg(key + mid) < uint32_t(r0 + r))
          lo = mid + 1;
        else
          hi = mid;
      }
      if (lo < bound[1] && __ldcg(key + lo) == uint32_t(r0 + r)) atomicOr(mask + (r >> 5), 1u << (r & 31));
    }
  }
  __syncthreads();
  float* g = p.grad + r0 * p.dim;
  if ((p.dim & 3) == 0) {
    const uint32_t per = uint32_t(p.dim >> 2), total = uint32_t(rows) * per;
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < total; i += blockDim.x) {
      const uint32_t r = i / per;
      if (!((mask[r >> 5] >> (r & 31u)) & 1u)) reinterpret_cast<float4*>(g)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  } else {
    const uint32_t per = uint32_t(p.dim), total = uint32_t(rows) * per;
    for (uint32_t i = threadIdx.x; i < total; i += blockDim.x) {
      const uint32_t r = i / per;
      if (!((mask[r >> 5] >> (r & 31u)) & 1u)) g[i] = 0.0f;
    }
  }
}

template <typename T, int V, bool DROP>
__global__ void __launch_bounds__(256, 4) embed_sum_kernel(const __grid_constant__ GradParams p) {
  __shared__ uint32_t s_key[kMaxChunk + 2];   // the chunk's keys between its neighbours'
  __shared__ uint32_t s_pos[kMaxChunk];
  __shared__ int64_t s_bound[2];
  ptx::griddep_wait();
  const uint32_t* key = p.key[(p.passes + 1) & 1];
  const uint32_t* pos = p.pos[(p.passes + 1) & 1];
  const int64_t n = p.tokens.n;
  const int64_t chunk = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  const int64_t s = chunk * p.chunk, e = min(n, s + p.chunk);
  if (chunk >= p.chunks) {   // the blocks after the sums'
    __shared__ uint32_t mask[kZeroMaskWords];
    const int64_t r0 = p.zero_first + ((chunk - p.chunks) * gridDim.x + blockIdx.x) * p.zero_rows;
    // (a grid of several z layers ends in spare blocks, also where nothing is to be zeroed)
    if (!p.accumulate && r0 < p.vocab) zero_untouched(p, key, r0, min(p.vocab, r0 + p.zero_rows), mask);
    return;
  }
  const uint32_t none = uint32_t(p.vocab);
  for (int i = int(threadIdx.x); i < int(e - s) + 2; i += int(blockDim.x)) {
    const int64_t at = s - 1 + i;
    s_key[i] = at < 0 || at >= n ? none : __ldcg(key + at);
    if (i >= 1 && i <= int(e - s)) s_pos[i - 1] = __ldcg(pos + at);
  }
  uint32_t key_after = none, key_before = none;   // see `reach`
  if (threadIdx.x < 32) {
    const int64_t after = (chunk + 1 + threadIdx.x) * p.chunk, prev = (chunk - int64_t(threadIdx.x)) * p.chunk - 1;
    if (after < n) key_after = __ldcg(key + after);
    if (prev >= 0) key_before = __ldcg(key + prev);
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
  constexpr int U = 4;
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
  // the chunks of the tokens that cross this chunk's ends
  const uint32_t head_key = s_key[1], tail_key = s_key[count];
  if (threadIdx.x < 32) {
    const int64_t c0 = from_before ? reach(p, key, head_key, chunk, key_before, -1) : chunk;
    const int64_t c1 = goes_on ? reach(p, key, tail_key, chunk, key_after, 1) : chunk;
    if (threadIdx.x == 0) {
      s_bound[0] = c0;
      s_bound[1] = c1;
    }
  }
  __syncthreads();
  const int64_t c0 = s_bound[0], c1 = s_bound[1];
  if (from_before) join<V>(p, head_key, chunk, c0, head ? c1 : chunk, col, live);   // (head: one token fills the chunk)
  if (goes_on && !head) join<V>(p, tail_key, chunk, chunk, c1, col, live);
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
cudaError_t lookup_as(const LookupParams& p, int sms, cudaStream_t stream) {
  if ((p.dim & 7) == 0) {
    const int64_t groups = p.dim / 8;
    unsigned x = 1;
    while (x < 256 && x < groups) x <<= 1;
    const unsigned y = 256 / x;
    // a few tokens a block: enough to load indexes ahead, and blocks that end at different times
    const int64_t blocks = std::min<int64_t>((p.tokens.n + y - 1) / y, int64_t(sms) * 40);
    const bool add = p.add != nullptr, drop = p.drop.threshold != 0;
    auto kern = add ? (drop ? embed_lookup_kernel<T, O, true, true> : embed_lookup_kernel<T, O, true, false>)
                    : (drop ? embed_lookup_kernel<T, O, false, true> : embed_lookup_kernel<T, O, false, false>);
    kern<<<unsigned(blocks), dim3(x, y), 0, stream>>>(p);
  } else {
    const int64_t groups = (p.tokens.n * p.dim + 7) / 8;
    embed_lookup_flat_kernel<T, O><<<unsigned((groups + 255) / 256), 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t sum_as(const GradParams& p, cudaStream_t stream) {
  const GradGrid g = grad_grid(p.tokens.n, p.dim);
  const int64_t zeros = p.accumulate ? 0 : (p.vocab - p.zero_first + p.zero_rows - 1) / p.zero_rows;
  const int64_t all = g.chunks + (zeros + g.col_blocks - 1) / g.col_blocks, y = all < 32768 ? all : 32768;
  // the launch overlaps the sort's end
  return launch_kernel(p.drop.threshold != 0 ? embed_sum_kernel<T, V, true> : embed_sum_kernel<T, V, false>,
                       dim3(unsigned(g.col_blocks), unsigned(y), unsigned((all + y - 1) / y)), dim3(unsigned(g.threads)), 0, 1,
                       true, stream, p);
}

cudaError_t launch_sums(const GradParams& p, bool dout_bf16, cudaStream_t stream) {
  const bool vec = (p.dim & 7) == 0;
  if (dout_bf16) return vec ? sum_as<uint16_t, 8>(p, stream) : sum_as<uint16_t, 1>(p, stream);
  return vec ? sum_as<float, 8>(p, stream) : sum_as<float, 1>(p, stream);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? dropout_as<uint16_t>(p, stream) : dropout_as<float>(p, stream);
}

cudaError_t launch_embed_lookup(const LookupParams& p, bool table_bf16, bool out_bf16, int sms, cudaStream_t stream) {
  if (table_bf16) return out_bf16 ? lookup_as<uint16_t, uint16_t>(p, sms, stream) : lookup_as<uint16_t, float>(p, sms, stream);
  return out_bf16 ? lookup_as<float, uint16_t>(p, sms, stream) : lookup_as<float, float>(p, sms, stream);
}

cudaError_t launch_embed_grad(const GradParams& p, bool dout_bf16, cudaStream_t stream) {
  static_assert(kSortSmem <= 227 * 1024, "shared memory");
  const size_t bins = size_t(1) << p.digit_bits;
  const size_t smem = sizeof(uint32_t) * (size_t(kSortWarps) * (bins + 1) + 2 * bins + kSortWarps);
  cudaError_t e;
  if (p.parts > 0) {   // many tokens
    if ((e = allow_smem(reinterpret_cast<const void*>(radix_scatter_kernel), kSortSmem)) != cudaSuccess) return e;
    for (int pass = 0; pass < p.passes; ++pass) {
      if ((e = launch_kernel(radix_count_kernel, dim3(unsigned(p.parts)), dim3(kSortThreads), 0, 1, pass > 0, stream, p, pass)) !=
              cudaSuccess ||
          (e = launch_kernel(radix_scan_kernel, dim3(unsigned(bins)), dim3(kSortThreads), 0, 1, true, stream, p, p.parts)) !=
              cudaSuccess ||
          (e = launch_kernel(radix_scatter_kernel, dim3(unsigned(p.parts)), dim3(kSortThreads), smem, 1, true, stream, p, pass)) !=
              cudaSuccess)
        return e;
    }
    return launch_sums(p, dout_bf16, stream);
  }
  if ((e = allow_smem(reinterpret_cast<const void*>(embed_sort_kernel), kSortSmem)) != cudaSuccess) return e;
  // few tokens sort faster without the cluster's barriers
  const int64_t ctas = p.tokens.n <= kOneCtaTokens ? 1 : 8;
  const int64_t zeros = p.accumulate ? 0 : (p.zero_first * p.dim * 4 + kZeroBytes - 1) / kZeroBytes;
  e = launch_kernel(embed_sort_kernel, dim3(unsigned(ctas + (zeros + ctas - 1) / ctas * ctas)), dim3(kSortThreads), smem,
                    unsigned(ctas), false, stream, p);
  if (e != cudaSuccess) return e;
  return launch_sums(p, dout_bf16, stream);
}

}  // namespace mo
