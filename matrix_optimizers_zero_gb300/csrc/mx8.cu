// 8-bit activation checkpoints: e4m3 codes with a power of two for each 32
// consecutive elements of a row, and what reads them on the way to a product.
//
//   code = e4m3(x 2^-e),  e the least with max |x| <= 448 2^e, e >= -127
//
// The scaling is exact, so a code is one rounding of x (at most 2^-4 of it, for
// elements above 2^-14 of the block's largest), and code 2^e is a bf16 number:
// products read the values without a second rounding.
#include <cuda_runtime.h>

#include "activation.cuh"
#include "launch.cuh"
#include "layer_kernels.h"

namespace mo {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t global_thread() { return int64_t(blockIdx.x) * kThreads + threadIdx.x; }

// Row and column of the first element of group g, where a row has `per_row`
// groups of eight. 64-bit divisions take longer than the rest of a thread.
__device__ __forceinline__ void place(int64_t g, uint32_t per_row, int64_t& row, int64_t& col) {
  if (g >> 32 == 0) {
    const uint32_t q = uint32_t(g) / per_row;
    row = q;
    col = int64_t(uint32_t(g) - q * per_row) * 8;
  } else {
    row = g / per_row;
    col = (g - row * per_row) * 8;
  }
}

// Groups of eight a thread, a block's threads apart: their loads are under way
// together. 8192 x 5120 bf16 in and out: 37 us for 31 of bytes.
constexpr int kQuantGroups = 4;

// Four lanes a block of 32, eight elements a lane. FLAT: rows of whole blocks,
// which need no row and column.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T* __restrict__ x, int64_t groups, int64_t k, uint32_t per_row,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t g0 = int64_t(blockIdx.x) * (kThreads * kQuantGroups) + threadIdx.x;
  float v[kQuantGroups][8];
#pragma unroll
  for (int q = 0; q < kQuantGroups; ++q) {
    const int64_t g = g0 + q * kThreads;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
    if (FLAT) {
      if (g < groups) load8(x + g * 8, v[q]);
    } else {
      int64_t row, col;
      place(g, per_row, row, col);
      if (g < groups && col < k) load8(x + row * k + col, v[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < kQuantGroups; ++q) {
    const int64_t g = g0 + q * kThreads;
    float top = fabsf(v[q][0]);
#pragma unroll
    for (int i = 1; i < 7; i += 2) top = top3(top, v[q][i], v[q][i + 1]);
    top = top2(top, fabsf(v[q][7]));
    top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (g >= groups) continue;   // (whole groups of four lanes)
    const uint32_t s = mx8_scale(top);
    const float down = mx8_down(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[q][i] *= down;
    *reinterpret_cast<uint2*>(codes + g * 8) =
        make_uint2(cvt_e4m3x4(v[q][0], v[q][1], v[q][2], v[q][3]), cvt_e4m3x4(v[q][4], v[q][5], v[q][6], v[q][7]));
    if ((g & 3) == 0) scales[g >> 2] = uint8_t(s);
  }
}

// Rows that are not 16-byte aligned: four neighbours a lane, element by element,
// eight lanes a block, kOddBlocks blocks a lane, loaded together. (An element a lane
// pays for the scale of its block each time: 16384 x 4097 bf16 143 us, so 63.)
constexpr int kOddBlocks = 2;

// f(q, block, row, first column) for a lane's blocks: a warp's lie side by side.
template <typename F>
__device__ __forceinline__ void each_odd(int64_t b0, int64_t blocks, uint32_t nb, F&& f) {
  int64_t row = b0 >> 32 == 0 ? int64_t(uint32_t(b0) / nb) : b0 / nb;
  int64_t at = b0 - row * nb;
#pragma unroll
  for (int q = 0; q < kOddBlocks; ++q) {
    if (b0 + 4 * q < blocks) f(q, b0 + 4 * q, row, at * 32 + (threadIdx.x & 7u) * 4u);
    for (at += 4; at >= nb; at -= nb) ++row;
  }
}
__device__ __forceinline__ int64_t first_odd() { return (global_thread() >> 5) * (4 * kOddBlocks) + ((threadIdx.x & 31u) >> 3); }

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_odd_kernel(const T* __restrict__ x, int64_t blocks, int64_t k, uint32_t nb,
                                                                uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t b0 = first_odd();
  float v[kOddBlocks][4] = {};
  each_odd(b0, blocks, nb, [&](int q, int64_t, int64_t row, int64_t col) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < k) v[q][i] = load1(x + row * k + col + i);
  });
#pragma unroll
  for (int q = 0; q < kOddBlocks; ++q) {
    float top = top2(top3(fabsf(v[q][0]), v[q][1], v[q][2]), fabsf(v[q][3]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const int64_t b = b0 + 4 * q;
    if (b >= blocks) continue;   // (whole groups of eight lanes)
    const uint32_t s = mx8_scale(top), sub = threadIdx.x & 7u;
    const float down = mx8_down(s);
    reinterpret_cast<uint32_t*>(codes)[b * 8 + sub] = cvt_e4m3x4(v[q][0] * down, v[q][1] * down, v[q][2] * down, v[q][3] * down);
    if (sub == 0) scales[b] = uint8_t(s);
  }
}

// Values of 8-bit codes into dense rows of whole blocks, eight a thread and group.
template <typename O>
__global__ void __launch_bounds__(kThreads) unpack_flat_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                               int64_t groups, O* __restrict__ out) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();   // (after the wait: act_grad_kernel)
  const int64_t g0 = int64_t(blockIdx.x) * (kThreads * kQuantGroups) + threadIdx.x;
  uint2 w[kQuantGroups];
  uint8_t s[kQuantGroups];
#pragma unroll
  for (int q = 0; q < kQuantGroups; ++q) {
    const int64_t g = g0 + q * kThreads;
    if (g < groups) {
      w[q] = *reinterpret_cast<const uint2*>(codes + g * 8);
      s[q] = scales[g >> 2];
    }
  }
#pragma unroll
  for (int q = 0; q < kQuantGroups; ++q) {
    const int64_t g = g0 + q * kThreads;
    if (g >= groups) break;
    const float up = mx8_up(s[q]);
    float a[4], b[4], v[8];
    e4m3x4_values(w[q].x, a);
    e4m3x4_values(w[q].y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i] * up;
      v[4 + i] = b[i] * up;
    }
    store8(out + g * 8, v);
  }
}

// Values of 8-bit codes, or of bf16 rows, into rows of `ld` elements: eight
// elements a thread where the output's rows are 16-byte aligned. Elements past
// k are not written.
template <bool MX8, typename O>
__device__ __forceinline__ void unpack_group(const void* src, const uint8_t* scales, int64_t g, int64_t k, uint32_t per_row, O* out,
                                             int64_t ld) {
  int64_t row, col;
  place(g, per_row, row, col);
  float v[8];
  if constexpr (MX8) {
    const uint32_t nb = uint32_t((k + 31) / 32);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(src) + (row * nb * 32 + col));
    const float up = mx8_up(scales[row * nb + (col >> 5)]);
    float a[4], b[4];
    e4m3x4_values(w.x, a);
    e4m3x4_values(w.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i] * up;
      v[4 + i] = b[i] * up;
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(src) + row * k + col;
    const int n = int(min(int64_t(8), k - col));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(s + i) : 0.0f;
  }
  O* o = out + row * ld + col;
  if (col + 8 <= k) {
    store8(o, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < k) store1(o + i, v[i]);
  }
}

template <typename O>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                          int64_t groups, int64_t k, uint32_t per_row, O* __restrict__ out, int64_t ld) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();   // (after the wait: act_grad_kernel)
  const int64_t g = global_thread();
  if (g < groups) unpack_group<true>(codes, scales, g, k, per_row, out, ld);
}

// Up to three operands of products, one behind the other.
struct LayOutParams {
  LayOut t[3];
  int64_t first[3];   // block
};
__global__ void __launch_bounds__(kThreads) lay_out_kernel(const LayOutParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();   // (after the wait: act_grad_kernel)
  const int i = int64_t(blockIdx.x) >= p.first[2] ? 2 : int64_t(blockIdx.x) >= p.first[1] ? 1 : 0;
  const LayOut& t = p.t[i];
  const int64_t g = (int64_t(blockIdx.x) - p.first[i]) * kThreads + threadIdx.x;
  const uint32_t per_row = uint32_t((t.cols + 7) / 8);
  if (g >= t.rows * per_row) return;
  if (t.src.dtype == MO_MX8)
    unpack_group<true>(t.src.data, t.src.scales, g, t.cols, per_row, t.out, t.ld);
  else
    unpack_group<false>(t.src.data, nullptr, g, t.cols, per_row, t.out, t.ld);
}

// 8-bit codes into rows that are not 16-byte aligned, as above.
template <typename O>
__global__ void __launch_bounds__(kThreads) unpack_odd_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                              int64_t blocks, int64_t k, uint32_t nb, O* __restrict__ out) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();   // (after the wait: act_grad_kernel)
  const int64_t b0 = first_odd();
  uint32_t c[kOddBlocks] = {};
  uint8_t s[kOddBlocks] = {};
#pragma unroll
  for (int q = 0; q < kOddBlocks; ++q) {
    const int64_t b = b0 + 4 * q;
    if (b >= blocks) break;
    c[q] = reinterpret_cast<const uint32_t*>(codes)[b * 8 + (threadIdx.x & 7u)];
    s[q] = scales[b];
  }
  each_odd(b0, blocks, nb, [&](int q, int64_t, int64_t row, int64_t col) {
    float v[4];
    e4m3x4_values(c[q], v);
    const float up = mx8_up(s[q]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < k) store1(out + row * k + col + i, v[i] * up);
  });
}

// dz = dout act'(pre) and its column sums: a block takes 256 columns, eight a
// thread, and `per` rows, eight at a time (one a warp); its warps' sums are
// joined in order. A launch of strips x parts blocks. dz is rounded to bf16, as an operand
// of the products; its sums are not. 8192 x 5120 with gelu_tanh and 8-bit pre: 38 us (gelu
// 44), by issue slots (61%) and latency; bytes alone 31.
constexpr int kRowsAhead = 2;   // of a warp, loaded together

template <bool MX8, int ACT>
__device__ __forceinline__ void act_grad_rows(const ActGradParams& p, int64_t row0, int64_t row1, int64_t col, F2 (&sum)[4]) {
  const int64_t n = p.rows;
  if (col >= n) return;
  // Pointers to this lane's elements of the next row, and what a warp's next row is further on: two
  // thirds of the time of a row are instructions.
  const int64_t pitch = MX8 ? (n + 31) / 32 * 32 : n, first = row0 + (threadIdx.x >> 5);
  const uint16_t* dout_at = p.dout + first * n + col;
  const uint8_t* pre_at = static_cast<const uint8_t*>(p.pre.data) + (first * pitch + col) * (MX8 ? 1 : 2);
  const uint8_t* scale_at = p.pre.scales + (first * pitch + col) / 32;
  uint16_t* dz_at = p.dz + first * p.ld + col;
  auto row = [&](const uint4& dout, const uint4& pre) {
    const uint32_t w[4] = {dout.x, dout.y, dout.z, dout.w};
    F2 d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = ptx::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    if constexpr (ACT != MO_ACT_NONE) {
      F2 z[4];
      if constexpr (MX8) {
        const F2 up = ptx::f2(mx8_up(pre.z));
        float a[4], b[4];
        e4m3x4_values(pre.x, a);
        e4m3x4_values(pre.y, b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          z[i] = ptx::mul2(ptx::f2(a[2 * i], a[2 * i + 1]), up);
          z[2 + i] = ptx::mul2(ptx::f2(b[2 * i], b[2 * i + 1]), up);
        }
      } else {
        const uint32_t v[4] = {pre.x, pre.y, pre.z, pre.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = ptx::f2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        F2 value;
        d[i] = ptx::mul2(d[i], act_slope<ACT>(z[i], &value));
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] = ptx::add2(sum[i], d[i]);
      const float2 y = ptx::parts(d[i]);
      o[i] = pack_bf16x2(y.x, y.y);
    }
    if (p.dz != nullptr) *reinterpret_cast<uint4*>(dz_at) = make_uint4(o[0], o[1], o[2], o[3]);
    dz_at += 8 * p.ld;
  };
  for (int64_t left = (row1 - first + 7) / 8; left > 0; left -= kRowsAhead) {
    uint4 dout[kRowsAhead], pre[kRowsAhead] = {};   // (pre: two words of 8-bit codes and the scale)
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (u >= left) break;
      dout[u] = *reinterpret_cast<const uint4*>(dout_at);
      if constexpr (ACT != MO_ACT_NONE) {
        if constexpr (MX8) {
          const uint2 c = *reinterpret_cast<const uint2*>(pre_at);
          pre[u] = make_uint4(c.x, c.y, *scale_at, 0u);
          scale_at += pitch / 4;
        } else {
          pre[u] = *reinterpret_cast<const uint4*>(pre_at);
        }
        pre_at += 8 * pitch * (MX8 ? 1 : 2);
      }
      dout_at += 8 * n;
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      if (u < left) row(dout[u], pre[u]);
  }
}

// Rows that are not 16-byte aligned: a thread's eight columns are a warp apart.
template <bool MX8, int ACT>
__device__ __forceinline__ void act_grad_rows_odd(const ActGradParams& p, int64_t row0, int64_t row1, int64_t col, float (&sum)[8]) {
  const int64_t n = p.rows;
  const uint32_t nb = uint32_t((n + 31) / 32);
  for (int64_t r = row0 + (threadIdx.x >> 5); r < row1; r += 8) {
    float d[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = col + 32 * i;
      d[i] = c < n ? load1(p.dout + r * n + c) : 0.0f;
      z[i] = 0.0f;
      if constexpr (ACT != MO_ACT_NONE) {
        if (c < n) {
          if constexpr (MX8)
            z[i] = e4m3_value(static_cast<const uint8_t*>(p.pre.data)[r * nb * 32 + c]) * mx8_up(p.pre.scales[r * nb + (c >> 5)]);
          else
            z[i] = load1(static_cast<const uint16_t*>(p.pre.data) + r * n + c);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float value;
      // (one rounding each, as in the pairs above: with and without dz the sums are the same)
      if constexpr (ACT != MO_ACT_NONE) d[i] = __fmul_rn(d[i], act_slope<ACT>(z[i], &value));
      sum[i] = __fadd_rn(sum[i], d[i]);
      if (p.dz != nullptr && col + 32 * i < n) store1(p.dz + r * p.ld + col + 32 * i, d[i]);
    }
  }
}

template <bool VEC, bool MX8>
__global__ void __launch_bounds__(kThreads, VEC ? 4 : 2) act_grad_kernel(const ActGradParams p) {
  __shared__ float sums[8][256];
  ptx::griddep_launch_dependents();
  // early: behind a launch that lays out operands and writes nothing that is read here. Its blocks let this
  // one come when they have waited, so what was before it has ended; and this one ends behind it.
  if (!p.early) ptx::griddep_wait();
  const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
  const int64_t col = int64_t(blockIdx.x) * 256 + (VEC ? lane * 8 : lane);
  const int64_t row0 = int64_t(blockIdx.y) * p.per, row1 = min(row0 + p.per, p.tokens);
  float sum[8] = {};
  with_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    if constexpr (VEC) {
      F2 pairs[4] = {ptx::f2(0.0f), ptx::f2(0.0f), ptx::f2(0.0f), ptx::f2(0.0f)};
      act_grad_rows<MX8, ACT>(p, row0, row1, col, pairs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 s = ptx::parts(pairs[i]);
        sum[2 * i] = s.x, sum[2 * i + 1] = s.y;
      }
    } else {
      act_grad_rows_odd<MX8, ACT>(p, row0, row1, col, sum);
    }
  });
  if (p.part != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][VEC ? lane * 8 + i : lane + 32 * i] = sum[i];
    __syncthreads();
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (c < p.rows) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
      p.part[int64_t(blockIdx.y) * p.rows + c] = t;
    }
  }
  if (p.early) ptx::griddep_wait();
}

// Column sums of part [parts, n]: a block takes 32 columns, each of its warps a
// run of rows in order, and the warps' sums are joined in order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const float* __restrict__ part, int64_t parts, int64_t n, float* out,
                                                               int accumulate) {
  __shared__ float sums[kJoinWarps][33];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  const int64_t per = (parts + kJoinWarps - 1) / kJoinWarps, r1 = min((warp + 1) * per, parts);
  float t = 0.0f;
  if (c < n) {
#pragma unroll 8
    for (int64_t r = warp * per; r < r1; ++r) t += part[r * n + c];
  }
  sums[warp][lane] = t;
  __syncthreads();
  // warp w: column w, a lane for each run
  t = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  const int64_t col = int64_t(blockIdx.x) * 32 + warp;
  if (lane == 0 && col < n) out[col] = accumulate ? out[col] + t : t;
}

unsigned blocks_of(int64_t threads) { return unsigned((threads + kThreads - 1) / kThreads); }

unsigned quant_blocks(int64_t groups) { return unsigned((groups + kThreads * kQuantGroups - 1) / (kThreads * kQuantGroups)); }

unsigned odd_blocks(int64_t blocks) { return blocks_of((blocks + 4 * kOddBlocks - 1) / (4 * kOddBlocks) * 32); }

template <typename T>
cudaError_t quantize_as(const T* x, int64_t rows, int64_t k, const Kept& q, cudaStream_t stream) {
  const int64_t nb = mx8_blocks(k);
  uint8_t* codes = static_cast<uint8_t*>(q.data);
  if (k % 8 == 0) {
    const int64_t groups = rows * nb * 4;
    auto kern = k % 32 == 0 ? quantize_kernel<T, true> : quantize_kernel<T, false>;
    return launch_kernel(kern, dim3(quant_blocks(groups)), dim3(kThreads), 0, 1, true, stream, x, groups, k, uint32_t(nb * 4), codes,
                         q.scales);
  }
  return launch_kernel(quantize_odd_kernel<T>, dim3(odd_blocks(rows * nb)), dim3(kThreads), 0, 1, true, stream, x, rows * nb, k,
                       uint32_t(nb), codes, q.scales);
}

template <typename O>
cudaError_t unpack_as(const Kept& src, int64_t rows, int64_t k, O* out, cudaStream_t stream) {
  const uint8_t* s = static_cast<const uint8_t*>(src.data);
  const uint8_t* scales = src.scales;
  if (k % 32 == 0)
    return launch_kernel(unpack_flat_kernel<O>, dim3(quant_blocks(rows * k / 8)), dim3(kThreads), 0, 1, true, stream, s, scales,
                         rows * k / 8, out);
  if (k % 8 == 0)
    return launch_kernel(unpack_kernel<O>, dim3(blocks_of(rows * k / 8)), dim3(kThreads), 0, 1, true, stream, s, scales, rows * k / 8, k,
                         uint32_t(k / 8), out, k);
  const int64_t nb = mx8_blocks(k);
  return launch_kernel(unpack_odd_kernel<O>, dim3(odd_blocks(rows * nb)), dim3(kThreads), 0, 1, true, stream, s, scales, rows * nb, k,
                       uint32_t(nb), out);
}

}  // namespace

cudaError_t launch_mx8_quantize(const void* x, bool bf16, int64_t rows, int64_t k, const Kept& q, cudaStream_t stream) {
  return bf16 ? quantize_as(static_cast<const uint16_t*>(x), rows, k, q, stream)
              : quantize_as(static_cast<const float*>(x), rows, k, q, stream);
}

cudaError_t launch_unpack(const Kept& src, int64_t rows, int64_t k, void* out, bool out_bf16, cudaStream_t stream) {
  return out_bf16 ? unpack_as(src, rows, k, static_cast<uint16_t*>(out), stream)
                  : unpack_as(src, rows, k, static_cast<float*>(out), stream);
}

cudaError_t launch_lay_out(const LayOut* t, int count, cudaStream_t stream) {
  if (count == 1 && t[0].src.dtype == MO_MX8 && t[0].ld == t[0].cols) return unpack_as(t[0].src, t[0].rows, t[0].cols, t[0].out, stream);
  LayOutParams p = {};
  int64_t blocks = 0;
  for (int i = 0; i < 3; ++i) {
    p.first[i] = i < count ? blocks : int64_t(1) << 62;
    if (i >= count) continue;
    p.t[i] = t[i];
    blocks += blocks_of(t[i].rows * ((t[i].cols + 7) / 8));
  }
  return launch_kernel(lay_out_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, 1, true, stream, p);
}

cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned((p.rows + 255) / 256), unsigned((p.tokens + p.per - 1) / p.per));
  const bool vec = p.rows % 8 == 0, mx8 = p.act != MO_ACT_NONE && p.pre.dtype == MO_MX8;
  auto kern = vec ? (mx8 ? act_grad_kernel<true, true> : act_grad_kernel<true, false>)
                  : (mx8 ? act_grad_kernel<false, true> : act_grad_kernel<false, false>);
  return launch_kernel(kern, grid, dim3(kThreads), 0, 1, true, stream, p);
}

cudaError_t launch_join(const float* part, int64_t parts, int64_t n, float* out, bool accumulate, cudaStream_t stream) {
  return launch_kernel(join_kernel, dim3(unsigned((n + 31) / 32)), dim3(32 * kJoinWarps), 0, 1, true, stream, part, parts, n, out,
                       accumulate ? 1 : 0);
}

}  // namespace mo
