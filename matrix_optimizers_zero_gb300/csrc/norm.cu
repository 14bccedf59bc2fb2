// Root-mean-square norm of rows, after the addition of a residual, and its
// backward pass:
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   g = dy w:  dx = r (g - s r mean(g s r)) + dres,  dw = sum over rows of dy s r
//
// A team of threads takes a row, eight elements a thread, and reads it once: the
// backward pass needs the two sums of s^2 and of g s, which one reduction
// gives. A team of the backward pass goes from row to row and adds its part of
// dw in registers; the teams' parts are joined in order, so results do not
// depend on scheduling.
#include <cuda_runtime.h>

#include <type_traits>

#include "activation.cuh"
#include "launch.cuh"
#include "layer_kernels.h"
#include "ptx_train.cuh"

namespace mo {
namespace {

// A team of TEAM threads holds a row of at most 8 TEAM elements, eight a thread:
// eight neighbours of every 8 TEAM where rows are 16-byte aligned (VEC), one of
// every TEAM otherwise. Either way 32 elements of a block lie in one warp.
template <int TEAM, bool VEC>
__device__ __forceinline__ int64_t column(int i, int t) {
  return VEC ? int64_t((i >> 3) * TEAM + t) * 8 + (i & 7) : int64_t(i) * TEAM + t;
}

template <int TEAM>
constexpr int kBlock = TEAM < 128 ? 128 : TEAM;

// Elements TEAM apart.
template <int TEAM, typename T>
__device__ __forceinline__ void store_row(T* p, int64_t dim, int t, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    if (c < dim) store1(p + c, v[i]);
  }
}

// A row in 8 bits. All threads of a warp come here together; elements past dim
// are zeros, and the codes of the last block past it too.
template <int TEAM, bool VEC>
__device__ __forceinline__ void store_row_mx8(uint8_t* codes, uint8_t* scales, int64_t end, int t, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += VEC ? 8 : 1) {
    const int64_t c = column<TEAM, VEC>(i, t);
    float top = fabsf(v[i]);
    if constexpr (VEC) {
#pragma unroll
      for (int j = 1; j < 7; j += 2) top = top3(top, v[i + j], v[i + j + 1]);
      top = top2(top, fabsf(v[i + 7]));
    }
#pragma unroll
    for (int o = VEC ? 2 : 16; o > 0; o >>= 1) top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (c >= end) continue;
    const uint32_t s = mx8_scale(top);
    const float down = mx8_down(s);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(codes + c) =
          make_uint2(cvt_e4m3x4(v[i] * down, v[i + 1] * down, v[i + 2] * down, v[i + 3] * down),
                     cvt_e4m3x4(v[i + 4] * down, v[i + 5] * down, v[i + 6] * down, v[i + 7] * down));
    } else {
      codes[c] = uint8_t(cvt_e4m3x2(v[i] * down, 0.0f));
    }
    if ((c & 31) == 0) scales[c >> 5] = uint8_t(s);
  }
}

// mean + eps where squares and products in fp32 say all: above what is lost where a
// square is below 2^-126, and finite. Others are computed again from scaled rows.
__device__ __forceinline__ bool usual(float mean_eps) { return mean_eps >= 0x1p-80f && mean_eps <= 3.402823466e38f; }
// (m: mean(g n); the same for the products of the backward pass)
__device__ __forceinline__ bool usual(float mean_eps, float m) { return usual(mean_eps) && fabsf(m) <= 0x1p100f; }

// 1 / sqrt(x), two units of 2^-23 off at most; infinite below 2^-126, which `usual` and
// scaled rows leave to rows of zeros (eps 0)
__device__ __forceinline__ float inverse_sqrt(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Sums of a and b over a team, in a fixed order, with one barrier: a row's warps
// leave theirs in one half of `shared`, the next row's in the other (parity). A
// team of a warp needs neither; teams of more are a whole block. From the first
// step on the upper half of a warp sums b and the lower a.
template <int TEAM>
__device__ __forceinline__ float2 team_sums(float a, float b, float (&shared)[2][64], int parity) {
  const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
  const bool upper = lane >= 16;
  float v = upper ? b : a;
  v += __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (TEAM > 32) {
    constexpr int kWarps = TEAM / 32;
    if ((lane & 15) == 0) shared[parity][(upper ? kWarps : 0) + warp] = v;
    __syncthreads();
    if constexpr (kWarps <= 16) {
      v = shared[parity][(upper ? kWarps : 0) + lane % kWarps];
    } else {
      v = shared[parity][(upper ? 32 : 0) + (lane & 15)] + shared[parity][(upper ? 48 : 16) + (lane & 15)];
    }
#pragma unroll
    for (int o = (kWarps <= 16 ? kWarps : 16) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
}

// Maxima of a and b over a team, likewise (a and b not negative; NaN does not count).
template <int TEAM>
__device__ __forceinline__ float2 team_max(float a, float b, float (&shared)[2][64], int parity) {
  const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    b = fmaxf(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
  }
  if constexpr (TEAM > 32) {
    constexpr int kWarps = TEAM / 32;
    if (lane == 0) shared[parity][warp] = a, shared[parity][32 + warp] = b;
    __syncthreads();
    a = shared[parity][lane % kWarps];
    b = shared[parity][32 + lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      b = fmaxf(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
    }
  }
  return make_float2(a, b);
}

// ------------------------------------------------------------------ rows out of range
//
// A row whose squares (or products with the gradient) leave fp32's range is scaled by
// a power of two, which loses nothing: with t = s 2^-e and the largest |t| (or the
// square root of eps) in [1, 4), r' = 1 / sqrt(mean(t^2) + eps 2^-2e) gives n = t r' = s r.
//
// The team's first sums have used one half of `shared` (parity); its maxima take the
// other, and the second sums the first again: between two uses of a half lies a barrier.

// The exponent of a magnitude, -126 to 126; 0 of 0 and of what is not finite.
__device__ __forceinline__ int exponent_of(float top) {
  const int e = int(__float_as_uint(top) >> 23);
  return top == 0.0f || e == 255 ? 0 : min(max(e, 1), 253) - 127;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }   // e: -126 to 127

// s becomes t; r'.
template <int TEAM>
__device__ __forceinline__ float scaled_row(float (&s)[8], float inv_dim, float eps, float (&shared)[2][64], int parity) {
  float top = 0.0f, squares = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(s[i]));
  top = team_max<TEAM>(top, 0.0f, shared, parity ^ 1).x;
  const float down = power_of_two(-exponent_of(fmaxf(top, sqrtf(eps))));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] *= down;
    squares = fmaf(s[i], s[i], squares);
  }
  return inverse_sqrt(fmaf(team_sums<TEAM>(squares, 0.0f, shared, parity).x, inv_dim, eps * down * down));
}

// s becomes n and w the gradient r (g - n mean(g n)); dy is scaled by its own power
// of two on the way.
template <int TEAM>
__device__ __forceinline__ void scaled_grad_row(float (&s)[8], const float (&dy)[8], float (&w)[8], float inv_dim, float eps,
                                                float (&shared)[2][64], int parity) {
  float top_s = 0.0f, top_d = 0.0f, squares = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top_s = fmaxf(top_s, fabsf(s[i]));
    top_d = fmaxf(top_d, fabsf(dy[i]));
  }
  const float2 top = team_max<TEAM>(top_s, top_d, shared, parity ^ 1);
  const int es = exponent_of(fmaxf(top.x, sqrtf(eps))), ed = exponent_of(top.y);
  const float down_s = power_of_two(-es), down_d = power_of_two(-ed);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] *= down_s;
    w[i] *= dy[i] * down_d;
    squares = fmaf(s[i], s[i], squares);
    dot = fmaf(w[i], s[i], dot);
  }
  const float2 sums = team_sums<TEAM>(squares, dot, shared, parity);
  const float r = inverse_sqrt(fmaf(sums.x, inv_dim, eps * down_s * down_s)), m = sums.y * r * inv_dim;
  const int c = ed - es;   // (in two steps: up to 2^252)
  const float c0 = power_of_two(c / 2), c1 = power_of_two(c - c / 2);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] *= r;
    w[i] = r * fmaf(-s[i], m, w[i]) * c0 * c1;
  }
}

// ------------------------------------------------------------------ aligned rows
//
// A thread copies its eight elements of the rows to come into slots of its own in
// shared memory (cp.async), up to three rows ahead, and reads them back when it
// gets there: no barrier, no registers, and enough bytes under way. With one row
// ahead in registers the backward pass of 16384 x 4096 took 101 us.
//
// 16384 x 4096 bf16 with a residual, the sum and an 8-bit result: 72 us, 6.5 TB/s,
// bound by memory. Backward from 8-bit rows with dres and dw: 77 us and 6 for the
// join, 71% of issue slots and 68% of DRAM's rate.
//
// Rows ahead where a row takes `slot` bytes a thread: 1024 threads' in 196 KB.
constexpr int rows_ahead(int slot) { return 192 / slot - 1 < 3 ? 192 / slot - 1 : 3; }

// Slots of BYTES bytes for each of THREADS threads and every row under way; 16
// bytes of neighbouring threads lie side by side, so a warp's accesses meet all
// banks.
template <int BYTES, int THREADS>
struct Slots {
  static constexpr int kUnit = BYTES < 16 ? BYTES : 16;
  static constexpr uint32_t kSlot = BYTES * THREADS;   // of one row
  uint32_t base;   // this thread's first
  __device__ __forceinline__ explicit Slots(uint32_t start) : base(start + threadIdx.x * kUnit) {}
  __device__ __forceinline__ uint32_t at(uint32_t slot, int unit) const { return base + slot * kSlot + uint32_t(unit) * THREADS * kUnit; }
  __device__ __forceinline__ void copy(uint32_t slot, const void* g) const {
#pragma unroll
    for (int i = 0; i < BYTES / kUnit; ++i) {
      const uint8_t* p = static_cast<const uint8_t*>(g) + i * kUnit;
      if constexpr (kUnit == 16)
        ptx::cp_async16(at(slot, i), p);
      else
        ptx::cp_async8(at(slot, i), p);
    }
  }
};
__device__ __forceinline__ void bf16_values(const uint4& w, F2 (&v)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = ptx::f2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xFFFF0000u));
}
template <int THREADS>
__device__ __forceinline__ void slot_values(const Slots<16, THREADS>& s, uint32_t slot, float, F2 (&v)[4]) {   // bf16
  bf16_values(ptx::ld_shared_v4(s.at(slot, 0)), v);
}
template <int THREADS>
__device__ __forceinline__ void slot_values(const Slots<32, THREADS>& s, uint32_t slot, float, F2 (&v)[4]) {   // fp32
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = ptx::ld_shared_v4(s.at(slot, i));
    v[2 * i] = ptx::f2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[2 * i + 1] = ptx::f2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}
template <int THREADS>
__device__ __forceinline__ void slot_values(const Slots<8, THREADS>& s, uint32_t slot, float up, F2 (&v)[4]) {   // 8 bits
  const uint2 w = ptx::ld_shared_v2(s.at(slot, 0));
  const F2 u = ptx::f2(up);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float a[4];
    e4m3x4_values(i == 0 ? w.x : w.y, a);
    v[2 * i] = ptx::mul2(ptx::f2(a[0], a[1]), u);
    v[2 * i + 1] = ptx::mul2(ptx::f2(a[2], a[3]), u);
  }
}
__device__ __forceinline__ void unpair(const F2 (&v)[4], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = ptx::parts(v[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ void pair(const float (&f)[8], F2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ptx::f2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const F2 (&v)[4]) {
  float f[8];
  unpair(v, f);
  store8(p, f);
}

template <typename T>
constexpr int kNormSlot = 2 * 8 * int(sizeof(T));
template <typename T>
constexpr int kNormAhead = rows_ahead(kNormSlot<T>);
template <typename T, bool MX8>
constexpr int kGradSlot = 2 * 8 * int(sizeof(T)) + (MX8 ? 8 : 8 * int(sizeof(T)));
template <typename T, bool MX8>
constexpr int kGradAhead = rows_ahead(kGradSlot<T, MX8>);
static_assert(kNormAhead<float> >= 1 && kGradAhead<float, true> >= 1 && kGradAhead<float, false> >= 1, "a row ahead");

// A row out of range, once more from its slots.
template <int TEAM, typename T>
__device__ __noinline__ void scaled_slot_row(const NormParams& p, int64_t row, uint32_t xs_at, uint32_t rs_at, float (&shared)[2][64], int parity) {
  const int t = int(threadIdx.x) % TEAM;
  const int64_t col = int64_t(t) * 8, nb = (p.dim + 31) / 32, at = row * p.dim + col;
  const bool in = col < p.dim;
  const Slots<8 * int(sizeof(T)), kBlock<TEAM>> xs(xs_at), rs(rs_at);
  float f[8] = {};
  if (in) {
    F2 s[4];
    slot_values(xs, 0, 0.0f, s);
    if (p.residual != nullptr) {
      F2 r[4];
      slot_values(rs, 0, 0.0f, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = ptx::add2(s[i], r[i]);
    }
    unpair(s, f);
  }
  const float r = scaled_row<TEAM>(f, 1.0f / float(p.dim), p.eps, shared, parity);
  if (in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * r * (p.weight != nullptr ? p.weight[col + i] : 1.0f);
    if (p.out != nullptr) {
      if (p.out_bf16)
        store8(static_cast<uint16_t*>(p.out) + at, f);
      else
        store8(static_cast<float*>(p.out) + at, f);
    }
  }
  if (p.out8.data != nullptr)
    store_row_mx8<TEAM, true>(static_cast<uint8_t*>(p.out8.data) + row * nb * 32, p.out8.scales + row * nb, nb * 32, t, f);
}

template <int TEAM, typename T>
__global__ void __launch_bounds__(kBlock<TEAM>, 1024 / kBlock<TEAM>) norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t slots[];
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM, kRow = 8 * int(sizeof(T)), kAhead = kNormAhead<T>;
  const int t = int(threadIdx.x) % TEAM;
  const int64_t team = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM, step = int64_t(gridDim.x) * kTeams;
  const int64_t col = int64_t(t) * 8, nb = (p.dim + 31) / 32;
  const bool in = col < p.dim;
  const float inv_dim = 1.0f / float(p.dim);
  const uint32_t start = ptx::smem_addr(slots);
  const Slots<kRow, kBlock<TEAM>> xs(start), rs(start + (kAhead + 1) * xs.kSlot);
  const T* x = static_cast<const T*>(p.x) + col;
  const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + col : nullptr;
  auto fetch = [&](int64_t row, uint32_t slot) {
    if (row < p.rows && in) {
      xs.copy(slot, x + row * p.dim);
      if (res != nullptr) rs.copy(slot, res + row * p.dim);
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(team + i * step, uint32_t(i));
  F2 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ptx::f2(1.0f);
  if (p.weight != nullptr && in) {
    float f[8];
    load8(p.weight + col, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::f2(f[2 * i], f[2 * i + 1]);
  }
  uint32_t slot = 0;
  int parity = 0;
  for (int64_t row = team; row < p.rows; row += step, parity ^= 1) {
    fetch(row + kAhead * step, slot == 0 ? kAhead : slot - 1);
    ptx::cp_async_wait_but<kAhead>();
    F2 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = ptx::f2(0.0f);
    if (in) {
      slot_values(xs, slot, 0.0f, s);
      if (res != nullptr) {
        F2 r[4];
        slot_values(rs, slot, 0.0f, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = ptx::add2(s[i], r[i]);
      }
      if (p.sum != nullptr) store_pairs(static_cast<T*>(p.sum) + row * p.dim + col, s);
    }
    F2 squares = ptx::mul2(s[0], s[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) squares = ptx::fma2(s[i], s[i], squares);
    const float2 half = ptx::parts(squares);
    const float mean = fmaf(team_sums<TEAM>(half.x + half.y, 0.0f, shared, parity).x, inv_dim, p.eps);
    const int64_t at = row * p.dim + col;
    const F2 r = ptx::f2(inverse_sqrt(mean));
    // (a thread past dim holds zeros; where r is not finite they have to stay so)
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = ptx::mul2(ptx::mul2(s[i], r), w[i]);
      if (p.out != nullptr) {
        if (p.out_bf16)
          store_pairs(static_cast<uint16_t*>(p.out) + at, s);
        else
          store_pairs(static_cast<float*>(p.out) + at, s);
      }
    }
    if (p.out8.data != nullptr) {
      float v[8];
      unpair(s, v);
      store_row_mx8<TEAM, true>(static_cast<uint8_t*>(p.out8.data) + row * nb * 32, p.out8.scales + row * nb, nb * 32, t, v);
    }
    if (!usual(mean))   // once more, from the slots: behind the row, where the check holds nothing up
      scaled_slot_row<TEAM, T>(p, row, start + slot * xs.kSlot, start + (kAhead + 1 + slot) * xs.kSlot, shared, parity);
    slot = slot == kAhead ? 0 : slot + 1;
  }
}

template <int TEAM, typename T, bool MX8>
__global__ void __launch_bounds__(kBlock<TEAM>, 1024 / kBlock<TEAM>) norm_grad_kernel(const NormGradParams p) {
  extern __shared__ __align__(16) uint8_t slots[];
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM, kRow = 8 * int(sizeof(T)), kAhead = kGradAhead<T, MX8>;
  const int t = int(threadIdx.x) % TEAM;
  const int64_t team = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM, step = int64_t(gridDim.x) * kTeams;
  const int64_t col = int64_t(t) * 8, nb = (p.dim + 31) / 32;
  const bool in = col < p.dim;
  const float inv_dim = 1.0f / float(p.dim);
  const uint32_t start = ptx::smem_addr(slots);
  const Slots<kRow, kBlock<TEAM>> ds(start), rs(start + (kAhead + 1) * ds.kSlot);
  const Slots<MX8 ? 8 : kRow, kBlock<TEAM>> xs(start + 2 * (kAhead + 1) * ds.kSlot);
  // The rows that are left, this thread's elements of the first of them, and how far the next are (of 8-bit
  // rows at8 and stride8): the instructions of a row take most of its time.
  int left = team < p.rows ? int((p.rows - team + step - 1) / step) : 0;
  int64_t at = team * p.dim + col, at8 = team * nb * 32 + col;
  const int64_t stride = step * p.dim, stride8 = step * nb * 32;
  auto fetch = [&](int ahead, uint32_t slot) {
    if (left > ahead && in) {
      ds.copy(slot, static_cast<const T*>(p.dy) + at + ahead * stride);
      if constexpr (MX8)
        xs.copy(slot, static_cast<const uint8_t*>(p.x.data) + at8 + ahead * stride8);
      else
        xs.copy(slot, static_cast<const T*>(p.x.data) + at + ahead * stride);
      if (p.dres != nullptr) rs.copy(slot, static_cast<const T*>(p.dres) + at + ahead * stride);
    }
    ptx::cp_async_commit();
  };
  // (a scale is one byte, too few for such a copy: one row ahead in a register)
  auto scale_of = [&](int ahead) { return MX8 && left > ahead && in ? p.x.scales[(at8 + ahead * stride8) >> 5] : uint8_t(0); };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i, uint32_t(i));
  uint8_t scale = scale_of(0);
  F2 w[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ptx::f2(1.0f), dw[i] = ptx::f2(0.0f);
  if (p.weight != nullptr && in) {
    float f[8];
    load8(p.weight + col, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::f2(f[2 * i], f[2 * i + 1]);
  }
  uint32_t slot = 0;
  int parity = 0;
  for (; left > 0; --left, at += stride, at8 += stride8, parity ^= 1) {
    fetch(kAhead, slot == 0 ? kAhead : slot - 1);
    ptx::cp_async_wait_but<kAhead>();
    F2 s[4], dy[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = ptx::f2(0.0f), dy[i] = ptx::f2(0.0f);
    if (in) {
      slot_values(ds, slot, 0.0f, dy);
      slot_values(xs, slot, MX8 ? mx8_up(scale) : 0.0f, s);
    }
    scale = scale_of(1);
    F2 squares = ptx::mul2(s[0], s[0]), dot = ptx::mul2(ptx::mul2(dy[0], w[0]), s[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      squares = ptx::fma2(s[i], s[i], squares);
      dot = ptx::fma2(ptx::mul2(dy[i], w[i]), s[i], dot);
    }
    const float2 hs = ptx::parts(squares), hd = ptx::parts(dot);
    const float2 sums = team_sums<TEAM>(hs.x + hs.y, hd.x + hd.y, shared, parity);
    const float mean = fmaf(sums.x, inv_dim, p.eps);
    float r = inverse_sqrt(mean), m = sums.y * r * inv_dim;   // m: mean(g s r)
    const bool fits = usual(mean, m);
    if (!fits) r = m = 0.0f;   // (adds nothing to dw)
    auto put = [&] {           // dy is the norm's gradient
      if (p.dres != nullptr) {
        slot_values(rs, slot, 0.0f, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) dy[i] = ptx::add2(dy[i], s[i]);
      }
      store_pairs(static_cast<T*>(p.dx) + at, dy);
    };
    if (in) {
      const F2 r2 = ptx::f2(r), m2 = ptx::f2(-m);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 n = ptx::mul2(s[i], r2);
        dw[i] = ptx::fma2(dy[i], n, dw[i]);
        dy[i] = ptx::mul2(r2, ptx::fma2(n, m2, ptx::mul2(dy[i], w[i])));
      }
      put();
    }
    if (!fits) {   // once more, from the slots: behind the row, where the check holds nothing up
      float fs[8] = {}, fd[8] = {}, fw[8];
      if (in) {
        slot_values(ds, slot, 0.0f, dy);
        slot_values(xs, slot, MX8 ? mx8_up(p.x.scales[at8 >> 5]) : 0.0f, s);
        unpair(s, fs);
        unpair(dy, fd);
      }
      unpair(w, fw);
      scaled_grad_row<TEAM>(fs, fd, fw, inv_dim, p.eps, shared, parity);
      if (in) {
        F2 n[4];
        pair(fs, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[i] = ptx::fma2(dy[i], n[i], dw[i]);
        pair(fw, dy);
        put();
      }
    }
    slot = slot == kAhead ? 0 : slot + 1;
  }
  if (p.part != nullptr && in) store_pairs(p.part + team * p.dim + col, dw);
}

// ------------------------------------------------------------------ other rows
//
// Rows that are not 16-byte aligned: elements TEAM apart, eight a thread, in the
// backward pass one row ahead in registers. Far from memory's rate, for its loads and
// stores of single elements: 16384 x 4097 bf16 154 us (40 of bytes), with residual, sum
// and 8-bit result 307 (71), its gradient 445 (59), from 8-bit rows with dres and dw 566
// (69).
// (2^-e, r') of a row out of range, from memory
template <int TEAM, typename T>
__device__ __noinline__ float2 scaled_odd_row(const T* x, const T* res, int64_t dim, float eps, float (&shared)[2][64]) {
  float top = 0.0f, squares = 0.0f;
#pragma unroll 1
  for (int64_t c = int(threadIdx.x) % TEAM; c < dim; c += TEAM)
    top = fmaxf(top, fabsf(load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f)));
  top = team_max<TEAM>(top, 0.0f, shared, 1).x;
  const float down = power_of_two(-exponent_of(fmaxf(top, sqrtf(eps))));
#pragma unroll 1
  for (int64_t c = int(threadIdx.x) % TEAM; c < dim; c += TEAM) {
    const float t = (load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f)) * down;
    squares = fmaf(t, t, squares);
  }
  const float mean = fmaf(team_sums<TEAM>(squares, 0.0f, shared, 0).x, 1.0f / float(dim), eps * down * down);
  return make_float2(down, inverse_sqrt(mean));
}

template <typename T>
__device__ __forceinline__ float kept_value(const Kept& x, int64_t row, int64_t dim, int64_t c) {
  const int64_t nb = (dim + 31) / 32;
  if (x.dtype == MO_MX8) return e4m3_value(static_cast<const uint8_t*>(x.data)[row * nb * 32 + c]) * mx8_up(x.scales[row * nb + (c >> 5)]);
  return load1(static_cast<const T*>(x.data) + row * dim + c);
}

template <int TEAM, typename T>
__global__ void __launch_bounds__(kBlock<TEAM>) norm_odd_kernel(const NormParams p) {
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM;
  const int t = int(threadIdx.x) % TEAM;
  const int64_t row = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM;
  if (row >= p.rows) return;   // a whole warp, and a whole block where teams are more than one
  const int64_t at = row * p.dim, nb = (p.dim + 31) / 32;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    s[i] = c < p.dim ? load1(static_cast<const T*>(p.x) + at + c) : 0.0f;
  }
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = column<TEAM, false>(i, t);
      if (c < p.dim) s[i] += load1(static_cast<const T*>(p.residual) + at + c);
    }
  }
  float squares = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) squares = fmaf(s[i], s[i], squares);
  const float mean = fmaf(team_sums<TEAM>(squares, 0.0f, shared, 0).x, 1.0f / float(p.dim), p.eps);
  float2 k = make_float2(1.0f, inverse_sqrt(mean));
  if (!usual(mean))
    k = scaled_odd_row<TEAM>(static_cast<const T*>(p.x) + at, p.residual != nullptr ? static_cast<const T*>(p.residual) + at : nullptr,
                             p.dim, p.eps, shared);
  if (p.sum != nullptr) store_row<TEAM>(static_cast<T*>(p.sum) + at, p.dim, t, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    // (past dim 0, also where r is not finite)
    const float n = s[i] * k.x * k.y;
    s[i] = c >= p.dim ? 0.0f : p.weight != nullptr ? n * p.weight[c] : n;
  }
  if (p.out != nullptr) {
    if (p.out_bf16)
      store_row<TEAM>(static_cast<uint16_t*>(p.out) + at, p.dim, t, s);
    else
      store_row<TEAM>(static_cast<float*>(p.out) + at, p.dim, t, s);
  }
  if (p.out8.data != nullptr)
    store_row_mx8<TEAM, false>(static_cast<uint8_t*>(p.out8.data) + row * nb * 32, p.out8.scales + row * nb, nb * 32, t, s);
}

// dx of a row if it is out of range, from memory; its dy n is added to `part` (null: not
// wanted), of which a thread adds to its own columns.
template <int TEAM, typename T>
__device__ __noinline__ void scaled_odd_grad(const NormGradParams& p, int64_t row, float* part, float (&shared)[2][64], int parity) {
  const int t = int(threadIdx.x) % TEAM;
  const float inv_dim = 1.0f / float(p.dim);
  float s[8], dy[8], g[8], squares = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    const bool in = c < p.dim;
    s[i] = in ? kept_value<T>(p.x, row, p.dim, c) : 0.0f;
    dy[i] = in ? load1(static_cast<const T*>(p.dy) + row * p.dim + c) : 0.0f;
    g[i] = p.weight != nullptr && in ? p.weight[c] : 1.0f;
    squares = fmaf(s[i], s[i], squares);   // (in the kernel's order: the same bits)
    dot = fmaf(dy[i] * g[i], s[i], dot);
  }
  const float2 sums = team_sums<TEAM>(squares, dot, shared, parity);
  const float mean = fmaf(sums.x, inv_dim, p.eps);
  if (usual(mean, sums.y * inverse_sqrt(mean) * inv_dim)) return;
  scaled_grad_row<TEAM>(s, dy, g, inv_dim, p.eps, shared, parity);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    if (c >= p.dim) continue;
    if (part != nullptr) part[c] = fmaf(dy[i], s[i], part[c]);
    if (p.dres != nullptr) g[i] += load1(static_cast<const T*>(p.dres) + row * p.dim + c);
    store1(static_cast<T*>(p.dx) + row * p.dim + c, g[i]);
  }
}

template <int TEAM, typename T, bool MX8>
__global__ void __launch_bounds__(kBlock<TEAM>) norm_grad_odd_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM;
  const int t = int(threadIdx.x) % TEAM;
  const int team = int(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM, step = int(gridDim.x) * kTeams;
  const int rows = int(p.rows);   // (2^30 at most; 64-bit counters cost registers that rows are kept in)
  const int64_t nb = (p.dim + 31) / 32;
  float w[8], dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = column<TEAM, false>(i, t);
    w[i] = p.weight != nullptr && c < p.dim ? p.weight[c] : 1.0f;
    dw[i] = 0.0f;
  }
  const float inv_dim = 1.0f / float(p.dim);
  T next_dy[8], next_res[8];
  typename std::conditional<MX8, uint8_t, T>::type next_x[8];
  uint8_t next_scale[8];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = column<TEAM, false>(i, t), at = row * p.dim + c;
      const bool in = c < p.dim;
      next_dy[i] = in ? static_cast<const T*>(p.dy)[at] : T(0);
      if constexpr (MX8) {
        next_x[i] = in ? static_cast<const uint8_t*>(p.x.data)[row * nb * 32 + c] : uint8_t(0);
        next_scale[i] = in ? p.x.scales[row * nb + (c >> 5)] : uint8_t(0);
      } else {
        next_x[i] = in ? static_cast<const T*>(p.x.data)[at] : T(0);
      }
      next_res[i] = in && p.dres != nullptr ? static_cast<const T*>(p.dres)[at] : T(0);
    }
  };
  if (team < p.rows) fetch(team);
  bool again = false;   // there are rows out of range
  int parity = 0;
  for (int row = team; row < rows; row += step, parity ^= 1) {
    float s[8], dy[8], res[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dy[i] = load1(&next_dy[i]);
      res[i] = load1(&next_res[i]);
      if constexpr (MX8)
        s[i] = e4m3_value(next_x[i]) * mx8_up(next_scale[i]);
      else
        s[i] = load1(&next_x[i]);
    }
    if (row + step < rows) fetch(row + step);
    float squares = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      squares = fmaf(s[i], s[i], squares);
      dot = fmaf(dy[i] * w[i], s[i], dot);
    }
    const float2 sums = team_sums<TEAM>(squares, dot, shared, parity);
    const float mean = fmaf(sums.x, inv_dim, p.eps);
    float r = inverse_sqrt(mean), m = sums.y * r * inv_dim;
    if (!usual(mean, m)) r = m = 0.0f;   // (adds nothing to dw, and is not stored: dx may be dy)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = s[i] * r;
      dw[i] = fmaf(dy[i], n, dw[i]);
      dy[i] = r * fmaf(-n, m, dy[i] * w[i]) + res[i];
    }
    if (r != 0.0f) store_row<TEAM>(static_cast<T*>(p.dx) + int64_t(row) * p.dim, p.dim, t, dy);
    again = again || r == 0.0f;
  }
  float* part = p.part != nullptr ? p.part + int64_t(team) * p.dim : nullptr;
  if (part != nullptr) store_row<TEAM>(part, p.dim, t, dw);
  if (again)
    for (int64_t row = team; row < p.rows; row += step, parity ^= 1) scaled_odd_grad<TEAM, T>(p, row, part, shared, parity);
}

// Rows that do not fit a team's registers: a block reads them twice, the second
// time from L2 or nearer. 8192 x 12288 bf16 81 us (59 of bytes), with residual, sum and
// 8-bit result 114 (89), its gradient 168 (89), from 8-bit rows with dres and dw 242 (104):
// two passes with nothing loaded ahead, and dw through shared memory once a row.
constexpr int kLong = 512;

template <typename T>
__global__ void __launch_bounds__(kLong, 3) norm_long_kernel(const NormParams p) {
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t at = int64_t(blockIdx.x) * p.dim;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + at : nullptr;
  float squares = 0.0f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
    const float s = load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f);
    squares = fmaf(s, s, squares);
  }
  const float mean = fmaf(team_sums<kLong>(squares, 0.0f, shared, 0).x, 1.0f / float(p.dim), p.eps);
  float2 k = make_float2(1.0f, inverse_sqrt(mean));
  if (!usual(mean)) k = scaled_odd_row<kLong>(x, res, p.dim, p.eps, shared);
  const int64_t nb = (p.dim + 31) / 32;
  uint8_t* codes = p.out8.data != nullptr ? static_cast<uint8_t*>(p.out8.data) + int64_t(blockIdx.x) * nb * 32 : nullptr;
  for (int64_t c = threadIdx.x; c < nb * 32; c += kLong) {   // whole warps
    const bool in = c < p.dim;
    const float s = in ? load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f) : 0.0f;
    const float n = s * k.x * k.y, y = !in ? 0.0f : p.weight != nullptr ? n * p.weight[c] : n;
    if (in && p.sum != nullptr) store1(static_cast<T*>(p.sum) + at + c, s);
    if (in && p.out != nullptr) {
      if (p.out_bf16)
        store1(static_cast<uint16_t*>(p.out) + at + c, y);
      else
        store1(static_cast<float*>(p.out) + at + c, y);
    }
    if (codes != nullptr) {
      float top = fabsf(y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const uint32_t e = mx8_scale(top);
      codes[c] = uint8_t(cvt_e4m3x2(y * mx8_down(e), 0.0f));
      if ((c & 31) == 0) p.out8.scales[int64_t(blockIdx.x) * nb + (c >> 5)] = uint8_t(e);
    }
  }
}

// A row's gradient, element by element: n = s down r, dx = r (dy down_d w - n m) c0 c1;
// dy n is added to `from` (null: nothing to add to) and left in `to` (null: not wanted).
struct LongGrad {
  float down = 1.0f, r, down_d = 1.0f, m, c0 = 1.0f, c1 = 1.0f;
};
template <typename T, int UNROLL>
__device__ __forceinline__ void put_long_grad(const NormGradParams& p, int64_t row, const LongGrad& l, const float* from, float* to) {
  const int64_t at = row * p.dim;
#pragma unroll UNROLL
  for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {   // a column is one thread's: no order to keep
    const float n = kept_value<T>(p.x, row, p.dim, c) * l.down * l.r, d = load1(static_cast<const T*>(p.dy) + at + c);
    if (to != nullptr) to[c] = from == nullptr ? d * n : fmaf(d, n, from[c]);
    float v = l.r * fmaf(-n, l.m, d * l.down_d * (p.weight != nullptr ? p.weight[c] : 1.0f)) * l.c0 * l.c1;
    if (p.dres != nullptr) v += load1(static_cast<const T*>(p.dres) + at + c);
    store1(static_cast<T*>(p.dx) + at + c, v);
  }
}
template <typename T>
__device__ __noinline__ void scaled_long_grad(const NormGradParams& p, int64_t row, float (&shared)[2][64], int parity, const float* from,
                                              float* to) {
  const T* dy = static_cast<const T*>(p.dy) + row * p.dim;
  LongGrad l;
  float top_s = 0.0f, top_d = 0.0f, squares = 0.0f, dot = 0.0f;
#pragma unroll 1
  for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
    top_s = fmaxf(top_s, fabsf(kept_value<T>(p.x, row, p.dim, c)));
    top_d = fmaxf(top_d, fabsf(load1(dy + c)));
  }
  const float2 top = team_max<kLong>(top_s, top_d, shared, parity ^ 1);
  const int es = exponent_of(fmaxf(top.x, sqrtf(p.eps))), ed = exponent_of(top.y);
  l.down = power_of_two(-es);
  l.down_d = power_of_two(-ed);
#pragma unroll 1
  for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
    const float t = kept_value<T>(p.x, row, p.dim, c) * l.down;
    squares = fmaf(t, t, squares);
    dot = fmaf(load1(dy + c) * l.down_d * (p.weight != nullptr ? p.weight[c] : 1.0f), t, dot);
  }
  const float2 sums = team_sums<kLong>(squares, dot, shared, parity);
  const float inv_dim = 1.0f / float(p.dim);
  l.r = inverse_sqrt(fmaf(sums.x, inv_dim, p.eps * l.down * l.down));
  l.m = sums.y * l.r * inv_dim;
  l.c0 = power_of_two((ed - es) / 2);
  l.c1 = power_of_two(ed - es - (ed - es) / 2);
  put_long_grad<T, 1>(p, row, l, from, to);
}

template <typename T>
__global__ void __launch_bounds__(kLong) norm_grad_long_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  float* part = p.part != nullptr ? p.part + int64_t(blockIdx.x) * p.dim : nullptr;
  const float inv_dim = 1.0f / float(p.dim);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.dim;
    float squares = 0.0f, dot = 0.0f;
    for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
      const float s = kept_value<T>(p.x, row, p.dim, c);
      squares = fmaf(s, s, squares);
      dot = fmaf(load1(dy + c) * (p.weight != nullptr ? p.weight[c] : 1.0f), s, dot);
    }
    const float2 sums = team_sums<kLong>(squares, dot, shared, parity);
    const float mean = fmaf(sums.x, inv_dim, p.eps);
    const float* from = row == int64_t(blockIdx.x) ? nullptr : part;
    LongGrad l;
    l.r = inverse_sqrt(mean);
    l.m = sums.y * l.r * inv_dim;
    if (usual(mean, l.m))
      put_long_grad<T, 4>(p, row, l, from, part);
    else
      scaled_long_grad<T>(p, row, shared, parity, from, part);
    parity ^= 1;
  }
}

// The same where rows are 16-byte aligned: eight neighbours a thread.
constexpr int kLongStep = kLong * 8;

template <typename T>
__device__ __forceinline__ void sum8(const T* x, const T* res, float (&s)[8]) {
  load8(x, s);
  if (res != nullptr) {
    float r[8];
    load8(res, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += r[i];
  }
}

// The sum of squares in two ranges, without a branch: of s 2^-75 (finite for 2^22
// numbers below 2^128, and accurate for a mean square from 2^24 on) and of s 2^40 (for
// less than that: its sum stays below 2^126; and down to 2^-206, where any eps but 0 is
// all that counts). Code for rows out of range would take registers from the others:
// 8192 x 12288 bf16 75 us with neither, 81 with this, 97 to 130 with that. eps > 0;
// other calls go to the kernel above.
constexpr float kHigh = 0x1p-75f, kLow = 0x1p40f;
// (f, r): n = s f r, where f is 1 if r is a normal number by itself
__device__ __forceinline__ float2 two_ranges(float2 sums, float inv_dim, float eps) {
  const bool low = sums.y <= 0x1p126f && eps <= 0x1p40f;
  const float f = low ? kLow : kHigh, r = inverse_sqrt(fmaf(low ? sums.y : sums.x, inv_dim, eps * f * f));
  return f * r >= 0x1p-126f ? make_float2(1.0f, f * r) : make_float2(f, r);
}

// (Four blocks an SM: 32 registers a thread, so columns are counted in 32 bits.)
template <typename T>
__global__ void __launch_bounds__(kLong, 4) norm_long_vec_kernel(const NormParams p) {
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int dim = int(p.dim), padded = (dim + 31) / 32 * 32;
  const int64_t at = int64_t(blockIdx.x) * dim;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + at : nullptr;
  F2 high = ptx::f2(0.0f), low = ptx::f2(0.0f);
#pragma unroll 2
  for (int c = threadIdx.x * 8; c < dim; c += kLongStep) {
    float s[8];
    sum8(x + c, res != nullptr ? res + c : nullptr, s);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const F2 v = ptx::f2(s[i], s[i + 1]), h = ptx::mul2(v, ptx::f2(kHigh)), l = ptx::mul2(v, ptx::f2(kLow));
      high = ptx::fma2(h, h, high);
      low = ptx::fma2(l, l, low);
    }
  }
  const float2 h = ptx::parts(high), l = ptx::parts(low);
  const float2 k = two_ranges(team_sums<kLong>(h.x + h.y, l.x + l.y, shared, 0), 1.0f / float(p.dim), p.eps);
  for (int first = 0; first < padded; first += kLongStep) {   // (whole warps: a block of 32 is four lanes)
    const int c = first + threadIdx.x * 8;
    float y[8] = {};
    if (c < dim) {
      sum8(x + c, res != nullptr ? res + c : nullptr, y);
      if (p.sum != nullptr) store8(static_cast<T*>(p.sum) + at + c, y);
      float w[8];
      if (p.weight != nullptr) load8(p.weight + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = y[i] * k.x * k.y;
        y[i] = p.weight != nullptr ? n * w[i] : n;
      }
      if (p.out != nullptr) {
        if (p.out_bf16)
          store8(static_cast<uint16_t*>(p.out) + at + c, y);
        else
          store8(static_cast<float*>(p.out) + at + c, y);
      }
    }
    if (p.out8.data != nullptr) {
      const int64_t q = int64_t(blockIdx.x) * padded + first;
      store_row_mx8<kLong, true>(static_cast<uint8_t*>(p.out8.data) + q, p.out8.scales + (q >> 5), padded - first, int(threadIdx.x), y);
    }
  }
}

// SHARED: the block's part of dw is kept in shared memory until its last row
// (4096 x 16384 with 8-bit rows: 184 us from row to row in `part`).
constexpr int64_t kLongShared = 100 * 1024;

template <typename T, bool SHARED>
__global__ void __launch_bounds__(kLong) norm_grad_long_vec_kernel(const __grid_constant__ NormGradParams p) {
  extern __shared__ __align__(16) uint8_t slots[];
  __shared__ float shared[2][64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t nb = (p.dim + 31) / 32;
  float* part = p.part != nullptr ? p.part + int64_t(blockIdx.x) * p.dim : nullptr;
  float* sum = SHARED ? reinterpret_cast<float*>(slots) : part;
  const float inv_dim = 1.0f / float(p.dim);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.dim;
    const T* dy = static_cast<const T*>(p.dy) + at;
    // x, dy and g = dy w of eight columns
    auto fetch = [&](int64_t c, float (&s)[8], float (&d)[8], float (&g)[8]) {
      if (p.x.dtype == MO_MX8) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x.data) + row * nb * 32 + c);
        const float up = mx8_up(p.x.scales[row * nb + (c >> 5)]);
        e4m3x4_values(q.x, *reinterpret_cast<float (*)[4]>(&s[0]));
        e4m3x4_values(q.y, *reinterpret_cast<float (*)[4]>(&s[4]));
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] *= up;
      } else {
        load8(static_cast<const T*>(p.x.data) + at + c, s);
      }
      load8(dy + c, d);
      if (p.weight != nullptr) load8(p.weight + c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = p.weight != nullptr ? d[i] * g[i] : d[i];
    };
    float squares = 0.0f, dot = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < p.dim; c += kLongStep) {
      float s[8], d[8], g[8];
      fetch(c, s, d, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        squares = fmaf(s[i], s[i], squares);
        dot = fmaf(g[i], s[i], dot);
      }
    }
    const float2 sums = team_sums<kLong>(squares, dot, shared, parity);
    const float mean = fmaf(sums.x, inv_dim, p.eps), r = inverse_sqrt(mean), m = sums.y * r * inv_dim;
    if (!usual(mean, m)) {
      scaled_long_grad<T>(p, row, shared, parity, row != int64_t(blockIdx.x) ? sum : nullptr,
                          part == nullptr ? nullptr : SHARED && row + gridDim.x < p.rows ? sum : part);
      parity ^= 1;
      continue;
    }
    parity ^= 1;
    for (int64_t c = threadIdx.x * 8; c < p.dim; c += kLongStep) {   // a column is one thread's: no order to keep
      float s[8], d[8], g[8];
      fetch(c, s, d, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] *= r;
      if (part != nullptr) {
        float q[8] = {};
        if (row != int64_t(blockIdx.x)) load8(sum + c, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = fmaf(d[i], s[i], q[i]);
        store8(SHARED && row + gridDim.x < p.rows ? sum + c : part + c, q);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = r * fmaf(-s[i], m, g[i]);
      if (p.dres != nullptr) {
        load8(static_cast<const T*>(p.dres) + at + c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += g[i];
      }
      store8(static_cast<T*>(p.dx) + at + c, d);
    }
  }
}

// Threads of the team that takes rows of `dim` elements, eight a thread; 0: rows
// that no team holds.
int team_of(int64_t dim) { return dim <= 256 ? 32 : dim <= 1024 ? 128 : dim <= 2048 ? 256 : dim <= 4096 ? 512 : dim <= 8192 ? 1024 : 0; }

// Teams of the backward pass: 1024 threads an SM, on 152 SMs (a number that does
// not depend on the device, so that the sums' order does not either).
int64_t grad_teams(int64_t rows, int64_t dim) {
  const int team = team_of(dim);
  return std::min<int64_t>(rows, 152 * (team == 0 ? 2 : 1024 / team));
}

template <typename F>
cudaError_t with_team(int64_t dim, F&& f) {
  switch (team_of(dim)) {
    case 32: return f(Act<32>());
    case 128: return f(Act<128>());
    case 256: return f(Act<256>());
    case 512: return f(Act<512>());
    default: return f(Act<1024>());
  }
}

template <typename T>
cudaError_t norm_as(const NormParams& p, cudaStream_t stream) {
  if (team_of(p.dim) == 0)
    return launch_kernel(p.dim % 8 == 0 && p.eps > 0.0f ? norm_long_vec_kernel<T> : norm_long_kernel<T>, dim3(unsigned(p.rows)), dim3(kLong),
                         0, 1, true, stream, p);
  return with_team(p.dim, [&](auto team) {
    constexpr int TEAM = decltype(team)::value, kTeams = kBlock<TEAM> / TEAM;
    if (p.dim % 8 != 0)
      return launch_kernel(norm_odd_kernel<TEAM, T>, dim3(unsigned((p.rows + kTeams - 1) / kTeams)), dim3(kBlock<TEAM>), 0, 1, true,
                           stream, p);
    constexpr size_t smem = size_t(kNormAhead<T> + 1) * kNormSlot<T> * kBlock<TEAM>;
    auto kern = norm_kernel<TEAM, T>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(unsigned(norm_parts(p.rows, p.dim) / kTeams)), dim3(kBlock<TEAM>), smem, 1, true, stream, p);
  });
}

template <typename T, bool MX8>
cudaError_t norm_grad_as(const NormGradParams& p, cudaStream_t stream) {
  const int64_t teams = norm_parts(p.rows, p.dim);
  if (team_of(p.dim) == 0) {
    const bool keep = p.dim % 8 == 0 && p.part != nullptr && p.dim * 4 <= kLongShared;
    auto kern = keep ? norm_grad_long_vec_kernel<T, true> : p.dim % 8 == 0 ? norm_grad_long_vec_kernel<T, false> : norm_grad_long_kernel<T>;
    const cudaError_t e = keep ? allow_smem(reinterpret_cast<const void*>(kern), kLongShared) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(unsigned(teams)), dim3(kLong), keep ? size_t(p.dim) * 4 : 0, 1, true, stream, p);
  }
  return with_team(p.dim, [&](auto team) {
    constexpr int TEAM = decltype(team)::value, kTeams = kBlock<TEAM> / TEAM;
    const dim3 grid(unsigned(teams / kTeams));
    if (p.dim % 8 != 0)
      return launch_kernel(norm_grad_odd_kernel<TEAM, T, MX8>, grid, dim3(kBlock<TEAM>), 0, 1, true, stream, p);
    constexpr size_t smem = size_t(kGradAhead<T, MX8> + 1) * kGradSlot<T, MX8> * kBlock<TEAM>;
    auto kern = norm_grad_kernel<TEAM, T, MX8>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, dim3(kBlock<TEAM>), smem, 1, true, stream, p);
  });
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t dim) {
  const int64_t teams = grad_teams(rows, dim), per = team_of(dim) == 32 ? kBlock<32> / 32 : 1;
  return (teams + per - 1) / per * per;
}

cudaError_t launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? norm_as<uint16_t>(p, stream) : norm_as<float>(p, stream);
}

cudaError_t launch_rms_norm_grad(const NormGradParams& p, bool bf16, cudaStream_t stream) {
  if (p.x.dtype == MO_MX8) return bf16 ? norm_grad_as<uint16_t, true>(p, stream) : norm_grad_as<float, true>(p, stream);
  return bf16 ? norm_grad_as<uint16_t, false>(p, stream) : norm_grad_as<float, false>(p, stream);
}

}  // namespace mo
