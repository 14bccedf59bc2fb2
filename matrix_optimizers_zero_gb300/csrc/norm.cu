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

namespace mo {
namespace {

// A team of TEAM threads holds a row of at most TEAM V elements, V a thread:
// eight neighbours of every 8 TEAM where rows are 16-byte aligned (VEC), one of
// every TEAM otherwise. Either way 32 elements of a block lie in one warp.
template <int TEAM, bool VEC>
__device__ __forceinline__ int64_t column(int i, int t) {
  return VEC ? int64_t((i >> 3) * TEAM + t) * 8 + (i & 7) : int64_t(i) * TEAM + t;
}

template <int TEAM>
constexpr int kBlock = TEAM < 128 ? 128 : TEAM;

template <int TEAM, int V, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T* p, int64_t dim, int t, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      float (&w)[8] = *reinterpret_cast<float (*)[8]>(&v[i]);
      const int64_t c = column<TEAM, VEC>(i, t);
      if (c < dim) {
        load8(p + c, w);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = column<TEAM, VEC>(i, t);
      v[i] = c < dim ? load1(p + c) : 0.0f;
    }
  }
}

template <int TEAM, int V, bool VEC, typename T>
__device__ __forceinline__ void store_row(T* p, int64_t dim, int t, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += VEC ? 8 : 1) {
    const int64_t c = column<TEAM, VEC>(i, t);
    if (c >= dim) continue;
    if constexpr (VEC)
      store8(p + c, *reinterpret_cast<const float (*)[8]>(&v[i]));
    else
      store1(p + c, v[i]);
  }
}

// A row in 8 bits. All threads of a warp come here together; elements past dim
// are zeros, and the codes of the last block past it too.
template <int TEAM, int V, bool VEC>
__device__ __forceinline__ void store_row_mx8(uint8_t* codes, uint8_t* scales, int64_t end, int t, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += VEC ? 8 : 1) {
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

// Sums of a and b over a team; the order is fixed. `shared` holds 2 x 32
// floats. (A team of a warp needs no shared memory; teams of more are a whole
// block.)
template <int TEAM>
__device__ __forceinline__ void team_sums(float& a, float& b, float* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if constexpr (TEAM > 32) {
    const int lane = int(threadIdx.x & 31), warp = int(threadIdx.x >> 5);
    if (lane == 0) {
      shared[warp] = a;
      shared[32 + warp] = b;
    }
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int w = 0; w < TEAM / 32; ++w) {
      a += shared[w];
      b += shared[32 + w];
    }
    __syncthreads();
  }
}

__device__ __forceinline__ float inverse_rms(float squares, int64_t dim, float eps) { return 1.0f / sqrtf(squares / float(dim) + eps); }

template <int TEAM, int V, bool VEC, typename T>
__global__ void __launch_bounds__(kBlock<TEAM>) norm_kernel(const NormParams p) {
  __shared__ float shared[64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM;
  const int t = int(threadIdx.x) % TEAM;
  const int64_t row = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM;
  if (row >= p.rows) return;   // a whole warp, and a whole block where teams are more than one
  const int64_t at = row * p.dim;
  float s[V];
  load_row<TEAM, V, VEC>(static_cast<const T*>(p.x) + at, p.dim, t, s);
  if (p.residual != nullptr) {
    float r[V];
    load_row<TEAM, V, VEC>(static_cast<const T*>(p.residual) + at, p.dim, t, r);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += r[i];
  }
  if (p.sum != nullptr) store_row<TEAM, V, VEC>(static_cast<T*>(p.sum) + at, p.dim, t, s);
  float squares = 0.0f, none = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) squares = fmaf(s[i], s[i], squares);
  team_sums<TEAM>(squares, none, shared);
  const float r = inverse_rms(squares, p.dim, p.eps);
  float w[V];
  if (p.weight != nullptr) load_row<TEAM, V, VEC>(p.weight, p.dim, t, w);
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = p.weight != nullptr ? s[i] * r * w[i] : s[i] * r;
  if (p.out != nullptr) {
    if (p.out_bf16)
      store_row<TEAM, V, VEC>(static_cast<uint16_t*>(p.out) + at, p.dim, t, s);
    else
      store_row<TEAM, V, VEC>(static_cast<float*>(p.out) + at, p.dim, t, s);
  }
  if (p.out8.data != nullptr) {
    const int64_t nb = (p.dim + 31) / 32;
    // (elements past dim are not zeros where r is not finite)
    if (column<TEAM, VEC>(V - 1, TEAM - 1) >= p.dim) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (column<TEAM, VEC>(i, t) >= p.dim) s[i] = 0.0f;
    }
    store_row_mx8<TEAM, V, VEC>(static_cast<uint8_t*>(p.out8.data) + row * nb * 32, p.out8.scales + row * nb, nb * 32, t, s);
  }
}

// A row as it lies in memory, loaded while the one before it is worked on.
template <int V, bool VEC, typename T>
struct RawRow {
  using Word = typename std::conditional<VEC, uint4, T>::type;
  static constexpr int kWords = VEC ? V * int(sizeof(T)) / 16 : V;
  Word w[kWords];
};
template <int V, bool VEC>
struct RawRow8 {
  using Word = typename std::conditional<VEC, uint2, uint8_t>::type;
  Word w[VEC ? V / 8 : V];
  uint8_t scale[VEC ? V / 8 : V];
};

template <int TEAM, int V, bool VEC, typename T>
__device__ __forceinline__ void fetch_row(const T* p, int64_t dim, int t, RawRow<V, VEC, T>& raw) {
  if constexpr (VEC) {
    constexpr int kPer = 8 * int(sizeof(T)) / 16;   // words of eight elements
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      const int64_t c = column<TEAM, VEC>(i, t);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        raw.w[i / 8 * kPer + j] = c < dim ? reinterpret_cast<const uint4*>(p + c)[j] : make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = column<TEAM, VEC>(i, t);
      raw.w[i] = c < dim ? p[c] : T(0);
    }
  }
}
template <int TEAM, int V, bool VEC>
__device__ __forceinline__ void fetch_row(const uint8_t* codes, const uint8_t* scales, int64_t dim, int t, RawRow8<V, VEC>& raw) {
#pragma unroll
  for (int i = 0; i < V; i += VEC ? 8 : 1) {
    const int64_t c = column<TEAM, VEC>(i, t);
    const int at = VEC ? i / 8 : i;
    if constexpr (VEC)
      raw.w[at] = c < dim ? *reinterpret_cast<const uint2*>(codes + c) : make_uint2(0u, 0u);
    else
      raw.w[at] = c < dim ? codes[c] : uint8_t(0);
    raw.scale[at] = c < dim ? scales[c >> 5] : uint8_t(0);
  }
}

template <int V, bool VEC, typename T>
__device__ __forceinline__ void row_values(const RawRow<V, VEC, T>& raw, float (&v)[V]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = load1(&raw.w[i]);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      const uint32_t u[4] = {raw.w[i].x, raw.w[i].y, raw.w[i].z, raw.w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      v[4 * i] = __uint_as_float(raw.w[i].x);
      v[4 * i + 1] = __uint_as_float(raw.w[i].y);
      v[4 * i + 2] = __uint_as_float(raw.w[i].z);
      v[4 * i + 3] = __uint_as_float(raw.w[i].w);
    }
  }
}
template <int V, bool VEC>
__device__ __forceinline__ void row_values(const RawRow8<V, VEC>& raw, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      const float up = mx8_up(raw.scale[i]);
      float a[4], b[4];
      e4m3x4_values(raw.w[i].x, a);
      e4m3x4_values(raw.w[i].y, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + j] = a[j] * up;
        v[8 * i + 4 + j] = b[j] * up;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e4m3_value(raw.w[i]) * mx8_up(raw.scale[i]);
  }
}

// The values are taken from the raw words again where they are used next, rather
// than kept: the compiler may not take this row's words for those it has
// converted already.
template <typename Raw>
__device__ __forceinline__ void forget(Raw& raw) {
  uint32_t* w = reinterpret_cast<uint32_t*>(raw.w);
  if constexpr (sizeof(raw.w) % 4 == 0 && sizeof(raw.w[0]) >= 8) {
#pragma unroll
    for (int i = 0; i < int(sizeof(raw.w) / 4); ++i) asm volatile("" : "+r"(w[i]));
  }
}

// Blocks an SM, and so registers a thread: 1024 threads an SM where a row is 16
// bytes a thread.
template <int TEAM, bool VEC, typename T>
constexpr int kGradBlocks = TEAM < 256 ? 4 : VEC && sizeof(T) == 2 ? 1024 / TEAM : TEAM > 512 ? 1 : 512 / TEAM;

// The backward pass. A team has the next row's loads under way while it works on
// one, and one barrier a row: the warps' sums go to one half of `shared` and the
// next row's to the other.
template <int TEAM, int V, bool VEC, typename T, bool MX8>
__global__ void __launch_bounds__(kBlock<TEAM>, kGradBlocks<TEAM, VEC, T>) norm_grad_kernel(const NormGradParams p) {
  __shared__ float2 shared[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM;
  const int t = int(threadIdx.x) % TEAM, lane = int(threadIdx.x & 31);
  const int64_t team = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM, step = int64_t(gridDim.x) * kTeams;
  const int64_t nb = (p.dim + 31) / 32;
  float w[V], dw[V];
  if (p.weight != nullptr) {
    load_row<TEAM, V, VEC>(p.weight, p.dim, t, w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.0f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.0f;
  struct Rows {
    RawRow<V, VEC, T> dy, res;
    typename std::conditional<MX8, RawRow8<V, VEC>, RawRow<V, VEC, T>>::type x;
  };
  Rows next;
  auto fetch = [&](int64_t row) {
    const int64_t at = row * p.dim;
    fetch_row<TEAM, V, VEC>(static_cast<const T*>(p.dy) + at, p.dim, t, next.dy);
    if constexpr (MX8)
      fetch_row<TEAM, V, VEC>(static_cast<const uint8_t*>(p.x.data) + row * nb * 32, p.x.scales + row * nb, p.dim, t, next.x);
    else
      fetch_row<TEAM, V, VEC>(static_cast<const T*>(p.x.data) + at, p.dim, t, next.x);
    if (p.dres != nullptr) fetch_row<TEAM, V, VEC>(static_cast<const T*>(p.dres) + at, p.dim, t, next.res);
  };
  if (team < p.rows) fetch(team);
  int parity = 0;
  for (int64_t row = team; row < p.rows; row += step, parity ^= 1) {
    Rows cur = next;
    if (row + step < p.rows) fetch(row + step);
    float squares = 0.0f, dot = 0.0f;
    {
      float s[V], dy[V];
      row_values(cur.dy, dy);
      row_values(cur.x, s);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        squares = fmaf(s[i], s[i], squares);
        dot = fmaf(dy[i] * w[i], s[i], dot);
      }
    }
    forget(cur.dy);
    forget(cur.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      squares += __shfl_xor_sync(0xFFFFFFFFu, squares, o);
      dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    }
    if constexpr (TEAM > 32) {
      if (lane == 0) shared[parity][threadIdx.x >> 5] = make_float2(squares, dot);
      __syncthreads();
      const float2 v = shared[parity][lane % (TEAM / 32)];
      squares = v.x;
      dot = v.y;
#pragma unroll
      for (int o = TEAM / 64; o > 0; o >>= 1) {
        squares += __shfl_xor_sync(0xFFFFFFFFu, squares, o);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      }
    }
    const float r = inverse_rms(squares, p.dim, p.eps);
    const float m = dot * r / float(p.dim);   // mean(g s r)
    float s[V], dy[V];
    row_values(cur.dy, dy);
    row_values(cur.x, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float n = s[i] * r;
      dw[i] = fmaf(dy[i], n, dw[i]);
      dy[i] = r * fmaf(-n, m, dy[i] * w[i]);
    }
    if (p.dres != nullptr) {
      row_values(cur.res, s);
#pragma unroll
      for (int i = 0; i < V; ++i) dy[i] += s[i];
    }
    store_row<TEAM, V, VEC>(static_cast<T*>(p.dx) + row * p.dim, p.dim, t, dy);
  }
  if (p.part != nullptr) store_row<TEAM, V, VEC>(p.part + team * p.dim, p.dim, t, dw);
}

// Rows that do not fit a team's registers: a block reads them twice, the second
// time from L2.
constexpr int kLong = 512;

template <typename T>
__global__ void __launch_bounds__(kLong) norm_long_kernel(const NormParams p) {
  __shared__ float shared[64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t at = int64_t(blockIdx.x) * p.dim;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* res = p.residual != nullptr ? static_cast<const T*>(p.residual) + at : nullptr;
  float squares = 0.0f, none = 0.0f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
    const float s = load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f);
    squares = fmaf(s, s, squares);
  }
  team_sums<kLong>(squares, none, shared);
  const float r = inverse_rms(squares, p.dim, p.eps);
  const int64_t nb = (p.dim + 31) / 32;
  uint8_t* codes = p.out8.data != nullptr ? static_cast<uint8_t*>(p.out8.data) + int64_t(blockIdx.x) * nb * 32 : nullptr;
  for (int64_t c = threadIdx.x; c < nb * 32; c += kLong) {   // whole warps
    const bool in = c < p.dim;
    const float s = in ? load1(x + c) + (res != nullptr ? load1(res + c) : 0.0f) : 0.0f;
    const float y = !in ? 0.0f : p.weight != nullptr ? s * r * p.weight[c] : s * r;
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
      const uint32_t k = mx8_scale(top);
      codes[c] = uint8_t(cvt_e4m3x2(y * mx8_down(k), 0.0f));
      if ((c & 31) == 0) p.out8.scales[int64_t(blockIdx.x) * nb + (c >> 5)] = uint8_t(k);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLong) norm_grad_long_kernel(const NormGradParams p) {
  __shared__ float shared[64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t nb = (p.dim + 31) / 32;
  float* part = p.part != nullptr ? p.part + int64_t(blockIdx.x) * p.dim : nullptr;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at = row * p.dim;
    auto x_at = [&](int64_t c) {
      if (p.x.dtype == MO_MX8)
        return e4m3_value(static_cast<const uint8_t*>(p.x.data)[row * nb * 32 + c]) * mx8_up(p.x.scales[row * nb + (c >> 5)]);
      return load1(static_cast<const T*>(p.x.data) + at + c);
    };
    auto w_at = [&](int64_t c) { return p.weight != nullptr ? p.weight[c] : 1.0f; };
    const T* dy = static_cast<const T*>(p.dy) + at;
    float squares = 0.0f, dot = 0.0f;
    for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {
      const float s = x_at(c);
      squares = fmaf(s, s, squares);
      dot = fmaf(load1(dy + c) * w_at(c), s, dot);
    }
    team_sums<kLong>(squares, dot, shared);
    const float r = inverse_rms(squares, p.dim, p.eps);
    const float m = dot * r / float(p.dim);
    for (int64_t c = threadIdx.x; c < p.dim; c += kLong) {   // a column is one thread's: no order to keep
      const float n = x_at(c) * r, d = load1(dy + c);
      if (part != nullptr) part[c] = row == int64_t(blockIdx.x) ? d * n : fmaf(d, n, part[c]);
      float v = r * fmaf(-n, m, d * w_at(c));
      if (p.dres != nullptr) v += load1(static_cast<const T*>(p.dres) + at + c);
      store1(static_cast<T*>(p.dx) + at + c, v);
    }
  }
}

// Threads of the team that takes rows of `dim` elements, eight a thread; 0: rows
// that no team holds.
int team_of(int64_t dim) { return dim <= 256 ? 32 : dim <= 1024 ? 128 : dim <= 2048 ? 256 : dim <= 4096 ? 512 : dim <= 8192 ? 1024 : 0; }

// Teams of the backward pass: 1024 threads an SM, on 152 SMs (a number that does
// not depend on the device, as results must not).
int64_t grad_teams(int64_t rows, int64_t dim) {
  const int team = team_of(dim);
  return std::min<int64_t>(rows, 152 * (team == 0 ? 2 : 1024 / team));
}

template <typename F>
cudaError_t with_team(int64_t dim, F&& f) {
  const bool vec = dim % 8 == 0;
  auto with = [&](auto team) { return vec ? f(team, std::true_type()) : f(team, std::false_type()); };
  switch (team_of(dim)) {
    case 32: return with(Act<32>());
    case 128: return with(Act<128>());
    case 256: return with(Act<256>());
    case 512: return with(Act<512>());
    default: return with(Act<1024>());
  }
}

template <typename T>
cudaError_t norm_as(const NormParams& p, cudaStream_t stream) {
  if (team_of(p.dim) == 0)
    return launch_kernel(norm_long_kernel<T>, dim3(unsigned(p.rows)), dim3(kLong), 0, 1, true, stream, p);
  return with_team(p.dim, [&](auto team, auto vec) {
    constexpr int TEAM = decltype(team)::value, kTeams = kBlock<TEAM> / TEAM;
    return launch_kernel(norm_kernel<TEAM, 8, decltype(vec)::value, T>, dim3(unsigned((p.rows + kTeams - 1) / kTeams)),
                         dim3(kBlock<TEAM>), 0, 1, true, stream, p);
  });
}

template <typename T>
cudaError_t norm_grad_as(const NormGradParams& p, cudaStream_t stream) {
  const int64_t teams = norm_parts(p.rows, p.dim);
  if (team_of(p.dim) == 0)
    return launch_kernel(norm_grad_long_kernel<T>, dim3(unsigned(teams)), dim3(kLong), 0, 1, true, stream, p);
  return with_team(p.dim, [&](auto team, auto vec) {
    constexpr int TEAM = decltype(team)::value, kTeams = kBlock<TEAM> / TEAM;
    constexpr bool VEC = decltype(vec)::value;
    auto kern = p.x.dtype == MO_MX8 ? norm_grad_kernel<TEAM, 8, VEC, T, true> : norm_grad_kernel<TEAM, 8, VEC, T, false>;
    return launch_kernel(kern, dim3(unsigned(teams / kTeams)), dim3(kBlock<TEAM>), 0, 1, true, stream, p);
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
  return bf16 ? norm_grad_as<uint16_t>(p, stream) : norm_grad_as<float>(p, stream);
}

}  // namespace mo
