// Root-mean-square norm of rows, after the addition of a residual, and its
// backward pass:
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   g = dy w:  dx = r (g - s r mean(g s r)) + dres,  dw = sum over rows of dy s r
//
// A team of threads takes a row, keeps it in registers and reads it once: the
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

template <int TEAM, int V, bool VEC>
__device__ __forceinline__ void load_row_mx8(const uint8_t* codes, const uint8_t* scales, int64_t dim, int t, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      const int64_t c = column<TEAM, VEC>(i, t);
      uint2 w = make_uint2(0u, 0u);
      float up = 0.0f;
      if (c < dim) {
        w = *reinterpret_cast<const uint2*>(codes + c);
        up = mx8_up(scales[c >> 5]);
      }
      float a[4], b[4];
      e4m3x4_values(w.x, a);
      e4m3x4_values(w.y, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + j] = a[j] * up;
        v[i + 4 + j] = b[j] * up;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = column<TEAM, VEC>(i, t);
      v[i] = c < dim ? e4m3_value(codes[c]) * mx8_up(scales[c >> 5]) : 0.0f;
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

template <int TEAM, int V, bool VEC, typename T>
__global__ void __launch_bounds__(kBlock<TEAM>) norm_grad_kernel(const NormGradParams p) {
  __shared__ float shared[64];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int kTeams = kBlock<TEAM> / TEAM;
  const int t = int(threadIdx.x) % TEAM;
  const int64_t team = int64_t(blockIdx.x) * kTeams + int(threadIdx.x) / TEAM;
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
  for (int64_t row = team; row < p.rows; row += int64_t(gridDim.x) * kTeams) {
    const int64_t at = row * p.dim;
    float s[V], dy[V];
    load_row<TEAM, V, VEC>(static_cast<const T*>(p.dy) + at, p.dim, t, dy);
    if (p.x.dtype == MO_MX8)
      load_row_mx8<TEAM, V, VEC>(static_cast<const uint8_t*>(p.x.data) + row * nb * 32, p.x.scales + row * nb, p.dim, t, s);
    else
      load_row<TEAM, V, VEC>(static_cast<const T*>(p.x.data) + at, p.dim, t, s);
    float squares = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      squares = fmaf(s[i], s[i], squares);
      dot = fmaf(dy[i] * w[i], s[i], dot);
    }
    team_sums<TEAM>(squares, dot, shared);
    const float r = inverse_rms(squares, p.dim, p.eps);
    const float m = dot * r / float(p.dim);   // mean(g s r)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float n = s[i] * r;
      dw[i] = fmaf(dy[i], n, dw[i]);
      dy[i] = r * fmaf(-n, m, dy[i] * w[i]);
    }
    if (p.dres != nullptr) {
      load_row<TEAM, V, VEC>(static_cast<const T*>(p.dres) + at, p.dim, t, s);
#pragma unroll
      for (int i = 0; i < V; ++i) dy[i] += s[i];
    }
    store_row<TEAM, V, VEC>(static_cast<T*>(p.dx) + at, p.dim, t, dy);
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

// The teams that take rows of `dim` elements.
struct Shape {
  int team, values;   // 0: rows that no team holds
};
Shape shape_of(int64_t dim) {
  if (dim <= 256) return {32, 8};
  if (dim <= 1024) return {128, 8};
  if (dim <= 2048) return {256, 8};
  if (dim <= 4096) return {256, 16};
  if (dim <= 8192) return {512, 16};
  return {0, 0};
}
// Teams of the backward pass: 16 of a warp an SM, or blocks as follows, on 152
// SMs (a number that does not depend on the device, as results must not).
int64_t grad_teams(int64_t rows, int64_t dim) {
  const int team = shape_of(dim).team;
  return std::min<int64_t>(rows, 152 * (team == 32 ? 16 : team == 128 ? 6 : team == 256 ? 2 : team == 512 ? 1 : 2));
}

template <typename F>
cudaError_t with_shape(int64_t dim, F&& f) {
  const bool vec = dim % 8 == 0;
  auto with = [&](auto team, auto values) {
    constexpr int TEAM = decltype(team)::value, V = decltype(values)::value;
    return vec ? f(Act<TEAM>(), Act<V>(), std::true_type()) : f(Act<TEAM>(), Act<V>(), std::false_type());
  };
  const Shape s = shape_of(dim);
  if (s.team == 32) return with(Act<32>(), Act<8>());
  if (s.team == 128) return with(Act<128>(), Act<8>());
  if (s.team == 512) return with(Act<512>(), Act<16>());
  return s.values == 8 ? with(Act<256>(), Act<8>()) : with(Act<256>(), Act<16>());
}

template <typename T>
cudaError_t norm_as(const NormParams& p, cudaStream_t stream) {
  if (shape_of(p.dim).team == 0)
    return launch_kernel(norm_long_kernel<T>, dim3(unsigned(p.rows)), dim3(kLong), 0, 1, true, stream, p);
  return with_shape(p.dim, [&](auto team, auto values, auto vec) {
    constexpr int TEAM = decltype(team)::value, V = decltype(values)::value;
    constexpr int kTeams = kBlock<TEAM> / TEAM;
    return launch_kernel(norm_kernel<TEAM, V, decltype(vec)::value, T>, dim3(unsigned((p.rows + kTeams - 1) / kTeams)),
                         dim3(kBlock<TEAM>), 0, 1, true, stream, p);
  });
}

template <typename T>
cudaError_t norm_grad_as(const NormGradParams& p, cudaStream_t stream) {
  const int64_t teams = norm_parts(p.rows, p.dim);
  if (shape_of(p.dim).team == 0)
    return launch_kernel(norm_grad_long_kernel<T>, dim3(unsigned(teams)), dim3(kLong), 0, 1, true, stream, p);
  return with_shape(p.dim, [&](auto team, auto values, auto vec) {
    constexpr int TEAM = decltype(team)::value, V = decltype(values)::value;
    constexpr int kTeams = kBlock<TEAM> / TEAM;
    return launch_kernel(norm_grad_kernel<TEAM, V, decltype(vec)::value, T>, dim3(unsigned(teams / kTeams)),
                         dim3(kBlock<TEAM>), 0, 1, true, stream, p);
  });
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t dim) {
  const int64_t teams = grad_teams(rows, dim), per = shape_of(dim).team == 32 ? kBlock<32> / 32 : 1;
  return (teams + per - 1) / per * per;
}

cudaError_t launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? norm_as<uint16_t>(p, stream) : norm_as<float>(p, stream);
}

cudaError_t launch_rms_norm_grad(const NormGradParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? norm_grad_as<uint16_t>(p, stream) : norm_grad_as<float>(p, stream);
}

}  // namespace mo
