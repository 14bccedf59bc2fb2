// Microscaled 4-bit quantisation: e2m1 codes with a scale for each block of
// consecutive elements (mx: 32 elements, e8m0; nv: 16 elements, e4m3, times a
// power of two g for the whole tensor).
//
// A block's scale is the smallest of its type, s, with which no element
// exceeds the largest code: max |x| <= 6 s g. Nothing saturates, so stochastic
// rounding stays unbiased. Both roundings are exact functions of the input:
// with mx (and g) a power of two the quotient x / (s g) is exact, with nv it
// is rounded once (see `quotient`).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "launch.cuh"
#include "philox.cuh"
#include "ptx_train.cuh"
#include "train_kernels.h"

namespace mo {
namespace {

// A 64 x 64 tile of x goes through shared memory, from which both
// orientations are quantised: x is read once for the operands of a forward and
// a backward product. (128 x 128 tiles, 256 threads: a tenth slower, as their
// last ones leave SMs idle.) 14336 x 4096 fp32 to mx, both orientations: 51 us for
// 297 MB, 5.8 TB/s. Others are bound by arithmetic, 8192 x 5120 bf16: mx 32 us,
// nv 41 us (quotients and a scale search for every 16 elements), stochastic 62
// and 81 us (the random numbers: 20 wide products for 8 elements). Row pitch in elements: 16 bytes more than the row, so
// that 32 threads reading 16 bytes of 32 rows meet all banks.
constexpr int kTile = kQuantTile;
constexpr int kThreads = 128;
template <typename T>
constexpr int kPitch = kTile + 16 / int(sizeof(T));

// max(|a|, |b|, |c|), NaN if any is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Value of e4m3 bits (0 - 126).
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(c)));
  return __half2float(__ushort_as_half(uint16_t(h)));
}

// The tensor's own scale of nv: the smallest power of two g with
// amax <= 6 * 448 g = 1.3125 * 2^11 g, from 2^-126; 1 for zeros (and for an
// amax that is not finite). Returns its exponent.
__device__ __forceinline__ int tensor_exponent(const float* amax) {
  if (amax == nullptr) return 0;
  const uint32_t b = abs_bits(*amax);
  if (b == 0u || b >= 0x7F800000u) return 0;
  int e = int(b >> 23) - 127 - 11 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) {   // -149 <= e <= 127
  return e >= -126 ? __uint_as_float(uint32_t(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// x / s for x = v[i] in fp32, correctly rounded: y = RN(1 / s), q = RN(x y), one
// correction with the exact remainder (Markstein, 1990). A plain product with
// the reciprocal would put exact ties on the wrong side.
__device__ __forceinline__ float quotient(float x, float s, float y) {
  const float q = x * y;
  return fmaf(fmaf(-q, s, x), y, q);
}

// Byte 3 of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Eight codes rounded up with the probability of the remainder in steps of
// 2^-16, |y| <= 6, signs from `sign`. In units of 2^-126 the numbers below 1 are
// subnormal, and the float's bits are the position on the grid (0, 0.5, 1,
// 1.5, 2, 3, 4, 6) in units of 2^22: the exponent's two low bits and the first
// mantissa bit are the code, linear in between. So the 16-bit number is added
// right below the code and the sum cut off: floor(position 2^16) + u, exactly.
__device__ __forceinline__ uint32_t stochastic_e2m1x8(const float (&y)[8], const float (&sign)[8], const uint4& g) {
  uint32_t t[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? (i < 2 ? g.x : g.y) : (i < 6 ? g.z : g.w);
    const uint32_t u = __byte_perm(w, 0u, (i & 1) ? 0x4324 : 0x4104);   // u 2^8
    t[i] = __float_as_uint(__fmul_rz(fabsf(y[i]), __uint_as_float(1u << 23))) * 4u + u;   // the code in byte 3
    s[i] = __float_as_uint(sign[i]);
  }
  return top_bytes(t[0], t[2], t[4], t[6]) + top_bytes(t[1], t[3], t[5], t[7]) * 16u +
         (((top_bytes(s[0], s[2], s[4], s[6]) >> 4) & 0x08080808u) | (top_bytes(s[1], s[3], s[5], s[7]) & 0x80808080u));
}

// Quantises 32 consecutive elements (one block of mx, two of nv): codes in four
// words, scale bits in the returned value (one byte a block). i0: index of the
// first element for the random numbers, a multiple of 32.
template <bool MX, bool STOCH>
__device__ __forceinline__ uint32_t quantize32(float (&v)[32], int gexp, const Philox& rng, uint64_t i0,
                                               uint32_t (&codes)[4]) {
  uint32_t bits = 0;
  constexpr int kBlock = MX ? 32 : 16;
#pragma unroll
  for (int b = 0; b < 32 / kBlock; ++b) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kBlock; i += 2) most = max_abs(most, v[b * kBlock + i], v[b * kBlock + i + 1]);
    const uint32_t top = __float_as_uint(most);
    float down, s = 1.0f, inv = 1.0f;
    uint32_t sc;
    if (MX) {
      // 6 = 1.5 * 2^2: the exponent of the maximum less two, one more where its mantissa exceeds 1.5
      const int e = int(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
      sc = top >= 0x7F800000u ? 0xFFu : uint32_t(max(e, 0));
      down = __uint_as_float((254u - min(sc, 253u)) << 23);
    } else {
      down = pow2(-gexp);
      const float a = __uint_as_float(top) * down;
      if (top >= 0x7F800000u) {
        sc = 0x7Fu;
      } else {
        // the e4m3 nearest to a / 6, and the next one where it is too small (448 s: saturated)
        uint16_t c16;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c16) : "f"(0.0f), "f"(a * (1.0f / 6.0f)));
        sc = c16;
        if (6.0f * e4m3_value(sc) < a && sc < 126u) ++sc;
        if (sc == 0u && top != 0u) sc = 1u;   // a underflowed
      }
      // x / (s g): with a tiny g the elements are scaled up first, so that no divisor is subnormal
      s = e4m3_value(min(sc, 126u));
      if (gexp < -100) {
#pragma unroll
        for (int i = 0; i < kBlock; ++i) v[b * kBlock + i] *= down;
      } else {
        s *= pow2(gexp);
      }
      inv = sc != 0u ? 1.0f / s : 0.0f;
    }
    bits |= sc << (8 * b);
    if (top >= 0x7F800000u) {   // the scale says NaN; codes 0
#pragma unroll
      for (int i = 0; i < kBlock; ++i) v[b * kBlock + i] = 0.0f;
    } else if (!MX && __uint_as_float(top) * down > 2688.0f) {
      // only a caller's too small amax lets elements exceed 6 s g: they saturate, however far they are
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        v[b * kBlock + i] = copysignf(fminf(fabsf(v[b * kBlock + i]), 6.0f * s), v[b * kBlock + i]);
    }
#pragma unroll
    for (int w = 0; w < kBlock / 8; ++w) {
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = y[i] = v[b * kBlock + 8 * w + i];
        y[i] = MX ? y[i] * down : quotient(y[i], s, inv);
      }
      const int k = b * (kBlock / 8) + w;
      codes[k] = STOCH ? stochastic_e2m1x8(y, x, rng.group(uint32_t(i0 >> 35), uint32_t(i0 >> 3) + uint32_t(k))) : ptx::cvt_e2m1x8(y);
    }
  }
  return bits;
}

__device__ __forceinline__ float as_float(uint16_t x) { return bf16_bits_to_float(x); }
__device__ __forceinline__ float as_float(float x) { return x; }

// Writes the codes (16 bytes) and the scale (mx) or scales (nv) of 32 elements of row `row` from
// element k0, a multiple of 32, on.
template <bool MX>
__device__ __forceinline__ void put32(const Fp4Out& q, int64_t row, int64_t k0, const uint32_t (&c)[4], uint32_t bits) {
  if (row < q.rows && k0 < q.k)
    *reinterpret_cast<uint4*>(q.codes + row * q.pitch + (k0 >> 1)) = make_uint4(c[0], c[1], c[2], c[3]);
  // rows and blocks outside the tensor have zeros in its last tiles (values and scale 0)
  const int64_t blk = MX ? k0 >> 5 : k0 >> 4;
  if ((blk >> 2) < q.tiles_k && (row >> 7) < q.tiles_r) {
    uint8_t* o = q.scales + ((row >> 7) * q.tiles_k + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
    if (MX)
      *o = uint8_t(bits);
    else
      *reinterpret_cast<uint16_t*>(o) = uint16_t(bits);
  }
}

template <typename T, bool MX, bool STOCH>
__global__ void __launch_bounds__(kThreads, 8) fp4_quantize_kernel(const QuantParams p) {
  extern __shared__ __align__(16) uint8_t tile_smem[];
  T* tile = reinterpret_cast<T*>(tile_smem);
  constexpr int P = kPitch<T>;
  constexpr int E = 16 / int(sizeof(T));        // elements of a 16-byte access
  constexpr int kVecs = kTile / E;              // accesses a row
  const int tid = int(threadIdx.x);
  const int64_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x - tr * p.tiles_c;
  const int64_t r0 = tr * kTile, c0 = tc * kTile;
  const T* x = static_cast<const T*>(p.x);
  ptx::griddep_launch_dependents();
  // after the launch that measured amax, which waited for whatever wrote x, x can be loaded at once
  if (!p.measured) ptx::griddep_wait();
  const bool full = r0 + kTile <= p.rows && c0 + kTile <= p.cols && p.vec;
  if (full) {
#pragma unroll 8
    for (int i = tid; i < kTile * kVecs; i += kThreads) {
      const int r = i / kVecs, c = (i - r * kVecs) * E;
      ptx::cp_async16(ptx::smem_addr(tile + r * P + c), x + (r0 + r) * p.cols + c0 + c);
    }
    ptx::cp_async_wait();
  } else {
    for (int i = tid; i < kTile * kTile; i += kThreads) {
      const int r = i / kTile, c = i - r * kTile;
      tile[r * P + c] = r0 + r < p.rows && c0 + c < p.cols ? x[(r0 + r) * p.cols + c0 + c] : T(0);
    }
  }
  if (p.measured) ptx::griddep_wait();
  const int gexp = MX ? 0 : tensor_exponent(p.amax);
  if (!MX && blockIdx.x == 0 && tid == 0) {
    if (p.row.amax != nullptr) *p.row.amax = *p.amax;
    if (p.col.amax != nullptr) *p.col.amax = *p.amax;
  }
  __syncthreads();
  const int line = tid & (kTile - 1), at = tid / kTile * 32;   // a row (a column) of the tile, 32 elements of it
  // One copy of the code serves both orientations: twice as long, with stochastic rounding, it no
  // longer fits the instruction cache.
  const int begin = p.row.codes != nullptr ? 0 : 1, end = p.col.codes != nullptr ? 2 : 1;
#pragma unroll 1
  for (int it = begin; it < end; ++it) {
    const bool by_row = it == 0;
    const Fp4Out& q = by_row ? p.row : p.col;
    float v[32];
    if (by_row) {
      const T* src = tile + line * P + at;
#pragma unroll
      for (int i = 0; i < 32 / E; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + i * E);
        const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int j = 0; j < E; ++j) v[i * E + j] = as_float(t[j]);
      }
    } else {
      const T* src = tile + at * P + line;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = as_float(src[i * P]);
    }
    const int64_t row = (by_row ? r0 : c0) + line, k0 = (by_row ? c0 : r0) + at;
    const Philox rng(p.rnd, by_row ? 0 : 1);   // the transposed tensor draws from the next offset
    uint32_t codes[4];
    const uint32_t bits = quantize32<MX, STOCH>(v, gexp, rng, uint64_t(row) * uint64_t(2 * q.pitch) + uint64_t(k0), codes);
    put32<MX>(q, row, k0, codes, bits);
  }
}

// Largest finite magnitude of x: an unsigned maximum of the bit patterns, so
// the order of the atomics does not matter. *amax is 0 on entry. A thread that
// meets a NaN or an infinity looks at its elements once more without them.
// 8192 x 5120 bf16: 16 us, 5.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(256, 8) fp4_amax_kernel(const T* x, int64_t n, uint32_t* amax) {
  constexpr int E = 16 / int(sizeof(T));
  constexpr int U = 4;
  ptx::griddep_launch_dependents();
  const int64_t full = n / E, stride = int64_t(gridDim.x) * blockDim.x;
  const int64_t i0 = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  float most = 0.0f;
  for (int64_t i = i0; i < full; i += U * stride) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i + u * stride < full) w[u] = __ldg(reinterpret_cast<const uint4*>(x) + i + u * stride);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      if constexpr (E == 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max_abs(most, __uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xFFFF0000u));
      } else {
        most = max_abs(most, __uint_as_float(q[0]), __uint_as_float(q[1]));
        most = max_abs(most, __uint_as_float(q[2]), __uint_as_float(q[3]));
      }
    }
  }
  if (i0 < n - full * E) most = max_abs(most, as_float(x[full * E + i0]), 0.0f);
  uint32_t top = __float_as_uint(most);
  if (top >= 0x7F800000u) {
    top = 0;
    auto take = [&](T v) {
      const uint32_t b = abs_bits(as_float(v));
      top = max(top, b < 0x7F800000u ? b : 0u);
    };
    for (int64_t i = i0; i < full; i += stride)
      for (int j = 0; j < E; ++j) take(x[i * E + j]);
    if (i0 < n - full * E) take(x[full * E + i0]);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  __shared__ uint32_t warp_top[8];
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) top = max(top, warp_top[i]);
    atomicMax(amax, top);
  }
}

// Values of a quantised tensor: a thread takes kDequantU groups of 16
// consecutive elements of a row (8 bytes of codes, one scale), 32 groups
// apart; 32 lanes by 8 rows a block, blocks down the rows first. Bound by
// memory: 14336 x 4096 to bf16 22 us for 148 MB, 6.7 TB/s.
constexpr int kDequantU = 2;

template <typename O, bool MX>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const Fp4In q, O* out, int vec) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int row = int(blockIdx.x) * 8 + int(threadIdx.y);
  if (row >= q.rows) return;
  const int k = int(q.k), g0 = int(blockIdx.y) * (32 * kDequantU) + int(threadIdx.x);
  const uint8_t* codes = q.codes + int64_t(row) * q.pitch;
  const uint8_t* scales = q.scales + int64_t(row >> 7) * q.tiles_k * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  O* o_row = out + int64_t(row) * k;
  const float g = MX ? 1.0f : pow2(tensor_exponent(q.amax));
  __shared__ O turns[8][32 * (sizeof(O) == 2 ? 18 : 17)];
  uint2 w[kDequantU] = {};
  uint32_t sc[kDequantU] = {};
#pragma unroll
  for (int u = 0; u < kDequantU; ++u) {
    const int at = g0 + 32 * u;
    if (16 * at < k) {
      w[u] = *reinterpret_cast<const uint2*>(codes + 8 * at);
      const int blk = MX ? at >> 1 : at;
      sc[u] = scales[(blk >> 2) * 512 + (blk & 3)];
    }
  }
#pragma unroll
  for (int u = 0; u < kDequantU; ++u) {
    const int k0 = 16 * (g0 + 32 * u);
    if (16 * (int(blockIdx.y) * (32 * kDequantU) + 32 * u) >= k) break;   // the whole warp
    if (vec && k0 >= k) break;
    const float s = sc[u] == (MX ? 0xFFu : 0x7Fu) ? __uint_as_float(0x7FC00000u) : MX ? pow2(int(sc[u]) - 127) : e4m3_value(sc[u]) * g;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t c = (j < 8 ? w[u].x : w[u].y) >> (4 * (j & 7));
      // the three magnitude bits are a tiny float: exponent field and first mantissa bit
      const float m = __uint_as_float((c & 7u) << 22) * __uint_as_float(253u << 23);   // 2^126
      v[j] = s * __uint_as_float(__float_as_uint(m) | (c & 8u) << 28);
    }
    O* o = o_row + k0;
    if (vec) {   // k is a multiple of 16 and the rows are 32-byte aligned
      if constexpr (sizeof(O) == 2) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        ptx::st_global_v8(o, r);
      } else {
        uint32_t r[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[8 * h + j]);
          ptx::st_global_v8(o + 8 * h, r);
        }
      }
    } else {   // rows that start anywhere: the warp's 512 elements in order, a whole warp a store
      O* turn = turns[threadIdx.y];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if constexpr (sizeof(O) == 2)
          turn[threadIdx.x * 18 + j] = float_to_bf16_bits(v[j]);
        else
          turn[threadIdx.x * 17 + j] = v[j];
      }
      __syncwarp();
      const int first = 16 * (g0 - int(threadIdx.x) + 32 * u), count = min(512, k - first);
      for (int j = int(threadIdx.x); j < count; j += 32) o_row[first + j] = turn[(j >> 4) * (sizeof(O) == 2 ? 18 : 17) + (j & 15)];
    }
  }
}

template <typename T, bool MX, bool STOCH>
cudaError_t quantize_as(const QuantParams& p, cudaStream_t stream) {
  constexpr size_t smem = size_t(kTile) * kPitch<T> * sizeof(T);
  auto kern = fp4_quantize_kernel<T, MX, STOCH>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (p.rows + 127) / 128 * (128 / kTile) * p.tiles_c;   // whole scale tiles
  return launch_kernel(kern, dim3(unsigned(tiles)), dim3(kThreads), smem, 1, true, stream, p);
}

}  // namespace

cudaError_t launch_fp4_quantize(const QuantParams& p, bool bf16, bool mx, bool stochastic, cudaStream_t stream) {
  if (bf16) {
    if (mx) return stochastic ? quantize_as<uint16_t, true, true>(p, stream) : quantize_as<uint16_t, true, false>(p, stream);
    return stochastic ? quantize_as<uint16_t, false, true>(p, stream) : quantize_as<uint16_t, false, false>(p, stream);
  }
  if (mx) return stochastic ? quantize_as<float, true, true>(p, stream) : quantize_as<float, true, false>(p, stream);
  return stochastic ? quantize_as<float, false, true>(p, stream) : quantize_as<float, false, false>(p, stream);
}

cudaError_t launch_fp4_amax(const void* x, bool bf16, int64_t n, float* amax, int sms, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(amax, 0, sizeof(float), stream);
  if (e != cudaSuccess) return e;
  const int64_t want = (n / (bf16 ? 8 : 4) + 1023) / 1024;
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(want, int64_t(sms) * 8)));
  if (bf16)
    fp4_amax_kernel<uint16_t><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x), n, reinterpret_cast<uint32_t*>(amax));
  else
    fp4_amax_kernel<float><<<grid, 256, 0, stream>>>(static_cast<const float*>(x), n, reinterpret_cast<uint32_t*>(amax));
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(const Fp4In& q, bool mx, void* out, bool out_bf16, cudaStream_t stream) {
  const dim3 grid(unsigned((q.rows + 7) / 8), unsigned((q.k + 16 * 32 * kDequantU - 1) / (16 * 32 * kDequantU)));
  const dim3 block(32, 8);
  const int vec = q.k % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  if (out_bf16) {
    uint16_t* o = static_cast<uint16_t*>(out);
    return launch_kernel(mx ? fp4_dequantize_kernel<uint16_t, true> : fp4_dequantize_kernel<uint16_t, false>, grid, block, 0, 1,
                         true, stream, q, o, vec);
  }
  float* o = static_cast<float*>(out);
  return launch_kernel(mx ? fp4_dequantize_kernel<float, true> : fp4_dequantize_kernel<float, false>, grid, block, 0, 1, true,
                       stream, q, o, vec);
}

}  // namespace mo
