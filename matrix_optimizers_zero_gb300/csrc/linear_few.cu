// bf16 products of one or two rows (see linear_pair.cu for what they compute): the
// reading of the weights and nothing else. A warp takes a column of the output (of
// gate and up: the same of both), reads its weights in 16-byte pieces of
// neighbouring lanes, the next pieces under way while it multiplies the last (across
// columns too), and adds its lanes' sums in a fixed order. The rows lie in shared
// memory, read anew for every column.
//
// What the kernel of few rows spends on the way is saved: tensor memory, barriers,
// clusters that leave SMs idle, the sums' way out (1280 -> 5120: 5.5 us, by the other
// 6.3; 14336 -> 4096: 19.8 and 22.4, which are 5.9 and 5.2 TB/s).
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "linear_gemm.cuh"

namespace mo {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 2;                  // an SM
constexpr int64_t kRowBytes = 112 * 1024;   // of shared memory for the rows

struct FewParams {
  const uint16_t* x;
  const uint16_t* w[2];
  int64_t x_ld, w_ld;
  int64_t n;
  uint32_t pieces;   // 16 bytes of a row each
  int32_t act, early;
  const float* bias;
  const void* add;
  void* out;
  int64_t ld, add_ld;
  int32_t out_bf16, add_bf16;
};

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void pairs(const uint4& v, F2 (&f)[4]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = ptx::f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}

template <Epilogue EPI, int T>
__global__ void __launch_bounds__(kThreads, kBlocks) linear_few_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint4 rows[];   // [T][pieces]
  constexpr int kPanels = EPI == kEpiGated ? 2 : 1, kAhead = 4 / kPanels;   // pieces of a lane and panel under way
  const uint32_t lane = threadIdx.x & 31u;
  const int64_t step = int64_t(gridDim.x) * kWarps;
  int64_t col = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  uint4 next[kPanels][kAhead];
  auto load = [&](int64_t c, uint32_t first) {
#pragma unroll
    for (int i = 0; i < kPanels; ++i) {
      const uint4* w = reinterpret_cast<const uint4*>(p.w[i] + c * p.w_ld) + first + lane;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c < p.n && first + uint32_t(u) * 32u + lane < p.pieces) next[i][u] = load_once(w + u * 32);
    }
  };
  // (weights that no launch of this call writes need not wait for the one before this, as in
  // linear_narrow_kernel)
  if (p.early) load(col, 0);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (!p.early) load(col, 0);
  for (uint32_t i = threadIdx.x; i < uint32_t(T) * p.pieces; i += kThreads) {
    const uint32_t t = T == 1 ? 0u : i / p.pieces;
    rows[i] = reinterpret_cast<const uint4*>(p.x + t * p.x_ld)[i - t * p.pieces];
  }
  __syncthreads();
  for (; col < p.n; col += step) {
    F2 acc[kPanels][T];
#pragma unroll
    for (int i = 0; i < kPanels; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[i][t] = ptx::f2(0.0f);
#pragma unroll 1
    for (uint32_t first = 0; first < p.pieces; first += 32 * kAhead) {
      uint4 now[kPanels][kAhead];
#pragma unroll
      for (int i = 0; i < kPanels; ++i)
#pragma unroll
        for (int u = 0; u < kAhead; ++u) now[i][u] = next[i][u];
      const bool last = first + 32 * kAhead >= p.pieces;
      load(last ? col + step : col, last ? 0 : first + 32 * kAhead);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t at = first + uint32_t(u) * 32u + lane;
        if (at >= p.pieces) break;
        F2 w[kPanels][4];
#pragma unroll
        for (int i = 0; i < kPanels; ++i) pairs(now[i][u], w[i]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          F2 x[4];
          pairs(rows[uint32_t(t) * p.pieces + at], x);
#pragma unroll
          for (int i = 0; i < kPanels; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][t] = ptx::fma2(w[i][j], x[j], acc[i][t]);
        }
      }
    }
    // lane t finishes row t
    float mine[kPanels] = {};
#pragma unroll
    for (int i = 0; i < kPanels; ++i)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float2 s = ptx::parts(acc[i][t]);
        float v = s.x + s.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == uint32_t(t)) mine[i] = v;
      }
    if (lane >= uint32_t(T)) continue;
    float y;
    if constexpr (EPI == kEpiGated) {
      with_act(p.act, [&](auto act) { y = act_value<decltype(act)::value>(mine[0]) * mine[1]; });
    } else {
      y = mine[0] + (p.bias != nullptr ? p.bias[col] : 0.0f);
      with_act(p.act, [&](auto act) { y = act_value<decltype(act)::value>(y); });
      if (p.add != nullptr) y += get(p.add, p.add_bf16 != 0, lane * p.add_ld + col);
    }
    put(p.out, p.out_bf16 != 0, lane * p.ld + col, y);
  }
}

template <Epilogue EPI>
auto kernel_for(int64_t rows) {
  return rows == 1 ? linear_few_kernel<EPI, 1> : linear_few_kernel<EPI, 2>;
}

}  // namespace

// One or two rows; a third costs more instructions than the weights leave time for (one, two, three and four
// tokens of the 8B block: 55, 57, 67 and 90 us, by the kernel of few rows 61 each). Below k = 512 the adding
// of the lanes' sums takes over, unless every warp has one column at most (256 -> 50304: 10.6 and 9.7 us by
// the other kernel; 256 -> 4096: 2.5 and 3.6; 512 -> 50304: 12.2 and 13.4).
bool is_few(const Product& q, int sms) {
  const Target& t = q.t[0];
  return t.m <= 2 && q.count == 1 && q.segments == 1 && !q.a_mn && !q.b_mn && q.epi != kEpiGatedGrad && q.pre.data == nullptr && q.start[0] == nullptr &&
         q.k % 8 == 0 && t.m * q.k * 2 <= kRowBytes && (q.k >= 512 || t.n <= int64_t(kBlocks) * kWarps * sms);
}

cudaError_t launch_few(const Product& q, int sms, cudaStream_t stream) {
  const Target& t = q.t[0];
  FewParams p = {};
  p.x = static_cast<const uint16_t*>(q.a[0].p);
  p.x_ld = q.a[0].ld;
  for (int i = 0; i < (q.epi == kEpiGated ? 2 : 1); ++i) p.w[i] = static_cast<const uint16_t*>(q.b[i].p);
  p.w_ld = q.b[0].ld;
  p.n = t.n;
  p.pieces = uint32_t(q.k / 8);
  p.act = q.act;
  p.early = q.early;
  p.bias = q.bias;
  p.add = t.add;
  p.out = t.out;
  p.ld = t.ld;
  p.add_ld = t.add_ld;
  p.out_bf16 = t.out_bf16;
  p.add_bf16 = t.add_bf16;
  auto kern = q.epi == kEpiGated ? kernel_for<kEpiGated>(t.m) : kernel_for<kEpiLinear>(t.m);
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kRowBytes);
  if (e != cudaSuccess) return e;
  const int64_t blocks = std::min<int64_t>((t.n + kWarps - 1) / kWarps, kBlocks * sms);
  return launch_kernel(kern, dim3(unsigned(blocks)), dim3(kThreads), size_t(t.m) * p.pieces * 16, 1, true, stream, p);
}

}  // namespace mo
