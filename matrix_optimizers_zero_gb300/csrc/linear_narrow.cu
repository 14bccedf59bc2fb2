// bf16 products of few rows (see linear_pair.cu for what they compute): a CTA
// multiplies 128 columns' operand by NT rows' over its part of the reduction,
// and the CTAs of a cluster, which hold the parts of one tile, add their sums
// through distributed shared memory in rank order. Accumulator lanes are
// columns of the output; after the addition a lane has four neighbours of a row,
// and eight lanes a block of an 8-bit tensor.
//
// With few rows a product is the reading of its weights, so K is split until all
// SMs have loads under way: 64 x 4096 -> 14336 22 us (5.3 TB/s). What else it takes
// is latency: about 6 us for one k block (launch, tensor memory, first loads, the
// join), 8.7 for 512 x 512 over 2048.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "linear_gemm.cuh"

namespace mo {
namespace {

// Two warps load and multiply; eight (four for 16 rows) move the sums.
template <int NT>
constexpr int kThreads = NT == 16 ? 192 : 320;
constexpr uint32_t kPanel = 128 * kBlockK * 2;   // 128 columns' operand
constexpr uint32_t kPitch = 132;                 // of the fp32 sums [NT][128] in shared memory

template <Epilogue EPI>
constexpr int kPanels = EPI == kEpiGated ? 2 : 1;   // gate and up
template <Epilogue EPI, int NT>
constexpr uint32_t kStage = kPanels<EPI> * kPanel + NT * kBlockK * 2;
// Stages (p.stages): two CTAs an SM where the sums and enough of them fit; with gate
// and up one CTA and all its memory (a token of the 8B block: 63 -> 60 us). Where all
// clusters fit with one CTA an SM, each takes all memory too (100 x 14336 -> 4096: 30
// -> 26 us).
constexpr size_t kCtrl = 256;
template <Epilogue EPI, int NT>
constexpr int kDeep = std::min(12, int((227 * 1024 - 1024 - kCtrl) / kStage<EPI, NT>));
template <Epilogue EPI, int NT>
constexpr int kStages = EPI == kEpiGated ? kDeep<EPI, NT> : (NT == 16 ? 6 : NT == 64 ? 4 : 3);
template <Epilogue EPI, int NT>
constexpr size_t smem_of(int stages) { return 1024 + size_t(stages) * kStage<EPI, NT> + kCtrl; }
template <Epilogue EPI, int NT>
constexpr uint32_t kCols = kPanels<EPI> * NT < 32 ? 32 : kPanels<EPI> * NT;   // of TMEM
template <Epilogue EPI, int NT>
constexpr bool kFits = kStages<EPI, NT> * kStage<EPI, NT> >= kPanels<EPI> * NT * kPitch * 4 && smem_of<EPI, NT>(kDeep<EPI, NT>) <= 227 * 1024;
static_assert(kFits<kEpiLinear, 16> && kFits<kEpiLinear, 64> && kFits<kEpiLinear, 128> && kFits<kEpiGated, 16> &&
                  kFits<kEpiGated, 64> && kFits<kEpiGated, 128>,
              "sums in the stages' memory");

// Four neighbours of a row, the first at `at` of a multiple of 4; `live` of them
// inside it. VEC: rows of a multiple of 4.
__device__ __forceinline__ void put4(void* out, bool bf16, int64_t at, int live, bool vec, const float (&v)[4]) {
  if (vec) {
    if (live <= 0) return;
    if (bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < live) put(out, bf16, at + i, v[i]);
}
__device__ __forceinline__ void get4(const void* p, bool bf16, int64_t at, int live, bool vec, float (&v)[4]) {
  if (vec && live > 0) {
    if (bf16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
      v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
      v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < live ? get(p, bf16, at + i) : 0.0f;
}

// Kept values of four neighbours: in 8 bits eight lanes hold a block.
__device__ __forceinline__ void keep4(const Kept& q, int64_t row, int64_t col, int64_t n, int live, bool vec, const float (&v)[4]) {
  if (q.dtype != MO_MX8) {
    put4(q.data, true, row * n + col, live, vec, v);
    return;
  }
  float x[4], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = i < live ? v[i] : 0.0f;
    top = top2(top, fabsf(x[i]));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = top2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const int64_t nb = (n + 31) / 32;
  if ((col & ~int64_t(31)) >= n) return;
  const uint32_t s = mx8_scale(top);
  const float down = mx8_down(s);
  *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(q.data) + row * nb * 32 + col) =
      cvt_e4m3x4(x[0] * down, x[1] * down, x[2] * down, x[3] * down);
  if ((col & 31) == 0) q.scales[row * nb + (col >> 5)] = uint8_t(s);
}

// What follows the sums of four neighbours of a row; a warp has 128.
template <Epilogue EPI>
__device__ __forceinline__ void finish(const GemmParams& p, const GemmTarget& t, int64_t row, int64_t col, float (&x)[4], float (&y)[4]) {
  const int live = int(max(int64_t(0), min(int64_t(4), t.n - col)));
  const bool vec = (t.n & 3) == 0;
  if (p.start[0] != nullptr && live > 0) {
    add_start(p.start[0] + row * p.start_ld + col, x);
    if (EPI == kEpiGated) add_start(p.start[1] + row * p.start_ld + col, y);
  }
  if constexpr (EPI == kEpiLinear) {
    if (p.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < live) x[i] += p.bias[col + i];
    }
    if (p.pre.data != nullptr) keep4(p.pre, row, col, t.n, live, vec, x);
    with_act(p.act, [&](auto act) { act_all<decltype(act)::value>(x); });
    if (t.add != nullptr) {
      float a[4];
      get4(t.add, t.add_bf16 != 0, row * t.add_ld + col, live, vec, a);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += a[i];
    }
    put4(t.out, t.out_bf16 != 0, row * t.ld + col, live, vec, x);
  } else if constexpr (EPI == kEpiGated) {
    if (p.pre.data != nullptr) {
      keep4(p.pre, row, col, t.n, live, vec, x);
      keep4(p.pre2, row, col, t.n, live, vec, y);
    }
    with_act(p.act, [&](auto act) { gate_all<decltype(act)::value>(x, y); });
    put4(t.out, true, row * t.ld + col, live, vec, x);
  } else {
    if (live <= 0) return;
    float g[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = i < live ? kept_at(p.pre, row, col + i, t.n) : 0.0f;
      u[i] = i < live ? kept_at(p.pre2, row, col + i, t.n) : 0.0f;
    }
    with_act(p.act, [&](auto act) { gate_grad_all<decltype(act)::value>(g, u, x); });
    const int64_t at = row * t.ld + col;
    put4(t.out, true, at, live, vec, g);
    put4(p.out2, true, at, live, vec, x);
    put4(p.out3, true, at, live, vec, u);
  }
}

// Q: the rows' operand (A of the product), P: the columns' (B).
template <Epilogue EPI, bool Q_MN, bool P_MN, int NT>
__global__ void __launch_bounds__(kThreads<NT>) linear_narrow_kernel(const __grid_constant__ GemmParams p) {
  static_assert(!Q_MN || NT == 128, "whole boxes");
  extern __shared__ uint8_t smem_raw[];
  constexpr uint32_t kStg = kStage<EPI, NT>;
  constexpr int kWarps = kThreads<NT> / 32, kShares = (kWarps - 2) / 4;   // warps; of a quarter of the lanes
  const int stages = p.stages;
  constexpr uint32_t kQ = kPanels<EPI> * kPanel;   // of the rows' operand in a stage
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t bars = base + uint32_t(stages) * kStg;
  constexpr uint32_t kBars = 2 * kDeep<EPI, NT> + 2;
  static_assert(8 * kBars + 8 <= kCtrl, "control block");
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + 8 * kBars);
  uint32_t* tmem_slot = ctrl;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 1);
  float* sums = reinterpret_cast<float*>(smem_raw + (base - raw));
  auto full_bar = [&](int s) { return bars + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bars + 8u * uint32_t(stages + s); };
  const uint32_t done_bar = bars + 8u * uint32_t(2 * stages);
  const uint32_t drain_bar = bars + 8u * uint32_t(2 * stages + 1);

  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  const uint32_t parts = gridDim.x / uint32_t(p.tiles);   // CTAs of a cluster
  const uint32_t rank = ptx::cluster_ctarank();
  const int32_t tile = int32_t(blockIdx.x / parts);
  const int q = target_of(p, tile);
  const GemmTarget& t = p.t[q];
  const int32_t tn = (tile - t.tile0) / t.tiles_m, tm = (tile - t.tile0) - tn * t.tiles_m;   // 128 columns, NT rows
  const int64_t blocks = int64_t(p.blocks) * p.segments;
  const int32_t k0 = int32_t(blocks * rank / parts), k1 = int32_t(blocks * (rank + 1) / parts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(done_bar, 1);
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_one(ptx::smem_addr(tmem_slot), kCols<EPI, NT>);
    ptx::tmem_relinquish_one();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Weights that no launch of this call writes need not wait for the one before this: its blocks let
  // this kernel come only after they have waited in their turn, when all earlier launches had ended.
  uint32_t n_issued = 0;
  bool mma_issued = false;
  auto load_p = [&](int32_t kb, uint32_t fb, uint32_t sp) {
    const int seg = kb >= p.blocks ? 1 : 0;
    const int32_t at = (kb - seg * p.blocks) * kBlockK;
#pragma unroll
    for (int i = 0; i < kPanels<EPI>; ++i) {
      const CUtensorMap* mp = &p.b[EPI == kEpiGated ? i : p.segments > 1 ? seg : q];
      const uint32_t s = sp + uint32_t(i) * kPanel;
      if (P_MN) {
        ptx::tma_load_2d(s, mp, fb, tn * 128, at);
        ptx::tma_load_2d(s + kBox, mp, fb, tn * 128 + 64, at);
      } else {
        ptx::tma_load_2d(s, mp, fb, at, tn * 128);
      }
    }
  };
  int32_t ahead = k0;   // stages whose columns' operand is under way already
  if (p.early && warp == 0 && lane == 0)
    for (; ahead < min(k1, k0 + stages); ++ahead) {
      const uint32_t fb = full_bar(ahead - k0);
      ptx::mbar_arrive_expect_tx(fb, kStg);
      load_p(ahead, fb, base + uint32_t(ahead - k0) * kStg);
    }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();   // with the TMEM held: the next kernel's blocks take theirs before they wait

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      for (int32_t kb = k0; kb < k1; ++kb) {
        // (stages that are under way were free: nothing may leave them half filled)
        if (kb >= ahead && !mbar_wait_bounded(empty_bar(stage), ph ^ 1u, abort_flag, p.status, p.timeout_ns)) break;
        const int seg = kb >= p.blocks ? 1 : 0;
        const int32_t at = (kb - seg * p.blocks) * kBlockK;
        const int op = p.segments > 1 ? seg : q;
        const uint32_t fb = full_bar(stage);
        const uint32_t sp = base + uint32_t(stage) * kStg, sq = sp + kQ;
        if (kb >= ahead) {
          ptx::mbar_arrive_expect_tx(fb, kStg);
          load_p(kb, fb, sp);
        }
        if (Q_MN) {
          ptx::tma_load_2d(sq, &p.a[op], fb, tm * NT, at);
          ptx::tma_load_2d(sq + kBox, &p.a[op], fb, tm * NT + 64, at);
        } else {
          ptx::tma_load_2d(sq, &p.a[op], fb, at, tm * NT);
        }
        ++n_issued;
        if (++stage == stages) {
          stage = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, NT, P_MN ? 1u : 0u, Q_MN ? 1u : 0u);
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int32_t kb = k0; kb < k1; ++kb) {
        if (!mbar_wait_bounded(full_bar(stage), ph, abort_flag, p.status, p.timeout_ns)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sp = base + uint32_t(stage) * kStg, sq = sp + kQ;
#pragma unroll
        for (int i = 0; i < kPanels<EPI>; ++i) {
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk) {
            const uint32_t s = sp + uint32_t(i) * kPanel;
            const uint64_t pd = P_MN ? ptx::smem_desc_sw128(s + uint32_t(kk) * 2048u, kBox, 1024u)
                                     : ptx::smem_desc_sw128(s + uint32_t(kk) * 32u, 16u, 1024u);
            const uint64_t qd = Q_MN ? ptx::smem_desc_sw128(sq + uint32_t(kk) * 2048u, kBox, 1024u)
                                     : ptx::smem_desc_sw128(sq + uint32_t(kk) * 32u, 16u, 1024u);
            ptx::umma_bf16_one(tmem + uint32_t(i) * NT, pd, qd, idesc, kb > k0 || kk > 0 ? 1u : 0u);
          }
        }
        ptx::umma_commit_one(empty_bar(stage));
        mma_issued = true;
        if (++stage == stages) {
          stage = 0;
          ph ^= 1u;
        }
      }
      if (ok) ptx::umma_commit_one(done_bar);
    }
  } else {
    const int quarter = warp & 3;
    bool ok = mbar_wait_bounded(done_bar, 0u, abort_flag, p.status, p.timeout_ns);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
      ptx::tc_fence_after();
      // lane l of a quarter holds column quarter 32 + l; the sums go to the memory of the stages, which
      // have all been read
      const int rows = int(min(int64_t(NT), t.m - int64_t(tm) * NT));
#pragma unroll 1
      for (int i = 0; i < kPanels<EPI>; ++i)
#pragma unroll 1
        for (int c = (warp - 2) / 4 * 16; c < rows; c += 16 * kShares) {
          uint32_t r[16];
          __syncwarp();
          ptx::tmem_ld_32x32b_x16(tmem + uint32_t(i * NT + c) + (uint32_t(quarter * 32) << 16), r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            sums[uint32_t(i * NT + c + j) * kPitch + uint32_t(quarter * 32 + lane)] = __uint_as_float(r[j]);
        }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0) {   // settle what is in flight before the memory is given back
    if (warp == 1 && lane == 0 && mma_issued) {
      ptx::umma_commit_one(drain_bar);
      mbar_wait_drain(drain_bar, 0u, p.timeout_ns);
    }
    if (threadIdx.x == 0)
      for (uint32_t n = uint32_t(stages), j = n_issued > n ? n_issued - n : 0u; j < n_issued; ++j)
        mbar_wait_drain(full_bar(int(j % n)), (j / n) & 1u, p.timeout_ns);
    __syncthreads();
  }
  if (parts > 1) ptx::cluster_sync();   // every part's sums are in place
  {
    // this CTA's share of the tile, a row a warp, four columns a lane, parts added in rank order
    const uint32_t sums_addr = ptx::smem_addr(sums);
    const int64_t row0 = int64_t(tm) * NT, col = int64_t(tn) * 128 + 4 * lane;
    const uint32_t rows = uint32_t(min(int64_t(NT), t.m - row0));
#pragma unroll 2
    for (uint32_t j = rank * kWarps + uint32_t(warp); j < rows; j += parts * kWarps) {
      float v[2][4];
#pragma unroll
      for (int i = 0; i < kPanels<EPI>; ++i) {
        const uint32_t at = (uint32_t(i) * NT + j) * kPitch + 4u * uint32_t(lane);
        float4 x[8];
#pragma unroll
        for (uint32_t s = 0; s < 8; ++s)
          if (s < parts)
            x[s] = parts == 1 ? *reinterpret_cast<const float4*>(sums + at)
                              : ptx::ld_shared_cluster_v4(ptx::mapa_shared(sums_addr + 4u * at, s));
        float4 f = x[0];
#pragma unroll
        for (uint32_t s = 1; s < 8; ++s)
          if (s < parts) f.x += x[s].x, f.y += x[s].y, f.z += x[s].z, f.w += x[s].w;
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
      }
      finish<EPI>(p, t, row0 + j, col, v[0], v[kPanels<EPI> - 1]);
    }
  }
  if (parts > 1) ptx::cluster_sync();   // the peers have read this CTA's sums
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_one(tmem, kCols<EPI, NT>);
}

// The reduction in as many parts (2^log) as leave all clusters resident and four stages a CTA. Clusters of 4
// and 8 do not fill the GPU's parts evenly: with a CTA an SM (all its memory), 36 and 15 of 38 and 19 fit on
// 152 SMs, with two twice as many. One cluster more than fit takes another round (512 x 512 over 4096 in 16
// clusters of 8: 15.8 us, with two CTAs an SM 10.3).
template <Epilogue EPI, int NT>
struct Split {
  int64_t tiles = 0;
  int log = 0;
  bool deep;   // one CTA an SM, with all its memory
  Split(const Product& q, int sms) {
    for (int i = 0; i < q.count; ++i) tiles += (q.t[i].m + NT - 1) / NT * ((q.t[i].n + 127) / 128);
    const int64_t per_sm = smem_of<EPI, NT>(kStages<EPI, NT>) <= 113 * 1024 ? 2 : 1;
    const int64_t fit[4] = {sms, sms / 2, sms * 47 / 200, sms * 18 / 200}, blocks = (q.k + kBlockK - 1) / kBlockK * q.segments;
    for (int i = 1; i < 4 && tiles <= fit[i] * per_sm && blocks >= (4 << i); ++i) log = i;
    deep = tiles <= fit[log];
  }
};

template <Epilogue EPI, bool Q_MN, bool P_MN, int NT>
cudaError_t narrow_as(const Product& q, GemmParams& p, int sms, cudaStream_t stream) {
  const int n = std::max(q.count, q.segments);
  for (int i = 0; i < 3; ++i) {
    if (i < n && !encode_operand(&p.a[i], q.a[i], Q_MN ? 64 : NT)) return cudaErrorInvalidValue;
    if (i < (EPI == kEpiGated ? 2 : n) && !encode_operand(&p.b[i], q.b[i], P_MN ? 64 : 128)) return cudaErrorInvalidValue;
  }
  int64_t tiles = 0;
  for (int i = 0; i < q.count; ++i) {
    GemmTarget& t = p.t[i];
    t.tile0 = int32_t(tiles);
    t.tiles_m = int32_t((t.m + NT - 1) / NT);
    t.tiles_n = int32_t((t.n + 127) / 128);
    tiles += int64_t(t.tiles_m) * t.tiles_n;
  }
  p.tiles = int32_t(tiles);
  const Split<EPI, NT> split(q, sms);
  const unsigned parts = 1u << split.log;
  p.stages = split.deep ? kDeep<EPI, NT> : kStages<EPI, NT>;
  auto kern = linear_narrow_kernel<EPI, Q_MN, P_MN, NT>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem_of<EPI, NT>(kDeep<EPI, NT>));
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(unsigned(tiles * parts)), dim3(kThreads<NT>), smem_of<EPI, NT>(p.stages), parts, true, stream, p);
}

// f(variant) for the kernel that a product takes.
template <Epilogue EPI, bool Q_MN, bool P_MN, int NT>
struct Variant {
  static int64_t parts(const Product& q, int sms) { return int64_t(1) << Split<EPI, NT>(q, sms).log; }
  static cudaError_t launch(const Product& q, GemmParams& p, int sms, cudaStream_t stream) {
    return narrow_as<EPI, Q_MN, P_MN, NT>(q, p, sms, stream);
  }
};
template <Epilogue EPI, bool P_MN, typename F>
auto with_rows(const Product& q, F&& f) {
  if (q.t[0].m <= 16) return f(Variant<EPI, false, P_MN, 16>());
  if (q.t[0].m <= 64) return f(Variant<EPI, false, P_MN, 64>());
  return f(Variant<EPI, false, P_MN, 128>());
}
template <typename F>
auto with_variant(const Product& q, F&& f) {
  if (q.epi == kEpiGated) return with_rows<kEpiGated, false>(q, f);
  if (q.epi == kEpiGatedGrad) return with_rows<kEpiGatedGrad, true>(q, f);
  if (q.a_mn) return f(Variant<kEpiLinear, true, true, 128>());
  return q.b_mn ? with_rows<kEpiLinear, true>(q, f) : with_rows<kEpiLinear, false>(q, f);
}

}  // namespace

int64_t narrow_parts(const Product& q, int sms) {
  return with_variant(q, [&](auto v) { return decltype(v)::parts(q, sms); });
}

cudaError_t launch_narrow(const Product& q, GemmParams& p, int sms, cudaStream_t stream) {
  return with_variant(q, [&](auto v) { return decltype(v)::launch(q, p, sms, stream); });
}

}  // namespace mo
