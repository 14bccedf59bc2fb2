// bf16 products of the feed-forward operators on the 5th-generation tensor
// cores, sums in fp32, everything that follows a sum in its epilogue:
//
//   out[m, n] = act(sum_k A[m, k] B[n, k] + bias[n]) + add[m, n]      kEpiLinear
//   out = act(g) u of two sums g and u with the same A                 kEpiGated
//   out = dh u act'(g), dh act(g) and act(g) u of one sum dh           kEpiGatedGrad
//
// 256 x 256 tiles on CTA pairs (cta_group::2), persistent, as the Newton-Schulz
// products: warp 0 loads this CTA's 128-row halves of both operands by TMA
// (128-byte swizzle) into 32 KB stages, the even CTA's warp 1 issues the
// instructions, the others drain 128 lanes x 256 columns; two accumulators let a
// tile's epilogue run under the next tile's products. Either operand's rows may
// run along k (K-major) or along its own index (MN-major: the transposed
// operands of the gradients, as they lie in memory).
//
// Where it stands: 8192 x 1280 x 5120 with gelu_tanh and an 8-bit copy 72 us (1.49
// PFLOP/s, 68% of the tensor pipe's cycles), the gradients of the same 73 and 74 us
// (83% and 76%; a last round of 8 and of 24 tiles on 76 pairs, and L2). The gated block
// of 8192 x 4096 x 14336: gate and up 930 us and down 500 in runs of milliseconds (96 and
// 97% of the tensor pipe's cycles), 1080 and 570 in runs of seconds, where the power cap
// lowers the clock.
//
// kEpiGated: the even CTA's half of B is 128 rows of the gate weight, the odd
// CTA's the same rows of the up weight. Both CTAs' accumulators then hold g in
// columns 0-127 and u in 128-255 for their own rows of A, and one thread has
// both.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "launch.cuh"
#include "linear_gemm.cuh"

namespace mo {
namespace {

// Epilogue warps: two a quarter of the lanes, or four where the reduction is short
// (see launch_pair), which take the memory of the sixth stage.
constexpr int kMostWarps = 16;
constexpr uint32_t kHalf = 128 * kBlockK * 2;   // 16 KB: 128 rows of an operand
constexpr uint32_t kStage = 2 * kHalf;
constexpr uint32_t kCodes = 32 * 32;            // a chunk of 32 rows in 8 bits
constexpr uint32_t kScratch = 2048 + 2 * kCodes;   // of an epilogue warp: what it stores by TMA, or turns
template <int WARPS>
constexpr int kStages = WARPS == kMostWarps ? 5 : 6;
constexpr uint32_t kBars = 2 * 6 + 5;
constexpr uint32_t kCtrl = 256;
template <int WARPS>
constexpr size_t kSmem = 1024 + size_t(kStages<WARPS>) * kStage + size_t(WARPS) * kScratch + kCtrl;
static_assert(8 * kBars + 16 <= kCtrl && kSmem<8> <= 227 * 1024 && kSmem<kMostWarps> <= 227 * 1024 && kTurn * 4 <= kScratch,
              "shared memory");

// A chunk of 32 columns of an accumulator, a row a lane.
__device__ __forceinline__ void tmem_chunk(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  __syncwarp();
  ptx::tmem_ld_32x32b_x32(taddr, r);
  ptx::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The 32 rows from row0 on (lane l has row0 + l) of the `width` accumulator
// columns from TMEM column `tb` on: chunks of 32 (or 16) columns, every PARTSth one
// this warp's, from `part` on. col0: the first column of the output.
//
// What is written in bf16 or 8 bits goes through the warp's scratch and out by TMA
// wherever its rows are 16-byte aligned: a store of a row a lane touches 32 lines an
// instruction, and those are what the load-store unit counts.
template <Epilogue EPI, int PARTS>
__device__ __forceinline__ void epilogue(const GemmParams& p, const GemmTarget& t, int q, int64_t row0, int64_t col0, int width, int part,
                                         uint32_t tb, uint32_t scratch, float* turn) {
  const int lane = int(threadIdx.x & 31);
  const int64_t row = row0 + lane;
  auto reuse = [&] {   // the scratch: its last copies have read it
    if (lane == 0) ptx::bulk_wait_read();
    __syncwarp();
  };
  if constexpr (EPI == kEpiLinear) {
#pragma unroll 1
    for (int c = part * 32; c < width; c += 32 * PARTS) {
      const int64_t col = col0 + c;
      float v[32];
      tmem_chunk(tb + uint32_t(c), v);
      if (row0 >= t.m || col >= t.n) continue;
      if (PARTS == 2 && p.start[0] != nullptr && row < t.m) add_start(p.start[0] + row * p.start_ld + col, v);
      reuse();
      if (p.bias != nullptr) {
        if (col + 32 <= t.n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 b = reinterpret_cast<const float4*>(p.bias + col)[j];
            const float2 lo = ptx::parts(ptx::add2(ptx::f2(v[4 * j], v[4 * j + 1]), ptx::f2(b.x, b.y)));
            const float2 hi = ptx::parts(ptx::add2(ptx::f2(v[4 * j + 2], v[4 * j + 3]), ptx::f2(b.z, b.w)));
            v[4 * j] = lo.x, v[4 * j + 1] = lo.y, v[4 * j + 2] = hi.x, v[4 * j + 3] = hi.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (col + i < t.n) v[i] += p.bias[col + i];
        }
      }
      if (p.pre.data != nullptr) keep_chunk(p.pre, p.pre_bulk != 0, p.pre_align, row0, t.m, col, t.n, v, scratch + 2048, turn);
      if (p.act != MO_ACT_NONE)
        with_act(p.act, [&](auto act) { act_all<decltype(act)::value>(v); });
      if (t.bulk) {
        if (t.add != nullptr && row < t.m) {   // (whole chunks)
          float x[32];
          if (t.add_bf16)
            load32(static_cast<const uint16_t*>(t.add) + row * t.add_ld + col, t.align, x);
          else
            load32(static_cast<const float*>(t.add) + row * t.add_ld + col, t.align, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += x[i];
        }
        put_bf16(scratch, v);
      }
      ptx::fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (t.bulk) ptx::tma_store_2d(&p.so[q], scratch, int32_t(col), int32_t(row0));
        if (p.pre_bulk) ptx::tma_store_2d(&p.sk[0], scratch + 2048, int32_t(col), int32_t(row0));
        ptx::bulk_commit();
      }
      if (!t.bulk) {
        reuse();   // (what is turned takes all of the scratch)
        store_chunk(t.out, t.out_bf16 != 0, t.ld, t.add, t.add_bf16 != 0, t.add_ld, t.align, row0, t.m, col, t.n, v, turn);
      }
    }
  } else if constexpr (EPI == kEpiGated) {
#pragma unroll 1
    for (int c = part * 32; c < width / 2; c += 32 * PARTS) {
      const int64_t col = col0 + c;
      float g[32], u[32];
      tmem_chunk(tb + uint32_t(c), g);
      tmem_chunk(tb + uint32_t(width / 2 + c), u);
      if (row0 >= t.m || col >= t.n) continue;
      if (p.start[0] != nullptr && row < t.m) {
        add_start(p.start[0] + row * p.start_ld + col, g);
        add_start(p.start[1] + row * p.start_ld + col, u);
      }
      reuse();
      if (p.pre.data != nullptr) {
        keep_chunk(p.pre, p.pre_bulk != 0, p.pre_align, row0, t.m, col, t.n, g, scratch + 2048, turn);
        keep_chunk(p.pre2, p.pre_bulk != 0, p.pre_align, row0, t.m, col, t.n, u, scratch + 2048 + kCodes, turn);
      }
      with_act(p.act, [&](auto act) { gate_all<decltype(act)::value>(g, u); });
      put_bf16(scratch, g);   // h in bf16, as the next product's operand
      ptx::fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        ptx::tma_store_2d(&p.so[0], scratch, int32_t(col), int32_t(row0));
        if (p.pre_bulk) {
          ptx::tma_store_2d(&p.sk[0], scratch + 2048, int32_t(col), int32_t(row0));
          ptx::tma_store_2d(&p.sk[1], scratch + 2048 + kCodes, int32_t(col), int32_t(row0));
        }
        ptx::bulk_commit();
      }
    }
  } else {
    // The next chunk's g and u are loaded while one is worked on.
    RawChunk rg = {}, ru = {};
    auto fetch = [&](int c) {
      const int64_t col = col0 + c;
      if (row < t.m && col < t.n) {
        fetch_kept(p.pre, p.pre_align, row, col, t.n, rg);
        fetch_kept(p.pre2, p.pre_align, row, col, t.n, ru);
      }
    };
    fetch(part * 16);
#pragma unroll 1
    for (int c = part * 16; c < width; c += 16 * PARTS) {
      const int64_t col = col0 + c;
      float g[16], u[16], dh[16];
      kept_values(p.pre, rg, g);
      kept_values(p.pre2, ru, u);
      if (c + 16 * PARTS < width) fetch(c + 16 * PARTS);
      uint32_t r[16];
      __syncwarp();
      ptx::tmem_ld_32x32b_x16(tb + uint32_t(c), r);
      ptx::tmem_ld_wait();
      if (row0 >= t.m || col >= t.n) continue;
      reuse();
#pragma unroll
      for (int i = 0; i < 16; ++i) dh[i] = __uint_as_float(r[i]);
      if (PARTS == 2 && p.start[0] != nullptr && row < t.m) add_start(p.start[0] + row * p.start_ld + col, dh);
      with_act(p.act, [&](auto act) { gate_grad_all<decltype(act)::value>(g, u, dh); });
      put_bf16(scratch, g);   // dg, du and h in bf16, as the next products' operands
      put_bf16(scratch + 1024, dh);
      put_bf16(scratch + 2048, u);
      ptx::fence_async_shared();
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) ptx::tma_store_2d(&p.so[i], scratch + uint32_t(i) * 1024u, int32_t(col), int32_t(row0));
        ptx::bulk_commit();
      }
    }
  }
}

// A tile of the launch: the first are 256 columns wide, the last ones cut into
// p.cut parts.
struct Tile {
  int q;              // target
  int32_t tm, tn;
  int32_t width, sub;   // accumulator columns, part
};
__device__ __forceinline__ Tile tile_of(const GemmParams& p, int32_t i) {
  Tile t;
  const int32_t over = i - p.whole;
  const int32_t tile = over < 0 ? i : p.whole + over / p.cut;
  t.sub = over < 0 ? 0 : over % p.cut;
  t.width = over < 0 ? 256 : 256 / p.cut;
  t.q = target_of(p, tile);
  tile_at(p.t[t.q], tile, t.tm, t.tn);
  return t;
}

template <Epilogue EPI, bool A_MN, bool B_MN, int WARPS>
__global__ void __launch_bounds__(64 + 32 * WARPS, 1) linear_pair_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  // stages (1024-byte aligned), the epilogue warps' scratch, control
  constexpr int kStgs = kStages<WARPS>;
  const uint32_t bars = base + uint32_t(kStgs) * kStage + uint32_t(WARPS) * kScratch;
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + 8 * kBars);
  uint32_t* tmem_slot = ctrl;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 1);
  volatile uint32_t* peer_report = ctrl + 2;   // [0] the peer gave up, [1] stages its producer issued
  auto full_bar = [&](int s) { return bars + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bars + 8u * uint32_t(kStgs + s); };
  auto tfull_bar = [&](int s) { return bars + 8u * uint32_t(2 * kStgs + s); };
  auto tempty_bar = [&](int s) { return bars + 8u * uint32_t(2 * kStgs + 2 + s); };
  const uint32_t drain_bar = bars + 8u * uint32_t(2 * kStgs + 4);

  const int warp = int(threadIdx.x >> 5);
  const int lane = int(threadIdx.x & 31);
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStgs; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(tfull_bar(s), 1);
      ptx::mbar_init(tempty_bar(s), 2 * WARPS);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    peer_report[0] = 0u;
    peer_report[1] = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // All of the above overlaps the previous kernel's end. The next one may come only now: its blocks
  // take their TMEM before they wait for this grid, and this block has its own.
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  const int32_t first = int32_t(ptx::cluster_id_x()), step = int32_t(ptx::nclusters_x());
  const int32_t blocks = p.blocks * p.segments;
  uint32_t n_issued = 0;
  bool mma_issued = false;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer (both CTAs)
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int32_t i = first; ok && i < p.tiles; i += step) {
        const Tile t = tile_of(p, i);
        const int32_t ra = t.tm * 256 + int32_t(rank) * 128;
        const int32_t half = t.width / 2;   // this CTA's rows of B
        const int32_t rb = EPI == kEpiGated ? t.tn * 128 + t.sub * half : t.tn * 256 + t.sub * t.width + int32_t(rank) * half;
        for (int32_t kb = 0; kb < blocks; ++kb) {
          if (!mbar_wait_bounded(empty_bar(stage), ph ^ 1u, abort_flag, p.status, p.timeout_ns)) {
            ok = false;
            break;
          }
          const int seg = kb >= p.blocks ? 1 : 0;
          const int32_t k0 = (kb - seg * p.blocks) * kBlockK;
          const int op = p.segments > 1 ? seg : t.q, opb = EPI == kEpiGated ? int(rank) : op;
          const CUtensorMap* ma = &p.a[op];
          const uint32_t fb_local = full_bar(stage);
          if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2 * (kHalf + uint32_t(half) * 128u));
          const uint32_t fb = ptx::mapa_shared(fb_local, 0);
          const uint32_t sa = base + uint32_t(stage) * kStage, sb = sa + kHalf;
          if (A_MN) {
            ptx::tma_load_2d_pair(sa, ma, fb, ra, k0);
            ptx::tma_load_2d_pair(sa + kBox, ma, fb, ra + 64, k0);
          } else {
            ptx::tma_load_2d_pair(sa, ma, fb, k0, ra);
          }
          if (B_MN) {
            const CUtensorMap* mb = &p.b[opb];
            ptx::tma_load_2d_pair(sb, mb, fb, rb, k0);
            if (half == 128) ptx::tma_load_2d_pair(sb + kBox, mb, fb, rb + 64, k0);
          } else if (half == 128) {
            ptx::tma_load_2d_pair(sb, &p.b[opb], fb, k0, rb);
          } else {
            for (int32_t j = 0; j < half; j += 32) ptx::tma_load_2d_pair(sb + uint32_t(j) * 128u, &p.bs[opb], fb, k0, rb + j);
          }
          ++n_issued;
          if (++stage == kStgs) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issuer (even CTA)
      const uint32_t a_lo = ptx::desc_lo(base, A_MN ? kBox : 16u), b_lo = ptx::desc_lo(base + kHalf, B_MN ? kBox : 16u);
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      int32_t n = 0;
      for (int32_t i = first; ok && i < p.tiles; i += step, ++n) {
        const int acc = n & 1;
        const uint32_t width = i < p.whole ? 256u : 256u / uint32_t(p.cut);
        const uint32_t idesc = ptx::idesc_bf16_f32(256, 0, A_MN ? 1u : 0u, B_MN ? 1u : 0u) | ((width >> 3) << 17);
        if (!mbar_wait_bounded<true>(tempty_bar(acc), (uint32_t(n >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc) * 256u;
        for (int32_t kb = 0; kb < blocks; ++kb) {
          // (the odd CTA's copies count on this barrier too)
          if (!mbar_wait_bounded(full_bar(stage), ph, abort_flag, p.status, p.timeout_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          // K = 16 an instruction: 32 bytes of K-major rows, 16 rows of MN-major ones
          const uint32_t at = uint32_t(stage) * (kStage / 16);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            ptx::umma_bf16_pair_lo(d, a_lo + at + uint32_t(kk) * (A_MN ? 128u : 2u), b_lo + at + uint32_t(kk) * (B_MN ? 128u : 2u), idesc,
                                   (kb | kk) != 0 ? 1u : 0u);
          ptx::umma_commit_pair(empty_bar(stage), 0x3);
          mma_issued = true;
          if (++stage == kStgs) {
            stage = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        ptx::umma_commit_pair(tfull_bar(acc), 0x3);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;
    const uint32_t scratch = base + uint32_t(kStgs) * kStage + uint32_t(warp - 2) * kScratch;
    float* turn = reinterpret_cast<float*>(smem_raw + (scratch - raw));
    int32_t n = 0;
    for (int32_t i = first; i < p.tiles; i += step, ++n) {
      const int acc = n & 1;
      const Tile t = tile_of(p, i);
      bool ok = mbar_wait_bounded(tfull_bar(acc), uint32_t(n >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const int64_t row0 = int64_t(t.tm) * 256 + int64_t(rank) * 128 + quarter * 32;
      const int64_t col0 = EPI == kEpiGated ? int64_t(t.tn) * 128 + t.sub * (t.width / 2) : int64_t(t.tn) * 256 + t.sub * t.width;
      epilogue<EPI, WARPS / 4>(p, p.t[t.q], t.q, row0, col0, t.width, part, tmem + uint32_t(acc) * 256u + (uint32_t(quarter * 32) << 16),
                               scratch, turn);
      // hand the accumulator back: its reads are complete (tcgen05.wait::ld) and fenced, and nothing
      // else of the tile has to be ordered inside the launch
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote_relaxed(ptx::mapa_shared(tempty_bar(acc), 0));
    }
    if (lane == 0) ptx::bulk_wait();
  }

  ptx::tc_fence_before();
  __syncthreads();
  // Both CTAs learn whether either gave up and how many stages its producer issued.
  if (threadIdx.x == 0)
    ptx::st_shared_cluster_v2(ptx::mapa_shared(ptx::smem_addr(const_cast<uint32_t*>(peer_report)), rank ^ 1u),
                              *abort_flag != 0 ? 1u : 0u, n_issued);
  ptx::cluster_sync();
  if (*abort_flag != 0 || peer_report[0] != 0u) {
    // Nothing may still write into either CTA's memory when they exit: the even CTA waits for its
    // instructions, then settles every stage that either producer left in flight (all copies of both
    // CTAs count their bytes on its full barriers; at most the last kStgs can be in flight).
    if (leader && warp == 1 && lane == 0 && mma_issued) {
      ptx::umma_commit_pair(drain_bar, 0x1);
      mbar_wait_drain(drain_bar, 0u, p.timeout_ns);
    }
    if (leader && threadIdx.x == 0) {
      const uint32_t L = n_issued, P = peer_report[1];
      const uint32_t most = L > P ? L : P;
      // stages of this pair's uncut tiles, which come first
      const uint32_t wide = first < p.whole ? uint32_t((p.whole - first + step - 1) / step) * uint32_t(blocks) : 0u;
      constexpr uint32_t stages = uint32_t(kStgs);
      for (uint32_t j = most > stages ? most - stages : 0u; j < most; ++j) {
        const int s = int(j % stages);
        const uint32_t bytes = kHalf + (j < wide ? kHalf : kHalf / uint32_t(p.cut));
        if (j >= L)
          ptx::mbar_arrive_expect_tx(full_bar(s), bytes);   // only the peer's half is coming
        else if (j >= P)
          ptx::mbar_complete_tx(full_bar(s), bytes);        // the peer's half never will
        mbar_wait_drain(full_bar(s), (j / stages) & 1u, p.timeout_ns);
      }
    }
    ptx::cluster_sync();
  }
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn tensor_map_encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Boxes of 32 rows of `cols` columns of an output, swizzled as put_row has them.
bool encode_box(CUtensorMap* map, void* p, int64_t rows, int64_t width, int64_t ld, int64_t size, uint32_t cols) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cuuint64_t(width), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld * size)};
  const cuuint32_t box[2] = {cols, 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Epilogue EPI, bool A_MN, bool B_MN>
cudaError_t launch_pair(const Product& q, GemmParams& p, int sms, cudaStream_t stream) {
  const int n = std::max(q.count, q.segments);
  for (int i = 0; i < 3; ++i) {
    if (i < n && !encode_operand(&p.a[i], q.a[i], A_MN ? 64 : 128)) return cudaErrorInvalidValue;
    if (i < (EPI == kEpiGated ? 2 : n) &&
        (!encode_operand(&p.b[i], q.b[i], B_MN ? 64 : 128) || (!B_MN && !encode_operand(&p.bs[i], q.b[i], 32))))
      return cudaErrorInvalidValue;
  }
  int64_t tiles = 0;
  for (int i = 0; i < q.count; ++i) {
    GemmTarget& t = p.t[i];
    t.tile0 = int32_t(tiles);
    t.tiles_m = int32_t((t.m + 255) / 256);
    t.tiles_n = int32_t(EPI == kEpiGated ? (t.n + 127) / 128 : (t.n + 255) / 256);
    tiles += int64_t(t.tiles_m) * t.tiles_n;
  }
  if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;
  // What is stored by TMA: bf16 rows that are 16-byte aligned (added to, whole chunks only), the padded
  // rows of the workspace, and 8-bit codes.
  if (EPI == kEpiLinear) {
    for (int i = 0; i < q.count; ++i) {
      GemmTarget& t = p.t[i];
      t.bulk = t.out_bf16 && t.align != 0 && (t.add == nullptr || t.n % 32 == 0);
      if (t.bulk && !encode_box(&p.so[i], t.out, t.m, t.n, t.ld, 2, 32)) return cudaErrorInvalidValue;
    }
  } else {
    void* outs[3] = {q.t[0].out, q.out2, q.out3};
    for (int i = 0; i < (EPI == kEpiGated ? 1 : 3); ++i)
      if (!encode_box(&p.so[i], outs[i], q.t[0].m, q.t[0].ld, q.t[0].ld, 2, EPI == kEpiGated ? 32 : 16)) return cudaErrorInvalidValue;
  }
  if (q.pre.data != nullptr && EPI != kEpiGatedGrad) {
    const bool mx8 = q.pre.dtype == MO_MX8;
    p.pre_bulk = mx8 || (EPI == kEpiLinear && p.pre_align != 0);
    const int64_t k = q.t[0].n, pitch = mx8 ? mx8_blocks(k) * 32 : k;
    const Kept* kept[2] = {&q.pre, &q.pre2};
    for (int i = 0; p.pre_bulk && i < (EPI == kEpiGated ? 2 : 1); ++i)
      if (!encode_box(&p.sk[i], kept[i]->data, q.t[0].m, mx8 ? pitch : k, pitch, mx8 ? 1 : 2, 32)) return cudaErrorInvalidValue;
  }
  // The tiles of a last round that leaves half of the pairs idle, or three quarters, are cut into as
  // many parts (us in quarters and in halves: 4096 x 1280 -> 5120 31.3 and 32.1, 2560 x 4096 -> 4096 53.9
  // and 55.9, 2560 x 1280 -> 4096 20.0 and 21.3; gate and up of 2048 x 8192 -> 2560 110 and 112, of 2048 x
  // 4096 -> 5120 96 and 95). Parts of 64 columns not where B's rows run along the output's columns: its
  // boxes are 64 wide a CTA.
  const int64_t pairs = sms / 2, last = tiles % pairs;
  p.cut = last * 2 > pairs || last == 0 ? 1 : !B_MN && last * 4 <= pairs ? 4 : 2;
  p.whole = int32_t(p.cut > 1 ? tiles - last : tiles);
  p.tiles = int32_t(p.cut > 1 ? tiles + last * (p.cut - 1) : tiles);
  // Short reductions: with eight warps an epilogue takes longer than the products of a tile (8192 tokens,
  // gelu_tanh and an 8-bit copy, 768 -> 3200: 48 us, with sixteen 37; 1280 -> 5120: 75 and 70). Long ones:
  // the sixteen's waiting and the stage they cost are more than they give (1600 -> 6400: 107 and 109; 2048
  // -> 8192: 168 and 176; gated block 8192 x 4096 x 14336: 1775 and 1850). Where sums only go out in bf16 it
  // turns earlier (768 -> 3200: 28 and 28; 1280 -> 5120: 57 and 60). (The gated block's figures here include the decoding
  // of its checkpoints.) Gate and up take more registers than
  // sixteen warps have (8192 x 1024 x 2816, both kept: 93, with sixteen 107); their gradients do not (131
  // with sixteen, 134 with eight).
  constexpr int kMost = EPI == kEpiGated ? 8 : kMostWarps;
  bool light = EPI == kEpiLinear && q.act == MO_ACT_NONE && q.pre.data == nullptr;
  for (int i = 0; i < q.count; ++i) light = light && p.t[i].bulk && p.t[i].add == nullptr;
  // (Sums so far belong to reductions that are longer still: eight warps.)
  const bool few = kMost == 8 || q.start[0] != nullptr || int64_t(p.blocks) * q.segments > (EPI == kEpiGatedGrad ? 32 : light ? 12 : 24);
  auto kern = few ? linear_pair_kernel<EPI, A_MN, B_MN, 8> : linear_pair_kernel<EPI, A_MN, B_MN, kMost>;
  const size_t smem = few ? kSmem<8> : kSmem<kMostWarps>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(2 * std::min<int64_t>(pairs, p.tiles));
  return launch_kernel(kern, dim3(grid), dim3(64 + 32 * (few ? 8 : kMostWarps)), smem, 2, true, stream, p);
}

}  // namespace

bool encode_operand(CUtensorMap* map, const Operand& o, uint32_t box_rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cuuint64_t(o.cols), cuuint64_t(o.rows)};
  const cuuint64_t strides[1] = {cuuint64_t(o.ld) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(o.p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Up to 64 rows, or few tiles and a reduction that is worth splitting: 16 blocks of 64, and half of the other
// kernel's tiles where they are more. In us by pairs and by the other kernel:
//   gated block of 4096 x 14336: 65 tokens 71 and 69, 100 73 and 73, 128 74 and 74, 129 80 and 98, 256 82 and 106
//   128 tokens 4096 -> 14336 28 and 28 (65: 27 and 25), 768 -> 16384 11 and 13, 1280 -> 50304 29 and 43
//   512 x 512 over 512 6 and 8, over 1024 7 and 7, over 2048 11 and 9; 1024 x 1024 over 1024 8 and 10, over 2048
//   12 and 11; 1024 x 2048 over 2048 13 and 14, over 8192 37 and 34
// Rows that are not 16-byte aligned take pairs longer to store: 777 x 515 over 1024 9 and 8, with a residual 15
// and 9.
bool is_narrow(const Product& q, int sms) {
  int64_t pair_tiles = 0, tiles = 0, rows = 0;
  bool odd = false;
  for (int i = 0; i < q.count; ++i) {
    const Target& t = q.t[i];
    pair_tiles += ((t.m + 255) / 256) * (q.epi == kEpiGated ? (t.n + 127) / 128 : (t.n + 255) / 256);
    tiles += ((t.m + 127) / 128) * ((t.n + 127) / 128);
    rows = std::max(rows, t.m);
    odd = odd || t.ld % (t.out_bf16 ? 8 : 4) != 0;
  }
  const int64_t blocks = (q.k + kBlockK - 1) / kBlockK * q.segments;
  return (rows <= 64 && !q.a_mn) || (pair_tiles * 2 < sms / 2 && blocks >= std::max<int64_t>(16, odd ? 0 : tiles / 2));
}

int64_t longest_sum(const Product& q, int sms) {
  if (is_few(q, sms)) return 0;
  const int64_t blocks = (q.k + kBlockK - 1) / kBlockK * q.segments, parts = is_narrow(q, sms) ? narrow_parts(q, sms) : 1;
  return (blocks + parts - 1) / parts * kBlockK;
}

cudaError_t launch_product(const Product& q, int sms, int* status, cudaStream_t stream) {
  if (is_few(q, sms)) return launch_few(q, sms, stream);
  GemmParams p = {};
  p.count = q.count;
  p.segments = q.segments;
  p.blocks = int32_t((q.k + kBlockK - 1) / kBlockK);
  p.act = q.act;
  p.bias = q.bias;
  p.start[0] = q.start[0];
  p.start[1] = q.start[1];
  p.start_ld = padded(q.t[0].n);
  p.pre = q.pre;
  p.pre2 = q.pre2;
  p.out2 = q.out2;
  p.out3 = q.out3;
  p.status = status;
  p.timeout_ns = kDefaultTimeoutNs;
  auto align_of = [](uintptr_t bits) { return (bits & 31) == 0 ? 32 : (bits & 15) == 0 ? 16 : 0; };
  p.early = q.early;
  for (int i = 0; i < q.count; ++i) {
    const Target& t = q.t[i];
    uintptr_t bits = reinterpret_cast<uintptr_t>(t.out) | uintptr_t(t.ld * (t.out_bf16 ? 2 : 4));
    if (t.add != nullptr) bits |= reinterpret_cast<uintptr_t>(t.add) | uintptr_t(t.add_ld * (t.add_bf16 ? 2 : 4));
    p.t[i] = {t.out, t.add, t.m, t.n, t.ld, t.add_ld, 0, 0, 0, align_of(bits), t.out_bf16, t.add_bf16};
  }
  if (q.pre.data != nullptr) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(q.pre.data) | reinterpret_cast<uintptr_t>(q.pre2.data);
    if (q.pre.dtype != MO_MX8) bits |= uintptr_t(q.t[0].n * 2);
    p.pre_align = align_of(bits);
  }
  if (is_narrow(q, sms)) return launch_narrow(q, p, sms, stream);
  if (q.epi == kEpiGated) return launch_pair<kEpiGated, false, false>(q, p, sms, stream);
  if (q.epi == kEpiGatedGrad) return launch_pair<kEpiGatedGrad, false, true>(q, p, sms, stream);
  if (q.a_mn) return launch_pair<kEpiLinear, true, true>(q, p, sms, stream);
  return q.b_mn ? launch_pair<kEpiLinear, false, true>(q, p, sms, stream) : launch_pair<kEpiLinear, false, false>(q, p, sms, stream);
}

}  // namespace mo
