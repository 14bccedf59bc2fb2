// Products of 4-bit block-scaled tensors on the 5th-generation tensor cores:
// D[m, n] = gA gB sum_k A[m, k] B[n, k], with A and B as e2m1 codes under a
// scale for each block of their rows, accumulated in fp32 in TMEM, rounded
// once to the output's type.
//
// Scales reach the tensor core through TMEM; their 512-byte tiles arrive in
// shared memory by TMA. The narrow kernel's issuing thread copies them to TMEM
// columns (tcgen05.cp) in front of the instructions that use them, in issue
// order. The pair kernel's scale warps store them there from registers
// (tcgen05.st) and hand them to the issuing thread through a barrier.
//
//   fp4_pair_kernel    256 x 256 tiles on CTA pairs, persistent: the large products.
//                      8192 x 14336 x 4096: mx 168 us = 5.7 PFLOP/s at 1.92 GHz,
//                      nv 185 us = 5.2 at 1.82, both under the 1.4 kW power cap;
//                      where the cap does not bind, by the issue of instructions
//                      (about 720 cycles a stage of four that take 530)
//   fp4_narrow_kernel  128 (rows of B) x NT (rows of A) tiles on single CTAs, K
//                      split over a cluster whose CTAs add their sums through
//                      distributed shared memory in rank order: few rows. Bound by
//                      latencies: 1 x 14336 x 4096 nv 10 us, 33 MB
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "device_common.cuh"
#include "launch.cuh"
#include "ptx_train.cuh"
#include "train_kernels.h"

namespace mo {
namespace {

constexpr int kStageK = 256;                         // elements of K a stage: 128 bytes of codes, one swizzle row
constexpr uint32_t kPanelBytes = 128 * kStageK / 2;  // 128 rows of codes
// 512-byte scale tiles of 128 rows in a stage, and K = 64 instructions a tile serves
template <bool MX>
constexpr int kSfTiles = MX ? 2 : 4;
template <bool MX>
constexpr int kStepsPerTile = MX ? 2 : 1;
template <bool MX>
constexpr uint32_t kSfBytes = 512u * kSfTiles<MX>;

struct ProductParams {
  CUtensorMap a, b, sa, sb;   // codes (128-byte swizzle) and scale tiles of both operands
  void* out;
  const float* amax_a;
  const float* amax_b;
  int* status;
  int64_t m, n;
  int32_t steps;              // K = 64 instructions: ceil(k / 64)
  int32_t stages;             // ceil(k / 256)
  int32_t tiles_k;            // scale tiles along K
  int32_t tiles_m, tiles_n;   // output tiles
  int32_t align;              // of D's rows: 32, 16 or 0 (element stores)
  uint64_t timeout_ns;
};

// Exponent of a tensor's own scale g (a power of two, 2^-126 to 2^117).
__device__ __forceinline__ int scale_exponent(const float* amax) {
  if (amax == nullptr) return 0;
  const uint32_t b = __float_as_uint(*amax) & 0x7FFFFFFFu;
  if (b == 0u || b >= 0x7F800000u) return 0;
  return max(int(b >> 23) - 138 + ((b & 0x7FFFFFu) > 0x280000u ? 1 : 0), -126);
}

// gA gB as two powers of two, applied one after the other: their product, 2^-252
// to 2^234, is no float at either end, where the sums times it may be (a sum of
// 0 always is). A sum that is not 0 is at least 2^-20 (the smallest codes and
// scales), so the first product, with no less than 2^-100, is exact; what the
// second cuts off below 2^-226 rounds to 0 whatever the sum.
struct Factor {
  float first, second;
  __device__ __forceinline__ Factor(const float* amax_a, const float* amax_b) {
    const int e = scale_exponent(amax_a) + scale_exponent(amax_b), e1 = min(max(e, -100), 127), e2 = max(e - e1, -126);
    first = __uint_as_float(uint32_t(e1 + 127) << 23);
    second = __uint_as_float(uint32_t(e2 + 127) << 23);
  }
  __device__ __forceinline__ float operator()(float sum) const { return sum * first * second; }
};

__device__ __forceinline__ void put(uint16_t* o, float v) { *o = float_to_bf16_bits(v); }
__device__ __forceinline__ void put(float* o, float v) { *o = v; }

// Stores a chunk of 32 columns, a row a lane, of the 32 rows from `row0` on.
// Rows that are 16-byte aligned and a whole chunk: vectors, 32 bytes wide
// where the rows allow it. Others (an odd n, the last columns) would store
// element by element into 32 rows at a time, so the chunk is turned in shared
// memory, and a warp stores one row after the other.
constexpr uint32_t kTurnWords = 17 * 32;   // a warp's: 32 rows of 16 words, each a word apart from the next

__device__ __forceinline__ void store_chunk(uint16_t* out, int64_t row0, int64_t m, int64_t col, int64_t n, int align,
                                            const float (&v)[32], uint32_t* turn) {
  const int lane = int(threadIdx.x & 31);
  uint32_t w[2][8];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j >> 3][j & 7] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  if (align != 0 && col + 32 <= n) {
    if (row0 + lane >= m) return;
    uint16_t* o = out + (row0 + lane) * n + col;
    if (align == 32) {
      ptx::st_global_v8(o, w[0]);
      ptx::st_global_v8(o + 16, w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<uint4*>(o)[j] = make_uint4(w[j >> 1][4 * (j & 1)], w[j >> 1][4 * (j & 1) + 1],
                                                    w[j >> 1][4 * (j & 1) + 2], w[j >> 1][4 * (j & 1) + 3]);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j) turn[lane * 17 + j] = w[j >> 3][j & 7];
  __syncwarp();
  const int rows = int(min(int64_t(32), m - row0));
  if (col + lane < n) {
    uint16_t* o = out + row0 * n + col + lane;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) o[r * n] = uint16_t(turn[r * 17 + (lane >> 1)] >> (16 * (lane & 1)));
  }
}

__device__ __forceinline__ void store_chunk(float* out, int64_t row0, int64_t m, int64_t col, int64_t n, int align,
                                            const float (&v)[32], uint32_t* turn) {
  const int lane = int(threadIdx.x & 31);
  if (align != 0 && col + 32 <= n) {
    if (row0 + lane >= m) return;
    float* o = out + (row0 + lane) * n + col;
    if (align == 32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * q + j]);
        ptx::st_global_v8(o + 8 * q, w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<float4*>(o)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    return;
  }
  const int rows = int(min(int64_t(32), m - row0));
#pragma unroll
  for (int h = 0; h < 2; ++h) {   // 16 columns at a time: two rows a store
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) turn[lane * 17 + j] = __float_as_uint(v[16 * h + j]);
    __syncwarp();
    const int64_t c = col + 16 * h + (lane & 15);
    if (c < n)
#pragma unroll 8
      for (int r = lane >> 4; r < rows; r += 2) out[(row0 + r) * n + c] = __uint_as_float(turn[r * 17 + (lane & 15)]);
  }
}

// ------------------------------------------------------------------ pairs
//
// Warp 0 of each CTA loads its 128-row halves of A and B, warp 18 its A scales
// and all 256 rows' B scales; warps 10-17 put the scales into TMEM; the even CTA's
// warp 1 issues the instructions; warps 2-9 drain 128 lanes x 256 columns.
//
// Scales: the tensor core's own copy (tcgen05.cp) runs in its instruction
// stream, about 30 cycles for each of the six to twelve 512-byte tiles of a
// stage beside 125 for each of its four instructions. Stores from registers
// (tcgen05.st) run beside it (8192^3: mx 267 -> 201 us, nv 357 -> 211 us).
//
// The issuing thread bounds a stage as much as the tensor core does: with
// operand descriptors put together for every instruction 8192^3 takes 201 us
// (mx), with precomputed halves 180. For the same reason tiles 192 wide, whose
// last round of tiles is fuller, take as long a stage as these.
//
// TMEM: an accumulator takes 256 columns and a stage's scales 24 (mx) or 48
// (nv), and a stage's scales are written while the last one's are in use. So
// the two accumulators overlap in 96 columns, [160, 256): the epilogue drains
// those first, and the next tile starts as soon as they are free.
constexpr int kEpiWarps = 8;
constexpr int kSfWarps = 4;    // a stage's: one a lane quarter
constexpr int kSfGroups = 2;
constexpr int kSfWarp0 = 2 + kEpiWarps;
constexpr int kSfLoader = kSfWarp0 + kSfGroups * kSfWarps;
constexpr int kPairThreads = 32 * (kSfLoader + 1);
constexpr int kSfStages = 8;   // scales run farther ahead: they have one step more to go

constexpr int kPairStages = 5;
constexpr uint32_t kAccStep = 160;
constexpr uint32_t kSfCol = 416;
template <bool MX>
constexpr uint32_t kSfCols = 12 * kSfTiles<MX>;    // A 4 columns, B 8, for every scale tile of a stage
template <bool MX>
constexpr int kSfSlots = int(96 / kSfCols<MX>);    // stages whose scales TMEM holds
constexpr uint32_t kPairBars = 2 * kPairStages + 7 + 2 * kSfStages + 4;
template <bool MX>
constexpr size_t kPairSmem = 1024 + size_t(kPairStages) * 2 * kPanelBytes + size_t(kSfStages) * 3 * kSfBytes<MX> + 384 +
                             kEpiWarps * 4 * kTurnWords;
static_assert(kAccStep + 256 <= kSfCol && kSfCol + 96 <= 512, "TMEM columns");
static_assert(8 * kPairBars + 32 <= 384, "control block");
static_assert(kPairSmem<false> <= 227 * 1024, "shared memory");

// Output tiles in groups of 8 tile rows, column by column: the tiles in
// flight share operand panels.
__device__ __forceinline__ void tile_at(int32_t t, int32_t tiles_m, int32_t tiles_n, int32_t& tm, int32_t& tn) {
  const int32_t group = t / (8 * tiles_n), first = group * 8;
  const int32_t height = min(8, tiles_m - first), in = t - group * 8 * tiles_n;
  tm = first + in % height;
  tn = in / height;
}

template <bool MX, typename O>
__global__ void __launch_bounds__(kPairThreads, 1) fp4_pair_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr uint32_t kStage = 2 * kPanelBytes;   // codes; their bytes count on the even CTA's barriers
  constexpr int kSlots = kSfSlots<MX>;
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  // panels first (1024-byte aligned), then the scale tiles of every stage, then control
  const uint32_t sf_base = base + uint32_t(kPairStages) * kStage;
  const uint32_t bars = sf_base + uint32_t(kSfStages) * 3u * kSfBytes<MX>;
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + 8 * kPairBars);
  uint32_t* tmem_slot = ctrl;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 1);
  volatile uint32_t* peer_report = ctrl + 2;   // [0] the peer gave up, [1] stages its producer issued
  auto full_bar = [&](int s) { return bars + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bars + 8u * uint32_t(kPairStages + s); };
  auto tfull_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + s); };
  auto tempty_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + 2 + s); };
  auto over_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + 4 + s); };
  const uint32_t drain_bar = bars + 8u * uint32_t(2 * kPairStages + 6);
  auto sf_full_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + 7 + s); };    // scales in shared memory
  auto sf_empty_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + 7 + kSfStages + s); };
  auto sf_ready_bar = [&](int s) { return bars + 8u * uint32_t(2 * kPairStages + 7 + 2 * kSfStages + s); };   // in TMEM, both CTAs

  const int warp = int(threadIdx.x >> 5);
  const int lane = int(threadIdx.x & 31);
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int s = 0; s < kSfStages; ++s) {
      ptx::mbar_init(sf_full_bar(s), 1);
      ptx::mbar_init(sf_empty_bar(s), kSfWarps);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(tfull_bar(s), 1);
      ptx::mbar_init(tempty_bar(s), 2 * kEpiWarps);
      ptx::mbar_init(over_bar(s), 2 * kEpiWarps);
    }
    for (int s = 0; s < kSlots; ++s) ptx::mbar_init(sf_ready_bar(s), 2 * kSfWarps);
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

  const int32_t ntiles = p.tiles_m * p.tiles_n;
  const int32_t first = int32_t(ptx::cluster_id_x()), step = int32_t(ptx::nclusters_x());
  uint32_t n_issued = 0, sf_issued = 0;
  bool mma_issued = false;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer (both CTAs)
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int32_t t = first; ok && t < ntiles; t += step) {
        int32_t tm, tn;
        tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
        const int32_t ra = tm * 256 + int32_t(rank) * 128, rb = tn * 256 + int32_t(rank) * 128;
        for (int32_t kb = 0; kb < p.stages; ++kb) {
          if (!mbar_wait_bounded(empty_bar(stage), ph ^ 1u, abort_flag, p.status, p.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = full_bar(stage);
          if (leader) ptx::mbar_arrive_expect_tx(fb_local, 2 * kStage);
          const uint32_t fb = ptx::mapa_shared(fb_local, 0);
          const uint32_t sa = base + uint32_t(stage) * kStage;
          ptx::tma_load_2d_pair(sa, &p.a, fb, kb * 128, ra);
          ptx::tma_load_2d_pair(sa + kPanelBytes, &p.b, fb, kb * 128, rb);
          ++n_issued;
          if (++stage == kPairStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issuer (even CTA)
      int stage = 0, slot = 0;
      uint32_t sph = 0;
      bool ok = true, seen = false;   // seen: the stage is known to be complete
      const uint32_t desc_lo = ptx::desc_lo_sw128(base);
      int32_t i = 0;
      for (int32_t t = first; ok && t < ntiles; t += step, ++i) {
        const int acc = i & 1;
        // the accumulator's previous tile is drained, and the columns shared with the last one
        if (!mbar_wait_bounded<true>(tempty_bar(acc), (uint32_t(i >> 1) & 1u) ^ 1u, abort_flag, p.status, p.timeout_ns)) break;
        if (i > 0 && !mbar_wait_bounded<true>(over_bar(acc ^ 1), uint32_t((i - 1) >> 1) & 1u, abort_flag, p.status, p.timeout_ns))
          break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc) * kAccStep;
        int32_t left = p.steps;
        for (int32_t kb = 0; kb < p.stages; ++kb) {
          // (a stage's scales are reported only once its codes have landed too)
          if (!seen && !mbar_wait_bounded<true>(sf_ready_bar(slot), sph, abort_flag, p.status, p.timeout_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a_lo = desc_lo + uint32_t(stage) * (kStage / 16), b_lo = a_lo + kPanelBytes / 16;
          const uint32_t sf = tmem + kSfCol + uint32_t(slot) * kSfCols<MX>;
          const uint32_t bar = empty_bar(stage);
          if (++slot == kSlots) {
            slot = 0;
            sph ^= 1u;
          }
          if (++stage == kPairStages) stage = 0;
          // instruction kk: 32 bytes of codes, its scales
          auto issue = [&](int kk) {
            const uint32_t c = sf + 12u * uint32_t(kk / kStepsPerTile<MX>);
            ptx::umma_fp4<true, MX>(d, a_lo + 2u * uint32_t(kk), b_lo + 2u * uint32_t(kk), ptx::kDescHiSw128,
                                    ptx::idesc_fp4(256, 256, MX, MX && (kk & 1) ? 2 : 0), c, c + 4, kk > 0 || kb > 0);
          };
          issue(0);
          if (left >= 4) {
            issue(1);
            issue(2);
            issue(3);
          } else {
            for (int kk = 1; kk < left; ++kk) issue(kk);
          }
          left -= 4;
          ptx::umma_commit_pair(bar, 0x3);
          // the next stage is looked at while these are under way
          seen = ptx::mbar_peek_cluster(sf_ready_bar(slot), sph);
          mma_issued = true;
        }
        if (!ok) break;
        ptx::umma_commit_pair(tfull_bar(acc), 0x3);
      }
    }
  } else if (warp == kSfLoader) {
    if (lane == 0) {
      // ------------------------------------------------------------ scale loads (both CTAs)
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int32_t t = first; ok && t < ntiles; t += step) {
        int32_t tm, tn;
        tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
        const int32_t ra = tm * 2 + int32_t(rank), rb = tn * 2;
        for (int32_t kb = 0; kb < p.stages; ++kb) {
          if (!mbar_wait_bounded(sf_empty_bar(stage), ph ^ 1u, abort_flag, p.status, p.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t sf = sf_base + uint32_t(stage) * 3u * kSfBytes<MX>;
          const uint32_t sfb = sf_full_bar(stage);
          const int32_t at = kb * kSfTiles<MX>;
          ptx::mbar_arrive_expect_tx(sfb, 3 * kSfBytes<MX>);
          ptx::tma_load_2d(sf, &p.sa, sfb, 0, (ra * p.tiles_k + at) * 2);
          ptx::tma_load_2d(sf + kSfBytes<MX>, &p.sb, sfb, 0, (rb * p.tiles_k + at) * 2);
          ptx::tma_load_2d(sf + 2 * kSfBytes<MX>, &p.sb, sfb, 0, ((rb + 1) * p.tiles_k + at) * 2);
          ++sf_issued;
          if (++stage == kSfStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp >= kSfWarp0) {
    // -------------------------------------------------------------- scales (both CTAs)
    // Lane l of every quarter holds, column by column, the scales of rows l, 32 + l, 64 + l, 96 + l
    // of a 512-byte tile: 16 consecutive bytes of it.
    // Warps 10-13 take every other stage, 14-17 the ones between: a stage's chain of waits, loads,
    // stores and the arrive is longer than its instructions.
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t total = first < ntiles ? uint32_t((ntiles - first + step - 1) / step) * uint32_t(p.stages) : 0u;
    for (uint32_t j = uint32_t(warp - kSfWarp0) >> 2; j < total; j += kSfGroups) {
      const uint32_t stage = j % kSfStages, slot = j % kSlots;
      bool ok = mbar_wait_bounded(sf_full_bar(int(stage)), (j / kSfStages) & 1u, abort_flag, p.status, p.timeout_ns);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const uint8_t* src = smem_raw + (sf_base - raw) + stage * 3u * kSfBytes<MX> + 16 * lane;
      uint32_t w[kSfCols<MX>];
#pragma unroll
      for (int a = 0; a < kSfTiles<MX>; ++a)
#pragma unroll
        for (int o = 0; o < 3; ++o)
          *reinterpret_cast<uint4*>(w + 12 * a + 4 * o) = *reinterpret_cast<const uint4*>(src + o * kSfBytes<MX> + 512 * a);
      if (j >= uint32_t(kSlots)) {   // the slot's last stage has been multiplied
        const uint32_t u = j - uint32_t(kSlots);
        ok = mbar_wait_bounded(empty_bar(int(u % kPairStages)), (u / kPairStages) & 1u, abort_flag, p.status, p.timeout_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
      }
      const uint32_t c = tmem + kSfCol + slot * kSfCols<MX> + lanes;
      ptx::tc_fence_after();
      ptx::tmem_st_32x32b_x16(c, w);
      if constexpr (MX) {
        ptx::tmem_st_32x32b_x8(c + 16, w + 16);
      } else {
        ptx::tmem_st_32x32b_x16(c + 16, w + 16);
        ptx::tmem_st_32x32b_x16(c + 32, w + 32);
      }
      // The shared memory goes back only after the stores: an arrive in front of them can pass loads
      // whose values nothing has used yet, and the next copy then overwrites what they read.
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sf_empty_bar(int(stage)));
      // The even CTA's warps report the stage when both CTAs' codes have landed as well, so that the
      // issuing thread has one barrier a stage to look at.
      if (leader) {
        ok = mbar_wait_bounded(full_bar(int(j % kPairStages)), (j / kPairStages) & 1u, abort_flag, p.status, p.timeout_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
      }
      // The TMEM stores are ordered by the wait and the fence above and the fence after the issuing
      // thread's wait, so the odd CTA's arrive is a relaxed one (8192^3 mx: 177 us; a cluster-scope
      // release in every stage nearly doubled the time). The even CTA's also passes on that the codes
      // have landed, to a thread of its own CTA. The issuing thread waits at cluster scope, which takes
      // 2% more than a wait at its own CTA's (173 us).
      if (lane == 0) {
        const uint32_t ready = ptx::mapa_shared(sf_ready_bar(int(slot)), 0);
        if (leader)
          ptx::mbar_arrive_remote_cta(ready);
        else
          ptx::mbar_arrive_remote_relaxed(ready);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const Factor scaled(p.amax_a, p.amax_b);
    uint32_t* turn = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + 384) + (warp - 2) * kTurnWords;
    int32_t i = 0;
    for (int32_t t = first; t < ntiles; t += step, ++i) {
      const int acc = i & 1;
      int32_t tm, tn;
      tile_at(t, p.tiles_m, p.tiles_n, tm, tn);
      bool ok = mbar_wait_bounded(tfull_bar(acc), uint32_t(i >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const int64_t row0 = int64_t(tm) * 256 + int64_t(rank) * 128 + quarter * 32;
      const int64_t col = int64_t(tn) * 256;
      const uint32_t tb = tmem + uint32_t(acc) * kAccStep + (uint32_t(quarter * 32) << 16);
      // Chunks of 32 columns, every other one each half's. Accumulator 0 ends in the shared columns
      // (chunks 7, 6, 5), accumulator 1 begins with them (0, 1, 2): each warp takes two chunks to
      // registers before it stores the first.
      auto chunk = [&](int s) { return acc == 0 ? 6 - 2 * s + half : 2 * s + half; };
#pragma unroll 1
      for (int s = 0; s < 4; s += 2) {
        uint32_t r[2][32];
        __syncwarp();
        ptx::tmem_ld_32x32b_x32(tb + uint32_t(chunk(s) * 32), r[0]);
        ptx::tmem_ld_32x32b_x32(tb + uint32_t(chunk(s + 1) * 32), r[1]);
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_relaxed(ptx::mapa_shared(s == 0 ? over_bar(acc) : tempty_bar(acc), 0));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t at = col + chunk(s + q) * 32;
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = scaled(__uint_as_float(r[q][j]));
          if (row0 < p.m && at < p.n) store_chunk(static_cast<O*>(p.out), row0, p.m, at, p.n, p.align, v, turn);
        }
      }
    }
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
    // CTAs count their bytes on its full barriers; at most the last kPairStages can be in flight).
    if (leader && warp == 1 && lane == 0 && mma_issued) {
      ptx::umma_commit_pair(drain_bar, 0x1);
      mbar_wait_drain(drain_bar, 0u, p.timeout_ns);
    }
    if (leader && threadIdx.x == 0) {
      const uint32_t L = n_issued, P = peer_report[1];
      const uint32_t most = L > P ? L : P;
      for (uint32_t j = most > uint32_t(kPairStages) ? most - uint32_t(kPairStages) : 0u; j < most; ++j) {
        const int s = int(j % uint32_t(kPairStages));
        if (j >= L)
          ptx::mbar_arrive_expect_tx(full_bar(s), kStage);   // only the peer's half is coming
        else if (j >= P)
          ptx::mbar_complete_tx(full_bar(s), kStage);        // the peer's half never will
        mbar_wait_drain(full_bar(s), (j / uint32_t(kPairStages)) & 1u, p.timeout_ns);
      }
    }
    // (each CTA's scales count on its own barriers)
    if (warp == kSfLoader && lane == 0)
      for (uint32_t j = sf_issued > uint32_t(kSfStages) ? sf_issued - uint32_t(kSfStages) : 0u; j < sf_issued; ++j)
        mbar_wait_drain(sf_full_bar(int(j % uint32_t(kSfStages))), (j / uint32_t(kSfStages)) & 1u, p.timeout_ns);
    ptx::cluster_sync();
  }
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ few rows
//
// A CTA multiplies 128 rows of B by NT rows of A over its part of K; the
// accumulator's lanes are the output's columns, so stores of a row of D are
// contiguous across lanes. The CTAs of a cluster hold the parts of one tile.
constexpr int kNarrowThreads = 192;
constexpr uint32_t kNarrowPitch = 132;   // of the fp32 sums [NT][128] in shared memory
template <int NT>
constexpr int kNarrowStages = NT <= 32 ? 4 : 3;   // two CTAs an SM
template <bool MX, int NT>
constexpr uint32_t kNarrowStageBytes = kPanelBytes + NT * (kStageK / 2) + 2 * kSfBytes<MX>;
template <bool MX, int NT>
constexpr size_t kNarrowSmem = 1024 + size_t(kNarrowStages<NT>) * kNarrowStageBytes<MX, NT> + 128;
template <int NT>
constexpr uint32_t kNarrowCols = NT <= 32 ? 64 : 2 * NT;   // TMEM: sums, then 8 columns of scales a tile
static_assert(2 * (kNarrowSmem<false, 128> + 1024) <= 228 * 1024 && 2 * kNarrowCols<128> <= 512, "two CTAs an SM");
static_assert(4 * kPanelBytes >= 32 * kNarrowPitch * 4 && 3 * (kPanelBytes + 64 * 128) >= 64 * kNarrowPitch * 4 &&
              3 * (kPanelBytes + 128 * 128) >= 128 * kNarrowPitch * 4, "sums in the stages' memory");

template <bool MX, int NT, typename O>
__global__ void __launch_bounds__(kNarrowThreads) fp4_narrow_kernel(const __grid_constant__ ProductParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr uint32_t kStage = kNarrowStageBytes<MX, NT>;
  constexpr int kStages = kNarrowStages<NT>;
  constexpr uint32_t kQBytes = NT * (kStageK / 2);
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sf_base = base + uint32_t(kStages) * (kPanelBytes + kQBytes);
  const uint32_t bars = sf_base + uint32_t(kStages) * 2u * kSfBytes<MX>;
  constexpr uint32_t kBars = 2 * kStages + 2;
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(smem_raw + (bars - raw) + 8 * kBars);
  uint32_t* tmem_slot = ctrl;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 1);
  float* sums = reinterpret_cast<float*>(smem_raw + (base - raw));
  auto full_bar = [&](int s) { return bars + 8u * uint32_t(s); };
  auto empty_bar = [&](int s) { return bars + 8u * uint32_t(kStages + s); };
  const uint32_t done_bar = bars + 8u * uint32_t(2 * kStages);
  const uint32_t drain_bar = bars + 8u * uint32_t(2 * kStages + 1);

  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  const uint32_t parts = gridDim.x / uint32_t(p.tiles_m * p.tiles_n);   // CTAs of a cluster
  const uint32_t rank = ptx::cluster_ctarank();
  const int32_t t = int32_t(blockIdx.x / parts);
  const int32_t tn = t / p.tiles_m, tm = t - tn * p.tiles_m;            // 128 columns of D, NT rows
  const int32_t k0 = int32_t(int64_t(p.stages) * rank / parts), k1 = int32_t(int64_t(p.stages) * (rank + 1) / parts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(done_bar, 1);
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_one(ptx::smem_addr(tmem_slot), kNarrowCols<NT>);
    ptx::tmem_relinquish_one();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_launch_dependents();   // after the TMEM is held, as above
  ptx::griddep_wait();
  const Factor scaled(p.amax_a, p.amax_b);

  uint32_t n_issued = 0;
  bool mma_issued = false;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      for (int32_t kb = k0; kb < k1; ++kb) {
        if (!mbar_wait_bounded(empty_bar(stage), ph ^ 1u, abort_flag, p.status, p.timeout_ns)) break;
        const uint32_t fb = full_bar(stage);
        ptx::mbar_arrive_expect_tx(fb, kStage);
        const uint32_t sp = base + uint32_t(stage) * (kPanelBytes + kQBytes);
        const uint32_t sf = sf_base + uint32_t(stage) * 2u * kSfBytes<MX>;
        ptx::tma_load_2d(sp, &p.b, fb, kb * 128, tn * 128);
        ptx::tma_load_2d(sp + kPanelBytes, &p.a, fb, kb * 128, tm * NT);
        const int32_t at = kb * kSfTiles<MX>;
        ptx::tma_load_2d(sf, &p.sb, fb, 0, (tn * p.tiles_k + at) * 2);
        ptx::tma_load_2d(sf + kSfBytes<MX>, &p.sa, fb, 0, (tm * p.tiles_k + at) * 2);
        ++n_issued;
        if (++stage == kStages) {
          stage = 0;
          ph ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      int32_t left = p.steps - 4 * k0;
      for (int32_t kb = k0; kb < k1; ++kb) {
        if (!mbar_wait_bounded(full_bar(stage), ph, abort_flag, p.status, p.timeout_ns)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sp = base + uint32_t(stage) * (kPanelBytes + kQBytes);
        const uint32_t sq = sp + kPanelBytes;
        const uint32_t sf = sf_base + uint32_t(stage) * 2u * kSfBytes<MX>;
#pragma unroll
        for (int a = 0; a < kSfTiles<MX>; ++a) {
          const uint32_t c = tmem + uint32_t(kNarrowCols<NT> == 64 ? 32 : NT) + uint32_t(a) * 8u;
          if (left > a * kStepsPerTile<MX>) {
            ptx::tmem_copy_scales(c, ptx::smem_desc_scales(sf + 512u * uint32_t(a)));
            ptx::tmem_copy_scales(c + 4, ptx::smem_desc_scales(sf + kSfBytes<MX> + 512u * uint32_t(a)));
          }
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < left) {
            const int a = kk / kStepsPerTile<MX>;
            const uint32_t c = tmem + uint32_t(kNarrowCols<NT> == 64 ? 32 : NT) + uint32_t(a) * 8u;
            ptx::umma_fp4<false, MX>(tmem, ptx::desc_lo_sw128(sp) + 2u * uint32_t(kk), ptx::desc_lo_sw128(sq) + 2u * uint32_t(kk),
                                     ptx::kDescHiSw128, ptx::idesc_fp4(128, NT, MX, MX && (kk & 1) ? 2 : 0), c, c + 4,
                                     kb > k0 || kk > 0);
          }
        }
        left -= 4;
        ptx::umma_commit_one(empty_bar(stage));
        mma_issued = true;
        if (++stage == kStages) {
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
      // lane l of a quarter holds column quarter 32 + l of the output. A CTA by itself stores it at
      // once; the parts of a cluster's tile go to the memory of the stages, which have all been read.
      const int64_t n_at = int64_t(tn) * 128 + quarter * 32 + lane;
      O* out = static_cast<O*>(p.out) + int64_t(tm) * NT * p.n + n_at;
      const int rows = int(min(int64_t(NT), p.m - int64_t(tm) * NT));
#pragma unroll 1
      for (int c = 0; c < rows; c += 16) {
        uint32_t r[16];
        __syncwarp();
        ptx::tmem_ld_32x32b_x16(tmem + uint32_t(c) + (uint32_t(quarter * 32) << 16), r);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (parts > 1)
            sums[uint32_t(c + j) * kNarrowPitch + uint32_t(quarter * 32 + lane)] = __uint_as_float(r[j]);
          else if (c + j < rows && n_at < p.n)
            put(out + int64_t(c + j) * p.n, scaled(__uint_as_float(r[j])));
        }
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
      for (uint32_t j = n_issued > uint32_t(kStages) ? n_issued - uint32_t(kStages) : 0u; j < n_issued; ++j)
        mbar_wait_drain(full_bar(int(j % uint32_t(kStages))), (j / uint32_t(kStages)) & 1u, p.timeout_ns);
    __syncthreads();
  }
  if (parts > 1) {
    ptx::cluster_sync();   // every part's sums are in place
    const uint32_t sums_addr = ptx::smem_addr(sums);
    const int64_t row0 = int64_t(tm) * NT, col0 = int64_t(tn) * 128;
    const bool vec = (p.n & 3) == 0;
    // this CTA's share of the tile, four columns a thread, parts added in rank order
    const uint32_t rows = uint32_t(min(int64_t(NT), p.m - row0)), share = (rows * 32u + parts - 1u) / parts;
    const uint32_t end = min(rows * 32u, (rank + 1u) * share);
    for (uint32_t i = rank * share + threadIdx.x; i < end; i += kNarrowThreads) {
      const uint32_t j = i >> 5, l = 4u * (i & 31u);
      float4 v[8];
#pragma unroll
      for (uint32_t s = 0; s < 8; ++s)
        if (s < parts) v[s] = ptx::ld_shared_cluster_v4(ptx::mapa_shared(sums_addr + 4u * (j * kNarrowPitch + l), s));
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (uint32_t s = 0; s < 8; ++s)
        if (s < parts) {
          t.x += v[s].x;
          t.y += v[s].y;
          t.z += v[s].z;
          t.w += v[s].w;
        }
      O* o = static_cast<O*>(p.out) + (row0 + j) * p.n + col0 + l;
      const float f[4] = {scaled(t.x), scaled(t.y), scaled(t.z), scaled(t.w)};
      if (vec && col0 + l + 4 <= p.n) {
        if constexpr (sizeof(O) == 2)
          *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
        else
          *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (col0 + l + q < p.n) put(o + q, f[q]);
      }
    }
    ptx::cluster_sync();   // the peers have read this CTA's sums
  }
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_one(tmem, kNarrowCols<NT>);
}

// ------------------------------------------------------------------ launches

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

// Codes as bytes [rows, pitch], boxes of 128 bytes (256 elements) by box_rows.
bool encode_codes(EncodeTiledFn enc, CUtensorMap* map, const Fp4In& q, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cuuint64_t(q.pitch), cuuint64_t(q.rows)};
  const cuuint64_t strides[1] = {cuuint64_t(q.pitch)};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q.codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as lines of 256 bytes, two a tile; a box is a stage's tiles of
// one 128-row panel. A box may run into the next panel's tiles (not used) or
// past the end (zeros).
bool encode_scales(EncodeTiledFn enc, CUtensorMap* map, const Fp4In& q, uint32_t tiles) {
  const cuuint64_t dims[2] = {64, cuuint64_t(q.tiles_r * q.tiles_k * 2)};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {64, 2 * tiles};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(q.scales), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A has more than one tile of rows only with NT = 128, so a tile's scales begin a scale tile; every
// CTA of a cluster has at least two stages.
template <bool MX, int NT, typename O>
cudaError_t narrow_as(ProductParams& p, int sms, cudaStream_t stream) {
  p.tiles_m = int32_t((p.m + NT - 1) / NT);
  p.tiles_n = int32_t((p.n + 127) / 128);
  const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
  // K in as many parts as leave all clusters resident (two CTAs an SM; clusters of 4 and 8 do not
  // fill the GPU's parts evenly: 72 of 76 and 30 of 38 fit on 152 SMs) and two stages for each CTA
  const int64_t most[4] = {0, sms, int64_t(sms) * 45 / 100, int64_t(sms) * 18 / 100};
  unsigned parts = 1;
  for (int i = 1; i < 4 && tiles <= most[i] && p.stages >= (2 << i); ++i) parts = 1u << i;
  auto kern = fp4_narrow_kernel<MX, NT, O>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kNarrowSmem<MX, NT>);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(unsigned(tiles * parts)), dim3(kNarrowThreads), kNarrowSmem<MX, NT>, parts, true, stream, p);
}

template <bool MX, typename O>
cudaError_t product_as(ProductParams& p, const Fp4In& a, const Fp4In& b, int sms, cudaStream_t stream) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const int64_t pairs = sms / 2;
  const int64_t pair_tiles = ((p.m + 255) / 256) * ((p.n + 255) / 256);
  // Few rows of A, or a long K and fewer tiles than half of the pairs: splitting K beats wider tiles
  // (1 x 4096 x 14336: 12 against 26 us, 128 x 4096 x 14336: 17 against 26; 1024 x 1024 x 1024, not
  // split: 11 against 8).
  const bool narrow = p.m <= 64 || (pair_tiles * 2 < pairs && p.stages >= 24);
  const uint32_t nt = !narrow ? 128 : p.m <= 16 ? 16 : p.m <= 32 ? 32 : p.m <= 64 ? 64 : 128;
  if (!encode_codes(enc, &p.a, a, nt) || !encode_codes(enc, &p.b, b, 128) ||
      !encode_scales(enc, &p.sa, a, kSfTiles<MX>) || !encode_scales(enc, &p.sb, b, kSfTiles<MX>))
    return cudaErrorInvalidValue;
  if (narrow) {
    if (nt == 16) return narrow_as<MX, 16, O>(p, sms, stream);
    if (nt == 32) return narrow_as<MX, 32, O>(p, sms, stream);
    if (nt == 64) return narrow_as<MX, 64, O>(p, sms, stream);
    return narrow_as<MX, 128, O>(p, sms, stream);
  }
  p.tiles_m = int32_t((p.m + 255) / 256);
  p.tiles_n = int32_t((p.n + 255) / 256);
  const unsigned grid = unsigned(2 * std::min(pairs, pair_tiles));
  auto kern = fp4_pair_kernel<MX, O>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kPairSmem<MX>);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid), dim3(kPairThreads), kPairSmem<MX>, 2, true, stream, p);
}

}  // namespace

cudaError_t launch_fp4_product(const Fp4In& a, const Fp4In& b, bool mx, void* out, bool out_bf16, int sms, int* status,
                               cudaStream_t stream) {
  ProductParams p = {};
  p.out = out;
  p.amax_a = a.amax;
  p.amax_b = b.amax;
  p.status = status;
  p.m = a.rows;
  p.n = b.rows;
  p.steps = int32_t((a.k + 63) / 64);
  p.stages = int32_t((a.k + kStageK - 1) / kStageK);
  p.tiles_k = int32_t(a.tiles_k);
  p.timeout_ns = kDefaultTimeoutNs;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(out) | uintptr_t(p.n * (out_bf16 ? 2 : 4));
  p.align = (mis & 31) == 0 ? 32 : (mis & 15) == 0 ? 16 : 0;
  if (out_bf16) return mx ? product_as<true, uint16_t>(p, a, b, sms, stream) : product_as<false, uint16_t>(p, a, b, sms, stream);
  return mx ? product_as<true, float>(p, a, b, sms, stream) : product_as<false, float>(p, a, b, sms, stream);
}

}  // namespace mo
