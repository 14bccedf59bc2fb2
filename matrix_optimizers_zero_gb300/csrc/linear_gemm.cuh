// What the two kernels of the bf16 products share: their parameters and the
// epilogue of a chunk of 32 columns.
#pragma once

#include <cuda.h>

#include "activation.cuh"
#include "layer_kernels.h"
#include "ptx_train.cuh"

namespace mo {

constexpr int kBlockK = 64;   // elements of the reduction a stage: 128 bytes, one swizzle row
constexpr uint32_t kBox = 64 * 64 * 2;

struct GemmTarget {
  void* out;
  const void* add;
  int64_t m, n, ld, add_ld;
  int32_t tiles_m, tiles_n, tile0;
  int32_t align;                 // of the rows of out and add: 32, 16 or 0 (elements)
  int32_t out_bf16, add_bf16;
  int32_t bulk;                  // pairs: out is stored by TMA
};

struct GemmParams {
  CUtensorMap a[3], b[3];
  CUtensorMap bs[3];             // pairs, K-major: b in boxes of 32 rows, for cut tiles
  CUtensorMap so[3], sk[2];      // pairs: boxes of 32 rows of a chunk of the outputs, and of what is kept
  GemmTarget t[3];
  int32_t count, segments;
  int32_t blocks;                // stages a segment
  int32_t tiles;                 // of all targets; pairs: with the cut ones counted as their parts
  int32_t whole;                 // pairs: tiles that are not cut, in front of the others
  int32_t cut;                   // pairs: parts of the others, side by side: 1, 2 or 4
  int32_t stages;                // of shared memory
  int32_t early;                 // narrow: the columns' operand may be read before the previous launch has ended
  int32_t act;
  const float* bias;
  const float* start[2];         // sums so far, or null
  int64_t start_ld;
  Kept pre, pre2;
  int32_t pre_align;             // of bf16 rows, as above; of 8-bit codes 32 or 16
  int32_t pre_bulk;              // pairs: they are stored by TMA
  uint16_t* out2;
  uint16_t* out3;
  int* status;
  uint64_t timeout_ns;
};

// The target of a tile, in order.
__device__ __forceinline__ int target_of(const GemmParams& p, int32_t tile) {
  return p.count > 2 && tile >= p.t[2].tile0 ? 2 : p.count > 1 && tile >= p.t[1].tile0 ? 1 : 0;
}

// Tiles in groups of 8 tile rows, column by column: those in flight share
// operand panels.
__device__ __forceinline__ void tile_at(const GemmTarget& t, int32_t tile, int32_t& tm, int32_t& tn) {
  const int32_t i = tile - t.tile0;
  const int32_t group = i / (8 * t.tiles_n), first = group * 8;
  const int32_t height = min(8, t.tiles_m - first), in = i - group * 8 * t.tiles_n;
  tm = first + in % height;
  tn = in / height;
}

// A warp's scratch of 16 columns of fp32: rows of 16 words, each a word apart
// from the next.
constexpr uint32_t kTurn = 17 * 32;

__device__ __forceinline__ void load32(const uint16_t* p, int align, float (&v)[32]) {
  uint32_t w[16];
  if (align == 32) {
    ptx::ld_global_v8(p, *reinterpret_cast<uint32_t (*)[8]>(&w[0]));
    ptx::ld_global_v8(p + 16, *reinterpret_cast<uint32_t (*)[8]>(&w[8]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[j];
      w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load32(const float* p, int align, float (&v)[32]) {
  if (align == 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[8];
      ptx::ld_global_v8(p + 8 * q, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * q + j] = __uint_as_float(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 q = reinterpret_cast<const float4*>(p)[j];
      v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
    }
  }
}

__device__ __forceinline__ void store32(uint16_t* p, int align, const float (&v)[32]) {
  uint32_t w[2][8];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j >> 3][j & 7] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  if (align == 32) {
    ptx::st_global_v8(p, w[0]);
    ptx::st_global_v8(p + 16, w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<uint4*>(p)[j] =
          make_uint4(w[j >> 1][4 * (j & 1)], w[j >> 1][4 * (j & 1) + 1], w[j >> 1][4 * (j & 1) + 2], w[j >> 1][4 * (j & 1) + 3]);
  }
}

__device__ __forceinline__ void store32(float* p, int align, const float (&v)[32]) {
  if (align == 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * q + j]);
      ptx::st_global_v8(p + 8 * q, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      reinterpret_cast<float4*>(p)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  }
}

// act of 32 (or 16) numbers, and times u
template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = ptx::parts(act_value<ACT>(ptx::f2(v[i], v[i + 1])));
    v[i] = y.x;
    v[i + 1] = y.y;
  }
}
template <int ACT, int N>
__device__ __forceinline__ void gate_all(float (&g)[N], const float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = ptx::parts(ptx::mul2(act_value<ACT>(ptx::f2(g[i], g[i + 1])), ptx::f2(u[i], u[i + 1])));
    g[i] = y.x;
    g[i + 1] = y.y;
  }
}
// dg, du and h of g, u and dh, in their places
template <int ACT, int N>
__device__ __forceinline__ void gate_grad_all(float (&g)[N], float (&u)[N], float (&dh)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const F2 u2 = ptx::f2(u[i], u[i + 1]), d2 = ptx::f2(dh[i], dh[i + 1]);
    F2 a;
    const F2 slope = act_slope<ACT>(ptx::f2(g[i], g[i + 1]), &a);
    const float2 dg = ptx::parts(ptx::mul2(ptx::mul2(d2, u2), slope)), du = ptx::parts(ptx::mul2(d2, a)), h = ptx::parts(ptx::mul2(a, u2));
    g[i] = dg.x, g[i + 1] = dg.y;
    dh[i] = du.x, dh[i + 1] = du.y;
    u[i] = h.x, u[i + 1] = h.y;
  }
}

__device__ __forceinline__ void put(void* out, bool bf16, int64_t at, float v) {
  if (bf16)
    store1(static_cast<uint16_t*>(out) + at, v);
  else
    store1(static_cast<float*>(out) + at, v);
}
__device__ __forceinline__ float get(const void* p, bool bf16, int64_t at) {
  return bf16 ? load1(static_cast<const uint16_t*>(p) + at) : load1(static_cast<const float*>(p) + at);
}

// Stores a chunk of 32 columns, a row a lane, of the 32 rows from `row0` on,
// plus the chunk of `add`. Rows that are 16-byte aligned and a whole chunk:
// vectors. Others (an odd n, the last columns) are turned in shared memory, 16
// columns at a time, and stored two rows an instruction.
__device__ __forceinline__ void store_chunk(void* out, bool out_bf16, int64_t ld, const void* add, bool add_bf16, int64_t add_ld,
                                            int align, int64_t row0, int64_t m, int64_t col, int64_t n, float (&v)[32],
                                            float* turn) {
  const int lane = int(threadIdx.x & 31);
  if (align != 0 && col + 32 <= n) {
    const int64_t row = row0 + lane;
    if (row >= m) return;
    if (add != nullptr) {
      float x[32];
      if (add_bf16)
        load32(static_cast<const uint16_t*>(add) + row * add_ld + col, align, x);
      else
        load32(static_cast<const float*>(add) + row * add_ld + col, align, x);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += x[i];
    }
    if (out_bf16)
      store32(static_cast<uint16_t*>(out) + row * ld + col, align, v);
    else
      store32(static_cast<float*>(out) + row * ld + col, align, v);
    return;
  }
  const int rows = int(min(int64_t(32), m - row0));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) turn[lane * 17 + j] = v[16 * h + j];
    __syncwarp();
    const int64_t c = col + 16 * h + (lane & 15);
    if (c < n) {
#pragma unroll 4
      for (int r = lane >> 4; r < rows; r += 2) {
        float x = turn[r * 17 + (lane & 15)];
        if (add != nullptr) x += get(add, add_bf16, (row0 + r) * add_ld + c);
        put(out, out_bf16, (row0 + r) * ld + c, x);
      }
    }
  }
}

// A chunk in 8 bits: codes and scale.
__device__ __forceinline__ uint32_t mx8_chunk(const float (&v)[32], uint32_t (&w)[8]) {
  float top = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 31; i += 2) top = top3(top, v[i], v[i + 1]);
  top = top2(top, fabsf(v[31]));
  const uint32_t s = mx8_scale(top);
  const F2 down = ptx::f2(mx8_down(s));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = ptx::parts(ptx::mul2(ptx::f2(v[4 * i], v[4 * i + 1]), down));
    const float2 b = ptx::parts(ptx::mul2(ptx::f2(v[4 * i + 2], v[4 * i + 3]), down));
    w[i] = cvt_e4m3x4(a.x, a.y, b.x, b.y);
  }
  return s;
}

// A lane's row of a box of 32 rows, swizzled as the tensor map is: its 16-byte
// pieces change places from row to row, so that the lanes meet all banks.
template <int BYTES>
__device__ __forceinline__ void put_row(uint32_t box, const uint32_t (&w)[BYTES / 4]) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t turn = BYTES == 64 ? (lane >> 1) & 3u : (lane >> 2) & 1u;
#pragma unroll
  for (uint32_t i = 0; i < BYTES / 16; ++i)
    ptx::st_shared_v4(box + lane * BYTES + ((i ^ turn) * 16u), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}
template <int N>
__device__ __forceinline__ void put_bf16(uint32_t box, const float (&v)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  put_row<2 * N>(box, w);
}

// Keeps a chunk, in 8 bits or in bf16: into `box` for the copy that follows (bulk;
// the scales go out at once), or as it is.
__device__ __forceinline__ void keep_chunk(const Kept& q, bool bulk, int align, int64_t row0, int64_t m, int64_t col, int64_t n,
                                           float (&v)[32], uint32_t box, float* turn) {
  if (q.dtype != MO_MX8) {
    if (bulk) {
      put_bf16(box, v);
    } else {
      float x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = v[i];
      store_chunk(q.data, true, n, nullptr, false, 0, align, row0, m, col, n, x, turn);
      __syncwarp();
    }
    return;
  }
  // (rows of codes are 16-byte aligned, and always bulk; past n a sum is 0, or NaN where its row's operand
  // is not finite)
  if (col + 32 > n) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i >= n) v[i] = 0.0f;
  }
  uint32_t w[8];
  const uint32_t s = mx8_chunk(v, w);
  put_row<32>(box, w);
  const int64_t row = row0 + int64_t(threadIdx.x & 31), nb = (n + 31) / 32;
  if (row < m) q.scales[row * nb + (col >> 5)] = uint8_t(s);
}

// 16 kept columns' raw words, loaded ahead of their use: 8-bit codes in the first
// four and the scale, or bf16. bf16 that is not a whole chunk or not aligned is
// read element by element.
struct RawChunk {
  uint32_t w[8];
  uint32_t scale;
};
__device__ __forceinline__ void fetch_kept(const Kept& q, int align, int64_t row, int64_t col, int64_t n, RawChunk& raw) {
  if (q.dtype == MO_MX8) {
    const int64_t nb = (n + 31) / 32;
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(q.data) + row * nb * 32 + col);
    raw.w[0] = a.x, raw.w[1] = a.y, raw.w[2] = a.z, raw.w[3] = a.w;
    raw.scale = q.scales[row * nb + (col >> 5)];
  } else {
    const uint16_t* o = static_cast<const uint16_t*>(q.data) + row * n + col;
    if (align != 0 && col + 16 <= n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 a = reinterpret_cast<const uint4*>(o)[j];
        raw.w[4 * j] = a.x, raw.w[4 * j + 1] = a.y, raw.w[4 * j + 2] = a.z, raw.w[4 * j + 3] = a.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        raw.w[j] = (col + 2 * j < n ? uint32_t(o[2 * j]) : 0u) | (col + 2 * j + 1 < n ? uint32_t(o[2 * j + 1]) << 16 : 0u);
    }
  }
}
__device__ __forceinline__ void kept_values(const Kept& q, const RawChunk& raw, float (&v)[16]) {
  if (q.dtype == MO_MX8) {
    const float up = mx8_up(raw.scale);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      e4m3x4_values(raw.w[j], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * j + i] = x[i] * up;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = __uint_as_float(raw.w[j] << 16);
      v[2 * j + 1] = __uint_as_float(raw.w[j] & 0xFFFF0000u);
    }
  }
}
// One element of a kept tensor of rows of n.
__device__ __forceinline__ float kept_at(const Kept& q, int64_t row, int64_t col, int64_t n) {
  if (q.dtype == MO_MX8) {
    const int64_t nb = (n + 31) / 32;
    return e4m3_value(static_cast<const uint8_t*>(q.data)[row * nb * 32 + col]) * mx8_up(q.scales[row * nb + (col >> 5)]);
  }
  return load1(static_cast<const uint16_t*>(q.data) + row * n + col);
}

// The sums so far of N columns of a row, added; rows of a multiple of 64, so all of them are there.
template <int N>
__device__ __forceinline__ void add_start(const float* p, float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const float4 x = reinterpret_cast<const float4*>(p)[j];
    v[4 * j] += x.x, v[4 * j + 1] += x.y, v[4 * j + 2] += x.z, v[4 * j + 3] += x.w;
  }
}

// Few rows: tiles of 128 columns, the reduction split over clusters.
int64_t narrow_parts(const Product& q, int sms);   // of the reduction
cudaError_t launch_narrow(const Product& q, GemmParams& p, int sms, cudaStream_t stream);
cudaError_t launch_few(const Product& q, int sms, cudaStream_t stream);
bool encode_operand(CUtensorMap* map, const Operand& o, uint32_t box_rows);

}  // namespace mo
