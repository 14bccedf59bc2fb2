// Launch interface between the entry points of the training-step operators
// (train_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mo.h"
#include "philox.cuh"

namespace mo {

// ---------------------------------------------------------------- shared with abi.cu
// The current device's SM count and status word; MO_OK or an error status.
int current_device(int* sms, int** status);
// Records a failing runtime call for mo_last_cuda_error; MO_ERR_CUDA.
int report_cuda(cudaError_t e);

// ---------------------------------------------------------------- dropout, embedding
struct DropoutParams {
  const void* x;
  const void* residual;   // or null
  void* y;
  int64_t n;
  DropArgs drop;
};
cudaError_t launch_dropout(const DropoutParams& p, bool bf16, cudaStream_t stream);

struct TokenArgs {
  const void* ids;
  int64_t n;
  int64_t padding;   // index without a gradient, or -1
  int32_t wide;      // 64-bit indexes
};

struct LookupParams {
  const void* table;
  const void* add;       // rows added to token t's: t mod add_rows; or null
  void* out;
  int* status;
  int64_t vocab, dim, add_rows;
  TokenArgs tokens;
  DropArgs drop;
  float scale;
};
cudaError_t launch_embed_lookup(const LookupParams& p, bool table_bf16, bool out_bf16, int sms, cudaStream_t stream);

// Bits a pass of the gradient's radix sort: the fewest passes of at most
// kMaxDigitBits, then the fewest bits.
constexpr int kMaxDigitBits = 9;
constexpr int kMaxChunk = 64;
constexpr int64_t kZeroRowsMost = 4096;   // rows a block of launch 2 zeroes, at most

// From kManyTokens on the sort takes all SMs and three launches a pass; fewer
// are one cluster's in one launch. (65536 x 1024 of 50257 rows: uniform tokens
// 104 us by the cluster, 87 so, one token for all 80 and 83.) A part is a
// block of 32 warps, one part an SM: with 1024 small parts 2^20 x 64 takes 247
// us instead of 199, with 16 large ones 65536 x 1024 takes 94 instead of 85.
// (152 SMs, here and in grad_grid's four blocks for each: the workspace's size is
// computed on the host alone and results do not depend on the device, so neither
// asks it for its count.)
constexpr int64_t kManyTokens = 65536;
struct SortParts {
  int64_t per_warp;   // positions, a multiple of 32
  int32_t parts;
};
inline SortParts sort_parts(int64_t n) {
  if (n < kManyTokens) return {0, 0};
  const int64_t per_warp = (n + 152 * 1024 - 1) / (152 * 1024) * 32;
  return {per_warp, int32_t((n + 32 * per_warp - 1) / (32 * per_warp))};
}

// Launch shape of the gradient's sums: chunks of sorted positions by blocks of
// columns (eight a thread, or one where dim is not a multiple of 8). A chunk
// is 64 positions, fewer where that leaves too few blocks to fill the GPU.
struct GradGrid {
  int64_t chunk, chunks, col_blocks;
  int threads;
};
inline GradGrid grad_grid(int64_t n, int64_t dim) {
  GradGrid g;
  const int64_t items = (dim & 7) == 0 ? dim / 8 : dim;
  g.col_blocks = (items + 255) / 256;
  const int64_t per = (items + g.col_blocks - 1) / g.col_blocks;
  g.threads = int((per + 31) / 32 * 32);
  g.chunk = kMaxChunk;
  while (g.chunk > 8 && (n + g.chunk - 1) / g.chunk * g.col_blocks < 608) g.chunk /= 2;
  g.chunks = (n + g.chunk - 1) / g.chunk;
  return g;
}

struct GradParams {
  const void* dout;
  float* grad;
  int* status;
  uint32_t* key[2];       // [n] each; the sorted keys are in key[(passes - 1) & 1]
  uint32_t* pos[2];
  uint32_t* counter;      // arrivals of the join: two per slot and column block
  float* partial;         // [2 chunks, dim_pad] sums of tokens that cross chunks
  uint32_t* part_count;   // many tokens: [bins, parts] digit counts, then offsets
  uint32_t* bin_count;    // [bins]
  int64_t per_warp;       // positions of a warp of a part
  int32_t parts;          // 0: one cluster sorts
  int64_t counters;
  int64_t vocab, dim, dim_pad, chunk, chunks;
  int64_t zero_first;     // rows that launch 1 zeroes; launch 2 zeroes those of the others that no token names,
  int64_t zero_rows;      // so many a block
  TokenArgs tokens;
  DropArgs drop;
  float factor;           // scale times the dropout's factor
  int32_t passes;         // of the sort
  int32_t digit_bits;
  int32_t accumulate;
};
cudaError_t launch_embed_grad(const GradParams& p, bool dout_bf16, cudaStream_t stream);

// ---------------------------------------------------------------- 4-bit tensors
// Storage of a 4-bit tensor [rows, k]: codes, two a byte (the even element in
// the low half), rows of `pitch` = 16 ceil(k / 32) bytes; scales in tiles of
// 128 rows by 4 blocks, the 512-byte order that the tensor core's scale copy
// takes: row r, block b of a tile at byte (r % 32) 16 + (r / 32) 4 + b.
struct Fp4Out {
  uint8_t* codes;          // null: this orientation is not wanted
  uint8_t* scales;
  float* amax;             // nv: receives the magnitude that fixes the tensor's scale
  int64_t rows, k, pitch;
  int64_t tiles_r, tiles_k;
};
struct Fp4In {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* amax;       // or null: the tensor's own scale is 1
  int64_t rows, k, pitch;
  int64_t tiles_r, tiles_k;
};

constexpr int kQuantTile = 64;   // rows and columns of x a block takes
struct QuantParams {
  const void* x;           // [rows, cols]
  const float* amax;       // nv: its largest magnitude
  int64_t rows, cols, tiles_c;
  Fp4Out row, col;         // blocks along the rows of x, and along its columns (transposed)
  RandomArgs rnd;          // of stochastic rounding
  int32_t vec;             // rows are 16-byte aligned
  int32_t measured;        // the launch before this one, a normal one, writes *amax
};
cudaError_t launch_fp4_quantize(const QuantParams& p, bool bf16, bool mx, bool stochastic, cudaStream_t stream);
cudaError_t launch_fp4_amax(const void* x, bool bf16, int64_t n, float* amax, int sms, cudaStream_t stream);
cudaError_t launch_fp4_dequantize(const Fp4In& q, bool mx, void* out, bool out_bf16, cudaStream_t stream);
// out [a.rows, b.rows] = A B^T; a.k == b.k.
cudaError_t launch_fp4_product(const Fp4In& a, const Fp4In& b, bool mx, void* out, bool out_bf16, int sms, int* status,
                               cudaStream_t stream);

}  // namespace mo
