// Launch interface between the entry points of the feed-forward operators
// (layer_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mo.h"
#include "train_kernels.h"

namespace mo {

// A tensor [rows, k] as a kernel reads or writes it: elements, dense, or e4m3
// codes in rows of 32 ceil(k / 32) bytes with ceil(k / 32) scales a row.
struct Kept {
  void* data = nullptr;      // null: not there
  uint8_t* scales = nullptr;
  int32_t dtype = MO_BF16;
};
inline int64_t mx8_blocks(int64_t k) { return (k + 31) / 32; }

// Row pitch, in elements, of the bf16 matrices that the operators keep in
// their workspaces: whole 128-byte lines, so that a chunk of 32 columns is
// stored as it is.
inline int64_t padded(int64_t cols) { return (cols + 63) / 64 * 64; }

// ---------------------------------------------------------------- 8-bit tensors
// q = x in 8 bits.
cudaError_t launch_mx8_quantize(const void* x, bool bf16, int64_t rows, int64_t k, const Kept& q, cudaStream_t stream);
// out [rows, k] = the values of the 8-bit src.
cudaError_t launch_unpack(const Kept& src, int64_t rows, int64_t k, void* out, bool out_bf16, cudaStream_t stream);

// Operands of products, 8 bits or bf16 [rows, cols], as bf16 in rows of `ld`
// elements (a multiple of 8): up to three in one launch.
struct LayOut {
  Kept src;
  int64_t rows, cols;
  uint16_t* out;
  int64_t ld;
};
cudaError_t launch_lay_out(const LayOut* t, int count, cudaStream_t stream);

// dz [tokens, ld] = dout act'(pre), and part [parts, rows] its column sums over
// `per` tokens each. dz null: no output; act 0: dz is dout.
struct ActGradParams {
  const uint16_t* dout;
  Kept pre;
  uint16_t* dz;
  float* part;
  int64_t tokens, rows, ld;
  int64_t per;
  int32_t act;
  int32_t early;   // directly behind launch_lay_out, and may run beside it
};
cudaError_t launch_act_grad(const ActGradParams& p, cudaStream_t stream);
// out[i] (+)= the sum over part[0..parts)[i], in order.
cudaError_t launch_join(const float* part, int64_t parts, int64_t n, float* out, bool accumulate, cudaStream_t stream);

// Parts of launch_act_grad at most: 608 blocks (four an SM at 152, a number that
// does not depend on the device). A block is 256 columns wide, so few parts do for
// wide rows.
inline int64_t act_grad_most(int64_t rows) { return std::max<int64_t>(1, 608 / ((rows + 255) / 256)); }
// Tokens that a block takes, a multiple of 8.
inline int64_t act_grad_per(int64_t tokens, int64_t rows) {
  const int64_t parts = act_grad_most(rows);
  return std::max<int64_t>(8, ((tokens + parts - 1) / parts + 7) / 8 * 8);
}
// Parts that `tokens` or fewer need: more than `tokens` make where their blocks have
// just grown (4865 tokens of 256 columns: 305 parts, 4864: 608).
inline int64_t act_grad_room(int64_t tokens, int64_t rows) { return std::min((tokens + 7) / 8, act_grad_most(rows)); }

// ---------------------------------------------------------------- norm
struct NormParams {
  const void* x;
  const void* residual;   // or null
  const float* weight;    // or null: ones
  void* sum;              // or null
  void* out;              // or null
  Kept out8;
  int64_t rows, dim;
  float eps;
  int32_t out_bf16;
};
cudaError_t launch_rms_norm(const NormParams& p, bool bf16, cudaStream_t stream);

struct NormGradParams {
  const void* dy;
  Kept x;                 // of dy's type, or 8 bits
  const float* weight;    // or null: ones
  const void* dres;       // or null
  void* dx;
  float* part;            // [norm_parts(rows, dim), dim], or null: no gradient of the weight
  int64_t rows, dim;
  float eps;
};
// Rows of `part`: one for every team of threads that takes rows in turn.
int64_t norm_parts(int64_t rows, int64_t dim);
cudaError_t launch_rms_norm_grad(const NormGradParams& p, bool bf16, cudaStream_t stream);

// ---------------------------------------------------------------- products
// A bf16 operand of a product in memory: [rows, cols] with `ld` elements from
// row to row (a multiple of 8, base 16-byte aligned).
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
};

// What becomes of the sums.
enum Epilogue : int32_t {
  kEpiLinear,      // out = act(sum + bias) + add; pre = sum + bias
  kEpiGated,       // gate and up sums: out = act(g) u; pre = g, pre2 = u
  kEpiGatedGrad    // sum = dh: out = dh u act'(g), out2 = dh act(g), out3 = act(g) u, from pre = g, pre2 = u
};

struct Target {
  void* out;
  const void* add;     // or null
  int64_t m, n;        // rows and columns
  int64_t ld, add_ld;  // elements from row to row
  int32_t out_bf16, add_bf16;
};

// Up to three products with the same reduction length (one a target), or one
// product whose reduction runs over up to two pairs of operands.
struct Product {
  Epilogue epi = kEpiLinear;
  int32_t act = 0;
  bool a_mn = false, b_mn = false;   // the operand's rows run along the reduction
  int count = 1;                     // targets
  int segments = 1;                  // pairs of operands that one reduction runs over
  Operand a[3], b[3];                // kEpiGated: b[0] gate, b[1] up
  Target t[3];
  int64_t k = 0;
  const float* bias = nullptr;
  Kept pre, pre2;
  // sums so far, fp32 [m, padded(n)], which the product's are added to (kEpiGated: gate's and up's); one target
  const float* start[2] = {nullptr, nullptr};
  uint16_t* out2 = nullptr;          // kEpiGatedGrad, pitch t[0].ld
  uint16_t* out3 = nullptr;
  // b may be read while the previous launch runs: that launch is a product for which is_narrow or is_few
  // holds, and does not write b
  bool early = false;
};
// The most products that one accumulator of the tensor cores takes (0: the product does not use them).
int64_t longest_sum(const Product& q, int sms);
// Whether a product goes to the kernel for one or two rows, and otherwise to the one for few.
bool is_few(const Product& q, int sms);
bool is_narrow(const Product& q, int sms);
cudaError_t launch_product(const Product& p, int sms, int* status, cudaStream_t stream);

}  // namespace mo
