// extern "C" entry points of the training-step operators around the
// optimizer (include/mo.h): argument checks, workspace layout, launches. No
// entry point allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <cmath>

#include "mo.h"
#include "train_kernels.h"

namespace {

using mo::report_cuda;

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxVocab = (int64_t(1) << 31) - 2;
constexpr int64_t kMaxDim = int64_t(1) << 22;
constexpr int64_t kMaxElems = int64_t(1) << 42;

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool dtype_ok(int32_t d) { return d == MO_F32 || d == MO_BF16; }
size_t dtype_bytes(int32_t d) { return d == MO_BF16 ? 2 : 4; }

int random_args(const mo_random& r, mo::RandomArgs* out) {
  if (misaligned(r.d_offset, 8)) return MO_ERR_MISALIGNED;
  out->seed = r.seed;
  out->offset = r.offset;
  out->offset_dev = r.d_offset;
  return MO_OK;
}

int drop_args(const mo_dropout* d, mo::DropArgs* out) {
  *out = mo::DropArgs();
  if (d == nullptr) return MO_OK;
  if (!(d->p >= 0.0f && d->p <= 1.0f)) return MO_ERR_BAD_PARAM;
  const int st = random_args(d->random, &out->rnd);
  if (st != MO_OK) return st;
  out->threshold = uint32_t(std::lrint(65536.0 * double(d->p)));
  out->factor = out->threshold < 65536u ? 65536.0f / float(65536u - out->threshold) : 0.0f;
  return MO_OK;
}

int token_args(const mo_tokens* t, mo::TokenArgs* out) {
  if (t == nullptr) return MO_ERR_NULL_POINTER;
  if (t->n < 0 || t->n > kMaxTokens) return MO_ERR_BAD_SHAPE;
  if (t->bits != 32 && t->bits != 64) return MO_ERR_BAD_PARAM;
  if (t->n > 0 && t->ids == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(t->ids, uintptr_t(t->bits / 8))) return MO_ERR_MISALIGNED;
  out->ids = t->ids;
  out->n = t->n;
  out->padding = t->padding_idx;
  out->wide = t->bits == 64 ? 1 : 0;
  return MO_OK;
}

size_t token_bytes(const mo_tokens* t) { return size_t(t->n) * size_t(t->bits / 8); }

int table_shape(int64_t vocab, int64_t dim) {
  return vocab <= 0 || vocab > kMaxVocab || dim <= 0 || dim > kMaxDim ? MO_ERR_BAD_SHAPE : MO_OK;
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Workspace of embed_grad: two buffers of keys and of positions, the join's
// counters, the sums of tokens that cross chunks, the sort's digit counts.
struct GradLayout {
  size_t key[2], pos[2], counter, partial, part_count, bin_count, bytes;
  int64_t counters, dim_pad;
};
GradLayout grad_layout(int64_t n, int64_t dim) {
  GradLayout L;
  const mo::GradGrid g = mo::grad_grid(n, dim);
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    L.key[i] = at;
    at += align256(size_t(n) * 4);
    L.pos[i] = at;
    at += align256(size_t(n) * 4);
  }
  L.counters = 4 * g.chunks * g.col_blocks;
  L.counter = at;
  at += align256(size_t(L.counters) * 4);
  L.dim_pad = (dim + 7) / 8 * 8;
  L.partial = at;
  at += align256(size_t(2 * g.chunks) * size_t(L.dim_pad) * 4);
  L.part_count = at;
  at += align256(size_t(mo::sort_parts(n).parts) * (size_t(4) << mo::kMaxDigitBits));
  L.bin_count = at;
  at += size_t(4) << mo::kMaxDigitBits;
  L.bytes = at;
  return L;
}

// ---------------------------------------------------------------- 4-bit tensors
constexpr int64_t kMaxFp4Dim = int64_t(1) << 22;
constexpr int64_t kMaxFp4Elems = int64_t(1) << 37;   // scale tiles and their lines count in 31 bits

int fp4_shape(int64_t rows, int64_t k, int32_t format) {
  if (format != MO_FP4_MX && format != MO_FP4_NV) return MO_ERR_BAD_PARAM;
  if (rows < 0 || k < 0 || rows > kMaxFp4Dim || k > kMaxFp4Dim) return MO_ERR_BAD_SHAPE;
  return (rows + 127) / 128 * 128 * ((k + 127) / 128 * 128) > kMaxFp4Elems ? MO_ERR_BAD_SHAPE : MO_OK;
}

size_t fp4_codes_bytes(int64_t rows, int64_t k) { return size_t(rows) * size_t((k + 31) / 32 * 16); }
int64_t fp4_tiles_k(int64_t k, int32_t format) { return format == MO_FP4_MX ? (k + 127) / 128 : (k + 63) / 64; }
size_t fp4_scales_bytes(int64_t rows, int64_t k, int32_t format) {
  return size_t((rows + 127) / 128) * size_t(fp4_tiles_k(k, format)) * 512;
}

// A tensor that is written (or read): its storage's pointers.
int fp4_storage(const mo_fp4* q, bool need_amax) {
  const int st = fp4_shape(q->rows, q->k, q->format);
  if (st != MO_OK) return st;
  if (q->rows == 0 || q->k == 0) return MO_OK;
  if (q->codes == nullptr || q->scales == nullptr || (need_amax && q->format == MO_FP4_NV && q->amax == nullptr))
    return MO_ERR_NULL_POINTER;
  if (misaligned(q->codes, 16) || misaligned(q->scales, 16) || misaligned(q->amax, 4)) return MO_ERR_MISALIGNED;
  return MO_OK;
}

bool fp4_overlaps(const mo_fp4* q, const void* p, size_t bytes) {
  return overlap(q->codes, fp4_codes_bytes(q->rows, q->k), p, bytes) ||
         overlap(q->scales, fp4_scales_bytes(q->rows, q->k, q->format), p, bytes) ||
         (q->format == MO_FP4_NV && overlap(q->amax, 4, p, bytes));
}

mo::Fp4In fp4_in(const mo_fp4* q) {
  return {static_cast<const uint8_t*>(q->codes), static_cast<const uint8_t*>(q->scales),
          q->format == MO_FP4_NV ? q->amax : nullptr, q->rows, q->k, (q->k + 31) / 32 * 16, (q->rows + 127) / 128,
          fp4_tiles_k(q->k, q->format)};
}

mo::Fp4Out fp4_out(const mo_fp4* q) {
  return {static_cast<uint8_t*>(q->codes), static_cast<uint8_t*>(q->scales), q->format == MO_FP4_NV ? q->amax : nullptr,
          q->rows, q->k, (q->k + 31) / 32 * 16, (q->rows + 127) / 128, fp4_tiles_k(q->k, q->format)};
}

}  // namespace

extern "C" {

int dropout_apply(const void* x, const void* residual, void* y, int64_t n, int32_t dtype, const mo_dropout* dropout,
                  cudaStream_t stream) {
  if (dropout == nullptr) return MO_ERR_NULL_POINTER;
  mo::DropoutParams p = {};
  int st = drop_args(dropout, &p.drop);
  if (st != MO_OK) return st;
  if (!dtype_ok(dtype)) return MO_ERR_BAD_PARAM;
  if (n < 0 || n > kMaxElems) return MO_ERR_BAD_SHAPE;
  if (n == 0) return MO_OK;
  if (x == nullptr || y == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(y, 16)) return MO_ERR_MISALIGNED;
  const size_t bytes = size_t(n) * dtype_bytes(dtype);
  // in place is fine (an element is read before it is written, by one thread); a shifted overlap is not
  if ((y != x && overlap(y, bytes, x, bytes)) || (y != residual && overlap(y, bytes, residual, bytes)))
    return MO_ERR_OVERLAP;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  p.x = x;
  p.residual = residual;
  p.y = y;
  p.n = n;
  const cudaError_t e = mo::launch_dropout(p, dtype == MO_BF16, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

int embed_lookup(const void* table, int32_t table_dtype, int64_t vocab, int64_t dim, const mo_tokens* tokens, float scale,
                 const void* add, int64_t add_rows, const mo_dropout* dropout, void* out, int32_t out_dtype,
                 cudaStream_t stream) {
  mo::LookupParams p = {};
  int st = token_args(tokens, &p.tokens);
  if (st != MO_OK) return st;
  if ((st = table_shape(vocab, dim)) != MO_OK) return st;
  if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype) || !std::isfinite(scale)) return MO_ERR_BAD_PARAM;
  if ((st = drop_args(dropout, &p.drop)) != MO_OK) return st;
  if (add != nullptr && (add_rows <= 0 || add_rows > kMaxVocab)) return MO_ERR_BAD_SHAPE;
  if (tokens->n == 0) return MO_OK;
  if (table == nullptr || out == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(table, 16) || misaligned(add, 16) || misaligned(out, 16)) return MO_ERR_MISALIGNED;
  const size_t out_bytes = size_t(tokens->n) * size_t(dim) * dtype_bytes(out_dtype);
  if (overlap(out, out_bytes, table, size_t(vocab) * size_t(dim) * dtype_bytes(table_dtype)) ||
      overlap(out, out_bytes, add, size_t(add ? add_rows : 0) * size_t(dim) * dtype_bytes(table_dtype)) ||
      overlap(out, out_bytes, tokens->ids, token_bytes(tokens)))
    return MO_ERR_OVERLAP;
  int sms = 0;
  if ((st = mo::current_device(&sms, &p.status)) != MO_OK) return st;
  p.table = table;
  p.add = add;
  p.out = out;
  p.vocab = vocab;
  p.dim = dim;
  p.add_rows = add_rows;
  p.scale = scale;
  const cudaError_t e = mo::launch_embed_lookup(p, table_dtype == MO_BF16, out_dtype == MO_BF16, sms, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

size_t mo_embed_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  if (n < 0 || n > kMaxTokens || table_shape(vocab, dim) != MO_OK) return 0;
  return n == 0 ? 256 : grad_layout(n, dim).bytes;
}

int embed_grad(const void* dout, int32_t dout_dtype, const mo_tokens* tokens, int64_t vocab, int64_t dim, float scale,
               const mo_dropout* dropout, float* grad, int32_t accumulate, void* ws, size_t ws_bytes,
               cudaStream_t stream) {
  mo::GradParams p = {};
  int st = token_args(tokens, &p.tokens);
  if (st != MO_OK) return st;
  if ((st = table_shape(vocab, dim)) != MO_OK) return st;
  if (!dtype_ok(dout_dtype) || !std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return MO_ERR_BAD_PARAM;
  if ((st = drop_args(dropout, &p.drop)) != MO_OK) return st;
  if (grad == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(grad, 16)) return MO_ERR_MISALIGNED;
  const int64_t n = tokens->n;
  const size_t grad_bytes = size_t(vocab) * size_t(dim) * 4;
  if (n == 0) {   // the sum over no tokens
    if (accumulate) return MO_OK;
    int sms = 0;
    if ((st = mo::current_device(&sms, &p.status)) != MO_OK) return st;
    const cudaError_t e = cudaMemsetAsync(grad, 0, grad_bytes, stream);
    return e != cudaSuccess ? report_cuda(e) : MO_OK;
  }
  if (dout == nullptr || ws == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(dout, 16) || misaligned(ws, 256)) return MO_ERR_MISALIGNED;
  const GradLayout L = grad_layout(n, dim);
  if (ws_bytes < L.bytes) return MO_ERR_WORKSPACE_TOO_SMALL;
  const size_t dout_bytes = size_t(n) * size_t(dim) * dtype_bytes(dout_dtype);
  if (overlap(grad, grad_bytes, dout, dout_bytes) || overlap(grad, grad_bytes, tokens->ids, token_bytes(tokens)) ||
      overlap(grad, grad_bytes, ws, L.bytes) || overlap(ws, L.bytes, dout, dout_bytes) ||
      overlap(ws, L.bytes, tokens->ids, token_bytes(tokens)))
    return MO_ERR_OVERLAP;
  int sms = 0;
  if ((st = mo::current_device(&sms, &p.status)) != MO_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  for (int i = 0; i < 2; ++i) {
    p.key[i] = reinterpret_cast<uint32_t*>(w + L.key[i]);
    p.pos[i] = reinterpret_cast<uint32_t*>(w + L.pos[i]);
  }
  p.counter = reinterpret_cast<uint32_t*>(w + L.counter);
  p.partial = reinterpret_cast<float*>(w + L.partial);
  p.part_count = reinterpret_cast<uint32_t*>(w + L.part_count);
  p.bin_count = reinterpret_cast<uint32_t*>(w + L.bin_count);
  const mo::SortParts parts = mo::sort_parts(n);
  p.parts = parts.parts;
  p.per_warp = parts.per_warp;
  p.counters = L.counters;
  p.dim_pad = L.dim_pad;
  const mo::GradGrid grid = mo::grad_grid(n, dim);
  p.chunk = grid.chunk;
  p.chunks = grid.chunks;
  // launch 1 writes zeros for about as long as its sort takes (at 7 TB/s: 9 us, and 0.34 ns a token);
  // launch 2 in blocks of 128 KB, or of 256 KB where there are thousands (2.1 GB: 327 -> 317 us)
  // (all of them with many tokens, whose sort leaves launch 1 no time)
  p.zero_first = p.parts > 0 ? 0 : std::min(vocab, ((int64_t(60) << 20) + 2304 * n) / (4 * dim) + 1);
  // but no more than 1 KB a thread, as blocks of narrow rows have few (65536 x 63 of 128256: 88 -> 66 us)
  const int64_t block =
      std::min(int64_t(grid.threads) << 10, int64_t(grad_bytes) > (int64_t(1) << 30) ? int64_t(256) << 10 : int64_t(128) << 10);
  p.zero_rows = std::max(int64_t(1), std::min(mo::kZeroRowsMost, block / (4 * dim)));
  p.dout = dout;
  p.grad = grad;
  p.vocab = vocab;
  p.dim = dim;
  p.factor = scale * p.drop.factor;
  p.accumulate = accumulate;
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;   // the keys run from 0 to vocab
  p.passes = (bits + mo::kMaxDigitBits - 1) / mo::kMaxDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  if (p.digit_bits < 5) p.digit_bits = 5;   // a whole warp of bins
  const cudaError_t e = mo::launch_embed_grad(p, dout_dtype == MO_BF16, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

size_t mo_fp4_codes_bytes(int64_t rows, int64_t k) {
  return fp4_shape(rows, k, MO_FP4_MX) == MO_OK ? fp4_codes_bytes(rows, k) : 0;
}

size_t mo_fp4_scales_bytes(int64_t rows, int64_t k, int32_t format) {
  return fp4_shape(rows, k, format) == MO_OK ? fp4_scales_bytes(rows, k, format) : 0;
}

int fp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, const mo_fp4* by_row, const mo_fp4* by_col,
                 const float* amax, const mo_random* stochastic, cudaStream_t stream) {
  if (by_row == nullptr && by_col == nullptr) return MO_ERR_NULL_POINTER;
  if (!dtype_ok(dtype)) return MO_ERR_BAD_PARAM;
  const int32_t format = by_row != nullptr ? by_row->format : by_col->format;
  int st = fp4_shape(rows, cols, format);
  if (st != MO_OK) return st;
  for (const mo_fp4* q : {by_row, by_col}) {
    if (q == nullptr) continue;
    if (q->format != format) return MO_ERR_BAD_PARAM;
    if (q->rows != (q == by_row ? rows : cols) || q->k != (q == by_row ? cols : rows)) return MO_ERR_BAD_SHAPE;
    if ((st = fp4_storage(q, true)) != MO_OK) return st;
  }
  mo::QuantParams p = {};
  if (stochastic != nullptr && (st = random_args(*stochastic, &p.rnd)) != MO_OK) return st;
  if (misaligned(amax, 4)) return MO_ERR_MISALIGNED;
  if (rows == 0 || cols == 0) return MO_OK;
  if (x == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(x, 16)) return MO_ERR_MISALIGNED;
  const size_t x_bytes = size_t(rows) * size_t(cols) * dtype_bytes(dtype);
  for (const mo_fp4* q : {by_row, by_col})
    if (q != nullptr && (fp4_overlaps(q, x, x_bytes) ||
                         overlap(q->codes, fp4_codes_bytes(q->rows, q->k), q->scales, fp4_scales_bytes(q->rows, q->k, format))))
      return MO_ERR_OVERLAP;
  if (by_row != nullptr && by_col != nullptr &&
      (fp4_overlaps(by_row, by_col->codes, fp4_codes_bytes(cols, rows)) ||
       fp4_overlaps(by_row, by_col->scales, fp4_scales_bytes(cols, rows, format))))
    return MO_ERR_OVERLAP;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.tiles_c = (cols + 127) / 128 * (128 / mo::kQuantTile);   // whole scale tiles
  p.vec = cols % (16 / int64_t(dtype_bytes(dtype))) == 0 ? 1 : 0;
  if (by_row != nullptr) p.row = fp4_out(by_row);
  if (by_col != nullptr) p.col = fp4_out(by_col);
  cudaError_t e = cudaSuccess;
  if (format == MO_FP4_NV) {
    p.amax = amax;
    if (amax == nullptr) {
      float* top = p.row.amax != nullptr ? p.row.amax : p.col.amax;
      if ((e = mo::launch_fp4_amax(x, dtype == MO_BF16, rows * cols, top, sms, stream)) != cudaSuccess) return report_cuda(e);
      p.amax = top;
      p.measured = 1;
    }
  }
  e = mo::launch_fp4_quantize(p, dtype == MO_BF16, format == MO_FP4_MX, stochastic != nullptr, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

int fp4_dequantize(const mo_fp4* q, void* out, int32_t dtype, cudaStream_t stream) {
  if (q == nullptr) return MO_ERR_NULL_POINTER;
  if (!dtype_ok(dtype)) return MO_ERR_BAD_PARAM;
  int st = fp4_storage(q, true);
  if (st != MO_OK) return st;
  if (q->rows == 0 || q->k == 0) return MO_OK;
  if (out == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(out, 16)) return MO_ERR_MISALIGNED;
  if (fp4_overlaps(q, out, size_t(q->rows) * size_t(q->k) * dtype_bytes(dtype))) return MO_ERR_OVERLAP;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  const cudaError_t e = mo::launch_fp4_dequantize(fp4_in(q), q->format == MO_FP4_MX, out, dtype == MO_BF16, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

int fp4_product(const mo_fp4* a, const mo_fp4* b, void* out, int32_t dtype, cudaStream_t stream) {
  if (a == nullptr || b == nullptr) return MO_ERR_NULL_POINTER;
  if (!dtype_ok(dtype)) return MO_ERR_BAD_PARAM;
  int st = fp4_storage(a, true);
  if (st != MO_OK) return st;
  if ((st = fp4_storage(b, true)) != MO_OK) return st;
  if (a->format != b->format) return MO_ERR_BAD_PARAM;
  if (a->k != b->k) return MO_ERR_BAD_SHAPE;
  if (a->rows == 0 || b->rows == 0) return MO_OK;
  if (out == nullptr) return MO_ERR_NULL_POINTER;
  if (misaligned(out, 16)) return MO_ERR_MISALIGNED;
  const size_t out_bytes = size_t(a->rows) * size_t(b->rows) * dtype_bytes(dtype);
  if (fp4_overlaps(a, out, out_bytes) || fp4_overlaps(b, out, out_bytes)) return MO_ERR_OVERLAP;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  const cudaError_t e =
      a->k == 0 ? cudaMemsetAsync(out, 0, out_bytes, stream)   // the sum over nothing
                : mo::launch_fp4_product(fp4_in(a), fp4_in(b), a->format == MO_FP4_MX, out, dtype == MO_BF16, sms, status, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

}  // extern "C"
