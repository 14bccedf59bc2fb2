// extern "C" entry points of the feed-forward operators (include/mo.h):
// argument checks, workspace layout, launches. No entry point allocates device
// memory or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "layer_kernels.h"
#include "mo.h"

namespace {

using mo::Kept;
using mo::Operand;
using mo::padded;
using mo::report_cuda;

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxElems = int64_t(1) << 37;
constexpr int64_t kMaxReduction = int64_t(1) << 16;   // columns that a forward product sums over
// Longer sums are taken in slices of as many, joined in fp32: the tensor core's
// accumulator cuts what is added off below the running sum, and the loss grows with the
// number of additions (numbers of one sign, relative to the sum: 1.6e-4 over 32768
// products, 3.4e-4 over 65536, in two slices 1.6e-4).
constexpr int64_t kSlice = 32768;

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool plain_dtype(int32_t d) { return d == MO_F32 || d == MO_BF16; }
size_t bytes_of(int32_t d) { return d == MO_BF16 ? 2 : 4; }
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

int matrix_shape(int64_t rows, int64_t k) {
  if (rows < 0 || rows > kMaxTokens || k <= 0 || k > kMaxWidth) return MO_ERR_BAD_SHAPE;
  return rows > 0 && mo::mx8_blocks(k) * 32 > kMaxElems / rows ? MO_ERR_BAD_SHAPE : MO_OK;
}

// Memory that a call touches; a range that is written may overlap no other, but
// be one that it was given to replace. Operands of a product are read whole, by
// tiles that write other places, and a norm's weight is read by every row: an output
// replaces none of them, whatever else was given at the same address.
struct Range {
  const void* p;
  size_t bytes;
  bool written, operand;
  const void* in_place[2];   // ranges that may begin at the same place
};
struct Ranges {
  Range r[24];
  int n = 0;
  void add(const void* p, size_t bytes, bool written, bool operand, const void* same0 = nullptr, const void* same1 = nullptr) {
    if (p != nullptr && bytes > 0) r[n++] = {p, bytes, written, operand, {same0, same1}};
  }
  void reads(const void* p, size_t bytes) { add(p, bytes, false, false); }
  void operand(const void* p, size_t bytes) { add(p, bytes, false, true); }
  void writes(const void* p, size_t bytes, const void* same0 = nullptr, const void* same1 = nullptr) {
    add(p, bytes, true, false, same0, same1);
  }
  void kept(const mo_tensor* t, int64_t rows, int64_t k, bool written, bool operand = false) {
    if (t == nullptr) return;
    if (t->dtype == MO_MX8) {
      add(t->data, size_t(rows) * size_t(mo::mx8_blocks(k)) * 32, written, operand);
      add(t->scales, size_t(rows) * size_t(mo::mx8_blocks(k)), written, operand);
    } else {
      add(t->data, size_t(rows) * size_t(k) * bytes_of(t->dtype), written, operand);
    }
  }
  int check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j) {
        if (i == j || !r[i].written) continue;
        const uintptr_t x = reinterpret_cast<uintptr_t>(r[i].p), y = reinterpret_cast<uintptr_t>(r[j].p);
        if (!(x < y + r[j].bytes && y < x + r[i].bytes)) continue;
        const bool same = x == y && r[i].bytes == r[j].bytes && !r[j].written && !r[j].operand && (r[i].in_place[0] == r[j].p || r[i].in_place[1] == r[j].p);
        if (!same) return MO_ERR_OVERLAP;
      }
    return MO_OK;
  }
};

// A tensor of a call, of bf16 or 8 bits (or fp32 where `f32` allows it).
int kept_args(const mo_tensor* t, bool f32, Kept* out) {
  if (t->dtype != MO_MX8 && t->dtype != MO_BF16 && !(f32 && t->dtype == MO_F32)) return MO_ERR_BAD_PARAM;
  if (t->data == nullptr || (t->dtype == MO_MX8 && t->scales == nullptr)) return MO_ERR_NULL_POINTER;
  if (misaligned(t->data, 16)) return MO_ERR_MISALIGNED;
  out->data = t->data;
  out->scales = static_cast<uint8_t*>(t->scales);
  out->dtype = t->dtype;
  return MO_OK;
}

struct Workspace {
  uint8_t* base;
  size_t at = 0;
  void* take(size_t bytes) {
    void* p = base + at;
    at += align256(bytes);
    return p;
  }
};

// Runs launches until one fails.
struct Launches {
  cudaError_t error = cudaSuccess;
  void operator()(cudaError_t e) {
    if (error == cudaSuccess) error = e;
  }
  int status() const { return error == cudaSuccess ? MO_OK : report_cuda(error); }
};

// The bf16 operands of a call's products as TMA can read them: rows of a multiple
// of 16 bytes. Others, and those in 8 bits, are laid out in the workspace, all of
// a launch's in one go.
bool needs_copy(int64_t cols, int32_t dtype) { return dtype == MO_MX8 || cols % 8 != 0; }
size_t copy_bytes(int64_t rows, int64_t cols) { return align256(size_t(rows) * size_t(padded(cols)) * 2); }

struct Operands {
  Workspace& ws;
  mo::LayOut todo[3];
  int n = 0;
  Operand operator()(const Kept& t, int64_t rows, int64_t cols) {
    if (!needs_copy(cols, t.dtype)) return {t.data, rows, cols, cols};
    uint16_t* copy = static_cast<uint16_t*>(ws.take(size_t(rows) * size_t(padded(cols)) * 2));
    todo[n++] = {t, rows, cols, copy, padded(cols)};
    return {copy, rows, cols, padded(cols)};
  }
  Operand operator()(const void* p, int64_t rows, int64_t cols) {
    Kept t;
    t.data = const_cast<void*>(p);
    return (*this)(t, rows, cols);
  }
  void lay_out(Launches& run, cudaStream_t stream) {
    if (n > 0 && run.error == cudaSuccess) run(mo::launch_lay_out(todo, n, stream));
    n = 0;
  }
};

// Bytes of the partial sums of a product whose reduction is cut.
size_t slice_bytes(int64_t k, int64_t m, int64_t n) { return k > kSlice ? align256(size_t(m) * size_t(n) * 4) : 0; }

// An operand's part along the reduction: its rows, or (whole 128-byte lines in, so
// aligned as the operand is) its columns.
void cut(Operand& o, bool mn, int64_t k0, int64_t k) {
  if (mn) {
    o.p = static_cast<const uint16_t*>(o.p) + k0 * o.ld;
    o.rows = k;
  } else {
    o.p = static_cast<const uint16_t*>(o.p) + k0;
    o.cols = k;
  }
}

// Bytes of the sums that a product with an epilogue starts from where its reduction is
// cut: of `count` sums [m, n].
size_t start_bytes(int64_t k, int64_t m, int64_t n, int count) {
  return k > kSlice ? size_t(count) * align256(size_t(m) * size_t(padded(n)) * 4) : 0;
}

// Cuts a product's reduction where one accumulation would be too long: the slices but
// the last are summed in fp32 in `part`, each on top of the last one's, and q is left
// with the last slice, which starts from there.
void slice_ahead(mo::Product& q, float* part, int sms, int* status, Launches& run, cudaStream_t stream) {
  if (mo::longest_sum(q, sms) <= kSlice) return;
  const mo::Target whole = q.t[0];
  const int64_t ld = padded(whole.n);
  mo::Product s;
  s.a_mn = q.a_mn;
  s.b_mn = q.b_mn;
  s.count = q.epi == mo::kEpiGated ? 2 : 1;
  s.k = kSlice;
  int64_t k0 = 0;
  for (; q.k - k0 > kSlice && run.error == cudaSuccess; k0 += kSlice) {
    for (int i = 0; i < s.count; ++i) {
      float* sums = part + i * (align256(size_t(whole.m) * size_t(ld) * 4) / 4);
      s.a[i] = q.a[0];
      s.b[i] = q.b[i];
      cut(s.a[i], q.a_mn, k0, kSlice);
      cut(s.b[i], q.b_mn, k0, kSlice);
      s.t[i] = {sums, k0 > 0 ? sums : nullptr, whole.m, whole.n, ld, ld, 0, 0};
      q.start[i] = sums;
    }
    run(mo::launch_product(s, sms, status, stream));
  }
  q.k -= k0;
  cut(q.a[0], q.a_mn, k0, q.k);
  for (int i = 0; i < s.count; ++i) cut(q.b[i], q.b_mn, k0, q.k);
}

// A product without activation whose reduction runs over the rows of both
// operands (or, without a_mn, of the second alone), in slices where it is long:
// the first slices' sums go to `part` in fp32, each on top of the last one's.
void sliced_product(const mo::Product& whole, float* part, int sms, int* status, Launches& run, cudaStream_t stream) {
  const int64_t slices = (whole.k + kSlice - 1) / kSlice;
  for (int64_t s = 0; s < slices && run.error == cudaSuccess; ++s) {
    mo::Product q = whole;
    const int64_t k0 = s * kSlice;
    q.k = std::min(kSlice, whole.k - k0);
    float* sums = part;
    for (int i = 0; i < q.count; ++i) {
      if (slices > 1) {
        cut(q.a[i], q.a_mn, k0, q.k);
        cut(q.b[i], true, k0, q.k);
        mo::Target& t = q.t[i];
        if (s > 0) t.add = sums, t.add_ld = t.n, t.add_bf16 = 0;
        if (s + 1 < slices) t.out = sums, t.ld = t.n, t.out_bf16 = 0;
        sums += align256(size_t(t.m) * size_t(t.n) * 4) / 4;
      }
    }
    run(mo::launch_product(q, sms, status, stream));
  }
}

mo::Target target(void* out, int32_t dtype, int64_t m, int64_t n, const void* add = nullptr) {
  return {out, add, m, n, n, n, dtype == MO_BF16, dtype == MO_BF16};
}

int clear(void* p, size_t bytes, cudaStream_t stream) {
  const cudaError_t e = cudaMemsetAsync(p, 0, bytes, stream);
  return e != cudaSuccess ? report_cuda(e) : MO_OK;
}

bool known_act(int32_t act) { return act >= MO_ACT_NONE && act <= MO_ACT_SILU; }

int linear_shape(int64_t tokens, int64_t cols, int64_t rows) {
  if (tokens < 0 || tokens > kMaxTokens || cols <= 0 || cols > kMaxReduction || rows <= 0 || rows > kMaxWidth) return MO_ERR_BAD_SHAPE;
  const int64_t most = std::max(padded(cols), padded(rows));
  return tokens > 0 && most > kMaxElems / tokens ? MO_ERR_BAD_SHAPE : MO_OK;
}

int ffn_shape(int64_t tokens, int64_t dim, int64_t inner) {
  if (tokens < 0 || tokens > kMaxTokens || dim <= 0 || dim > kMaxReduction || inner <= 0 || inner > kMaxReduction / 2)
    return MO_ERR_BAD_SHAPE;
  const int64_t most = std::max(padded(dim), padded(inner));
  return tokens > 0 && most > kMaxElems / tokens ? MO_ERR_BAD_SHAPE : MO_OK;
}

// (No less for more tokens: a workspace of the largest batch serves the others.)
size_t linear_bytes(int64_t tokens, int64_t cols, int64_t rows, bool grad) {
  size_t b = copy_bytes(tokens, cols) + (cols % 8 != 0 ? copy_bytes(rows, cols) : 0) + start_bytes(cols, tokens, rows, 1);
  if (grad) {
    b += copy_bytes(tokens, rows);   // dz
    b += align256(size_t(mo::act_grad_room(tokens, rows)) * size_t(rows) * 4);
    b += std::max(slice_bytes(tokens, rows, cols), slice_bytes(rows, tokens, cols));
  }
  return std::max<size_t>(b, 256);
}

size_t ffn_bytes(int64_t tokens, int64_t dim, int64_t inner, bool grad) {
  size_t b = copy_bytes(tokens, dim) + copy_bytes(tokens, inner);   // x, h
  if (dim % 8 != 0) b += 2 * copy_bytes(inner, dim);
  if (inner % 8 != 0) b += copy_bytes(dim, inner);
  size_t sums = start_bytes(dim, tokens, inner, 2);   // of one launch at a time
  if (grad) {
    sums = std::max({sums, slice_bytes(2 * inner, tokens, dim), 3 * slice_bytes(tokens, inner, dim)});
    b += 2 * copy_bytes(tokens, inner);   // dg, du
    if (dim % 8 != 0) b += copy_bytes(tokens, dim);   // dout
  }
  return std::max<size_t>(b + sums, 256);
}

}  // namespace

extern "C" {

size_t mo_mx8_codes_bytes(int64_t rows, int64_t k) {
  return matrix_shape(rows, k) == MO_OK ? size_t(rows) * size_t(mo::mx8_blocks(k)) * 32 : 0;
}

size_t mo_mx8_scales_bytes(int64_t rows, int64_t k) {
  return matrix_shape(rows, k) == MO_OK ? size_t(rows) * size_t(mo::mx8_blocks(k)) : 0;
}

int mx8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, const mo_tensor* q, cudaStream_t stream) {
  if (q == nullptr) return MO_ERR_NULL_POINTER;
  if (!plain_dtype(dtype) || q->dtype != MO_MX8) return MO_ERR_BAD_PARAM;
  int st = matrix_shape(rows, k);
  if (st != MO_OK) return st;
  if (rows == 0) return MO_OK;
  Kept to;
  if (x == nullptr) return MO_ERR_NULL_POINTER;
  if ((st = kept_args(q, false, &to)) != MO_OK) return st;
  if (misaligned(x, 16)) return MO_ERR_MISALIGNED;
  Ranges mem;
  mem.reads(x, size_t(rows) * size_t(k) * bytes_of(dtype));
  mem.kept(q, rows, k, true);
  if ((st = mem.check()) != MO_OK) return st;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Launches run;
  run(mo::launch_mx8_quantize(x, dtype == MO_BF16, rows, k, to, stream));
  return run.status();
}

int mx8_dequantize(const mo_tensor* q, int64_t rows, int64_t k, void* out, int32_t dtype, cudaStream_t stream) {
  if (q == nullptr) return MO_ERR_NULL_POINTER;
  if (!plain_dtype(dtype) || q->dtype != MO_MX8) return MO_ERR_BAD_PARAM;
  int st = matrix_shape(rows, k);
  if (st != MO_OK) return st;
  if (rows == 0) return MO_OK;
  Kept from;
  if (out == nullptr) return MO_ERR_NULL_POINTER;
  if ((st = kept_args(q, false, &from)) != MO_OK) return st;
  if (misaligned(out, 16)) return MO_ERR_MISALIGNED;
  Ranges mem;
  mem.writes(out, size_t(rows) * size_t(k) * bytes_of(dtype));
  mem.kept(q, rows, k, false);
  if ((st = mem.check()) != MO_OK) return st;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Launches run;
  run(mo::launch_unpack(from, rows, k, out, dtype == MO_BF16, stream));
  return run.status();
}

int rms_norm(const void* x, const void* residual, int32_t dtype, int64_t rows, int64_t dim, const float* weight, float eps,
             void* sum, void* out, int32_t out_dtype, const mo_tensor* out8, cudaStream_t stream) {
  if (!plain_dtype(dtype) || (out != nullptr && !plain_dtype(out_dtype)) || (out8 != nullptr && out8->dtype != MO_MX8) ||
      !(eps >= 0.0f) || !std::isfinite(eps))
    return MO_ERR_BAD_PARAM;
  int st = matrix_shape(rows, dim);
  if (st != MO_OK) return st;
  if (rows == 0) return MO_OK;
  if (x == nullptr || (out == nullptr && out8 == nullptr)) return MO_ERR_NULL_POINTER;
  mo::NormParams p = {};
  if (out8 != nullptr && (st = kept_args(out8, false, &p.out8)) != MO_OK) return st;
  for (const void* q : {x, residual, static_cast<const void*>(weight), static_cast<const void*>(sum), static_cast<const void*>(out)})
    if (misaligned(q, 16)) return MO_ERR_MISALIGNED;
  const size_t n = size_t(rows) * size_t(dim);
  Ranges mem;
  mem.reads(x, n * bytes_of(dtype));
  mem.reads(residual, n * bytes_of(dtype));
  mem.operand(weight, size_t(dim) * 4);
  mem.writes(sum, n * bytes_of(dtype), x, residual);
  mem.writes(out, n * bytes_of(out_dtype), x, residual);
  mem.kept(out8, rows, dim, true);
  if ((st = mem.check()) != MO_OK) return st;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.sum = sum;
  p.out = out;
  p.rows = rows;
  p.dim = dim;
  p.eps = eps;
  p.out_bf16 = out_dtype == MO_BF16;
  Launches run;
  run(mo::launch_rms_norm(p, dtype == MO_BF16, stream));
  return run.status();
}

size_t mo_rms_norm_grad_workspace_bytes(int64_t rows, int64_t dim) {
  if (matrix_shape(rows, dim) != MO_OK) return 0;
  return std::max<size_t>(256, rows == 0 ? 0 : align256(size_t(mo::norm_parts(rows, dim)) * size_t(dim) * 4));
}

int rms_norm_grad(const void* dy, int32_t dtype, const mo_tensor* x, int64_t rows, int64_t dim, const float* weight,
                  float eps, const void* dresidual, void* dx, float* dweight, int32_t accumulate, void* ws,
                  size_t ws_bytes, cudaStream_t stream) {
  if (!plain_dtype(dtype) || !(eps >= 0.0f) || !std::isfinite(eps) || (accumulate != 0 && accumulate != 1)) return MO_ERR_BAD_PARAM;
  int st = matrix_shape(rows, dim);
  if (st != MO_OK) return st;
  if (misaligned(dweight, 16)) return MO_ERR_MISALIGNED;
  int sms = 0;
  int* status = nullptr;
  if (rows == 0) {   // the sum over no rows
    if (dweight == nullptr || accumulate) return MO_OK;
    if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
    return clear(dweight, size_t(dim) * 4, stream);
  }
  if (dy == nullptr || x == nullptr || dx == nullptr) return MO_ERR_NULL_POINTER;
  mo::NormGradParams p = {};
  if ((st = kept_args(x, true, &p.x)) != MO_OK) return st;
  if (x->dtype != MO_MX8 && x->dtype != dtype) return MO_ERR_BAD_PARAM;
  for (const void* q : {dy, static_cast<const void*>(weight), dresidual, static_cast<const void*>(dx)})
    if (misaligned(q, 16)) return MO_ERR_MISALIGNED;
  const size_t n = size_t(rows) * size_t(dim) * bytes_of(dtype);
  const size_t need = dweight != nullptr ? mo_rms_norm_grad_workspace_bytes(rows, dim) : 0;
  if (dweight != nullptr) {
    if (ws == nullptr) return MO_ERR_NULL_POINTER;
    if (misaligned(ws, 256)) return MO_ERR_MISALIGNED;
    if (ws_bytes < need) return MO_ERR_WORKSPACE_TOO_SMALL;
  }
  Ranges mem;
  mem.reads(dy, n);
  mem.kept(x, rows, dim, false);
  mem.operand(weight, size_t(dim) * 4);
  mem.reads(dresidual, n);
  mem.writes(dx, n, dy, dresidual);
  mem.writes(dweight, size_t(dim) * 4);
  mem.writes(ws, need);
  if ((st = mem.check()) != MO_OK) return st;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  p.dy = dy;
  p.weight = weight;
  p.dres = dresidual;
  p.dx = dx;
  p.part = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  p.rows = rows;
  p.dim = dim;
  p.eps = eps;
  Launches run;
  run(mo::launch_rms_norm_grad(p, dtype == MO_BF16, stream));
  if (dweight != nullptr && run.error == cudaSuccess)
    run(mo::launch_join(p.part, mo::norm_parts(rows, dim), dim, dweight, accumulate != 0, stream));
  return run.status();
}

size_t mo_linear_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t grad) {
  if (linear_shape(tokens, cols, rows) != MO_OK || (grad != 0 && grad != 1)) return 0;
  return linear_bytes(tokens, cols, rows, grad != 0);
}

int linear_forward(const mo_tensor* x, const void* w, int64_t tokens, int64_t cols, int64_t rows, const float* bias,
                   int32_t act, const void* residual, const mo_tensor* pre, void* out, int32_t out_dtype, void* ws,
                   size_t ws_bytes, cudaStream_t stream) {
  if (!known_act(act) || !plain_dtype(out_dtype) || (pre != nullptr && act == MO_ACT_NONE)) return MO_ERR_BAD_PARAM;
  int st = linear_shape(tokens, cols, rows);
  if (st != MO_OK) return st;
  if (tokens == 0) return MO_OK;
  if (x == nullptr || w == nullptr || out == nullptr || ws == nullptr) return MO_ERR_NULL_POINTER;
  Kept xk;
  mo::Product q;
  if ((st = kept_args(x, false, &xk)) != MO_OK) return st;
  if (pre != nullptr && (st = kept_args(pre, false, &q.pre)) != MO_OK) return st;
  for (const void* p : {w, static_cast<const void*>(bias), residual, static_cast<const void*>(out)})
    if (misaligned(p, 16)) return MO_ERR_MISALIGNED;
  if (misaligned(ws, 256)) return MO_ERR_MISALIGNED;
  const size_t need = linear_bytes(tokens, cols, rows, false), out_bytes = size_t(tokens) * size_t(rows) * bytes_of(out_dtype);
  if (ws_bytes < need) return MO_ERR_WORKSPACE_TOO_SMALL;
  Ranges mem;
  mem.kept(x, tokens, cols, false, true);
  mem.operand(w, size_t(rows) * size_t(cols) * 2);
  mem.reads(bias, size_t(rows) * 4);
  mem.reads(residual, out_bytes);
  mem.kept(pre, tokens, rows, true);
  mem.writes(out, out_bytes, residual);
  mem.writes(ws, need);
  if ((st = mem.check()) != MO_OK) return st;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Workspace space{static_cast<uint8_t*>(ws)};
  Launches run;
  q.act = act;
  Operands operand{space};
  q.a[0] = operand(xk, tokens, cols);
  q.b[0] = operand(w, rows, cols);
  operand.lay_out(run, stream);
  q.t[0] = target(out, out_dtype, tokens, rows, residual);
  q.k = cols;
  q.bias = bias;
  slice_ahead(q, static_cast<float*>(space.take(0)), sms, status, run, stream);
  if (run.error == cudaSuccess) run(mo::launch_product(q, sms, status, stream));
  return run.status();
}

int linear_grad(const void* dout, const mo_tensor* x, const void* w, int64_t tokens, int64_t cols, int64_t rows,
                int32_t act, const mo_tensor* pre, void* dx, int32_t dx_dtype, void* dw, int32_t dw_dtype, float* dbias,
                int32_t accumulate, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!known_act(act) || (dx != nullptr && !plain_dtype(dx_dtype)) || (dw != nullptr && !plain_dtype(dw_dtype)) ||
      (accumulate != 0 && accumulate != 1) || (pre != nullptr && act == MO_ACT_NONE))
    return MO_ERR_BAD_PARAM;
  int st = linear_shape(tokens, cols, rows);
  if (st != MO_OK) return st;
  if (tokens > 0 && dx == nullptr && dw == nullptr && dbias == nullptr) return MO_ERR_NULL_POINTER;
  for (const void* p : {static_cast<const void*>(dx), static_cast<const void*>(dw), static_cast<const void*>(dbias)})
    if (misaligned(p, 16)) return MO_ERR_MISALIGNED;
  int sms = 0;
  int* status = nullptr;
  const size_t dw_bytes = size_t(rows) * size_t(cols) * bytes_of(dw_dtype);
  if (tokens == 0) {   // sums over no tokens
    if (accumulate || (dw == nullptr && dbias == nullptr)) return MO_OK;
    if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
    if (dw != nullptr && (st = clear(dw, dw_bytes, stream)) != MO_OK) return st;
    return dbias != nullptr ? clear(dbias, size_t(rows) * 4, stream) : MO_OK;
  }
  if (dout == nullptr || ws == nullptr || (dw != nullptr && x == nullptr) || (dx != nullptr && w == nullptr) ||
      (act != MO_ACT_NONE && pre == nullptr))
    return MO_ERR_NULL_POINTER;
  Kept xk;
  mo::ActGradParams g = {};
  if (dw != nullptr && (st = kept_args(x, false, &xk)) != MO_OK) return st;
  if (pre != nullptr && (st = kept_args(pre, false, &g.pre)) != MO_OK) return st;
  if (misaligned(dout, 16) || misaligned(dx != nullptr ? w : nullptr, 16) || misaligned(ws, 256)) return MO_ERR_MISALIGNED;
  const size_t need = linear_bytes(tokens, cols, rows, true);
  if (ws_bytes < need) return MO_ERR_WORKSPACE_TOO_SMALL;
  Ranges mem;
  mem.reads(dout, size_t(tokens) * size_t(rows) * 2);
  if (dw != nullptr) mem.kept(x, tokens, cols, false);
  if (dx != nullptr) mem.reads(w, size_t(rows) * size_t(cols) * 2);
  mem.kept(pre, tokens, rows, false);
  mem.writes(dx, size_t(tokens) * size_t(cols) * bytes_of(dx_dtype));
  mem.writes(dw, dw_bytes);
  mem.writes(dbias, size_t(rows) * 4);
  mem.writes(ws, need);
  if ((st = mem.check()) != MO_OK) return st;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Workspace space{static_cast<uint8_t*>(ws)};
  Launches run;
  // dz, and its sums over tokens
  Operand dz = {dout, tokens, rows, rows};
  const bool products = dx != nullptr || dw != nullptr;
  g.dout = static_cast<const uint16_t*>(dout);
  g.tokens = tokens;
  g.rows = rows;
  g.act = act;
  g.per = mo::act_grad_per(tokens, rows);
  if (products && (act != MO_ACT_NONE || rows % 8 != 0)) {
    g.ld = padded(rows);
    g.dz = static_cast<uint16_t*>(space.take(size_t(tokens) * size_t(g.ld) * 2));
    dz = {g.dz, tokens, rows, g.ld};
  }
  const int64_t parts = (tokens + g.per - 1) / g.per;
  if (dbias != nullptr) g.part = static_cast<float*>(space.take(size_t(parts) * size_t(rows) * 4));
  Operands operand{space};
  const Operand xo = dw != nullptr ? operand(xk, tokens, cols) : Operand{};
  const Operand wo = dx != nullptr ? operand(w, rows, cols) : Operand{};
  g.early = operand.n > 0;
  operand.lay_out(run, stream);
  if ((g.dz != nullptr || g.part != nullptr) && run.error == cudaSuccess) run(mo::launch_act_grad(g, stream));
  if (dbias != nullptr && run.error == cudaSuccess) run(mo::launch_join(g.part, parts, rows, dbias, accumulate != 0, stream));
  float* part = reinterpret_cast<float*>(space.take(0));
  if (dx != nullptr) {
    mo::Product q;
    q.b_mn = true;
    q.a[0] = dz;
    q.b[0] = wo;
    q.t[0] = target(dx, dx_dtype, tokens, cols);
    q.k = rows;
    sliced_product(q, part, sms, status, run, stream);
  }
  if (dw != nullptr) {
    mo::Product q;
    q.a_mn = q.b_mn = true;
    q.a[0] = dz;
    q.b[0] = xo;
    q.t[0] = target(dw, dw_dtype, rows, cols, accumulate ? dw : nullptr);
    q.k = tokens;
    sliced_product(q, part, sms, status, run, stream);
  }
  return run.status();
}

size_t mo_gated_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t inner, int32_t grad) {
  if (ffn_shape(tokens, dim, inner) != MO_OK || (grad != 0 && grad != 1)) return 0;
  return ffn_bytes(tokens, dim, inner, grad != 0);
}

int gated_ffn_forward(const mo_tensor* x, const void* w_gate, const void* w_up, const void* w_down, int64_t tokens,
                      int64_t dim, int64_t inner, int32_t act, const void* residual, const mo_tensor* gate,
                      const mo_tensor* up, void* out, int32_t out_dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!known_act(act) || !plain_dtype(out_dtype)) return MO_ERR_BAD_PARAM;
  int st = ffn_shape(tokens, dim, inner);
  if (st != MO_OK) return st;
  if ((gate == nullptr) != (up == nullptr)) return MO_ERR_NULL_POINTER;
  if (tokens == 0) return MO_OK;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || w_down == nullptr || out == nullptr || ws == nullptr)
    return MO_ERR_NULL_POINTER;
  Kept xk;
  mo::Product q;
  if ((st = kept_args(x, false, &xk)) != MO_OK) return st;
  if (gate != nullptr) {
    if ((st = kept_args(gate, false, &q.pre)) != MO_OK || (st = kept_args(up, false, &q.pre2)) != MO_OK) return st;
    if (gate->dtype != up->dtype) return MO_ERR_BAD_PARAM;
  }
  for (const void* p : {w_gate, w_up, w_down, residual, static_cast<const void*>(out)})
    if (misaligned(p, 16)) return MO_ERR_MISALIGNED;
  if (misaligned(ws, 256)) return MO_ERR_MISALIGNED;
  const size_t need = ffn_bytes(tokens, dim, inner, false), out_bytes = size_t(tokens) * size_t(dim) * bytes_of(out_dtype);
  if (ws_bytes < need) return MO_ERR_WORKSPACE_TOO_SMALL;
  Ranges mem;
  mem.kept(x, tokens, dim, false);   // (out may replace it as the residual: the launch that writes out does not read x)
  for (const void* p : {w_gate, w_up, w_down}) mem.operand(p, size_t(inner) * size_t(dim) * 2);
  mem.reads(residual, out_bytes);
  mem.kept(gate, tokens, inner, true);
  mem.kept(up, tokens, inner, true);
  mem.writes(out, out_bytes, residual);
  mem.writes(ws, need);
  if ((st = mem.check()) != MO_OK) return st;
  int sms = 0;
  int* status = nullptr;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Workspace space{static_cast<uint8_t*>(ws)};
  Launches run;
  const int64_t ld = padded(inner);
  void* h = space.take(size_t(tokens) * size_t(ld) * 2);
  q.epi = mo::kEpiGated;
  q.act = act;
  Operands operand{space};
  q.a[0] = operand(xk, tokens, dim);
  q.b[0] = operand(w_gate, inner, dim);
  q.b[1] = operand(w_up, inner, dim);
  operand.lay_out(run, stream);
  q.t[0] = {h, nullptr, tokens, inner, ld, 0, 1, 0};
  q.k = dim;
  slice_ahead(q, static_cast<float*>(space.take(0)), sms, status, run, stream);
  if (run.error == cudaSuccess) run(mo::launch_product(q, sms, status, stream));
  mo::Product down;
  down.a[0] = {h, tokens, inner, ld};
  down.b[0] = operand(w_down, dim, inner);
  operand.lay_out(run, stream);
  down.early = !needs_copy(inner, MO_BF16) && (mo::is_few(q, sms) || mo::is_narrow(q, sms));
  down.t[0] = target(out, out_dtype, tokens, dim, residual);
  down.k = inner;
  if (run.error == cudaSuccess) run(mo::launch_product(down, sms, status, stream));
  return run.status();
}

int gated_ffn_grad(const void* dout, const mo_tensor* x, const mo_tensor* gate, const mo_tensor* up, const void* w_gate,
                   const void* w_up, const void* w_down, int64_t tokens, int64_t dim, int64_t inner, int32_t act,
                   void* dx, int32_t dx_dtype, void* dw_gate, void* dw_up, void* dw_down, int32_t dw_dtype,
                   int32_t accumulate, void* ws, size_t ws_bytes, cudaStream_t stream) {
  void* const dw[3] = {dw_gate, dw_up, dw_down};
  const bool any_dw = dw_gate != nullptr || dw_up != nullptr || dw_down != nullptr;
  if (!known_act(act) || (dx != nullptr && !plain_dtype(dx_dtype)) || (any_dw && !plain_dtype(dw_dtype)) ||
      (accumulate != 0 && accumulate != 1))
    return MO_ERR_BAD_PARAM;
  int st = ffn_shape(tokens, dim, inner);
  if (st != MO_OK) return st;
  if (tokens > 0 && dx == nullptr && !any_dw) return MO_ERR_NULL_POINTER;
  for (const void* p : {static_cast<const void*>(dx), static_cast<const void*>(dw_gate), static_cast<const void*>(dw_up),
                        static_cast<const void*>(dw_down)})
    if (misaligned(p, 16)) return MO_ERR_MISALIGNED;
  int sms = 0;
  int* status = nullptr;
  const size_t dw_bytes = size_t(inner) * size_t(dim) * bytes_of(dw_dtype);
  if (tokens == 0) {   // sums over no tokens
    if (accumulate || !any_dw) return MO_OK;
    if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
    for (void* p : dw)
      if (p != nullptr && (st = clear(p, dw_bytes, stream)) != MO_OK) return st;
    return MO_OK;
  }
  const bool need_x = dw_gate != nullptr || dw_up != nullptr;
  if (dout == nullptr || gate == nullptr || up == nullptr || w_down == nullptr || ws == nullptr || (need_x && x == nullptr) ||
      (dx != nullptr && (w_gate == nullptr || w_up == nullptr)))
    return MO_ERR_NULL_POINTER;
  Kept xk;
  mo::Product q;
  if (need_x && (st = kept_args(x, false, &xk)) != MO_OK) return st;
  if ((st = kept_args(gate, false, &q.pre)) != MO_OK || (st = kept_args(up, false, &q.pre2)) != MO_OK) return st;
  if (gate->dtype != up->dtype) return MO_ERR_BAD_PARAM;
  if (misaligned(dout, 16) || misaligned(w_down, 16) || misaligned(ws, 256) ||
      (dx != nullptr && (misaligned(w_gate, 16) || misaligned(w_up, 16))))
    return MO_ERR_MISALIGNED;
  const size_t need = ffn_bytes(tokens, dim, inner, true);
  if (ws_bytes < need) return MO_ERR_WORKSPACE_TOO_SMALL;
  Ranges mem;
  mem.reads(dout, size_t(tokens) * size_t(dim) * 2);
  if (need_x) mem.kept(x, tokens, dim, false);
  mem.kept(gate, tokens, inner, false);
  mem.kept(up, tokens, inner, false);
  mem.reads(w_down, size_t(inner) * size_t(dim) * 2);
  if (dx != nullptr)
    for (const void* p : {w_gate, w_up}) mem.reads(p, size_t(inner) * size_t(dim) * 2);
  mem.writes(dx, size_t(tokens) * size_t(dim) * bytes_of(dx_dtype));
  for (void* p : dw) mem.writes(p, dw_bytes);
  mem.writes(ws, need);
  if ((st = mem.check()) != MO_OK) return st;
  if ((st = mo::current_device(&sms, &status)) != MO_OK) return st;
  Workspace space{static_cast<uint8_t*>(ws)};
  Launches run;
  const int64_t ld = padded(inner);
  uint16_t* kept[3];   // dg, du, h
  for (uint16_t*& p : kept) p = static_cast<uint16_t*>(space.take(size_t(tokens) * size_t(ld) * 2));
  Operands operand{space};
  const Operand d = operand(dout, tokens, dim);
  q.epi = mo::kEpiGatedGrad;
  q.act = act;
  q.b_mn = true;
  q.a[0] = d;
  q.b[0] = operand(w_down, dim, inner);
  operand.lay_out(run, stream);
  q.t[0] = {kept[0], nullptr, tokens, inner, ld, 0, 1, 0};
  q.out2 = kept[1];
  q.out3 = kept[2];
  q.k = dim;
  slice_ahead(q, static_cast<float*>(space.take(0)), sms, status, run, stream);
  if (run.error == cudaSuccess) run(mo::launch_product(q, sms, status, stream));
  if (dx != nullptr) {
    mo::Product s;
    s.b_mn = true;
    s.segments = 2;
    const void* w[2] = {w_gate, w_up};
    for (int i = 0; i < 2; ++i) {
      s.a[i] = {kept[i], tokens, inner, ld};
      s.b[i] = operand(w[i], inner, dim);
    }
    operand.lay_out(run, stream);
    s.t[0] = target(dx, dx_dtype, tokens, dim);
    s.k = inner;
    if (mo::longest_sum(s, sms) > kSlice) {   // one after the other, joined in fp32
      float* sums = static_cast<float*>(space.take(0));
      s.segments = 1;
      s.t[0] = target(sums, MO_F32, tokens, dim);
      if (run.error == cudaSuccess) run(mo::launch_product(s, sms, status, stream));
      s.a[0] = s.a[1];
      s.b[0] = s.b[1];
      s.t[0] = {dx, sums, tokens, dim, dim, dim, dx_dtype == MO_BF16, 0};
    }
    if (run.error == cudaSuccess) run(mo::launch_product(s, sms, status, stream));
  }
  if (any_dw) {   // up to three products over the tokens, one launch
    const Operand xo = need_x ? operand(xk, tokens, dim) : Operand{};
    operand.lay_out(run, stream);
    mo::Product s;
    s.a_mn = s.b_mn = true;
    s.count = 0;
    for (int i = 0; i < 3; ++i) {
      if (dw[i] == nullptr) continue;
      s.a[s.count] = i < 2 ? Operand{kept[i], tokens, inner, ld} : d;
      s.b[s.count] = i < 2 ? xo : Operand{kept[2], tokens, inner, ld};
      s.t[s.count] = target(dw[i], dw_dtype, i < 2 ? inner : dim, i < 2 ? dim : inner, accumulate ? dw[i] : nullptr);
      ++s.count;
    }
    s.k = tokens;
    sliced_product(s, reinterpret_cast<float*>(space.take(0)), sms, status, run, stream);
  }
  return run.status();
}

}  // extern "C"
