"""Binding of the training-step operators around the optimizer (include/mo.h):
embedding lookup and its gradient, counter-based dropout, and microscaled 4-bit
quantisation with its product.

Tensors are contiguous CUDA tensors on the current device, fp32 or bf16;
outputs are written in place, on the current stream unless one is given:

    drop = mo.Dropout(0.1, seed=seed, offset=4 * step)     # drawn again in the backward pass
    mo.embed_lookup(table, tokens, x, scale=1.0, add=positions, dropout=drop)
    ws = mo.embed_grad_workspace(tokens.numel(), *table.shape)   # reuse it every step
    mo.embed_grad(dx, tokens, g, ws, scale=1.0, dropout=drop)    # g: the fp32 gradient adamw_tail_step reads
    mo.dropout_apply(h, y, drop, residual=x)               # forward; with dy for h the backward pass

    wq, wt = mo.Fp4Tensor(n, k, "mx"), mo.Fp4Tensor(k, n, "mx")   # "mx": 32-element blocks; "nv": 16
    mo.fp4_quantize(w, wq, wt)                             # both orientations from one pass over w
    mo.fp4_quantize(dy, dyq, dyt, stochastic=mo.Random(seed, 4 * step + 1))   # dyt takes 4 * step + 2
    mo.fp4_product(xq, wq, y)                              # y = x w^T
    mo.fp4_product(dyt, xt, dw)                            # dw = dy^T x: the bf16 gradient muon_owner_step reads

Every dropout and every stochastic rounding of a step has an offset of its own,
and a step's offsets begin behind the last one's: uses that share seed and
offset draw the same numbers. fp4_quantize takes offset + 1 too, for by_col.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _check, load_library
from . import _stream_ptr as _stream_handle

MO_F32, MO_BF16 = 0, 1


class Random(ctypes.Structure):
    """mo_random: seed and offset of the counter-based generator. offset_dev, a
    one-element int64 CUDA tensor, is added to offset when the kernel runs."""
    _fields_ = [("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("d_offset", ctypes.c_void_p)]

    def __init__(self, seed=0, offset=0, offset_dev=None):
        super().__init__(int(seed), int(offset), _offset_ptr(offset_dev))
        self.keep = offset_dev


class Dropout(ctypes.Structure):
    """mo_dropout: probability p and the random numbers of the mask."""
    _fields_ = [("p", ctypes.c_float), ("random", Random)]

    def __init__(self, p, seed=0, offset=0, offset_dev=None):
        super().__init__(p, Random(seed, offset, offset_dev))
        self.keep = offset_dev


class MoTokens(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("n", ctypes.c_int64), ("padding_idx", ctypes.c_int64),
                ("bits", ctypes.c_int32)]


def _offset_ptr(t):
    if t is None:
        return None
    import torch
    if t.dtype != torch.int64 or t.numel() != 1 or not t.is_cuda:
        raise TypeError("offset_dev must be a one-element int64 CUDA tensor")
    return t.data_ptr()


_raw_stream = None


def _stream_ptr(stream, t) -> int:
    """The stream's handle; None: the current one of t's device, by torch's
    plain-integer query where it has one (2.8 us less a call than the Stream
    object on the Grace CPU)."""
    global _raw_stream
    if stream is not None:
        return _stream_handle(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(t.get_device())


def _dtype(t, name: str) -> int:
    import torch
    if t.dtype == torch.float32:
        code = MO_F32
    elif t.dtype == torch.bfloat16:
        code = MO_BF16
    else:
        raise TypeError(f"{name} must be fp32 or bf16")
    _dense(t, name)
    return code


def _dense(t, name: str) -> None:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _tokens(tokens, padding_idx: int = -1) -> MoTokens:
    import torch
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError("tokens must be int32 or int64")
    _dense(tokens, "tokens")
    return MoTokens(tokens.data_ptr(), tokens.numel(), padding_idx, 64 if tokens.dtype == torch.int64 else 32)


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def dropout_apply(x, out, dropout: Dropout, residual=None, stream=None) -> None:
    """out = drop(x) (+ residual); out may be x or residual. With dy for x and
    no residual it is the backward pass."""
    code = _dtype(x, "x")
    if _dtype(out, "out") != code or out.numel() != x.numel():
        raise ValueError("x and out must have equal types and sizes")
    if residual is not None and (_dtype(residual, "residual") != code or residual.numel() != x.numel()):
        raise ValueError("x and residual must have equal types and sizes")
    st = load_library().dropout_apply(x.data_ptr(), None if residual is None else residual.data_ptr(), out.data_ptr(),
                                      x.numel(), code, ctypes.byref(dropout), _stream_ptr(stream, x))
    _check(st, "dropout_apply")


def embed_lookup(table, tokens, out, scale: float = 1.0, add=None, dropout: Optional[Dropout] = None,
                 stream=None) -> None:
    """out[t] = drop(scale * table[tokens[t]] + add[t % len(add)]) for every
    token, in the order of the flattened tokens."""
    code, out_code = _dtype(table, "table"), _dtype(out, "out")
    if table.dim() != 2:
        raise ValueError("table must be [vocab, dim]")
    vocab, dim = table.shape
    if out.numel() != tokens.numel() * dim:
        raise ValueError("out must have dim elements for every token")
    if add is not None and (_dtype(add, "add") != code or add.dim() != 2 or add.shape[1] != dim):
        raise ValueError("add must be [rows, dim] of the table's type")
    tk = _tokens(tokens)
    st = load_library().embed_lookup(table.data_ptr(), code, vocab, dim, ctypes.byref(tk), scale,
                                     None if add is None else add.data_ptr(), 0 if add is None else add.shape[0],
                                     _ref(dropout), out.data_ptr(), out_code, _stream_ptr(stream, out))
    _check(st, "embed_lookup")


def mo_embed_grad_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    return int(load_library().mo_embed_grad_workspace_bytes(n, vocab, dim))


def embed_grad_workspace(n: int, vocab: int, dim: int, device=None):
    """A torch uint8 device tensor large enough for embed_grad of n tokens."""
    import torch
    return torch.empty(max(mo_embed_grad_workspace_bytes(n, vocab, dim), 256), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def embed_grad(dout, tokens, grad, workspace, scale: float = 1.0, padding_idx: int = -1, accumulate: bool = False,
               dropout: Optional[Dropout] = None, stream=None) -> None:
    """grad[v] (+)= scale * sum of dout[t] over the tokens t = v, under the
    forward pass's dropout; grad is fp32 [vocab, dim]. Without accumulate the
    rows no token names become 0."""
    import torch
    code = _dtype(dout, "dout")
    if grad.dtype != torch.float32 or grad.dim() != 2:
        raise TypeError("grad must be fp32 [vocab, dim]")
    _dense(grad, "grad")
    vocab, dim = grad.shape
    if dout.numel() != tokens.numel() * dim:
        raise ValueError("dout must have dim elements for every token")
    _dense(workspace, "workspace")
    tk = _tokens(tokens, padding_idx)
    st = load_library().embed_grad(dout.data_ptr(), code, ctypes.byref(tk), vocab, dim, scale, _ref(dropout),
                                   grad.data_ptr(), int(accumulate), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_ptr(stream, grad))
    _check(st, "embed_grad")


# ---------------------------------------------------------------- 4-bit tensors

FP4_FORMATS = {"mx": 0, "nv": 1}   # mo_fp4_format


class MoFp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("format", ctypes.c_int32)]


def mo_fp4_codes_bytes(rows: int, k: int) -> int:
    return int(load_library().mo_fp4_codes_bytes(rows, k))


def mo_fp4_scales_bytes(rows: int, k: int, fmt: str = "mx") -> int:
    return int(load_library().mo_fp4_scales_bytes(rows, k, FP4_FORMATS[fmt]))


class Fp4Tensor:
    """Storage of a microscaled 4-bit tensor [rows, k] (mo_fp4): uint8 `codes`
    and `scales` and, for "nv", a one-element fp32 `amax`. Allocated when not
    given; reuse it every step. Given codes and scales hold zeros in their
    padding, as fp4_quantize leaves it: fp4_product reads it."""

    def __init__(self, rows: int, k: int, fmt: str = "mx", codes=None, scales=None, amax=None, device=None):
        import torch
        if fmt not in FP4_FORMATS:
            raise ValueError('format must be "mx" or "nv"')
        device = device or torch.device("cuda")
        sizes = mo_fp4_codes_bytes(rows, k), mo_fp4_scales_bytes(rows, k, fmt)
        if rows and k and not all(sizes):
            raise ValueError("rows and k must be 0 to 2^22, with at most 2^37 elements")
        got = []
        for t, nbytes, name in ((codes, sizes[0], "codes"), (scales, sizes[1], "scales")):
            if t is None:
                t = torch.empty(nbytes, dtype=torch.uint8, device=device)
            if t.dtype != torch.uint8 or t.numel() != nbytes:
                raise ValueError(f"{name} must be {nbytes} uint8 elements")
            _dense(t, name)
            got.append(t)
        self.codes, self.scales = got
        if amax is None and fmt == "nv":
            amax = torch.ones(1, dtype=torch.float32, device=device)
        self.amax = _amax(amax)
        self.rows, self.k, self.format = rows, k, fmt
        self.arg = MoFp4(self.codes.data_ptr(), self.scales.data_ptr(), None if amax is None else amax.data_ptr(), rows, k,
                         FP4_FORMATS[fmt])


def _amax(t):
    import torch
    if t is not None and (t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda):
        raise TypeError("amax must be a one-element fp32 CUDA tensor")
    return t


def fp4_quantize(x, by_row: Optional[Fp4Tensor] = None, by_col: Optional[Fp4Tensor] = None, amax=None,
                 stochastic: Optional[Random] = None, stream=None) -> None:
    """Quantises x [rows, cols] into by_row [rows, cols] and, transposed, into
    by_col [cols, rows]. "nv" tensors take their scale from amax (a one-element
    fp32 CUDA tensor) or from x itself."""
    code = _dtype(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2D")
    st = load_library().fp4_quantize(x.data_ptr(), code, x.shape[0], x.shape[1],
                                     None if by_row is None else ctypes.byref(by_row.arg),
                                     None if by_col is None else ctypes.byref(by_col.arg),
                                     None if amax is None else _amax(amax).data_ptr(), _ref(stochastic), _stream_ptr(stream, x))
    _check(st, "fp4_quantize")


def fp4_dequantize(q: Fp4Tensor, out, stream=None) -> None:
    """out [rows, k] = the values q stands for."""
    code = _dtype(out, "out")
    if out.numel() != q.rows * q.k:
        raise ValueError("out must be [rows, k]")
    _check(load_library().fp4_dequantize(ctypes.byref(q.arg), out.data_ptr(), code, _stream_ptr(stream, out)), "fp4_dequantize")


def fp4_product(a: Fp4Tensor, b: Fp4Tensor, out, stream=None) -> None:
    """out [a.rows, b.rows] = a b^T over k; out is bf16 or fp32."""
    code = _dtype(out, "out")
    if out.numel() != a.rows * b.rows:
        raise ValueError("out must be [a.rows, b.rows]")
    _check(load_library().fp4_product(ctypes.byref(a.arg), ctypes.byref(b.arg), out.data_ptr(), code, _stream_ptr(stream, out)),
           "fp4_product")
