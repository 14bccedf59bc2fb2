"""Binding of the feed-forward operators (include/mo.h): root-mean-square norm
with the residual's addition, matrix products with bias, activation and residual
in their epilogue, the gated feed-forward block, and the 8-bit activation
checkpoints that their backward passes read.

Tensors are contiguous CUDA tensors on the current device; outputs are written
in place, on the current stream unless one is given. Weights and the
activations of products are bf16; `Mx8Tensor` stands wherever an activation may
be in 8 bits. One layer's second half, s being the residual stream:

    n8, s8 = mo.Mx8Tensor(t, d), mo.Mx8Tensor(t, d)
    g8, u8 = mo.Mx8Tensor(t, f), mo.Mx8Tensor(t, f)
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)              # reuse it every step
    mo.rms_norm(attn, weight=w, residual=s, sum_out=s, out8=n8)  # s += attn; n8: the block's input and its checkpoint
    mo.mx8_quantize(s, s8)                                       # the norm's checkpoint
    mo.gated_ffn(n8, wg, wu, wd, s, residual=s, gate=g8, up=u8, workspace=ws)
    # backward, ds: the gradient of the stream
    mo.gated_ffn_grad(ds, n8, g8, u8, wg, wu, wd, dx=dn, dw_gate=Gg, dw_up=Gu, dw_down=Gd, workspace=ws)
    mo.rms_norm_grad(dn, s8, ds, weight=w, dresidual=ds, dweight=gw, workspace=norm_ws)

Gg, Gu and Gd are the bf16 gradients muon_owner_step reads, gw the fp32 one of
adamw_tail_step. A GPT-2 style block is two calls of `linear`:

    mo.linear(x, w1, h, bias=b1, activation="gelu_tanh", pre=z8, workspace=ws)
    mo.linear(h, w2, s, bias=b2, residual=s, workspace=ws)
    mo.linear_grad(ds, h, w2, dx=dh, dw=G2, dbias=gb2, workspace=ws)
    mo.linear_grad(dh, x, w1, dx=dx, dw=G1, dbias=gb1, activation="gelu_tanh", pre=z8, workspace=ws)
"""
from __future__ import annotations

import ctypes
import math

from . import _check, load_library
from .train_ops import MO_BF16, MO_F32, _dense, _stream_ptr

MO_MX8 = 2
ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}   # mo_activation


class MoTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("dtype", ctypes.c_int32)]


def mo_mx8_codes_bytes(rows: int, k: int) -> int:
    return int(load_library().mo_mx8_codes_bytes(rows, k))


def mo_mx8_scales_bytes(rows: int, k: int) -> int:
    return int(load_library().mo_mx8_scales_bytes(rows, k))


class Mx8Tensor:
    """Storage of an 8-bit tensor [rows, k] (mo_tensor of MO_MX8): uint8
    `codes` [rows, 32 ceil(k / 32)] and `scales` [rows, ceil(k / 32)].
    Allocated when not given; reuse it every step."""

    def __init__(self, rows: int, k: int, codes=None, scales=None, device=None):
        import torch
        if not (0 <= rows <= 1 << 30 and 1 <= k <= 1 << 22) or (rows and not mo_mx8_codes_bytes(rows, k)):
            raise ValueError("rows must be 0 to 2^30 and k 1 to 2^22, with at most 2^37 elements")
        device = device or torch.device("cuda")
        blocks = -(-k // 32)
        self.rows, self.k = rows, k
        self.codes, self.scales = (torch.empty((rows, width), dtype=torch.uint8, device=device) if t is None else t
                                   for t, width in ((codes, 32 * blocks), (scales, blocks)))
        self._look()

    def _look(self):
        """Checks the storage and takes its addresses."""
        import torch
        blocks = -(-self.k // 32)
        for t, width, name in ((self.codes, 32 * blocks, "codes"), (self.scales, blocks, "scales")):
            if t.dtype != torch.uint8 or t.numel() != self.rows * width:
                raise ValueError(f"{name} must be {self.rows * width} uint8 elements")
            _dense(t, name)
        if self.codes.get_device() != self.scales.get_device():
            raise ValueError("codes and scales must be on one device")
        self.device_index = self.codes.get_device()
        self.at, self.scales_at = self.codes.data_ptr(), self.scales.data_ptr()
        self.arg = MoTensor(self.at, self.scales_at, MO_MX8)

    def address(self) -> MoTensor:
        """mo_tensor of the storage where it is now: codes or scales may have been replaced or moved."""
        if self.codes.data_ptr() != self.at or self.scales.data_ptr() != self.scales_at:
            self._look()
        return self.arg

    def numel(self) -> int:
        return self.rows * self.k

    def get_device(self) -> int:
        return self.device_index


# A call of one token takes a few microseconds on the GPU, and as many here: each
# tensor is asked once for what is checked of it.

_dtypes = None          # {torch dtype: mo_dtype}, from the first call on
_current_device = None


def _here() -> int:
    """The current device, which the library launches on and all tensors must be on."""
    global _dtypes, _current_device
    if _dtypes is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _dtypes = {torch.float32: MO_F32, torch.bfloat16: MO_BF16}   # last: another thread that sees it finds both
    return _current_device()


def _refuse(t, name: str, here: int, types: str):
    if t.dtype not in _dtypes:
        raise TypeError(f"{name} must be {types}")
    if t.get_device() < 0 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    raise ValueError(f"{name} must be on the current device ({here})")


def _plain(t, name: str, here: int):
    """(pointer, type) of an fp32 or bf16 tensor."""
    code = _dtypes.get(t.dtype)
    if code is None or t.get_device() != here or not t.is_contiguous():
        _refuse(t, name, here, "fp32 or bf16")
    return t.data_ptr(), code


def _sized(t, shape, name: str):
    """Refuses a tensor of another size than `shape`, or one that lies as the transposed matrix does. Views of
    the same rows ([batch, tokens, heads, width of a head] or all in one dimension) are as good as
    [tokens, width]."""
    numel, ends, at = math.prod(shape), {1}, 1
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements")
    for n in t.shape:
        at *= n
        ends.add(at)
    if len(shape) > 1 and shape[-1] in ends and numel // max(shape[-1], 1) not in ends:
        raise ValueError(f"{name} must be {list(shape)}, not its transpose")


def _typed(t, name: str, here: int, code: int, shape):
    """Pointer of a tensor that must have a type and a shape; None for none."""
    if t is None:
        return None
    if _dtypes.get(t.dtype) != code:
        raise TypeError(f"{name} must be {'bf16' if code == MO_BF16 else 'fp32'}")
    if t.get_device() != here or not t.is_contiguous():
        _refuse(t, name, here, "")
    if t.shape != shape:
        _sized(t, shape, name)
    return t.data_ptr()


def _matrix(t, shape, name: str, here: int):
    """Pointer of a bf16 matrix of a shape."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if _dtypes.get(t.dtype) != MO_BF16:
        raise TypeError(f"{name} must be bf16")
    if t.get_device() != here or not t.is_contiguous():
        _refuse(t, name, here, "")
    return t.data_ptr()


def _rows(t, width: int, name: str) -> int:
    """Rows of a tensor whose rows have `width` elements."""
    if isinstance(t, Mx8Tensor):
        if t.k == width:
            return t.rows
    else:
        shape = t.shape
        if len(shape) and shape[-1] == width:
            return shape[0] if len(shape) == 2 else t.numel() // width
    raise ValueError(f"rows of {name} must have {width} elements")


def _kept(t, name: str, here: int, f32: bool = False):
    """mo_tensor of a plain or an 8-bit tensor."""
    if isinstance(t, Mx8Tensor):
        arg = t.address()
        if t.device_index != here:
            raise ValueError(f"{name} must be on the current device ({here})")
        return arg
    code = _dtypes.get(t.dtype)
    if code != MO_BF16 and not (f32 and code == MO_F32):
        raise TypeError(f"{name} must be bf16 or an Mx8Tensor")
    if t.get_device() != here or not t.is_contiguous():
        _refuse(t, name, here, "")
    return MoTensor(t.data_ptr(), None, code)


def _kept_rows(t, width: int, rows: int, name: str, here: int, f32: bool = False):
    """The same, of a tensor with so many rows."""
    if _rows(t, width, name) != rows:
        raise ValueError(f"{name} must have {rows} rows")
    return _kept(t, name, here, f32)


def _result(t, shape, name: str, here: int):
    """Pointer and type of an output; (None, bf16) for none."""
    if t is None:
        return None, MO_BF16
    got = _plain(t, name, here)
    if t.shape != shape:
        _sized(t, shape, name)
    return got


def _scratch(t, name: str, here: int):
    if t is None:
        raise ValueError(f"a workspace is needed ({name})")
    if t.get_device() != here or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the current device")
    return t.data_ptr(), t.nbytes


def _act(name):
    code = ACTIVATIONS.get(name)   # (0: none)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(str(k) for k in ACTIVATIONS)}")
    return code


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _workspace(nbytes: int, device):
    import torch
    if not nbytes:
        raise ValueError("sizes out of range")
    return torch.empty(nbytes, dtype=torch.uint8, device=device or torch.device("cuda"))


# ---------------------------------------------------------------- 8-bit tensors

def mx8_quantize(x, q: Mx8Tensor, stream=None) -> None:
    """q = x [rows, k], fp32 or bf16, in 8 bits."""
    here = _here()
    arg = _kept(q, "q", here)
    ptr, code = _plain(x, "x", here)
    if _rows(x, q.k, "x") != q.rows:
        raise ValueError("x and q must have equal sizes")
    _check(load_library().mx8_quantize(ptr, code, q.rows, q.k, ctypes.byref(arg), _stream_ptr(stream, x)), "mx8_quantize")


def mx8_dequantize(q: Mx8Tensor, out, stream=None) -> None:
    """out [rows, k], fp32 or bf16, = the values q stands for."""
    here = _here()
    arg = _kept(q, "q", here)
    ptr, code = _result(out, (q.rows, q.k), "out", here)
    _check(load_library().mx8_dequantize(ctypes.byref(arg), q.rows, q.k, ptr, code, _stream_ptr(stream, out)), "mx8_dequantize")


# ---------------------------------------------------------------- norm

def rms_norm(x, out=None, weight=None, eps: float = 1e-6, residual=None, sum_out=None, out8=None, stream=None) -> None:
    """y = s / sqrt(mean(s^2) + eps) * weight over the rows (the last dimension)
    of s = x + residual, into out (fp32 or bf16), out8 (an Mx8Tensor), or both;
    s into sum_out. sum_out and out may each be x or residual."""
    here = _here()
    ptr, code = _plain(x, "x", here)
    shape, numel = x.shape, x.numel()
    dim = shape[-1] if len(shape) else 0
    if dim == 0:
        raise ValueError("rows of x must have elements")
    rows = numel // dim
    if out is None and out8 is None:
        raise ValueError("out or out8 must be given")
    out_ptr, out_code = _result(out, shape, "out", here)
    arg8 = None
    if out8 is not None:
        if not isinstance(out8, Mx8Tensor) or (out8.rows, out8.k) != (rows, dim):
            raise ValueError(f"out8 must be an Mx8Tensor of [{rows}, {dim}]")
        arg8 = ctypes.byref(_kept(out8, "out8", here))
    st = load_library().rms_norm(ptr, _typed(residual, "residual", here, code, shape), code, rows, dim,
                                 _typed(weight, "weight", here, MO_F32, (dim,)), eps, _typed(sum_out, "sum_out", here, code, shape), out_ptr,
                                 out_code, arg8, _stream_ptr(stream, x))
    _check(st, "rms_norm")


def mo_rms_norm_grad_workspace_bytes(rows: int, dim: int) -> int:
    return int(load_library().mo_rms_norm_grad_workspace_bytes(rows, dim))


def rms_norm_grad_workspace(rows: int, dim: int, device=None):
    """A torch uint8 device tensor for rms_norm_grad with a dweight."""
    return _workspace(mo_rms_norm_grad_workspace_bytes(rows, dim), device)


def rms_norm_grad(dy, x, dx, weight=None, eps: float = 1e-6, dresidual=None, dweight=None, workspace=None,
                  accumulate: bool = False, stream=None) -> None:
    """Gradients of rms_norm from dy and s, the rows it normalised (x: of dy's
    type, or an Mx8Tensor): dx (+ dresidual; it may be dy or dresidual) and the
    fp32 dweight, added to with accumulate, for which the workspace is needed."""
    here = _here()
    ptr, code = _plain(dy, "dy", here)
    shape, numel = dy.shape, dy.numel()
    dim = shape[-1] if len(shape) else 0
    if dim == 0:
        raise ValueError("rows of dy must have elements")
    rows = numel // dim
    arg = _kept_rows(x, dim, rows, "x", here, f32=True)
    if arg.dtype not in (MO_MX8, code):
        raise TypeError("x must have the type of dy, or be an Mx8Tensor")
    ws, nbytes = (None, 0) if dweight is None else _scratch(workspace, "rms_norm_grad_workspace", here)
    st = load_library().rms_norm_grad(ptr, code, ctypes.byref(arg), rows, dim, _typed(weight, "weight", here, MO_F32, (dim,)), eps,
                                      _typed(dresidual, "dresidual", here, code, shape), _typed(dx, "dx", here, code, shape),
                                      _typed(dweight, "dweight", here, MO_F32, (dim,)), int(accumulate), ws, nbytes, _stream_ptr(stream, dy))
    _check(st, "rms_norm_grad")


# ---------------------------------------------------------------- products

def mo_linear_workspace_bytes(tokens: int, cols: int, rows: int, grad: bool = False) -> int:
    return int(load_library().mo_linear_workspace_bytes(tokens, cols, rows, int(grad)))


def linear_workspace(tokens: int, cols: int, rows: int, grad: bool = False, device=None):
    """A torch uint8 device tensor for linear (and, with grad, linear_grad) of a weight [rows, cols]."""
    return _workspace(mo_linear_workspace_bytes(tokens, cols, rows, grad), device)


def linear(x, w, out, bias=None, activation=None, residual=None, pre=None, workspace=None, stream=None) -> None:
    """out = act(x w^T + bias) + residual: x bf16 or an Mx8Tensor [tokens, cols],
    w bf16 [rows, cols], bias fp32, out (fp32 or bf16) and residual of one type (out
    may be residual, but not x). pre: bf16 or an Mx8Tensor [tokens, rows] that
    receives x w^T + bias for linear_grad. One launch, and one more where x is in 8
    bits or cols is no multiple of 8."""
    here = _here()
    act = _act(activation)
    shape = w.shape
    if len(shape) != 2:
        raise ValueError("w must be [rows, cols]")
    rows, cols = shape
    wp = _matrix(w, shape, "w", here)
    tokens = _rows(x, cols, "x")
    xk = _kept(x, "x", here)
    out_shape = tokens, rows
    ptr, code = _result(out, out_shape, "out", here)
    pk = None
    if pre is not None:
        if not act:
            raise ValueError("pre goes with an activation")
        pk = ctypes.byref(_kept_rows(pre, rows, tokens, "pre", here))
    ws, nbytes = _scratch(workspace, "linear_workspace", here)
    st = load_library().linear_forward(ctypes.byref(xk), wp, tokens, cols, rows, _typed(bias, "bias", here, MO_F32, (rows,)), act,
                                       _typed(residual, "residual", here, code, out_shape), pk, ptr, code, ws, nbytes,
                                       _stream_ptr(stream, out))
    _check(st, "linear")


def linear_grad(dout, x, w, dx=None, dw=None, dbias=None, activation=None, pre=None, workspace=None, accumulate: bool = False,
                stream=None) -> None:
    """Gradients of linear from dout (bf16) and what was kept: dx, dw (fp32 or
    bf16) and the fp32 dbias, whichever are given; dw and dbias are added to with
    accumulate. x may be None without dw, and an Mx8Tensor in place of the x that
    linear was given."""
    here = _here()
    act = _act(activation)
    shape = w.shape
    if len(shape) != 2:
        raise ValueError("w must be [rows, cols]")
    rows, cols = shape
    wp = _matrix(w, shape, "w", here)
    if dx is None and dw is None and dbias is None:
        raise ValueError("dx, dw or dbias must be given")
    tokens = _rows(dout, rows, "dout")
    dp = _typed(dout, "dout", here, MO_BF16, (tokens, rows))
    xk = None
    if dw is not None:
        if x is None:
            raise ValueError("dw needs x")
        xk = ctypes.byref(_kept_rows(x, cols, tokens, "x", here))
    if bool(act) != (pre is not None):
        raise ValueError("pre goes with an activation, and an activation with pre")
    pk = ctypes.byref(_kept_rows(pre, rows, tokens, "pre", here)) if act else None
    dxp, dx_code = _result(dx, (tokens, cols), "dx", here)
    dwp, dw_code = _result(dw, shape, "dw", here)
    ws, nbytes = _scratch(workspace, "linear_workspace", here)
    st = load_library().linear_grad(dp, xk, wp, tokens, cols, rows, act, pk, dxp, dx_code, dwp, dw_code,
                                    _typed(dbias, "dbias", here, MO_F32, (rows,)), int(accumulate), ws, nbytes, _stream_ptr(stream, dout))
    _check(st, "linear_grad")


# ---------------------------------------------------------------- gated feed-forward block

def mo_gated_ffn_workspace_bytes(tokens: int, dim: int, inner: int, grad: bool = False) -> int:
    return int(load_library().mo_gated_ffn_workspace_bytes(tokens, dim, inner, int(grad)))


def gated_ffn_workspace(tokens: int, dim: int, inner: int, grad: bool = False, device=None):
    """A torch uint8 device tensor for gated_ffn (and, with grad, gated_ffn_grad)."""
    return _workspace(mo_gated_ffn_workspace_bytes(tokens, dim, inner, grad), device)


def _gated_weights(w_gate, w_up, w_down, here: int):
    shape = w_gate.shape
    if len(shape) != 2:
        raise ValueError("w_gate must be [inner, dim]")
    inner, dim = shape
    return dim, inner, (_matrix(w_gate, shape, "w_gate", here), _matrix(w_up, shape, "w_up", here),
                        _matrix(w_down, (dim, inner), "w_down", here))


def _gated_kept(gate, up, tokens: int, inner: int, here: int):
    gk, uk = _kept_rows(gate, inner, tokens, "gate", here), _kept_rows(up, inner, tokens, "up", here)
    if gk.dtype != uk.dtype:
        raise TypeError("gate and up must be of one type")
    return gk, uk


def gated_ffn(x, w_gate, w_up, w_down, out, activation="silu", residual=None, gate=None, up=None, workspace=None,
              stream=None) -> None:
    """out = (act(x w_gate^T) * (x w_up^T)) w_down^T + residual: x bf16 or an
    Mx8Tensor [tokens, dim], bf16 weights [inner, dim] and [dim, inner], out (fp32
    or bf16) and residual of one type (out may be residual, and both x). gate and up: bf16 or
    Mx8Tensors [tokens, inner] that receive the two projections for gated_ffn_grad."""
    here = _here()
    act = _act(activation)
    dim, inner, w = _gated_weights(w_gate, w_up, w_down, here)
    tokens = _rows(x, dim, "x")
    xk = _kept(x, "x", here)
    out_shape = tokens, dim
    ptr, code = _result(out, out_shape, "out", here)
    if (gate is None) != (up is None):
        raise ValueError("gate and up go together")
    gk, uk = (None, None) if gate is None else _gated_kept(gate, up, tokens, inner, here)
    ws, nbytes = _scratch(workspace, "gated_ffn_workspace", here)
    st = load_library().gated_ffn_forward(ctypes.byref(xk), *w, tokens, dim, inner, act,
                                          _typed(residual, "residual", here, code, out_shape), _ref(gk), _ref(uk), ptr, code, ws, nbytes,
                                          _stream_ptr(stream, out))
    _check(st, "gated_ffn")


def gated_ffn_grad(dout, x, gate, up, w_gate, w_up, w_down, activation="silu", dx=None, dw_gate=None, dw_up=None, dw_down=None,
                   workspace=None, accumulate: bool = False, stream=None) -> None:
    """Gradients of gated_ffn from dout (bf16) and the kept gate and up: dx
    (fp32 or bf16) and those of the weights (of one type), whichever are given; the
    weights' are added to with accumulate. x may be None without dw_gate and dw_up."""
    here = _here()
    act = _act(activation)
    dim, inner, w = _gated_weights(w_gate, w_up, w_down, here)
    tokens = _rows(dout, dim, "dout")
    dp = _typed(dout, "dout", here, MO_BF16, (tokens, dim))
    grads = [_result(t, s, n, here) for t, s, n in ((dw_gate, (inner, dim), "dw_gate"), (dw_up, (inner, dim), "dw_up"), (dw_down, (dim, inner), "dw_down"))]
    codes = {code for t, (_, code) in zip((dw_gate, dw_up, dw_down), grads) if t is not None}
    if len(codes) > 1:
        raise TypeError("the weights' gradients must be of one type")
    if dx is None and not codes:
        raise ValueError("dx or a weight's gradient must be given")
    xk = None
    if dw_gate is not None or dw_up is not None:
        if x is None:
            raise ValueError("dw_gate and dw_up need x")
        xk = ctypes.byref(_kept_rows(x, dim, tokens, "x", here))
    gk, uk = _gated_kept(gate, up, tokens, inner, here)
    dxp, dx_code = _result(dx, (tokens, dim), "dx", here)
    ws, nbytes = _scratch(workspace, "gated_ffn_workspace", here)
    st = load_library().gated_ffn_grad(dp, xk, ctypes.byref(gk), ctypes.byref(uk), *w, tokens, dim, inner, act, dxp, dx_code, grads[0][0],
                                       grads[1][0], grads[2][0], codes.pop() if codes else MO_BF16, int(accumulate), ws, nbytes,
                                       _stream_ptr(stream, dout))
    _check(st, "gated_ffn_grad")
