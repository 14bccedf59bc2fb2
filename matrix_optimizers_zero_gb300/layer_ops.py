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

from . import _check, load_library
from .train_ops import MO_BF16, MO_F32, _dense, _dtype, _stream_ptr

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
        got = []
        for t, width, name in ((codes, 32 * blocks, "codes"), (scales, blocks, "scales")):
            if t is None:
                t = torch.empty((rows, width), dtype=torch.uint8, device=device)
            if t.dtype != torch.uint8 or t.numel() != rows * width:
                raise ValueError(f"{name} must be {rows * width} uint8 elements")
            _dense(t, name)
            got.append(t)
        self.codes, self.scales = got
        if self.codes.get_device() != self.scales.get_device():
            raise ValueError("codes and scales must be on one device")
        self.rows, self.k = rows, k
        self.arg = MoTensor(self.codes.data_ptr(), self.scales.data_ptr(), MO_MX8)

    def numel(self) -> int:
        return self.rows * self.k

    def get_device(self) -> int:
        return self.codes.get_device()


def _here(*tensors) -> None:
    """All on the current device, which the library launches on."""
    import torch
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError("tensors must be on the current device")


def _rows(t, width: int, name: str) -> int:
    """Rows of a tensor whose rows have `width` elements."""
    if (t.k if isinstance(t, Mx8Tensor) else t.shape[-1] if t.dim() else 0) != width:
        raise ValueError(f"rows of {name} must have {width} elements")
    return t.rows if isinstance(t, Mx8Tensor) else t.numel() // width


def _kept(t, name: str, f32: bool = False):
    """mo_tensor of a plain or an 8-bit tensor."""
    if isinstance(t, Mx8Tensor):
        return t.arg
    code = _dtype(t, name)
    if code == MO_F32 and not f32:
        raise TypeError(f"{name} must be bf16 or an Mx8Tensor")
    return MoTensor(t.data_ptr(), None, code)


def _matrix(t, rows: int, cols: int, name: str):
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bf16")
    _dense(t, name)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    return t.data_ptr()


def _vector(t, n: int, name: str):
    import torch
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be fp32")
    _dense(t, name)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements")
    return t.data_ptr()


def _same(t, like, code: int, name: str):
    if t is None:
        return None
    if _dtype(t, name) != code or t.numel() != like.numel():
        raise ValueError(f"{name} must have the type and size of the tensor it goes with")
    return t.data_ptr()


def _result(t, rows: int, cols: int, name: str):
    """Pointer and type of an output of rows * cols elements; (None, bf16) for none."""
    if t is None:
        return None, MO_BF16
    code = _dtype(t, name)
    if t.numel() != rows * cols:
        raise ValueError(f"{name} must have {rows} x {cols} elements")
    return t.data_ptr(), code


def _scratch(t):
    _dense(t, "workspace")
    return t.data_ptr(), t.numel() * t.element_size()


def _act(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(str(k) for k in ACTIVATIONS)}")
    return ACTIVATIONS[name]


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
    code = _dtype(x, "x")
    if _rows(x, q.k, "x") != q.rows:
        raise ValueError("x and q must have equal sizes")
    _here(x, q)
    _check(load_library().mx8_quantize(x.data_ptr(), code, q.rows, q.k, ctypes.byref(q.arg), _stream_ptr(stream, x)), "mx8_quantize")


def mx8_dequantize(q: Mx8Tensor, out, stream=None) -> None:
    """out [rows, k], fp32 or bf16, = the values q stands for."""
    ptr, code = _result(out, q.rows, q.k, "out")
    _here(q, out)
    _check(load_library().mx8_dequantize(ctypes.byref(q.arg), q.rows, q.k, ptr, code, _stream_ptr(stream, out)), "mx8_dequantize")


# ---------------------------------------------------------------- norm

def rms_norm(x, out=None, weight=None, eps: float = 1e-6, residual=None, sum_out=None, out8=None, stream=None) -> None:
    """y = s / sqrt(mean(s^2) + eps) * weight over the rows (the last dimension)
    of s = x + residual, into out (fp32 or bf16), out8 (an Mx8Tensor), or both;
    s into sum_out. sum_out and out may each be x or residual."""
    code = _dtype(x, "x")
    dim = x.shape[-1] if x.dim() else 0
    if dim == 0:
        raise ValueError("rows of x must have elements")
    rows = x.numel() // dim
    if out is None and out8 is None:
        raise ValueError("out or out8 must be given")
    ptr, out_code = _result(out, rows, dim, "out")
    if out8 is not None and (not isinstance(out8, Mx8Tensor) or (out8.rows, out8.k) != (rows, dim)):
        raise ValueError(f"out8 must be an Mx8Tensor of [{rows}, {dim}]")
    _here(x, out, weight, residual, sum_out, out8)
    st = load_library().rms_norm(x.data_ptr(), _same(residual, x, code, "residual"), code, rows, dim, _vector(weight, dim, "weight"),
                                 eps, _same(sum_out, x, code, "sum_out"), ptr, out_code,
                                 None if out8 is None else ctypes.byref(out8.arg), _stream_ptr(stream, x))
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
    code = _dtype(dy, "dy")
    dim = dy.shape[-1] if dy.dim() else 0
    if dim == 0:
        raise ValueError("rows of dy must have elements")
    rows = dy.numel() // dim
    if _rows(x, dim, "x") != rows:
        raise ValueError("dy and x must have equal sizes")
    arg = _kept(x, "x", f32=True)
    if arg.dtype not in (MO_MX8, code):
        raise TypeError("x must have the type of dy, or be an Mx8Tensor")
    if dweight is not None and workspace is None:
        raise ValueError("dweight needs a workspace (rms_norm_grad_workspace)")
    ws, nbytes = _scratch(workspace) if workspace is not None else (None, 0)
    _here(dy, x, dx, weight, dresidual, dweight, workspace)
    st = load_library().rms_norm_grad(dy.data_ptr(), code, ctypes.byref(arg), rows, dim, _vector(weight, dim, "weight"), eps,
                                      _same(dresidual, dy, code, "dresidual"), _same(dx, dy, code, "dx"),
                                      _vector(dweight, dim, "dweight"), int(accumulate), ws, nbytes, _stream_ptr(stream, dy))
    _check(st, "rms_norm_grad")


# ---------------------------------------------------------------- products

def mo_linear_workspace_bytes(tokens: int, cols: int, rows: int, grad: bool = False) -> int:
    return int(load_library().mo_linear_workspace_bytes(tokens, cols, rows, int(grad)))


def linear_workspace(tokens: int, cols: int, rows: int, grad: bool = False, device=None):
    """A torch uint8 device tensor for linear (and, with grad, linear_grad) of a weight [rows, cols]."""
    return _workspace(mo_linear_workspace_bytes(tokens, cols, rows, grad), device)


def linear(x, w, out, bias=None, activation=None, residual=None, pre=None, workspace=None, stream=None) -> None:
    """out = act(x w^T + bias) + residual, in one launch: x bf16 or an Mx8Tensor
    [tokens, cols], w bf16 [rows, cols], bias fp32, out (fp32 or bf16) and residual
    of one type (out may be residual). pre: bf16 or an Mx8Tensor [tokens, rows]
    that receives x w^T + bias for linear_grad."""
    act = _act(activation)
    rows, cols = w.shape if w.dim() == 2 else (0, 0)
    wp = _matrix(w, rows, cols, "w")
    tokens = _rows(x, cols, "x")
    xk = _kept(x, "x")
    ptr, code = _result(out, tokens, rows, "out")
    pk = None if pre is None else _kept(pre, "pre")
    if pre is not None and _rows(pre, rows, "pre") != tokens:
        raise ValueError("pre must have a row for every token")
    if pre is not None and not act:
        raise ValueError("pre goes with an activation")
    if workspace is None:
        raise ValueError("a workspace is needed (linear_workspace)")
    ws, nbytes = _scratch(workspace)
    _here(x, w, out, bias, residual, pre, workspace)
    st = load_library().linear_forward(ctypes.byref(xk), wp, tokens, cols, rows, _vector(bias, rows, "bias"), act,
                                       _same(residual, out, code, "residual"), _ref(pk), ptr, code, ws, nbytes,
                                       _stream_ptr(stream, out))
    _check(st, "linear")


def linear_grad(dout, x, w, dx=None, dw=None, dbias=None, activation=None, pre=None, workspace=None, accumulate: bool = False,
                stream=None) -> None:
    """Gradients of linear from dout (bf16) and what was kept: dx, dw (fp32 or
    bf16) and the fp32 dbias, whichever are given; dw and dbias are added to with
    accumulate. x may be None without dw, and an Mx8Tensor in place of the x that
    linear was given."""
    act = _act(activation)
    rows, cols = w.shape if w.dim() == 2 else (0, 0)
    wp = _matrix(w, rows, cols, "w")
    if dx is None and dw is None and dbias is None:
        raise ValueError("dx, dw or dbias must be given")
    tokens = _rows(dout, rows, "dout")
    dk = _kept(dout, "dout")
    if dk.dtype != MO_BF16:
        raise TypeError("dout must be bf16")
    if dw is not None and x is None:
        raise ValueError("dw needs x")
    xk = None
    if dw is not None:
        if _rows(x, cols, "x") != tokens:
            raise ValueError("dout and x must have a row for every token")
        xk = _kept(x, "x")
    if bool(act) != (pre is not None):
        raise ValueError("pre goes with an activation, and an activation with pre")
    pk = None
    if act:
        if _rows(pre, rows, "pre") != tokens:
            raise ValueError("pre must have a row for every token")
        pk = _kept(pre, "pre")
    dxp, dx_code = _result(dx, tokens, cols, "dx")
    dwp, dw_code = _result(dw, rows, cols, "dw")
    if workspace is None:
        raise ValueError("a workspace is needed (linear_workspace)")
    ws, nbytes = _scratch(workspace)
    _here(dout, x if dw is not None else None, w, dx, dw, dbias, pre, workspace)
    st = load_library().linear_grad(dk.data, _ref(xk), wp, tokens, cols, rows, act, _ref(pk), dxp, dx_code, dwp, dw_code,
                                    _vector(dbias, rows, "dbias"), int(accumulate), ws, nbytes, _stream_ptr(stream, dout))
    _check(st, "linear_grad")


# ---------------------------------------------------------------- gated feed-forward block

def mo_gated_ffn_workspace_bytes(tokens: int, dim: int, inner: int, grad: bool = False) -> int:
    return int(load_library().mo_gated_ffn_workspace_bytes(tokens, dim, inner, int(grad)))


def gated_ffn_workspace(tokens: int, dim: int, inner: int, grad: bool = False, device=None):
    """A torch uint8 device tensor for gated_ffn (and, with grad, gated_ffn_grad)."""
    return _workspace(mo_gated_ffn_workspace_bytes(tokens, dim, inner, grad), device)


def _gated_weights(w_gate, w_up, w_down):
    inner, dim = w_gate.shape if w_gate.dim() == 2 else (0, 0)
    return dim, inner, (_matrix(w_gate, inner, dim, "w_gate"), _matrix(w_up, inner, dim, "w_up"), _matrix(w_down, dim, inner, "w_down"))


def _gated_kept(gate, up, tokens: int, inner: int):
    gk, uk = _kept(gate, "gate"), _kept(up, "up")
    if gk.dtype != uk.dtype:
        raise TypeError("gate and up must be of one type")
    if _rows(gate, inner, "gate") != tokens or _rows(up, inner, "up") != tokens:
        raise ValueError("gate and up must have a row for every token")
    return gk, uk


def gated_ffn(x, w_gate, w_up, w_down, out, activation="silu", residual=None, gate=None, up=None, workspace=None,
              stream=None) -> None:
    """out = (act(x w_gate^T) * (x w_up^T)) w_down^T + residual: x bf16 or an
    Mx8Tensor [tokens, dim], bf16 weights [inner, dim] and [dim, inner], out (fp32
    or bf16) and residual of one type (out may be residual). gate and up: bf16 or
    Mx8Tensors [tokens, inner] that receive the two projections for gated_ffn_grad."""
    act = _act(activation)
    dim, inner, w = _gated_weights(w_gate, w_up, w_down)
    tokens = _rows(x, dim, "x")
    xk = _kept(x, "x")
    ptr, code = _result(out, tokens, dim, "out")
    if (gate is None) != (up is None):
        raise ValueError("gate and up go together")
    gk, uk = (None, None) if gate is None else _gated_kept(gate, up, tokens, inner)
    if workspace is None:
        raise ValueError("a workspace is needed (gated_ffn_workspace)")
    ws, nbytes = _scratch(workspace)
    _here(x, w_gate, w_up, w_down, out, residual, gate, up, workspace)
    st = load_library().gated_ffn_forward(ctypes.byref(xk), *w, tokens, dim, inner, act, _same(residual, out, code, "residual"),
                                          _ref(gk), _ref(uk), ptr, code, ws, nbytes, _stream_ptr(stream, out))
    _check(st, "gated_ffn")


def gated_ffn_grad(dout, x, gate, up, w_gate, w_up, w_down, activation="silu", dx=None, dw_gate=None, dw_up=None, dw_down=None,
                   workspace=None, accumulate: bool = False, stream=None) -> None:
    """Gradients of gated_ffn from dout (bf16) and the kept gate and up: dx
    (fp32 or bf16) and those of the weights (of one type), whichever are given; the
    weights' are added to with accumulate. x may be None without dw_gate and dw_up."""
    act = _act(activation)
    dim, inner, w = _gated_weights(w_gate, w_up, w_down)
    tokens = _rows(dout, dim, "dout")
    dk = _kept(dout, "dout")
    if dk.dtype != MO_BF16:
        raise TypeError("dout must be bf16")
    grads = [_result(t, *s, n) for t, s, n in ((dw_gate, (inner, dim), "dw_gate"), (dw_up, (inner, dim), "dw_up"),
                                               (dw_down, (dim, inner), "dw_down"))]
    codes = {code for p, code in grads if p is not None}
    if len(codes) > 1:
        raise TypeError("the weights' gradients must be of one type")
    if dx is None and not codes:
        raise ValueError("dx or a weight's gradient must be given")
    need_x = dw_gate is not None or dw_up is not None
    if need_x and x is None:
        raise ValueError("dw_gate and dw_up need x")
    xk = None
    if need_x:
        if _rows(x, dim, "x") != tokens:
            raise ValueError("dout and x must have a row for every token")
        xk = _kept(x, "x")
    gk, uk = _gated_kept(gate, up, tokens, inner)
    dxp, dx_code = _result(dx, tokens, dim, "dx")
    if workspace is None:
        raise ValueError("a workspace is needed (gated_ffn_workspace)")
    ws, nbytes = _scratch(workspace)
    _here(dout, x if need_x else None, gate, up, w_gate, w_up, w_down, dx, dw_gate, dw_up, dw_down, workspace)
    st = load_library().gated_ffn_grad(dk.data, _ref(xk), ctypes.byref(gk), ctypes.byref(uk), *w, tokens, dim, inner, act, dxp,
                                       dx_code, grads[0][0], grads[1][0], grads[2][0], codes.pop() if codes else MO_BF16,
                                       int(accumulate), ws, nbytes, _stream_ptr(stream, dout))
    _check(st, "gated_ffn_grad")
