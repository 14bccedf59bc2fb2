"""What the binding of the feed-forward operators checks of its tensors (no GPU
needed: stand-ins for CUDA tensors, and one for the library that records its
calls)."""
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from matrix_optimizers_zero_gb300 import layer_ops

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


class Tensor:
    def __init__(self, shape, dtype=BF16, device=0, contiguous=True):
        self.shape, self.dtype, self.device_index, self._contiguous = torch.Size(shape), dtype, device, contiguous
        self.is_cuda = device >= 0

    def is_contiguous(self):
        return self._contiguous

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device_index


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *args: 256
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(layer_ops, "load_library", lambda: lib)
    monkeypatch.setattr(layer_ops, "_stream_ptr", lambda stream, t: 0)
    monkeypatch.setattr(layer_ops, "_here", lambda: 0)
    monkeypatch.setattr(layer_ops, "_dtypes", {F32: 0, BF16: 1})
    return lib


def mx8(rows, k, device=0):
    nb = -(-k // 32)
    return mo.Mx8Tensor(rows, k, codes=Tensor((rows, 32 * nb), U8, device), scales=Tensor((rows, nb), U8, device))


WS = dict(workspace=Tensor((256,), U8))
T, D, F = 6, 40, 72


def calls():
    """name -> (function, keyword arguments of a call that is right)"""
    t = Tensor
    return {
        "mx8_quantize": (mo.mx8_quantize, dict(x=t((T, D), F32), q=mx8(T, D))),
        "mx8_dequantize": (mo.mx8_dequantize, dict(q=mx8(T, D), out=t((T, D)))),
        "rms_norm": (mo.rms_norm, dict(x=t((T, D)), out=t((T, D), F32), weight=t((D,), F32), residual=t((T, D)), sum_out=t((T, D)), out8=mx8(T, D))),
        "rms_norm_grad": (mo.rms_norm_grad, dict(dy=t((T, D)), x=mx8(T, D), dx=t((T, D)), weight=t((D,), F32), dresidual=t((T, D)),
                                                 dweight=t((D,), F32), **WS)),
        "linear": (mo.linear, dict(x=t((T, D)), w=t((F, D)), out=t((T, F), F32), bias=t((F,), F32), activation="gelu", residual=t((T, F), F32),
                                   pre=mx8(T, F), **WS)),
        "linear_grad": (mo.linear_grad, dict(dout=t((T, F)), x=mx8(T, D), w=t((F, D)), dx=t((T, D), F32), dw=t((F, D)), dbias=t((F,), F32),
                                             activation="gelu", pre=t((T, F)), **WS)),
        "gated_ffn": (mo.gated_ffn, dict(x=mx8(T, D), w_gate=t((F, D)), w_up=t((F, D)), w_down=t((D, F)), out=t((T, D)), residual=t((T, D)),
                                         gate=mx8(T, F), up=mx8(T, F), **WS)),
        "gated_ffn_grad": (mo.gated_ffn_grad, dict(dout=t((T, D)), x=t((T, D)), gate=t((T, F)), up=t((T, F)), w_gate=t((F, D)), w_up=t((F, D)),
                                                   w_down=t((D, F)), dx=t((T, D), F32), dw_gate=t((F, D)), dw_up=t((F, D)), dw_down=t((D, F)),
                                                   **WS)),
    }


SYMBOL = {"linear": "linear_forward", "gated_ffn": "gated_ffn_forward"}
NAMES = ["mx8_quantize", "mx8_dequantize", "rms_norm", "rms_norm_grad", "linear", "linear_grad", "gated_ffn", "gated_ffn_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_the_right_call_reaches_the_library(library, name):
    f, kw = calls()[name]
    f(**kw)
    assert [n for n, _ in library.calls] == [SYMBOL.get(name, name)]


def every(name_list):
    for name in name_list:
        for arg in TENSOR_ARGS[name]:
            yield name, arg


TENSOR_ARGS = {
    "mx8_quantize": ["x"], "mx8_dequantize": ["out"], "rms_norm": ["x", "out", "weight", "residual", "sum_out"],
    "rms_norm_grad": ["dy", "dx", "weight", "dresidual", "dweight", "workspace"],
    "linear": ["x", "w", "out", "bias", "residual", "workspace"], "linear_grad": ["dout", "w", "dx", "dw", "dbias", "pre", "workspace"],
    "gated_ffn": ["w_gate", "w_up", "w_down", "out", "residual", "workspace"],
    "gated_ffn_grad": ["dout", "x", "gate", "up", "w_gate", "w_up", "w_down", "dx", "dw_gate", "dw_up", "dw_down", "workspace"]}


@pytest.mark.parametrize("fault", ["host", "other device", "strided"])
@pytest.mark.parametrize("name,arg", list(every(NAMES)))
def test_refuses_tensors_from_elsewhere(library, name, arg, fault):
    f, kw = calls()[name]
    v = kw[arg]
    kw[arg] = Tensor(v.shape, v.dtype, {"host": -1, "other device": 1}.get(fault, 0), fault != "strided")
    with pytest.raises(ValueError, match="CUDA tensor|device"):
        f(**kw)
    assert not library.calls


@pytest.mark.parametrize("name,arg", [(n, a) for n, a in every(NAMES) if a != "workspace"])
def test_refuses_other_types_and_sizes(library, name, arg):
    f, kw = calls()[name]
    v = kw[arg]
    kw[arg] = Tensor(v.shape, torch.float16)
    with pytest.raises(TypeError):
        f(**kw)
    kw[arg] = Tensor((*v.shape[:-1], v.shape[-1] + 1), v.dtype)
    with pytest.raises(ValueError):
        f(**kw)
    assert not library.calls


@pytest.mark.parametrize("name,arg", [("mx8_quantize", "q"), ("mx8_dequantize", "q"), ("rms_norm", "out8"), ("rms_norm_grad", "x"), ("linear", "pre"),
                                      ("linear_grad", "x"), ("gated_ffn", "x"), ("gated_ffn", "gate"), ("gated_ffn", "up")])
def test_refuses_8_bit_tensors_of_other_sizes_and_devices(library, name, arg):
    f, kw = calls()[name]
    q = kw[arg]
    for bad in (mx8(q.rows + 1, q.k), mx8(q.rows, q.k + 1), mx8(q.rows, q.k, device=1)):
        kw[arg] = bad
        with pytest.raises(ValueError):
            f(**kw)
    assert not library.calls


@pytest.mark.parametrize("name,kw,error", [
    ("rms_norm", dict(out=None, out8=None), ValueError), ("rms_norm", dict(out8=Tensor((T, D))), ValueError), ("rms_norm", dict(x=Tensor(())), ValueError),
    ("rms_norm", dict(residual=Tensor((T, D), F32)), TypeError), ("rms_norm_grad", dict(workspace=None), ValueError),
    ("rms_norm_grad", dict(x=Tensor((T, D), F32)), TypeError), ("linear", dict(activation="tanh"), ValueError), ("linear", dict(activation=None), ValueError),
    ("linear", dict(workspace=None), ValueError), ("linear", dict(x=Tensor((T, D), F32)), TypeError), ("linear", dict(residual=Tensor((T, F))), TypeError),
    ("linear", dict(w=Tensor((F * D,))), ValueError), ("linear_grad", dict(x=None), ValueError), ("linear_grad", dict(pre=None), ValueError),
    ("linear_grad", dict(activation=None), ValueError), ("linear_grad", dict(dx=None, dw=None, dbias=None), ValueError),
    ("gated_ffn", dict(gate=None), ValueError), ("gated_ffn", dict(up=Tensor((T, F))), TypeError), ("gated_ffn", dict(w_down=Tensor((F, D))), ValueError),
    ("gated_ffn_grad", dict(x=None), ValueError), ("gated_ffn_grad", dict(dw_up=Tensor((F, D), F32)), TypeError),
    ("gated_ffn_grad", dict(dx=None, dw_gate=None, dw_up=None, dw_down=None), ValueError), ("gated_ffn_grad", dict(gate="8 bits"), TypeError)])
def test_refuses_calls_that_do_not_fit_together(library, name, kw, error):
    f, good = calls()[name]
    kw = {k: mx8(T, F) if isinstance(v, str) and v == "8 bits" else v for k, v in kw.items()}
    with pytest.raises(error):
        f(**{**good, **kw})
    assert not library.calls


@pytest.mark.parametrize("kw", [dict(rows=-1, k=4), dict(rows=2, k=0), dict(rows=(1 << 30) + 1, k=4), dict(rows=2, k=(1 << 22) + 1)])
def test_8_bit_tensor_sizes(kw):
    with pytest.raises(ValueError):
        mo.Mx8Tensor(**kw)


def test_8_bit_tensor_storage():
    for codes, scales in ((Tensor((2, 64), U8), Tensor((2, 1), U8)), (Tensor((2, 64), torch.int8), Tensor((2, 2), U8)),
                          (Tensor((2, 40), U8), Tensor((2, 2), U8)), (Tensor((2, 64), U8), Tensor((2, 2), U8, device=1)),
                          (Tensor((2, 64), U8, device=-1), Tensor((2, 2), U8)), (Tensor((2, 64), U8, contiguous=False), Tensor((2, 2), U8))):
        with pytest.raises(ValueError):
            mo.Mx8Tensor(2, 40, codes=codes, scales=scales)
    q = mo.Mx8Tensor(2, 40, codes=Tensor((2, 64), U8), scales=Tensor((2, 2), U8))
    assert (q.arg.dtype, q.numel()) == (2, 80)
