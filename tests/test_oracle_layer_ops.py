"""Pins of the float64 oracle of the feed-forward operators, and the argument
checks of their entry points (no GPU needed: a call is refused before anything
is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from matrix_optimizers_zero_gb300 import build as mo_build
from matrix_optimizers_zero_gb300.layer_ops import MoTensor
from oracle import layer_ops as ol

NULL, SHAPE, ALIGN, PARAM, WS, OVERLAP = -1, -2, -3, -4, -5, -6
F32, BF16, MX8 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    mo_build.build()
    return mo.load_library()


# ---------------------------------------------------------------- oracle

def test_e4m3_table_is_the_type():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ol.E4M3[:127])


def test_quantised_values_are_nearest_with_ties_to_even():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 70)) * np.exp(3 * rng.normal(size=(5, 1)))
    x[0, :32] = 0.0
    x[1, 0], x[1, 1] = 448.0, 17.0          # 17: halfway between 16 and 18, of which 16 is even
    x[1, 2:32] = 0.5
    codes, scales, values = ol.mx8_quantize(x)
    assert scales[0, 0] == 0 and scales[1, 0] == 127 and values[1, 1] == 16.0
    assert np.array_equal(ol.mx8_values(codes, scales, 70), values)
    top = np.abs(np.pad(x, ((0, 0), (0, 26))).reshape(5, 3, 32)).max(2)
    s = 2.0 ** (scales.astype(float) - 127)
    assert (top <= 448 * s).all() and ((top > 224 * s) | (scales == 0)).all()
    t = torch.from_numpy(np.pad(x, ((0, 0), (0, 26))) / np.repeat(s, 32, 1)).float()
    np.testing.assert_allclose(t.numpy(), np.pad(x, ((0, 0), (0, 26))) / np.repeat(s, 32, 1), rtol=2 ** -23)
    want = t.to(torch.float8_e4m3fn).double().numpy() * np.repeat(s, 32, 1)
    assert np.array_equal(want[:, :70], values)


@pytest.mark.parametrize("name", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_activations_match_torch(name):
    z = torch.linspace(-9, 9, 301, dtype=torch.float64).requires_grad_()
    f = {None: lambda v: v * 1.0, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    y = f(z)
    y.sum().backward()
    value, slope = ol.act(z.detach().numpy(), name)
    np.testing.assert_allclose(value, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(slope, z.grad.numpy(), rtol=1e-12, atol=1e-13)


def double(*shape, seed=0):
    return torch.from_numpy(np.random.default_rng(seed + sum(shape)).normal(size=shape)).requires_grad_()


def test_norm_gradients_match_autograd():
    x, r, w, dy = double(5, 13), double(5, 13, seed=1), double(13), double(5, 13, seed=2).detach()
    s = x + r
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-5) * w
    y.backward(dy)
    oy, os = ol.rms_norm(x.detach().numpy(), w.detach().numpy(), 1e-5, r.detach().numpy())
    dx, dw = ol.rms_norm_grad(dy.numpy(), os, w.detach().numpy(), 1e-5)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-12)


@pytest.mark.parametrize("name", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_product_gradients_match_autograd(name):
    f = {None: lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    x, w, b, dy = double(6, 7), double(9, 7), double(9), double(6, 9, seed=3).detach()
    f(x @ w.T + b).backward(dy)
    n = [t.detach().numpy() for t in (x, w, b)]
    _, z = ol.linear(*n, activation=name)
    for got, want in zip(ol.linear_grad(dy.numpy(), n[0], n[1], name, z), (x, w, b)):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)
    x, wg, wu, wd, dy = double(6, 7), double(11, 7), double(11, 7, seed=1), double(7, 11), double(6, 7, seed=4).detach()
    ((f(x @ wg.T) * (x @ wu.T)) @ wd.T).backward(dy)
    n = [t.detach().numpy() for t in (x, wg, wu, wd)]
    _, g, u = ol.gated_ffn(*n, activation=name)
    for got, want in zip(ol.gated_ffn_grad(dy.numpy(), n[0], g, u, *n[1:], activation=name), (x, wg, wu, wd)):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)


# ---------------------------------------------------------------- sizes

def test_storage_sizes(lib):
    assert lib.mo_mx8_codes_bytes(3, 33) == 3 * 64 and lib.mo_mx8_scales_bytes(3, 33) == 6
    assert lib.mo_mx8_codes_bytes(0, 33) == 0
    for rows, k in ((-1, 32), (2 ** 30 + 1, 32), (4, 0), (4, 2 ** 22 + 1), (2 ** 30, 2 ** 22)):
        assert lib.mo_mx8_codes_bytes(rows, k) == 0 and lib.mo_mx8_scales_bytes(rows, k) == 0


def test_workspace_sizes(lib):
    assert lib.mo_linear_workspace_bytes(8, 64, 64, 0) >= 8 * 64 * 2
    assert lib.mo_linear_workspace_bytes(8, 65, 64, 0) >= (8 + 64) * 65 * 2
    assert lib.mo_linear_workspace_bytes(8, 64, 64, 1) > lib.mo_linear_workspace_bytes(8, 64, 64, 0)
    assert lib.mo_linear_workspace_bytes(40000, 64, 64, 1) >= 2 * 40000 * 64 * 2 + 64 * 64 * 4
    assert lib.mo_gated_ffn_workspace_bytes(8, 64, 128, 1) >= 8 * (64 + 3 * 128) * 2
    for bad in ((-1, 64, 64, 0), (8, 0, 64, 0), (8, 64, 0, 0), (8, 2 ** 16 + 1, 64, 0), (8, 64, 2 ** 22 + 1, 0), (8, 64, 64, 2),
                (2 ** 30, 2 ** 16, 64, 0)):
        assert lib.mo_linear_workspace_bytes(*bad) == 0
    for bad in ((-1, 64, 64, 0), (8, 2 ** 16 + 1, 64, 0), (8, 64, 2 ** 15 + 1, 0)):
        assert lib.mo_gated_ffn_workspace_bytes(*bad) == 0
    assert lib.mo_rms_norm_grad_workspace_bytes(0, 8) == 256 and lib.mo_rms_norm_grad_workspace_bytes(5, 0) == 0


# ---------------------------------------------------------------- refusals

A, B, C, D, E, F, G, H, I, J, K, L = (0x100000000 * k for k in range(1, 13))   # far apart, aligned, never read
BIG = 1 << 30


def ten(data=A, scales=None, dtype=BF16):
    return MoTensor(data, scales, dtype)


def q8(data=A, scales=B):
    return MoTensor(data, scales, MX8)


def ref(t):
    return None if t is None else ctypes.byref(t)


def call_quantize(lib, x=C, dtype=BF16, rows=4, k=40, q=q8()):
    return lib.mx8_quantize(x, dtype, rows, k, ref(q), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(q=q8(None)), NULL), (dict(q=q8(A, None)), NULL), (dict(dtype=2), PARAM),
    (dict(q=ten()), PARAM), (dict(rows=-1), SHAPE), (dict(rows=2 ** 30 + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=2 ** 22 + 1), SHAPE),
    (dict(x=C + 8), ALIGN), (dict(q=q8(A + 8)), ALIGN), (dict(q=q8(C + 16)), OVERLAP), (dict(q=q8(A, C)), OVERLAP),
    (dict(q=q8(A, A + 64)), OVERLAP), (dict(rows=2 ** 20, k=2 ** 18), SHAPE),
])
def test_quantize_refusals(lib, kw, status):
    assert call_quantize(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), NULL), (dict(q=None), NULL), (dict(q=q8(None)), NULL), (dict(q=q8(A, None)), NULL), (dict(dtype=2), PARAM),
    (dict(q=ten()), PARAM), (dict(rows=-1), SHAPE), (dict(k=0), SHAPE), (dict(out=C + 8), ALIGN), (dict(q=q8(A + 8)), ALIGN),
    (dict(q=q8(C + 16)), OVERLAP), (dict(q=q8(A, C)), OVERLAP),
])
def test_dequantize_refusals(lib, kw, status):
    a = dict(dict(q=q8(), rows=4, k=40, out=C, dtype=BF16), **kw)
    assert lib.mx8_dequantize(ref(a["q"]), a["rows"], a["k"], a["out"], a["dtype"], None) == status


def call_norm(lib, x=A, res=None, dtype=BF16, rows=4, dim=40, w=B, eps=1e-6, sum_=None, out=C, odt=BF16, out8=None):
    return lib.rms_norm(x, res, dtype, rows, dim, w, eps, sum_, out, odt, ref(out8), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(out8=q8(D, None)), NULL), (dict(dtype=2), PARAM), (dict(odt=2), PARAM),
    (dict(eps=-1.0), PARAM), (dict(eps=float("nan")), PARAM), (dict(eps=float("inf")), PARAM), (dict(out8=ten(D)), PARAM),
    (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=2 ** 22 + 1), SHAPE), (dict(x=A + 2), ALIGN), (dict(w=B + 4), ALIGN),
    (dict(out=C + 8), ALIGN), (dict(res=D + 8), ALIGN), (dict(sum_=D + 8), ALIGN), (dict(out=A + 16), OVERLAP), (dict(out=B), OVERLAP),
    (dict(out=A, odt=F32), OVERLAP), (dict(sum_=C), OVERLAP), (dict(sum_=A, out=A), OVERLAP), (dict(out8=q8(C, D)), OVERLAP),
    (dict(out8=q8(D, A)), OVERLAP),
])
def test_norm_refusals(lib, kw, status):
    assert call_norm(lib, **kw) == status


def call_norm_grad(lib, dy=A, dtype=BF16, x=ten(B), rows=4, dim=40, w=C, eps=1e-6, dres=None, dx=D, dw=E, acc=0, ws=F, nbytes=BIG):
    return lib.rms_norm_grad(dy, dtype, ref(x), rows, dim, w, eps, dres, dx, dw, acc, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(dx=None), NULL), (dict(ws=None), NULL), (dict(x=q8(B, None)), NULL),
    (dict(x=ten(B, None, F32)), PARAM), (dict(dtype=2), PARAM), (dict(acc=2), PARAM), (dict(eps=-1e-9), PARAM), (dict(rows=-1), SHAPE),
    (dict(dim=0), SHAPE), (dict(dy=A + 2), ALIGN), (dict(x=ten(B + 2)), ALIGN), (dict(dw=E + 4), ALIGN), (dict(ws=F + 16), ALIGN),
    (dict(dres=G + 4), ALIGN), (dict(nbytes=16), WS), (dict(dx=B), OVERLAP), (dict(dx=A + 16), OVERLAP), (dict(dw=C), OVERLAP),
    (dict(ws=A), OVERLAP), (dict(dw=D), OVERLAP),
])
def test_norm_grad_refusals(lib, kw, status):
    assert call_norm_grad(lib, **kw) == status


def call_linear(lib, x=ten(A), w=B, t=8, k=64, n=32, bias=None, act=0, res=None, pre=None, out=C, odt=BF16, ws=D, nbytes=BIG):
    return lib.linear_forward(ref(x), w, t, k, n, bias, act, res, ref(pre), out, odt, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(x=q8(A, None)), NULL),
    (dict(act=1, pre=ten(None)), NULL), (dict(x=ten(A, None, F32)), PARAM), (dict(act=5), PARAM), (dict(act=-1), PARAM),
    (dict(odt=2), PARAM), (dict(pre=ten(E)), PARAM), (dict(act=1, pre=ten(E, None, F32)), PARAM), (dict(t=-1), SHAPE),
    (dict(k=0), SHAPE), (dict(k=2 ** 16 + 1), SHAPE), (dict(n=0), SHAPE), (dict(n=2 ** 22 + 1), SHAPE), (dict(t=2 ** 30 + 1), SHAPE),
    (dict(x=ten(A + 2)), ALIGN), (dict(w=B + 8), ALIGN), (dict(bias=E + 4), ALIGN), (dict(out=C + 4), ALIGN), (dict(ws=D + 128), ALIGN),
    (dict(res=E + 2), ALIGN), (dict(nbytes=64), WS), (dict(out=A + 16), OVERLAP), (dict(out=B), OVERLAP), (dict(res=C + 16), OVERLAP),
    (dict(ws=A), OVERLAP), (dict(act=1, pre=ten(C)), OVERLAP), (dict(bias=C), OVERLAP),
])
def test_linear_refusals(lib, kw, status):
    assert call_linear(lib, **kw) == status


def call_linear_grad(lib, dout=A, x=ten(B), w=C, t=8, k=64, n=32, act=0, pre=None, dx=D, dxt=BF16, dw=E, dwt=BF16, db=F, acc=0, ws=G,
                     nbytes=BIG):
    return lib.linear_grad(dout, ref(x), w, t, k, n, act, ref(pre), dx, dxt, dw, dwt, db, acc, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(act=1), NULL),
    (dict(dx=None, dw=None, db=None), NULL), (dict(act=7), PARAM), (dict(pre=ten(H)), PARAM), (dict(acc=-1), PARAM), (dict(dxt=2), PARAM),
    (dict(dwt=3), PARAM), (dict(x=ten(B, None, F32)), PARAM), (dict(act=1, pre=ten(H, None, F32)), PARAM), (dict(t=-1), SHAPE),
    (dict(k=2 ** 16 + 1), SHAPE), (dict(dout=A + 2), ALIGN), (dict(dx=D + 2), ALIGN), (dict(dw=E + 2), ALIGN), (dict(db=F + 4), ALIGN),
    (dict(w=C + 2), ALIGN), (dict(ws=G + 8), ALIGN), (dict(nbytes=128), WS), (dict(dx=A), OVERLAP), (dict(dw=B), OVERLAP),
    (dict(dw=C), OVERLAP), (dict(db=E), OVERLAP), (dict(ws=E), OVERLAP), (dict(dx=E), OVERLAP),
])
def test_linear_grad_refusals(lib, kw, status):
    assert call_linear_grad(lib, **kw) == status


def call_ffn(lib, x=ten(A), wg=B, wu=C, wd=D, t=8, d=64, f=96, act=4, res=None, gate=None, up=None, out=E, odt=BF16, ws=F, nbytes=BIG):
    return lib.gated_ffn_forward(ref(x), wg, wu, wd, t, d, f, act, res, ref(gate), ref(up), out, odt, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(wg=None), NULL), (dict(wu=None), NULL), (dict(wd=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(gate=ten(G)), NULL), (dict(up=ten(G)), NULL), (dict(gate=ten(G), up=q8(H, I)), PARAM), (dict(act=9), PARAM), (dict(odt=2), PARAM),
    (dict(x=ten(A, None, F32)), PARAM), (dict(t=-1), SHAPE), (dict(d=0), SHAPE), (dict(f=2 ** 15 + 1), SHAPE), (dict(d=2 ** 16 + 1), SHAPE),
    (dict(wg=B + 2), ALIGN), (dict(wu=C + 2), ALIGN), (dict(wd=D + 2), ALIGN), (dict(out=E + 2), ALIGN), (dict(ws=F + 2), ALIGN),
    (dict(nbytes=512), WS), (dict(out=A), OVERLAP), (dict(ws=D), OVERLAP), (dict(gate=ten(G), up=ten(G)), OVERLAP),
    (dict(gate=ten(E), up=ten(H)), OVERLAP), (dict(res=E + 16), OVERLAP),
])
def test_gated_ffn_refusals(lib, kw, status):
    assert call_ffn(lib, **kw) == status


def call_ffn_grad(lib, dout=A, x=ten(B), gate=ten(C), up=ten(D), wg=E, wu=F, wd=G, t=8, d=64, f=96, act=4, dx=H, dxt=BF16, dwg=I, dwu=J,
                  dwd=K, dwt=BF16, acc=0, ws=L, nbytes=BIG):
    return lib.gated_ffn_grad(dout, ref(x), ref(gate), ref(up), wg, wu, wd, t, d, f, act, dx, dxt, dwg, dwu, dwd, dwt, acc, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), NULL), (dict(x=None), NULL), (dict(gate=None), NULL), (dict(up=None), NULL), (dict(wd=None), NULL), (dict(wg=None), NULL),
    (dict(ws=None), NULL), (dict(dx=None, dwg=None, dwu=None, dwd=None), NULL), (dict(up=q8(D, 13 * A)), PARAM), (dict(act=-2), PARAM),
    (dict(dxt=2), PARAM), (dict(dwt=2), PARAM), (dict(acc=5), PARAM), (dict(f=0), SHAPE), (dict(dout=A + 2), ALIGN), (dict(dwu=J + 4), ALIGN),
    (dict(wd=G + 2), ALIGN), (dict(ws=L + 32), ALIGN), (dict(nbytes=1000), WS), (dict(dx=A), OVERLAP), (dict(dwg=J), OVERLAP),
    (dict(dwd=G), OVERLAP), (dict(ws=C), OVERLAP), (dict(dx=D), OVERLAP),
])
def test_gated_ffn_grad_refusals(lib, kw, status):
    assert call_ffn_grad(lib, **kw) == status


def test_no_tokens_is_no_work(lib):
    """Empty tensors have no address."""
    assert call_linear(lib, x=ten(None), t=0, out=None) == 0
    assert call_ffn(lib, x=ten(None), t=0, out=None) == 0
    assert call_norm(lib, x=None, out=None, rows=0) == 0
    assert call_quantize(lib, x=None, q=q8(None, None), rows=0) == 0
    assert call_linear_grad(lib, dout=None, x=ten(None), t=0, dx=None, dw=None, db=None) == 0
    assert call_linear_grad(lib, dout=None, x=ten(None), t=0, dx=None, acc=1) == 0
    assert call_norm_grad(lib, dy=None, x=ten(None), rows=0, dx=None, dw=None) == 0
