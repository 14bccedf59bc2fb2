"""Pins of the float64 oracle of the training-step operators, and the argument
checks of their entry points (no GPU needed: a call is refused before anything
is enqueued)."""
import ctypes

import numpy as np
import pytest

import matrix_optimizers_zero_gb300 as mo
from matrix_optimizers_zero_gb300 import build as mo_build
from matrix_optimizers_zero_gb300.train_ops import MoTokens
from oracle import train_ops as ot

NULL, SHAPE, ALIGN, PARAM, WS, OVERLAP = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    mo_build.build()
    return mo.load_library()


# ---------------------------------------------------------------- oracle

@pytest.mark.parametrize("counter,key,expect", [
    # the generator's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, expect):
    assert tuple(ot.philox4x32_10(counter, key)) == expect


def test_random16_is_philox_by_element():
    seed, offset, first = 0x1234567890ABCDEF, (7 << 32) + 3, 8 * (1 << 32) - 5   # counters on both sides of 2^32
    got = ot.random16(21, seed, offset, first)
    for i in range(21):
        e = first + i
        j = e // 8
        w = ot.philox4x32_10((j & ot.M32, j >> 32, offset & ot.M32, offset >> 32), (seed & ot.M32, seed >> 32))
        k = e % 8
        assert got[i] == (w[k // 2] >> (16 * (k % 2))) & 0xFFFF


def test_dropout_oracle_rate_and_mean():
    n, p = 400000, 0.1
    f = ot.dropout_factors((n,), p, seed=11)
    T = round(65536 * p)
    q = T / 65536
    sd = (q * (1 - q) / n) ** 0.5
    assert abs((f == 0).mean() - q) < 5 * sd             # five standard deviations of a binomial share
    assert abs(f.mean() - 1.0) < 5 * sd / (1 - q)        # kept ones carry 1 / (1 - q)


def test_embed_grad_oracle_is_the_lookups_transpose():
    rng = np.random.default_rng(0)
    V, d, n = 13, 5, 40
    E, D = rng.normal(size=(V, d)), rng.normal(size=(V, d))
    tok = rng.integers(0, V, n)
    dout = rng.normal(size=(n, d))
    drop = (0.3, 5, 2)
    g = ot.embed_grad(dout, tok, V, scale=1.5, drop=drop)
    diff = ot.embed_lookup(E + D, tok, 1.5, drop=drop) - ot.embed_lookup(E, tok, 1.5, drop=drop)
    np.testing.assert_allclose((diff * dout).sum(), (g * D).sum(), rtol=1e-12)


# ---------------------------------------------------------------- refusals

A, B, C, D_, E_ = (0x100000000 * k for k in range(1, 6))   # far apart, aligned, never read


def tok(n=16, ids=E_, bits=64, pad=-1):
    return MoTokens(ids, n, pad, bits)


def drop(p=0.1, **kw):
    d = mo.Dropout(p, seed=1)
    for k, v in kw.items():
        setattr(d.random, k, v)
    return d


def call_dropout(lib, x=A, res=None, y=B, n=64, dtype=0, d=drop()):
    return lib.dropout_apply(x, res, y, n, dtype, ctypes.byref(d) if d is not None else None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=A + 8), ALIGN), (dict(y=B + 4), ALIGN),
    (dict(res=C + 2), ALIGN), (dict(n=-1), SHAPE), (dict(dtype=2), PARAM), (dict(d=drop(1.5)), PARAM),
    (dict(d=drop(-0.1)), PARAM), (dict(d=drop(float("nan"))), PARAM), (dict(y=A + 16), OVERLAP),
    (dict(res=B + 16), OVERLAP), (dict(d=drop(d_offset=C + 4)), ALIGN),
])
def test_dropout_refusals(lib, kw, status):
    assert call_dropout(lib, **kw) == status


def call_lookup(lib, table=A, tdt=0, V=100, dim=8, t=None, scale=1.0, add=None, add_rows=0, d=None, out=B, odt=1):
    return lib.embed_lookup(table, tdt, V, dim, ctypes.byref(t if t is not None else tok()), scale, add, add_rows,
                            ctypes.byref(d) if d is not None else None, out, odt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), NULL), (dict(out=None), NULL), (dict(t=tok(ids=None)), NULL), (dict(V=0), SHAPE),
    (dict(V=2 ** 31), SHAPE), (dict(dim=0), SHAPE), (dict(dim=2 ** 22 + 1), SHAPE), (dict(t=tok(n=-1)), SHAPE),
    (dict(t=tok(n=2 ** 30 + 1)), SHAPE), (dict(t=tok(bits=16)), PARAM), (dict(t=tok(ids=E_ + 4)), ALIGN),
    (dict(table=A + 4), ALIGN), (dict(out=B + 8), ALIGN), (dict(add=C + 8, add_rows=4), ALIGN),
    (dict(add=C, add_rows=0), SHAPE), (dict(tdt=3), PARAM), (dict(odt=-1), PARAM), (dict(scale=float("inf")), PARAM),
    (dict(d=drop(2.0)), PARAM), (dict(out=A + 16), OVERLAP), (dict(out=E_), OVERLAP), (dict(add=B + 16, add_rows=2), OVERLAP),
])
def test_lookup_refusals(lib, kw, status):
    assert call_lookup(lib, **kw) == status


def call_grad(lib, dout=A, dt=0, t=None, V=100, dim=8, scale=1.0, d=None, grad=B, acc=0, ws=C, wsb=1 << 20):
    return lib.embed_grad(dout, dt, ctypes.byref(t if t is not None else tok()), V, dim, scale,
                          ctypes.byref(d) if d is not None else None, grad, acc, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), NULL), (dict(grad=None), NULL), (dict(ws=None), NULL), (dict(dout=A + 8), ALIGN),
    (dict(grad=B + 4), ALIGN), (dict(ws=C + 16), ALIGN), (dict(V=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dt=7), PARAM),
    (dict(acc=2), PARAM), (dict(scale=float("nan")), PARAM), (dict(wsb=16), WS), (dict(dout=B + 16), OVERLAP),
    (dict(ws=B), OVERLAP), (dict(ws=E_), OVERLAP), (dict(t=tok(ids=B)), OVERLAP),
])
def test_grad_refusals(lib, kw, status):
    assert call_grad(lib, **kw) == status


def test_empty_calls_are_no_ops(lib):
    assert call_dropout(lib, n=0, x=None, y=None) == 0
    assert call_lookup(lib, t=tok(n=0, ids=None)) == 0
    assert call_grad(lib, t=tok(n=0, ids=None), acc=1) == 0


def test_grad_workspace_bytes(lib):
    assert mo.mo_embed_grad_workspace_bytes(-1, 100, 8) == 0
    assert mo.mo_embed_grad_workspace_bytes(5, 0, 8) == 0
    assert mo.mo_embed_grad_workspace_bytes(5, 100, 0) == 0
    sizes = [mo.mo_embed_grad_workspace_bytes(n, 128256, 4096) for n in (0, 1, 1000, 16384, 1 << 20)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    # keys and positions twice, and two partial rows for every 64 positions
    assert sizes[-1] >= 16 * (1 << 20) + 2 * (1 << 14) * 4096 * 4


def test_status_names_the_bad_token(lib):
    assert "token" in mo.mo_status_string(-11)


# ---------------------------------------------------------------- 4-bit tensors

@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_fp4_oracle_rounds_to_nearest_and_never_saturates(fmt):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(40, 100)) * np.exp(2 * rng.normal(size=(40, 1)))
    codes, bits, values = ot.fp4_quantize(x, fmt)
    s = ot.fp4_scale_values(fmt)[bits] * (ot.fp4_tensor_scale(np.abs(x).max()) if fmt == "nv" else 1.0)
    B = ot.FP4_BLOCK[fmt]
    for r in range(40):
        for k in range(100):
            grid = np.concatenate([-ot.FP4_GRID, ot.FP4_GRID]) * s[r, k // B]
            assert abs(values[r, k] - x[r, k]) <= np.abs(grid - x[r, k]).min() * (1 + 1e-12)
            assert abs(x[r, k]) <= 6 * s[r, k // B]
    # the next smaller scale would not do
    for r in range(40):
        for b in range(bits.shape[1]):
            if bits[r, b] > 0:
                smaller = s[r, b] * ot.fp4_scale_values(fmt)[bits[r, b] - 1] / ot.fp4_scale_values(fmt)[bits[r, b]]
                assert np.abs(x[r, b * B:(b + 1) * B]).max() > 6 * smaller * (1 - 1e-15)


def test_fp4_oracle_ties_go_to_the_even_code():
    # scale 1 (the block's maximum is 6): the midpoints of the grid
    x = np.zeros((1, 32))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    codes, bits, values = ot.fp4_quantize(x, "mx")
    assert bits[0, 0] == 127
    assert list(values[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4]


def test_fp4_oracle_stochastic_rounding_is_unbiased():
    n = 32 * 4000
    x = np.tile(np.linspace(-6, 6, 32), 4000).reshape(4000, 32)
    _, _, values = ot.fp4_quantize(x, "mx", (5, 6))
    mean = values.mean(axis=0)
    # the widest step is 2: a standard deviation of at most 1 an element
    assert np.all(np.abs(mean - x[0]) < 5 / np.sqrt(4000) + 2 ** -15)


@pytest.mark.parametrize("amax,g", [(2688.0, 1.0), (2688.1, 2.0), (1344.0, 0.5), (0.0, 1.0), (1e-45, 2.0 ** -126)])
def test_fp4_oracle_tensor_scale(amax, g):
    assert ot.fp4_tensor_scale(amax) == g


class Fp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("format", ctypes.c_int32)]


def q4(rows=64, k=96, fmt=0, codes=C, scales=D_, amax=E_):
    return Fp4(codes, scales, amax, rows, k, fmt)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def call_quantize(lib, x=A, dt=0, rows=64, cols=96, row=q4(), col=None, amax=None, rnd=None):
    return lib.fp4_quantize(x, dt, rows, cols, ref(row), ref(col), amax, ref(rnd), None)


@pytest.mark.parametrize("kw,status", [
    (dict(row=None), NULL), (dict(x=None), NULL), (dict(row=q4(codes=None)), NULL), (dict(row=q4(scales=None)), NULL),
    (dict(row=q4(fmt=1, amax=None)), NULL), (dict(dt=5), PARAM), (dict(row=q4(fmt=2)), PARAM),
    (dict(col=q4(96, 64, 1, B, B + 65536)), PARAM), (dict(rows=-1), SHAPE), (dict(row=q4(63)), SHAPE),
    (dict(col=q4(64, 96, 0, B, B + 65536)), SHAPE), (dict(cols=2 ** 22 + 1), SHAPE), (dict(x=A + 8), ALIGN),
    (dict(row=q4(codes=C + 8)), ALIGN), (dict(row=q4(scales=D_ + 4)), ALIGN), (dict(amax=E_ + 2), ALIGN),
    (dict(rnd=mo.Random(1), row=q4(fmt=1, amax=E_ + 1)), ALIGN), (dict(row=q4(codes=A + 64)), OVERLAP),
    (dict(row=q4(scales=C + 16)), OVERLAP), (dict(col=q4(96, 64, 0, C + 16, B)), OVERLAP),
])
def test_quantize_refusals(lib, kw, status):
    assert call_quantize(lib, **kw) == status


def call_product(lib, a=None, b=None, out=B, dt=1):
    a = a if a is not None else q4()
    b = b if b is not None else q4(32, 96, 0, A, A + 65536)
    return lib.fp4_product(ref(a), ref(b), out, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(a=q4(codes=None)), NULL), (dict(out=None), NULL), (dict(a=q4(fmt=1)), PARAM), (dict(dt=9), PARAM),
    (dict(a=q4(k=64)), SHAPE), (dict(a=q4(rows=-3)), SHAPE), (dict(a=q4(2 ** 22, 2 ** 22)), SHAPE), (dict(out=B + 8), ALIGN),
    (dict(out=C), OVERLAP), (dict(out=A + 65536), OVERLAP),
])
def test_product_refusals(lib, kw, status):
    assert call_product(lib, **kw) == status


def test_dequantize_refusals(lib):
    assert lib.fp4_dequantize(None, B, 0, None) == NULL
    assert lib.fp4_dequantize(ref(q4()), None, 0, None) == NULL
    assert lib.fp4_dequantize(ref(q4()), B, 3, None) == PARAM
    assert lib.fp4_dequantize(ref(q4()), B + 4, 0, None) == ALIGN
    assert lib.fp4_dequantize(ref(q4()), C, 0, None) == OVERLAP
    assert lib.fp4_dequantize(ref(q4(k=-1)), B, 0, None) == SHAPE


def test_fp4_empty_calls_are_no_ops(lib):
    assert call_quantize(lib, rows=0, row=q4(0, 96)) == 0
    assert call_product(lib, a=q4(0)) == 0
    assert lib.fp4_dequantize(ref(q4(0, 96)), None, 0, None) == 0


def test_fp4_storage_sizes(lib):
    assert mo.mo_fp4_codes_bytes(3, 33) == 3 * 32
    assert mo.mo_fp4_scales_bytes(129, 129, "mx") == 2 * 2 * 512
    assert mo.mo_fp4_scales_bytes(1, 65, "nv") == 2 * 512
    assert mo.mo_fp4_codes_bytes(-1, 4) == 0 and mo.mo_fp4_scales_bytes(4, 2 ** 23, "nv") == 0
