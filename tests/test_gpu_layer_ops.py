"""Feed-forward operators on the GPU against the float64 oracle.

Bounds, element by element. A product's sum of K terms: each addition in fp32
is off by at most 2^-23 of the magnitudes so far (truncation counted), so
K 2^-23 of the sum of the terms' magnitudes. A rounding to a type: eps / 2 of
the value. A logistic function: its exponent's argument is off by a few units
of 2^-24 of itself and the fast exponential by (2 + 1.2 |x|) 2^-23, so
(8 + 4 |u|) 2^-23 of the value with u the argument. gelu's normal distribution is
a published approximation (Abramowitz and Stegun 7.1.26): erfc within 1.5e-7, so
0.75e-7 < 2^-23 times the argument, and 2 y^2 2^-23 for the exponent. What an
error passes through multiplies it by at most its slope (|act'| <= 1.13)."""
import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from gpu_util import f64
from oracle import layer_ops as ol

pytestmark = pytest.mark.gpu
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16
TINY = 1e-37   # below the smallest normal number


def dev():
    return torch.device("cuda")


def data(*shape, dtype=BF16, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g) * std).to(dtype).to(dev())


def empty8(rows, k, fill=0x5A):
    q = mo.Mx8Tensor(rows, k)
    q.codes.fill_(fill)      # whatever was there before
    q.scales.fill_(fill)
    return q


def packed(x):
    """(tensor, values) of x in 8 bits, by the oracle."""
    codes, scales, values = ol.mx8_quantize(f64(x))
    q = mo.Mx8Tensor(*x.shape, codes=torch.from_numpy(codes).to(dev()), scales=torch.from_numpy(scales).to(dev()))
    q.codes.view(x.shape[0], -1)[:, x.shape[1]:] = 0x7F   # nothing looks past k
    return q, values


def values(q):
    return ol.mx8_values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.k)


def within(got, want, tol, what=""):
    got = f64(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = np.max(np.abs(got - want) / (tol + TINY)) if want.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def within8(q, want, tol, what=""):
    """q holds values that are off by `tol` at most before their rounding: each block's scale fits its largest
    magnitude, each value is within half a step, and the padding is zeros."""
    rows, k = want.shape
    nb = -(-k // 32)
    scales = q.scales.cpu().numpy().reshape(rows, nb)
    pad = lambda v: np.pad(v, ((0, 0), (0, nb * 32 - k))).reshape(rows, nb, 32)   # noqa: E731
    s = np.exp2(scales.astype(np.float64) - 127)
    top, slack = pad(np.abs(want)).max(2), pad(np.broadcast_to(tol, want.shape)).max(2)
    assert (top - slack <= 448 * s).all() and ((top + slack > 224 * s) | (scales == 0)).all(), what
    step = np.repeat(s, 32, 1)[:, :k]
    within(values(q), want, tol + np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * step), what)
    codes = q.codes.cpu().numpy().reshape(rows, nb * 32)
    assert (codes[:, k:] == 0).all(), what


def act_error(z, name):
    """Bound on the error of act and act' at z."""
    a = np.minimum(np.abs(z), 64.0)
    u = 1.6 * (a + 0.045 * a ** 3) if name == "gelu_tanh" else a
    wide = (1 + a) * (1 + 0.14 * a * a if name == "gelu_tanh" else 1.0)
    return np.zeros_like(z) if name in (None, "relu") else (16 + 4 * u + 2 * a * a) * 2.0 ** -23 * wide


def clean():
    torch.cuda.synchronize()
    assert mo.mo_last_device_error() == 0


# ---------------------------------------------------------------- 8-bit tensors

SHAPES8 = [(1, 1), (1, 32), (3, 33), (5, 8), (130, 257), (127, 64), (64, 1000), (31, 4096), (257, 40)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,k", SHAPES8)
def test_quantize_exact(rows, k, dtype):
    x = data(rows, k, dtype=dtype) * torch.exp(4 * torch.randn(rows, 1, generator=torch.Generator().manual_seed(k))).to(dev()).to(dtype)
    q = empty8(rows, k)
    mo.mx8_quantize(x, q)
    clean()
    codes, scales, want = ol.mx8_quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    for out_dtype in (F32, BF16):
        out = torch.full((rows, k), 7.0, dtype=out_dtype, device=dev())
        mo.mx8_dequantize(q, out)
        assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("k", [32, 64, 37])
def test_quantize_ends_of_the_range(k):
    special = [0.0, -0.0, 448.0, 449.0, 448.5, 17.0, 19.0, -17.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 3.3e38, 2.0 ** -126, 2.0 ** -130,
               2.0 ** -149, float("inf"), float("nan"), -float("inf"), 2.0 ** -118, 448 * 2.0 ** -127, 449 * 2.0 ** -127]
    x = torch.zeros(len(special), k, device=dev())
    for i, v in enumerate(special):
        x[i] = torch.linspace(-1, 1, k, device=dev()) * (abs(v) if np.isfinite(v) else 1.0)
        x[i, i % k] = v
    q = empty8(len(special), k)
    mo.mx8_quantize(x, q)
    clean()
    codes, scales, want = ol.mx8_quantize(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    live = ~np.repeat(scales == 255, 32, 1)
    assert np.array_equal(q.codes.cpu().numpy()[live], codes[live])
    out = torch.empty(len(special), k, device=dev())
    mo.mx8_dequantize(q, out)
    got = f64(out)
    # 3.3e38 lies above the middle of 240 2^120 and 256 2^120, and the latter, 2^128, is infinite in fp32
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)
    assert np.isinf(want).sum() == np.isinf(got).sum() > 0
    off = [(special[i], got[i, j], want[i, j]) for i in range(len(special)) for j in range(k) if not np.array_equal(got[i, j], want[i, j], equal_nan=True)]
    assert not off, off[:8]


def test_every_code_comes_back():
    codes = torch.arange(256, dtype=torch.uint8, device=dev()).reshape(1, 256)
    for e in (0, 1, 63, 127, 200, 246):
        q = mo.Mx8Tensor(1, 256, codes=codes, scales=torch.full((1, 8), e, dtype=torch.uint8, device=dev()))
        out = torch.empty(1, 256, device=dev())
        mo.mx8_dequantize(q, out)
        assert np.array_equal(f64(out), values(q), equal_nan=True)


# ---------------------------------------------------------------- norm

DIMS = [1, 7, 8, 32, 33, 256, 257, 264, 1000, 1024, 1280, 1999, 2048, 4096, 4100, 4104, 8192, 8200, 20001]


def norm_tol(y):
    # the sum of squares: at most 64 additions in a row, then a few roundings
    return 80 * 2.0 ** -24 * np.abs(y)


@pytest.mark.parametrize("dtype,out,residual,mx8", [(BF16, BF16, True, False), (BF16, None, True, True), (F32, F32, False, False),
                                                    (F32, BF16, True, True), (BF16, F32, False, True)])
@pytest.mark.parametrize("dim", DIMS)
def test_norm(dim, dtype, out, residual, mx8):
    rows = 9 if dim < 2000 else 3
    x, r = data(rows, dim, dtype=dtype, std=3.0), data(rows, dim, dtype=dtype, seed=1) if residual else None
    w = data(dim, dtype=F32, seed=2)
    o = torch.full((rows, dim), 9.0, dtype=out, device=dev()) if out else None
    s = torch.empty_like(x) if residual else None
    q = empty8(rows, dim) if mx8 else None
    mo.rms_norm(x, o, weight=w, eps=1e-5, residual=r, sum_out=s, out8=q)
    clean()
    want, ws = ol.rms_norm(f64(x), f64(w), 1e-5, f64(r) if residual else None)
    tol = norm_tol(want)
    if residual:
        tol = tol + 2 * 2.0 ** -24 * np.abs(want)   # s itself is rounded to fp32
        within(s, ws, (ROUND[dtype] + 2.0 ** -24) * np.abs(ws), "sum")
    if o is not None:
        within(o, want, tol + ROUND[out] * (np.abs(want) + tol), "out")
    if mx8:
        within8(q, want, tol, "out8")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [48, 1001, 4096, 9000])
def test_norm_in_place(dim, dtype):
    """sum_out in the residual, out in x; no weight; a row of zeros."""
    x, r = data(6, dim, dtype=dtype), data(6, dim, dtype=dtype, seed=1)
    x[2], r[2] = 0, 0
    a, b = torch.empty_like(x), torch.empty_like(x)
    mo.rms_norm(x, a, residual=r, sum_out=b)
    mo.rms_norm(x, x, residual=r, sum_out=r)
    clean()
    assert torch.equal(x, a) and torch.equal(r, b) and not a[2].any() and not b[2].any()
    want, _ = ol.rms_norm(f64(data(6, dim, dtype=dtype)), None, 1e-6, f64(data(6, dim, dtype=dtype, seed=1)))
    keep = [0, 1, 3, 4, 5]
    within(f64(a)[keep], want[keep], norm_tol(want)[keep] + (2 * 2.0 ** -24 + ROUND[dtype] * 1.01) * np.abs(want)[keep])


@pytest.mark.parametrize("dtype,mx8,dres,accumulate", [(BF16, False, True, False), (BF16, True, True, True), (F32, False, False, True),
                                                       (F32, True, True, False)])
@pytest.mark.parametrize("rows,dim", [(1, 4096), (3, 1), (5, 8), (700, 33), (64, 256), (33, 1000), (40, 1280), (2000, 257), (19, 4104),
                                      (11, 8192), (400, 4096), (7, 12001), (5000, 64)])
def test_norm_grad(rows, dim, dtype, mx8, dres, accumulate):
    dy, x = data(rows, dim, dtype=dtype), data(rows, dim, dtype=dtype, seed=1, std=2.0)
    w, dw = data(dim, dtype=F32, seed=2), data(dim, dtype=F32, seed=3)
    start = f64(dw)
    d = data(rows, dim, dtype=dtype, seed=4) if dres else None
    q, xv = packed(x) if mx8 else (x, f64(x))
    dx = torch.full_like(dy, 5.0)
    ws = mo.rms_norm_grad_workspace(rows, dim)
    ws.fill_(0xFF)
    mo.rms_norm_grad(dy, q, dx, weight=w, eps=1e-5, dresidual=d, dweight=dw, workspace=ws, accumulate=accumulate)
    clean()
    dyv, wv = f64(dy), f64(w)
    want, want_w = ol.rms_norm_grad(dyv, xv, wv, 1e-5, f64(d) if dres else None)
    # both sums take at most 64 additions in a row; the projection's terms are bounded by the sum of their magnitudes
    r = 1 / np.sqrt(np.mean(xv * xv, 1, keepdims=True) + 1e-5)
    mag = r * (np.abs(dyv * wv) + np.abs(xv * r) * np.mean(np.abs(dyv * wv * xv * r), 1, keepdims=True)) + (np.abs(f64(d)) if dres else 0)
    tol = 240 * 2.0 ** -24 * mag
    within(dx, want, tol + ROUND[dtype] * (np.abs(want) + tol), "dx")
    n = np.abs(dyv * xv * r)
    want_w = want_w + (start if accumulate else 0)
    within(dw, want_w, (rows + 80) * 2.0 ** -24 * n.sum(0) + 2.0 ** -23 * np.abs(want_w), "dweight")
    # in place, without the weight's gradient, without a weight
    again, plain = dy.clone(), torch.empty_like(dy)
    mo.rms_norm_grad(again, q, again, weight=w, eps=1e-5, dresidual=d)
    assert torch.equal(again, dx)
    mo.rms_norm_grad(dy, q, plain, eps=1e-5, dresidual=d)
    ones = torch.empty_like(dy)
    mo.rms_norm_grad(dy, q, ones, weight=torch.ones(dim, device=dev()), eps=1e-5, dresidual=d)
    clean()
    assert torch.equal(plain, ones)


def test_norm_gradient_against_differences():
    rows, dim = 4, 40
    x, dy, w = data(rows, dim, dtype=F32), data(rows, dim, dtype=F32, seed=1), data(dim, dtype=F32, seed=2)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    mo.rms_norm_grad(dy, x, dx, weight=w, dweight=dw, workspace=mo.rms_norm_grad_workspace(rows, dim))
    clean()
    f = lambda xv, wv: (ol.rms_norm(xv, wv)[0] * f64(dy)).sum()   # noqa: E731
    rng = np.random.default_rng(0)
    h = 1e-5
    for _ in range(5):
        p, q = rng.normal(size=(rows, dim)), rng.normal(size=dim)
        slope = (f(f64(x) + h * p, f64(w) + h * q) - f(f64(x) - h * p, f64(w) - h * q)) / (2 * h)
        got = (f64(dx) * p).sum() + (f64(dw) * q).sum()
        assert abs(got - slope) <= 1e-5 * (np.abs(f64(dx) * p).sum() + np.abs(f64(dw) * q).sum())   # h^2 and fp32


# ---------------------------------------------------------------- linear

LINEAR = [(1, 1, 1), (1, 32, 32), (1, 1280, 5120), (2, 2048, 40), (5, 33, 47), (16, 64, 128), (17, 128, 130), (33, 4100, 24), (64, 100, 257),
          (65, 512, 512), (100, 1600, 300), (128, 256, 384), (129, 72, 520), (300, 1000, 264), (777, 1003, 515), (1000, 64, 2048),
          (257, 2056, 96), (520, 8, 600)]


def linear_data(t, k, n, mx8):
    x = data(t, k)
    q, xv = packed(x) if mx8 else (x, f64(x))
    return q, xv, data(n, k, seed=1, std=k ** -0.5)


@pytest.mark.parametrize("t,k,n", LINEAR)
@pytest.mark.parametrize("activation,bias,residual,pre,mx8,out", [
    (None, False, False, None, False, BF16), (None, True, True, None, True, F32), ("gelu_tanh", True, False, "mx8", False, BF16),
    ("silu", False, True, "bf16", True, BF16), ("gelu", True, True, None, False, F32), ("relu", True, False, "mx8", True, F32)])
def test_linear(t, k, n, activation, bias, residual, pre, mx8, out):
    x, xv, w = linear_data(t, k, n, mx8)
    b = data(n, dtype=F32, seed=2) if bias else None
    r = data(t, n, dtype=out, seed=3) if residual else None
    p = {None: None, "mx8": empty8(t, n), "bf16": torch.full((t, n), 3.0, dtype=BF16, device=dev())}[pre]
    o = torch.full((t, n), 9.0, dtype=out, device=dev())
    ws = mo.linear_workspace(t, k, n)
    ws.fill_(0xFF)
    mo.linear(x, w, o, bias=b, activation=activation, residual=r, pre=p, workspace=ws)
    clean()
    wv, bv, rv = f64(w), f64(b) if bias else None, f64(r) if residual else None
    want, z = ol.linear(xv, wv, bv, activation, rv)
    ez = k * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T) + 2.0 ** -23 * np.abs(z)
    e = 1.13 * ez + act_error(z, activation) + 2.0 ** -23 * np.abs(want)
    within(o, want, e + ROUND[out] * (np.abs(want) + e), "out")
    if pre == "mx8":
        within8(p, z, ez, "pre")
    elif pre:
        within(p, z, ez + ROUND[BF16] * (np.abs(z) + ez), "pre")
    if residual:   # in place
        mo.linear(x, w, r, bias=b, activation=activation, residual=r, pre=p, workspace=ws)
        clean()
        assert torch.equal(r, o)


GRAD = [(1, 1, 1), (1, 64, 96), (3, 33, 47), (16, 64, 128), (40, 1280, 72), (64, 100, 257), (65, 512, 512), (129, 72, 520), (300, 1000, 264),
        (777, 203, 515), (2000, 64, 40), (1030, 1032, 24)]


@pytest.mark.parametrize("t,k,n", GRAD)
@pytest.mark.parametrize("activation,pre,mx8,dtype,accumulate", [
    (None, None, False, BF16, False), (None, None, True, F32, True), ("gelu_tanh", "mx8", True, BF16, True),
    ("silu", "bf16", False, F32, False), ("gelu", "bf16", True, BF16, False), ("relu", "mx8", False, F32, True)])
def test_linear_grad(t, k, n, activation, pre, mx8, dtype, accumulate):
    x, xv, w = linear_data(t, k, n, mx8)
    dout = data(t, n, seed=5)
    z = data(t, n, seed=6, std=1.5)
    p, zv = (packed(z) if pre == "mx8" else (z, f64(z))) if pre else (None, None)
    dx = torch.full((t, k), 9.0, dtype=dtype, device=dev())
    dw, db = data(n, k, dtype=dtype, seed=7), data(n, dtype=F32, seed=8)
    dw0, db0 = (f64(dw), f64(db)) if accumulate else (0.0, 0.0)
    ws = mo.linear_workspace(t, k, n, grad=True)
    ws.fill_(0xFF)
    mo.linear_grad(dout, x, w, dx=dx, dw=dw, dbias=db, activation=activation, pre=p, workspace=ws, accumulate=accumulate)
    clean()
    dv, wv = f64(dout), f64(w)
    want = ol.linear_grad(dv, xv, wv, activation, zv)
    dz = np.abs(dv if activation is None else dv * ol.act(zv, activation)[1])
    es = np.abs(dv) * act_error(zv, activation) if activation else np.zeros_like(dv)
    ez = es + (ROUND[BF16] * (dz + es) if activation else 0.0)
    e = ez @ np.abs(wv) + n * 2.0 ** -23 * ((dz + ez) @ np.abs(wv))
    within(dx, want[0], e + ROUND[dtype] * (np.abs(want[0]) + e), "dx")
    e = ez.T @ np.abs(xv) + t * 2.0 ** -23 * ((dz + ez).T @ np.abs(xv))
    v = want[1] + dw0
    within(dw, v, e + (ROUND[dtype] + 2.0 ** -23) * (np.abs(v) + e), "dw")
    v = want[2] + db0
    within(db, v, es.sum(0) + t * 2.0 ** -24 * (dz + es).sum(0) + 2.0 ** -23 * (np.abs(v) + dz.sum(0)), "dbias")
    # one at a time they are the same
    for name, like in (("dx", dx), ("dw", dw), ("dbias", db)):
        one = torch.empty_like(like)
        if accumulate and name != "dx":
            one.copy_(data(n, k, dtype=dtype, seed=7) if name == "dw" else data(n, dtype=F32, seed=8))
        mo.linear_grad(dout, x if name == "dw" else None, w, activation=activation, pre=p, workspace=ws, accumulate=accumulate, **{name: one})
        clean()
        assert torch.equal(one, like), name


def test_linear_gradient_against_differences():
    t, k, n = 6, 40, 24
    x, w, b, dout = data(t, k), data(n, k, seed=1, std=0.2), data(n, dtype=F32, seed=2), data(t, n, seed=3)
    pre, out = torch.empty(t, n, dtype=BF16, device=dev()), torch.empty(t, n, device=dev())
    ws = mo.linear_workspace(t, k, n, grad=True)
    mo.linear(x, w, out, bias=b, activation="silu", pre=pre, workspace=ws)
    dx, dw, db = torch.empty(t, k, device=dev()), torch.empty(n, k, device=dev()), torch.empty(n, device=dev())
    mo.linear_grad(dout, x, w, dx=dx, dw=dw, dbias=db, activation="silu", pre=pre, workspace=ws)
    clean()
    f = lambda *a: (ol.linear(*a, activation="silu")[0] * f64(dout)).sum()   # noqa: E731
    rng = np.random.default_rng(1)
    base, grads, h = [f64(v) for v in (x, w, b)], [f64(v) for v in (dx, dw, db)], 1e-4
    for _ in range(5):
        steps = [rng.normal(size=v.shape) for v in base]
        slope = (f(*[v + h * s for v, s in zip(base, steps)]) - f(*[v - h * s for v, s in zip(base, steps)])) / (2 * h)
        got = sum((g * s).sum() for g, s in zip(grads, steps))
        # pre and dz are rounded to bf16: 2^-8 of each, the slope of act' at most 0.5 of a pre-activation's error
        assert abs(got - slope) <= 2 * 2.0 ** -8 * sum(np.abs(g * s).sum() for g, s in zip(grads, steps))


# ---------------------------------------------------------------- gated feed-forward block

FFN = [(1, 64, 96), (1, 512, 1376), (3, 33, 47), (16, 64, 128), (17, 40, 1000), (60, 1280, 136), (64, 100, 257), (128, 256, 384), (130, 264, 520),
       (300, 512, 1001), (513, 128, 320)]


def ffn_data(t, d, f, mx8):
    x = data(t, d)
    q, xv = packed(x) if mx8 else (x, f64(x))
    return q, xv, data(f, d, seed=1, std=1.3 * d ** -0.5), data(f, d, seed=2, std=1.3 * d ** -0.5), data(d, f, seed=3, std=f ** -0.5)


@pytest.mark.parametrize("t,d,f", FFN)
@pytest.mark.parametrize("activation,residual,save,mx8,out", [
    ("silu", True, "mx8", True, BF16), ("gelu_tanh", False, "bf16", False, F32), ("gelu", True, None, False, BF16), ("relu", False, "mx8", False, BF16),
    (None, True, "bf16", True, F32)])
def test_gated_ffn(t, d, f, activation, residual, save, mx8, out):
    x, xv, wg, wu, wd = ffn_data(t, d, f, mx8)
    r = data(t, d, dtype=out, seed=4) if residual else None
    make = {None: lambda: None, "mx8": lambda: empty8(t, f), "bf16": lambda: torch.full((t, f), 3.0, dtype=BF16, device=dev())}[save]
    g, u = make(), make()
    o = torch.full((t, d), 9.0, dtype=out, device=dev())
    ws = mo.gated_ffn_workspace(t, d, f)
    ws.fill_(0xFF)
    mo.gated_ffn(x, wg, wu, wd, o, activation=activation, residual=r, gate=g, up=u, workspace=ws)
    clean()
    vg, vu, vd = f64(wg), f64(wu), f64(wd)
    want, zg, zu = ol.gated_ffn(xv, vg, vu, vd, activation, f64(r) if residual else None)
    eg, eu = (d * 2.0 ** -23 * (np.abs(xv) @ np.abs(v).T) + 2.0 ** -23 * np.abs(z) for v, z in ((vg, zg), (vu, zu)))
    a = ol.act(zg, activation)[0]
    ea = 1.13 * eg + act_error(zg, activation)
    eh = ea * np.abs(zu) + (np.abs(a) + ea) * eu
    h = np.abs(a * zu)
    eh = eh + ROUND[BF16] * (h + eh) + 2.0 ** -23 * h
    e = eh @ np.abs(vd).T + f * 2.0 ** -23 * ((h + eh) @ np.abs(vd).T) + 2.0 ** -23 * np.abs(want)
    within(o, want, e + ROUND[out] * (np.abs(want) + e), "out")
    for q, z, ez, name in ((g, zg, eg, "gate"), (u, zu, eu, "up")):
        if save == "mx8":
            within8(q, z, ez, name)
        elif save:
            within(q, z, ez + ROUND[BF16] * (np.abs(z) + ez), name)
    if residual:   # in place
        mo.gated_ffn(x, wg, wu, wd, r, activation=activation, residual=r, gate=g, up=u, workspace=ws)
        clean()
        assert torch.equal(r, o)


@pytest.mark.parametrize("t,d,f", FFN)
@pytest.mark.parametrize("activation,save,mx8,dtype,accumulate", [
    ("silu", "mx8", True, BF16, False), ("gelu_tanh", "bf16", False, F32, True), ("gelu", "mx8", False, BF16, True),
    ("relu", "bf16", True, F32, False), (None, "bf16", False, BF16, False)])
def test_gated_ffn_grad(t, d, f, activation, save, mx8, dtype, accumulate):
    x, xv, wg, wu, wd = ffn_data(t, d, f, mx8)
    dout = data(t, d, seed=5)
    (g, gv), (u, uv) = ((packed(z) if save == "mx8" else (z, f64(z))) for z in (data(t, f, seed=6, std=1.3), data(t, f, seed=7, std=1.3)))
    dx = torch.full((t, d), 9.0, dtype=dtype, device=dev())
    start = [data(f, d, dtype=dtype, seed=8), data(f, d, dtype=dtype, seed=9), data(d, f, dtype=dtype, seed=10)]
    dw = [v.clone() for v in start]
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)
    ws.fill_(0xFF)
    call = dict(activation=activation, workspace=ws, accumulate=accumulate)
    mo.gated_ffn_grad(dout, x, g, u, wg, wu, wd, dx=dx, dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2], **call)
    clean()
    dv, vg, vu, vd = (f64(v) for v in (dout, wg, wu, wd))
    want = ol.gated_ffn_grad(dv, xv, gv, uv, vg, vu, vd, activation)
    a, slope = ol.act(gv, activation)
    ea = act_error(gv, activation)
    dh, edh = np.abs(dv @ vd), d * 2.0 ** -23 * (np.abs(dv) @ np.abs(vd))
    R = ROUND[BF16] + 4 * 2.0 ** -24
    mg, mu, mh = dh * np.abs(uv * slope), dh * np.abs(a), np.abs(a * uv)
    eg = np.abs(uv) * (edh * (np.abs(slope) + ea) + dh * ea)
    eu = edh * (np.abs(a) + ea) + dh * ea
    eh = ea * np.abs(uv)
    eg, eu, eh = eg + R * (mg + eg), eu + R * (mu + eu), eh + R * (mh + eh)
    e = eg @ np.abs(vg) + eu @ np.abs(vu) + 2 * f * 2.0 ** -23 * ((mg + eg) @ np.abs(vg) + (mu + eu) @ np.abs(vu))
    within(dx, want[0], e + ROUND[dtype] * (np.abs(want[0]) + e), "dx")
    for got, v, s, m, em, other in ((dw[0], want[1], start[0], mg, eg, xv), (dw[1], want[2], start[1], mu, eu, xv)):
        v = v + (f64(s) if accumulate else 0)
        e = em.T @ np.abs(other) + t * 2.0 ** -23 * ((m + em).T @ np.abs(other))
        within(got, v, e + (ROUND[dtype] + 2.0 ** -23) * (np.abs(v) + e), "dw_gate, dw_up")
    v = want[3] + (f64(start[2]) if accumulate else 0)
    e = np.abs(dv).T @ eh + t * 2.0 ** -23 * (np.abs(dv).T @ (mh + eh))
    within(dw[2], v, e + (ROUND[dtype] + 2.0 ** -23) * (np.abs(v) + e), "dw_down")
    # one at a time they are the same, and so is a second time
    for i, name in enumerate(("dw_gate", "dw_up", "dw_down", "dx")):
        one = (start[i].clone() if accumulate else torch.empty_like(start[i])) if i < 3 else torch.empty_like(dx)
        mo.gated_ffn_grad(dout, x if i < 2 else None, g, u, wg, wu, wd, **{name: one}, **call)
        clean()
        assert torch.equal(one, dw[i] if i < 3 else dx), name


def test_gated_ffn_gradient_against_differences():
    t, d, f = 6, 40, 24
    x, xv, wg, wu, wd = ffn_data(t, d, f, False)
    dout = data(t, d, seed=5)
    g, u = torch.empty(t, f, dtype=BF16, device=dev()), torch.empty(t, f, dtype=BF16, device=dev())
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)
    out = torch.empty(t, d, device=dev())
    mo.gated_ffn(x, wg, wu, wd, out, gate=g, up=u, workspace=ws)
    grads = [torch.empty_like(v, dtype=F32) for v in (x, wg, wu, wd)]
    mo.gated_ffn_grad(dout, x, g, u, wg, wu, wd, dx=grads[0], dw_gate=grads[1], dw_up=grads[2], dw_down=grads[3], workspace=ws)
    clean()
    fn = lambda *v: (ol.gated_ffn(*v)[0] * f64(dout)).sum()   # noqa: E731
    rng = np.random.default_rng(1)
    base, grads, h = [xv, f64(wg), f64(wu), f64(wd)], [f64(v) for v in grads], 1e-4
    for _ in range(5):
        steps = [rng.normal(size=v.shape) for v in base]
        slope = (fn(*[v + h * s for v, s in zip(base, steps)]) - fn(*[v - h * s for v, s in zip(base, steps)])) / (2 * h)
        got = sum((v * s).sum() for v, s in zip(grads, steps))
        # gate, up, dg, du and h are rounded to bf16
        assert abs(got - slope) <= 4 * 2.0 ** -8 * sum(np.abs(v * s).sum() for v, s in zip(grads, steps))
