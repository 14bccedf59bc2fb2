"""Feed-forward operators on the GPU: calls that the documentation allows beside
the usual ones, at both ends of the numbers' range and of the sizes."""
import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
import test_gpu_layer_ops as base
from gpu_util import f64
from oracle import layer_ops as ol
from test_gpu_layer_ops import BF16, F32, ROUND, clean, data, dev, empty8, norm_tol, packed, within, within8

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- in place

@pytest.mark.parametrize("t,d,f", [(1, 512, 1376), (2, 264, 4880), (3, 40, 72), (60, 1280, 136), (130, 1100, 1500), (300, 33, 1001), (2300, 1100, 1153)])
@pytest.mark.parametrize("save", [None, "mx8"])
def test_a_gated_block_replaces_its_input(t, d, f, save):
    """x is the residual and the output: s += block(s)."""
    s, _, wg, wu, wd = base.ffn_data(t, d, f, False)
    ws = mo.gated_ffn_workspace(t, d, f)
    kept = [dict(gate=empty8(t, f), up=empty8(t, f)) if save else {} for _ in range(2)]
    want = torch.empty(t, d, dtype=BF16, device=s.device)
    mo.gated_ffn(s, wg, wu, wd, want, residual=s, workspace=ws, **kept[0])
    mo.gated_ffn(s, wg, wu, wd, s, residual=s, workspace=ws, **kept[1])
    clean()
    assert torch.equal(s, want)
    for name in kept[0]:
        assert torch.equal(kept[0][name].codes, kept[1][name].codes) and torch.equal(kept[0][name].scales, kept[1][name].scales)


# ---------------------------------------------------------------- relative accuracy of activations

# gelu's Phi(-x) = e^(-x^2 / 2) t q(t). The fit: 1.6e-7 < 1.4 2^-23. t is off by 1.5 2^-23 (a reciprocal of one
# unit, a rounded sum), and t q(t) by at most 2.7 times that; Horner's 14 roundings of 2^-24, the magnitudes
# of its terms 1.9 times their sum at most: 14 2^-23 at the very worst. The exponent x^2 / 2 carries 2.5
# roundings of 2^-24, 0.63 x^2 2^-23; ex2 two units; three products. Together (24 + x^2) 2^-23.
# silu and gelu_tanh: (8 + 4 |u|) 2^-23 with u the logistic function's argument, as the products' tests have it.
def relative(z, name):
    a = np.abs(z)
    u = 1.6 * (a + 0.045 * a ** 3) if name == "gelu_tanh" else a
    return (24 + a * a if name == "gelu" else 8 + 4 * u) * 2.0 ** -23


def exact(z, name):
    """(value, slope) without cancellation: the oracle's 1 + tanh(u) has nothing left of 2 / (1 + e^(-2u)) far to
    the left."""
    if name != "gelu_tanh":
        return ol.act(z, name)
    a = 2 * ol.SQRT_2_PI
    s = 1 / (1 + np.exp(-a * (z + 0.044715 * z ** 3)))
    return z * s, s + z * s * (1 - s) * a * (1 + 3 * 0.044715 * z * z)


def arguments():
    """bf16 numbers from -13 to 13, and small ones."""
    z = torch.cat([torch.linspace(-13, 13, 4000), torch.linspace(-1, 1, 64) * 2.0 ** -20, torch.tensor([0.0] * 32)])
    return z.to(BF16).reshape(64, 64).to(dev())


@pytest.mark.parametrize("t", [1, 3, 64, 300])     # each kernel of the products
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_activations_keep_their_relative_accuracy(name, t):
    z, eye = arguments(), torch.eye(64, dtype=BF16, device=dev())
    z = z.repeat(-(-t // 64) or 1, 1)[:t] if t >= 64 else z[torch.arange(t, device=dev()) * 17]
    out = torch.empty(z.shape, device=dev())
    mo.linear(z, eye, out, activation=name, workspace=mo.linear_workspace(t, 64, 64))
    clean()
    want = exact(f64(z), name)[0]
    live = np.abs(want) > 1e-36     # (e^x below 2^-126 is 0)
    off = np.abs(f64(out) - want) / np.where(live, np.abs(want), 1)
    assert (off <= relative(f64(z), name))[live].all(), (off / relative(f64(z), name))[live].max()
    assert (np.abs(f64(out)) <= 2e-36)[~live].all()


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_slopes_keep_their_relative_accuracy(name):
    """dbias of one token is act'(pre) itself, in fp32. Where the slope's two terms cancel (it is 0 near -0.75 and
    -1.28), their magnitudes count."""
    z = arguments().reshape(1, -1)
    n = z.shape[1]
    db = torch.empty(n, device=dev())
    mo.linear_grad(torch.ones_like(z), None, torch.zeros(n, 8, dtype=BF16, device=dev()), dbias=db, activation=name, pre=z,
                   workspace=mo.linear_workspace(1, 8, n, grad=True))
    clean()
    v = f64(z)[0]
    value, want = exact(v, name)
    s = np.where(v == 0, 0.5, value / np.where(v == 0, 1, v))          # Phi or the logistic function
    size = np.abs(s) + np.abs(want - s)
    live = size > 1e-35
    tol = (4 * 2.0 ** -23 + 2 * relative(v, name)) * size
    assert (np.abs(f64(db) - want) <= tol)[live].all(), (np.abs(f64(db) - want) / tol)[live].max()


# ---------------------------------------------------------------- norms at both ends of fp32's range

# Sizes of a row and of its gradient: squares that overflow, that are 0, and products of the two that do; rows of
# ordinary size lie between them, in the same blocks.
SCALES = [(1.0, 1.0), (1e20, 1.0), (1.0, 1e-20), (1e-23, 1.0), (1e38, 1e38), (1.0, 1.0), (3e18, 1e30), (1e-38, 1e-6), (1e10, 1e32), (1e-20, 1e-25),
          (1e30, 1e-5), (1e-30, 1e-10), (1.0, 1e35)]
NORM_DIMS = [7, 48, 256, 257, 1000, 1001, 2048, 4096, 4099, 8192, 8200, 9001]


def scaled(rows, dim, which, dtype, seed):
    """Numbers of both signs, between half and twice their row's size."""
    g = torch.Generator().manual_seed(seed + dim)
    u = (torch.rand(rows, dim, generator=g) * 1.5 + 0.5) * torch.where(torch.rand(rows, dim, generator=g) < 0.5, -1.0, 1.0)
    size = torch.tensor([SCALES[i % len(SCALES)][which] for i in range(rows)], dtype=torch.float64)
    return (u.double() * size[:, None]).to(dtype).to(dev())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-35, 1e7, 1e30])
def test_norm_of_rows_of_every_size(dim, dtype, eps):
    rows = 2 * len(SCALES) + 1
    x, r, w = scaled(rows, dim, 0, dtype, 1), scaled(rows, dim, 0, dtype, 2) * 0.125, data(dim, dtype=F32, seed=3)
    eps = float(np.float32(eps))
    for residual in (None, r):
        o, q = torch.empty(rows, dim, device=dev()), empty8(rows, dim)
        mo.rms_norm(x, o, weight=w, eps=eps, residual=residual, out8=q)
        clean()
        want, _ = ol.rms_norm(f64(x), f64(w), eps, None if residual is None else f64(r))
        # (s is rounded to fp32; scaling is exact but for what is 2^-126 of the row's largest)
        tol = norm_tol(want) + 2 * 2.0 ** -24 * np.abs(want)
        within(o, want, tol + ROUND[F32] * np.abs(want), "out")
        within8(q, want, tol, "out8")


@pytest.mark.parametrize("dtype,mx8", [(F32, False), (BF16, False), (F32, True), (BF16, True)])
@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e30])
def test_norm_gradient_of_rows_of_every_size(dim, dtype, mx8, eps):
    rows = 2 * len(SCALES) + 1
    norm_gradient_case(rows, dim, dtype, mx8, float(np.float32(eps)))


@pytest.mark.parametrize("rows,dim", [(700, 4096), (650, 1001), (700, 8200), (640, 8193), (5000, 40)])
def test_norm_gradient_of_more_rows_than_blocks(rows, dim):
    """A block takes ordinary rows and others in turn."""
    norm_gradient_case(rows, dim, F32, False, 0.0)


def norm_gradient_case(rows, dim, dtype, mx8, eps):
    x, dy, w = scaled(rows, dim, 0, dtype, 1), scaled(rows, dim, 1, dtype, 2), data(dim, dtype=F32, seed=3)
    w = torch.sign(w) * (w.abs() + 0.1).clamp(max=4)
    q, xv = packed(x) if mx8 else (x, f64(x))
    dx, dw = torch.empty_like(dy), torch.empty(dim, device=dev())
    mo.rms_norm_grad(dy, q, dx, weight=w, eps=eps, dweight=dw, workspace=mo.rms_norm_grad_workspace(rows, dim))
    clean()
    dyv, wv = f64(dy), f64(w)
    want, _ = ol.rms_norm_grad(dyv, xv, wv, eps)
    r = 1 / np.sqrt(np.mean(xv * xv, 1, keepdims=True) + eps)
    mag = r * (np.abs(dyv * wv) + np.abs(xv * r) * np.mean(np.abs(dyv * wv * xv * r), 1, keepdims=True))
    # where the gradient itself leaves the type, or terms of it leave fp32, nothing is asked
    live = (mag < 1e38).all(1)
    assert live.sum() >= rows * 3 // 4
    tol = 240 * 2.0 ** -24 * mag
    within(f64(dx)[live], want[live], (tol + ROUND[dtype] * (np.abs(want) + tol))[live], "dx")
    # dweight: the rows' terms differ by 60 orders of magnitude; their sum is held by the largest. Columns whose
    # magnitudes add up to more than fp32 holds (several rows of 1e38) may be infinite
    n = np.abs(dyv * xv * r)
    fits = n.sum(0) < 3.4e38
    within(f64(dw)[fits], (dyv * xv * r).sum(0)[fits], (rows + 80) * 2.0 ** -24 * n.sum(0)[fits], "dweight")
    if dtype == F32 and not mx8:   # without them every column fits
        keep = np.flatnonzero(np.abs(dyv).max(1) < 1e37)
        part = mo.rms_norm_grad_workspace(len(keep), dim)
        mo.rms_norm_grad(dy[keep].contiguous(), x[keep].contiguous(), torch.empty(len(keep), dim, device=dev()), weight=w, eps=eps, dweight=dw,
                         workspace=part)
        clean()
        within(dw, (dyv * xv * r)[keep].sum(0), (rows + 80) * 2.0 ** -24 * n[keep].sum(0), "dweight of the others")
    if dtype == F32 and not mx8:   # each row alone gives the same, whatever its neighbours are
        for i in range(min(rows, len(SCALES))):
            if live[i]:
                one = torch.empty(1, dim, device=dev())
                mo.rms_norm_grad(dy[i:i + 1].clone(), x[i:i + 1].clone(), one, weight=w, eps=eps)
                assert torch.equal(one[0], dx[i]), i


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim", [(27, d) for d in NORM_DIMS] + [(700, 4096), (650, 1001), (700, 8200), (640, 8193)])
def test_norms_of_rows_of_every_size_in_place(rows, dim, dtype):
    """What replaces its input has the bits of what does not, and so has a gradient that another is added to."""
    x, r, w = scaled(rows, dim, 0, dtype, 1), scaled(rows, dim, 0, dtype, 2) * 0.125, data(dim, dtype=F32, seed=3)
    out, total = torch.empty_like(x), torch.empty_like(x)
    q8, p8 = empty8(rows, dim), empty8(rows, dim)
    mo.rms_norm(x, out, weight=w, eps=0.0, residual=r, sum_out=total, out8=q8)
    a, b = x.clone(), r.clone()
    mo.rms_norm(a, a, weight=w, eps=0.0, residual=b, sum_out=b, out8=p8)
    clean()
    assert torch.equal(a, out) and torch.equal(b, total) and torch.equal(q8.codes, p8.codes) and torch.equal(q8.scales, p8.scales)
    assert torch.equal(total, (x.float() + r.float()).to(dtype))
    dy, ws = scaled(rows, dim, 1, dtype, 4), mo.rms_norm_grad_workspace(rows, dim)
    plain, dx, dw, dv = torch.empty_like(x), torch.empty_like(x), torch.empty(dim, device=dev()), torch.empty(dim, device=dev())
    mo.rms_norm_grad(dy, x, plain, weight=w, eps=0.0, dweight=dw, workspace=ws)
    dres = (plain.float() * 0.5).nan_to_num(0, 0, 0).to(dtype)      # of each row's own size
    mo.rms_norm_grad(dy, x, dx, weight=w, eps=0.0, dresidual=dres, dweight=dv, workspace=ws)
    clean()
    assert torch.equal(dw.view(torch.int32), dv.view(torch.int32))
    live = torch.isfinite(plain) & (plain.abs() < 1e38) & (plain.abs() > 1e-36)
    got, want = f64(dx)[live.cpu().numpy()], (f64(plain) + f64(dres))[live.cpu().numpy()]
    # plain is rounded to its type; dx is not before dres is added
    assert (np.abs(got - want) <= (2 * ROUND[dtype] + 2.0 ** -22) * np.abs(f64(plain) * 1.5)[live.cpu().numpy()]).all()
    for same in (dy, dres):
        again = same.clone()
        mo.rms_norm_grad(again if same is dy else dy, x, again, weight=w, eps=0.0, dresidual=again if same is dres else dres, dweight=dv, workspace=ws)
        clean()
        assert torch.equal(again.view(torch.uint8), dx.view(torch.uint8)) and torch.equal(dw.view(torch.int32), dv.view(torch.int32))


def test_rows_of_zeros_and_no_numbers_stay_what_they_were():
    """Rows that scaling says nothing of: zeros give zeros where eps is not 0, and infinities stay in their row."""
    for dim in (48, 1001, 4096, 8200, 9001):
        x, w = data(5, dim, dtype=F32), data(dim, dtype=F32, seed=1)
        alone = torch.empty_like(x)
        mo.rms_norm(x, alone, weight=w, eps=0.0)
        x[1] = 0
        x[2, 3] = float("inf")
        x[3, 5] = float("nan")
        o, dx = torch.empty_like(x), torch.empty_like(x)
        for eps in (1e-6, 1e-38):
            mo.rms_norm(x, o, weight=w, eps=eps)
            mo.rms_norm_grad(torch.ones_like(x), x, dx, weight=w, eps=eps)
            clean()
            assert not o[1].any() and torch.isfinite(dx[1]).all()
            assert torch.isnan(o[2, 3]) and torch.isnan(o[3]).all()
            assert torch.isfinite(o[[0, 4]]).all() and torch.isfinite(dx[[0, 4]]).all() and not torch.isfinite(dx[3]).any()
        mo.rms_norm(x, o, weight=w, eps=0.0)
        clean()
        assert torch.equal(o[[0, 4]], alone[[0, 4]])


# ---------------------------------------------------------------- long reductions

SLICE = 32768


def large(*shape, dtype=BF16, seed=0, std=1.0):
    """data, made on the GPU."""
    g = torch.Generator(dev()).manual_seed(seed + sum(shape))
    return (torch.randn(shape, generator=g, device=dev()) * std).to(dtype)


def positive(*shape, seed=0, std=1.0):
    return (large(*shape, seed=seed, std=std).abs() + std / 2).to(BF16)


# CTA pairs (more than 38 tiles of 256), clusters that are too many to split the reduction, and the kernels that
# split it by themselves (few columns; one row).
@pytest.mark.parametrize("t,k,n", [(520, 65536, 4900), (520, 40001, 4900), (64, 40000, 20004), (12, 33000, 20001), (300, 65536, 256), (1, 65536, 300)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_long_forward_sums_are_joined_in_fp32(t, k, n, out):
    """No accumulation is longer than 32768 products: the call gives the bits of a call for each slice, the second
    on top of the first. (The split kernels' own slices are shorter; theirs is the bound alone.)"""
    x, w, b = positive(t, k), positive(n, k, seed=1, std=k ** -0.5), large(n, dtype=F32, seed=2)
    o = torch.empty(t, n, dtype=out, device=dev())
    mo.linear(x, w, o, bias=b, workspace=mo.linear_workspace(t, k, n))
    first, two = torch.empty(t, n, device=dev()), torch.empty(t, n, device=dev())
    x0, x1, w0, w1 = (v.contiguous() for v in (x[:, :SLICE], x[:, SLICE:], w[:, :SLICE], w[:, SLICE:]))
    ws = mo.linear_workspace(t, SLICE, n)
    mo.linear(x0, w0, first, workspace=ws)
    mo.linear(x1, w1, two, residual=first, workspace=mo.linear_workspace(t, k - SLICE, n))
    clean()
    if t > 1 and n > 300:
        assert torch.equal(o, (two + b).to(out))
    # terms of one sign: an addition of 16 products cuts off at most 2^-22 of the sum so far, which is half of the
    # last one on average
    rows = slice(0, min(t, 64))
    want = f64(x[rows].double() @ w.double().T + b.double())
    size = f64(x[rows].double() @ w.double().T)
    tol = (SLICE / 16 + 4) * 2.0 ** -23 * size + 2.0 ** -23 * np.abs(want)
    within(f64(o[rows]), want, tol + ROUND[out] * (np.abs(want) + tol))


@pytest.mark.parametrize("t,k,n", [(520, 40000, 4864), (64, 40001, 19500)])
def test_long_forward_sums_with_activation_and_copies(t, k, n):
    """What follows the sum follows the joined one."""
    x, w, b, r = large(t, k), large(n, k, seed=1, std=k ** -0.5), large(n, dtype=F32, seed=2), large(t, n, dtype=F32, seed=3)
    ws = mo.linear_workspace(t, k, n)
    z, pre, z8, o = torch.empty(t, n, dtype=BF16, device=dev()), torch.empty(t, n, dtype=BF16, device=dev()), empty8(t, n), torch.empty(t, n, device=dev())
    mo.linear(x, w, z, bias=b, workspace=ws)
    mo.linear(x, w, o, bias=b, activation="relu", residual=r, pre=pre, workspace=ws)
    clean()
    assert torch.equal(z, pre)
    wide = torch.empty(t, n, device=dev())
    mo.linear(x, w, wide, bias=b, workspace=ws)
    assert torch.equal(o, torch.relu(wide) + r)
    mo.linear(x, w, r, bias=b, activation="relu", residual=r, pre=z8, workspace=ws)
    q = empty8(t, n)
    mo.mx8_quantize(wide, q)
    clean()
    assert torch.equal(r, o) and torch.equal(q.codes, z8.codes) and torch.equal(q.scales, z8.scales)


@pytest.mark.parametrize("t,d,f", [(520, 33000, 2500), (48, 40000, 9999), (70, 33001, 300)])
def test_gated_block_of_long_rows(t, d, f):
    """gate and up are the sums that linear gives, and the backward pass's dh is taken in slices too."""
    x, wg, wu, wd = large(t, d), large(f, d, seed=1, std=d ** -0.5), large(f, d, seed=2, std=d ** -0.5), large(d, f, seed=3, std=f ** -0.5)
    gate, up, o = torch.empty(t, f, dtype=BF16, device=dev()), torch.empty(t, f, dtype=BF16, device=dev()), torch.empty(t, d, device=dev())
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)
    mo.gated_ffn(x, wg, wu, wd, o, gate=gate, up=up, workspace=ws)
    clean()
    D = torch.float64
    g, u = x.to(D) @ wg.to(D).T, x.to(D) @ wu.to(D).T
    size = [x.to(D).abs() @ v.to(D).abs().T for v in (wg, wu)]
    for got, want, s in ((gate, g, size[0]), (up, u, size[1])):
        tol = f64((d / 16 + 4) * 2.0 ** -23 * s)
        within(got, f64(want), tol + ROUND[BF16] * (np.abs(f64(want)) + tol))
    # backward from the kept values, as they are
    dout = large(t, d, seed=5)
    dw = [torch.empty(v.shape, device=dev()) for v in (wg, wu, wd)]
    dx = torch.empty(t, d, device=dev())
    mo.gated_ffn_grad(dout, x, gate, up, wg, wu, wd, activation="relu", dx=dx, dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2], workspace=ws)
    clean()
    gv, uv, dv = gate.to(D), up.to(D), dout.to(D)
    dh, edh = dv @ wd.to(D), (d / 16 + 4) * 2.0 ** -23 * (dv.abs() @ wd.to(D).abs())
    on = (gv > 0).to(D)
    dg, du = dh * uv * on, dh * gv * on
    eg, eu = edh * (uv * on).abs(), edh * (gv * on).abs()
    R = ROUND[BF16] + 2.0 ** -22
    eg, eu = eg + R * (dg.abs() + eg), eu + R * (du.abs() + eu)
    e = eg @ wg.to(D).abs() + eu @ wu.to(D).abs() + (2 * f / 16 + 8) * 2.0 ** -23 * ((dg.abs() + eg) @ wg.to(D).abs() + (du.abs() + eu) @ wu.to(D).abs())
    want = dg @ wg.to(D) + du @ wu.to(D)
    within(dx, f64(want), f64(e + 2.0 ** -23 * want.abs()), "dx")
    for got, m, em in ((dw[0], dg, eg), (dw[1], du, eu)):
        want = m.T @ x.to(D)
        e = em.T @ x.to(D).abs() + (t / 16 + 4) * 2.0 ** -23 * ((m.abs() + em).T @ x.to(D).abs())
        within(got, f64(want), f64(e + 2.0 ** -23 * want.abs()), "dw")


@pytest.mark.parametrize("t,d,f", [(520, 4900, 32768), (520, 4864, 20001), (64, 20004, 32768), (300, 256, 32768), (3, 33, 32768)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_input_gradient_of_a_wide_block(t, d, f, dtype):
    """Both halves of dx together are longer than one accumulation may be."""
    dout, gate, up = positive(t, d, seed=5), positive(t, f, seed=6), positive(t, f, seed=7)
    wg, wu, wd = positive(f, d, seed=1, std=f ** -0.5), positive(f, d, seed=2, std=f ** -0.5), positive(d, f, seed=3, std=d ** -0.5)
    dx = torch.empty(t, d, dtype=dtype, device=dev())
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)
    ws.fill_(0xFF)
    mo.gated_ffn_grad(dout, None, gate, up, wg, wu, wd, activation=None, dx=dx, workspace=ws)
    clean()
    D = torch.float64
    rows = slice(0, min(t, 64))
    dh = dout[rows].to(D) @ wd.to(D)
    edh = (d / 16 + 4) * 2.0 ** -23 * dh
    a, b = dh * up[rows].to(D), dh * gate[rows].to(D)
    ea, eb = ((ROUND[BF16] + 2.0 ** -22) * (v + e) + e for v, e in ((a, edh * up[rows].to(D)), (b, edh * gate[rows].to(D))))
    want = a @ wg.to(D) + b @ wu.to(D)
    # roundings of a and b go either way; they are a sixteenth of their bound together (a sum of thousands): all of it is allowed
    e = ea @ wg.to(D) + eb @ wu.to(D) + (SLICE / 16 + 8) * 2.0 ** -23 * 1.01 * want
    within(f64(dx[rows]), f64(want), f64(e + ROUND[dtype] * (want + e)))


# ---------------------------------------------------------------- one output at a time

@pytest.mark.parametrize("t,k,n,activation,pre", [(512, 2, 3082, "silu", "bf16"), (973, 312, 2421, "gelu_tanh", "bf16"), (2560, 8, 2346, "gelu", "mx8"),
                                                  (600, 8, 2344, "gelu", "bf16")])
def test_a_bias_gradient_does_not_depend_on_what_else_is_wanted(t, k, n, activation, pre):
    """Several rows a warp, of widths that are and are no multiples of 8."""
    x, w, dout, z = data(t, k), data(n, k, seed=1, std=k ** -0.5), data(t, n, seed=5), data(t, n, seed=6, std=1.5)
    if pre == "mx8":
        q = empty8(t, n)
        mo.mx8_quantize(z, q)
        z = q
    ws = mo.linear_workspace(t, k, n, grad=True)
    got = []
    for more in (dict(), dict(dx=torch.empty(t, k, device=dev())), dict(dw=torch.empty(n, k, device=dev()))):
        got.append(torch.empty(n, device=dev()))
        mo.linear_grad(dout, x, w, dbias=got[-1], activation=activation, pre=z, workspace=ws, **more)
    clean()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
