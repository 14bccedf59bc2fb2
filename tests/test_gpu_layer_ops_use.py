"""The feed-forward operators as programs use them: one after the other in the
example's model, in graphs, on other streams, with buffers that end where the
call ends, with values that are not numbers, with sums that are cut and offsets
past 32 bits, and at sizes that take every variant of the products."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
import test_gpu_layer_ops as base
from gpu_util import f64
from oracle import layer_ops as ol
from test_gpu_layer_ops import BF16, F32, ROUND, act_error, clean, data, dev, empty8, norm_tol, values, within, within8

pytestmark = pytest.mark.gpu
U8 = torch.uint8


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward_step.py")
    spec = importlib.util.spec_from_file_location("feed_forward_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# ---------------------------------------------------------------- every variant of the products

# Tiles of 256 columns (128 of gate and up) on 76 pairs: a last round of 14, 24 and 5 tiles (cut into 4, 2
# and 4 parts), of 32 and more (not cut); reductions above and below 32 blocks of 64; rows that are and are
# not aligned. All with at least 38 tiles, so that nothing is split.

@pytest.mark.parametrize("t,k,n,activation,bias,residual,pre,mx8,out", [
    (2400, 1100, 2304, "gelu_tanh", True, False, "mx8", False, BF16),
    (2500, 2100, 2500, "silu", True, True, "bf16", False, BF16),
    (2300, 2080, 2301, "relu", False, True, "mx8", False, F32),
    (2050, 1032, 2184, None, True, True, None, False, F32),
    (2050, 1029, 2177, "silu", True, False, "mx8", False, BF16),
    (2305, 520, 2248, "relu", False, True, "bf16", False, BF16),
    (4000, 2056, 777, None, False, True, None, False, BF16)])
def test_linear_tiles(t, k, n, activation, bias, residual, pre, mx8, out):
    base.test_linear(t, k, n, activation, bias, residual, pre, mx8, out)


@pytest.mark.parametrize("t,k,n,activation,pre,mx8,dtype,accumulate", [
    (2400, 2300, 2200, "silu", "bf16", False, BF16, True), (2304, 2304, 1000, "relu", "bf16", False, F32, False),
    (1100, 2050, 2301, None, None, False, BF16, False)])
def test_linear_grad_tiles(t, k, n, activation, pre, mx8, dtype, accumulate):
    base.test_linear_grad(t, k, n, activation, pre, mx8, dtype, accumulate)


@pytest.mark.parametrize("t,d,f,activation,residual,save,mx8,out", [
    (2300, 1100, 1153, "silu", True, "mx8", False, BF16), (1800, 2112, 1600, "gelu_tanh", True, "bf16", False, F32),
    (1800, 2112, 1601, "silu", False, "mx8", False, BF16)])
def test_gated_ffn_tiles(t, d, f, activation, residual, save, mx8, out):
    base.test_gated_ffn(t, d, f, activation, residual, save, mx8, out)


@pytest.mark.parametrize("t,d,f,activation,save,mx8,dtype,accumulate", [
    (2300, 1100, 2296, "silu", "bf16", False, BF16, False), (2060, 2100, 1301, "silu", "bf16", False, F32, True)])
def test_gated_ffn_grad_tiles(t, d, f, activation, save, mx8, dtype, accumulate):
    base.test_gated_ffn_grad(t, d, f, activation, save, mx8, dtype, accumulate)


# Reductions that are split: clusters of 2, 4 and 8, one and two CTAs an SM, every operand order.

@pytest.mark.parametrize("t,k,n,activation,bias,residual,pre,mx8,out", [
    (500, 2112, 520, "silu", True, True, "bf16", False, BF16), (300, 4100, 1000, None, False, True, None, False, F32),
    (1000, 1604, 700, "gelu_tanh", True, False, "mx8", False, BF16), (1300, 4200, 1100, "relu", False, False, "mx8", False, F32),
    (72, 8200, 2050, None, True, True, None, False, BF16), (128, 1100, 1030, "silu", False, False, "mx8", False, BF16)])
def test_linear_splits(t, k, n, activation, bias, residual, pre, mx8, out):
    base.test_linear(t, k, n, activation, bias, residual, pre, mx8, out)


@pytest.mark.parametrize("t,k,n,activation,pre,mx8,dtype,accumulate", [
    (2100, 500, 520, "silu", "bf16", False, BF16, True), (4100, 300, 1001, None, None, False, F32, True),
    (140, 1030, 4200, "relu", "bf16", False, BF16, False)])
def test_linear_grad_splits(t, k, n, activation, pre, mx8, dtype, accumulate):
    base.test_linear_grad(t, k, n, activation, pre, mx8, dtype, accumulate)


@pytest.mark.parametrize("t,d,f", [(200, 2112, 700), (130, 1100, 1500), (90, 4104, 264)])
def test_gated_ffn_splits(t, d, f):
    base.test_gated_ffn(t, d, f, "silu", True, "mx8", False, BF16)
    base.test_gated_ffn(t, d, f, "gelu_tanh", False, "bf16", False, F32)
    base.test_gated_ffn_grad(t, d, f, "silu", "bf16", False, BF16, True)


# One and two rows, which have a kernel of their own where nothing is kept: reductions that end inside a
# warp's pieces, columns past every warp's first, the longest rows it takes and longer ones.

@pytest.mark.parametrize("t,k,n", [(1, 8, 5), (2, 264, 4863), (1, 256, 4864), (2, 256, 4865), (1, 512, 9999), (2, 520, 4870), (1, 4096, 33),
                                   (2, 28672, 40), (1, 57344, 17), (2, 28680, 16), (1, 57352, 16), (3, 1280, 100), (1, 1283, 90)])
@pytest.mark.parametrize("activation,bias,residual,mx8,out", [(None, False, False, False, BF16), ("silu", True, True, True, F32),
                                                              ("gelu", False, True, False, BF16)])
def test_one_and_two_rows(t, k, n, activation, bias, residual, mx8, out):
    base.test_linear(t, k, n, activation, bias, residual, None, mx8, out)


@pytest.mark.parametrize("t,d,f", [(1, 8, 16), (2, 264, 4880), (1, 520, 9728), (2, 1280, 1003), (2, 1003, 1288), (1, 512, 5000), (2, 64, 30000)])
@pytest.mark.parametrize("activation,residual,mx8,out", [("silu", True, False, BF16), ("gelu_tanh", False, True, F32)])
def test_gated_block_of_one_and_two_rows(t, d, f, activation, residual, mx8, out):
    base.test_gated_ffn(t, d, f, activation, residual, None, mx8, out)


# Rows that no team of threads holds, aligned and not; more of them than blocks, so that a block's rows add up.

@pytest.mark.parametrize("dim", [8193, 8200, 12288, 16392, 40001])
@pytest.mark.parametrize("dtype,out,residual,mx8", [(BF16, BF16, True, True), (F32, None, False, True)])
def test_long_rows(dim, dtype, out, residual, mx8):
    base.test_norm(dim, dtype, out, residual, mx8)
    base.test_norm_in_place(dim, dtype)


@pytest.mark.parametrize("rows,dim", [(3, 16392), (700, 8200), (650, 8195)])
@pytest.mark.parametrize("dtype,mx8", [(BF16, True), (BF16, False), (F32, True)])
def test_gradients_of_long_rows(rows, dim, dtype, mx8):
    base.test_norm_grad(rows, dim, dtype, mx8, True, rows == 700)


# ---------------------------------------------------------------- sums that are cut, offsets past 32 bits

@pytest.mark.parametrize("t,k,n,accumulate", [(40000, 24, 40, True), (70001, 33, 17, False), (32769, 8, 8, True)])
def test_weight_gradient_over_many_tokens(t, k, n, accumulate):
    base.test_linear_grad(t, k, n, None, None, False, BF16, accumulate)
    base.test_linear_grad(t, k, n, "relu", "bf16", False, F32, accumulate)


@pytest.mark.parametrize("n", [33000, 70001])
def test_input_gradient_over_many_rows(n):
    base.test_linear_grad(9, 24, n, None, None, False, F32, False)
    base.test_linear_grad(130, 16, n, "relu", "bf16", False, BF16, True)


@pytest.mark.parametrize("t,d,f", [(33000, 24, 40), (70001, 9, 17)])
def test_gated_gradients_over_many_tokens(t, d, f):
    base.test_gated_ffn_grad(t, d, f, "relu", "bf16", False, BF16, True)


LONG = 600_000   # rows of 4096: 2.46e9 elements


def test_rows_past_32_bit_offsets():
    """The last rows of a long call are what a call of those rows alone gives."""
    d = 4096
    x = torch.empty(LONG, d, dtype=BF16, device=dev()).normal_(generator=torch.Generator(dev()).manual_seed(1))
    w, tail = data(d, dtype=F32), slice(LONG - 5, LONG)
    q, one = mo.Mx8Tensor(LONG, d), empty8(5, d)
    mo.mx8_quantize(x, q)
    mo.mx8_quantize(x[tail], one)
    assert torch.equal(q.codes[tail], one.codes) and torch.equal(q.scales[tail], one.scales)
    back = torch.empty_like(x)
    mo.mx8_dequantize(q, back)
    assert np.array_equal(f64(back[tail]), values(one))
    mo.rms_norm(x, back, weight=w, out8=q)
    want = ol.rms_norm(f64(x[tail]), f64(w))[0]
    within(back[tail], want, norm_tol(want) + ROUND[BF16] * 1.01 * np.abs(want))
    one.codes.copy_(q.codes[tail])
    one.scales.copy_(q.scales[tail])
    within8(one, want, norm_tol(want))
    mo.rms_norm_grad(back, x, back, weight=w)
    clean()
    dy = want   # (rounded to bf16 where it was stored)
    g, _ = ol.rms_norm_grad(dy, f64(x[tail]), f64(w))
    r = 1 / np.sqrt(np.mean(f64(x[tail]) ** 2, 1, keepdims=True) + 1e-6)
    m = np.abs(dy * f64(w))
    mag = r * (m + np.abs(f64(x[tail]) * r) * np.mean(m * np.abs(f64(x[tail]) * r), 1, keepdims=True))
    within(back[tail], g, (1.01 * 2.0 ** -8 + 320 * 2.0 ** -24) * mag + ROUND[BF16] * 1.01 * np.abs(g))


def test_products_past_32_bit_offsets():
    t, k, n = LONG, 64, 4096
    x, w = data(t, k), data(n, k, seed=1, std=0.125)
    out, pre = torch.empty(t, n, dtype=BF16, device=dev()), mo.Mx8Tensor(t, n)
    mo.linear(x, w, out, activation="silu", pre=pre, workspace=mo.linear_workspace(t, k, n))
    tail = slice(t - 300, t)
    one, p = torch.empty(300, n, dtype=BF16, device=dev()), empty8(300, n)
    ws = mo.linear_workspace(300, k, n, grad=True)
    mo.linear(x[tail], w, one, activation="silu", pre=p, workspace=ws)
    clean()
    assert torch.equal(out[tail], one) and torch.equal(pre.codes[tail], p.codes) and torch.equal(pre.scales[tail], p.scales)
    dx, alone = torch.empty(t, k, dtype=BF16, device=dev()), torch.empty(300, k, device=dev())
    mo.linear_grad(out, None, w, dx=dx, activation="silu", pre=pre, workspace=mo.linear_workspace(t, k, n, grad=True))
    mo.linear_grad(out[tail], None, w, dx=alone, activation="silu", pre=p, workspace=ws)   # (its reduction may be cut otherwise)
    clean()
    dz = np.abs(f64(one) * ol.act(values(p), "silu")[1])
    within(dx[tail], f64(alone), 1.01 * 2 * n * 2.0 ** -23 * (dz @ np.abs(f64(w))) + ROUND[BF16] * np.abs(f64(alone)))


def test_gated_block_past_32_bit_offsets():
    t, d, f = LONG, 64, 4096
    x, wg, wu, wd = data(t, d), data(f, d, seed=1, std=0.125), data(f, d, seed=2, std=0.125), data(d, f, seed=3, std=1 / 64)
    g, u, out = mo.Mx8Tensor(t, f), mo.Mx8Tensor(t, f), torch.empty(t, d, device=dev())
    mo.gated_ffn(x, wg, wu, wd, out, gate=g, up=u, workspace=mo.gated_ffn_workspace(t, d, f))
    tail = slice(t - 300, t)
    want, zg, zu = ol.gated_ffn(f64(x[tail]), f64(wg), f64(wu), f64(wd))
    xv, a = np.abs(f64(x[tail])), np.abs(ol.act(zg, "silu")[0])
    eg, eu = (2.0 ** -23 * (d * (xv @ np.abs(f64(v)).T) + np.abs(z)) for v, z in ((wg, zg), (wu, zu)))
    ea = 1.13 * eg + act_error(zg, "silu")
    eh = ea * np.abs(zu) + (a + ea) * eu
    a = a * np.abs(zu)
    eh = eh + (ROUND[BF16] + 2.0 ** -23) * (a + eh)
    within(out[tail], want, eh @ np.abs(f64(wd)).T + f * 2.0 ** -23 * ((a + eh) @ np.abs(f64(wd)).T) + 2.0 ** -23 * np.abs(want))
    for q, z, e in ((g, zg, eg), (u, zu, eu)):
        within8(mo.Mx8Tensor(300, f, codes=q.codes[tail], scales=q.scales[tail]), z, e)
    dout = data(t, d, seed=5)
    dx = torch.empty(t, d, device=dev())
    mo.gated_ffn_grad(dout, None, g, u, wg, wu, wd, dx=dx, workspace=mo.gated_ffn_workspace(t, d, f, grad=True))
    alone = torch.empty(300, d, device=dev())
    g1, u1 = (mo.Mx8Tensor(300, f, codes=q.codes[tail], scales=q.scales[tail]) for q in (g, u))
    mo.gated_ffn_grad(dout[tail], None, g1, u1, wg, wu, wd, dx=alone, workspace=mo.gated_ffn_workspace(300, d, f, grad=True))
    clean()
    # dh is a sum over one block of 64 in both, and dg and du the same bits; their sums may be cut otherwise
    gv, uv, dv = values(g1), values(u1), np.abs(f64(dout[tail]))
    dh = np.abs(f64(dout[tail]) @ f64(wd)) + d * 2.0 ** -23 * (dv @ np.abs(f64(wd)))
    av, slope = ol.act(gv, "silu")
    ea = act_error(gv, "silu")
    m = (dh * np.abs(uv) * (np.abs(slope) + ea)) @ np.abs(f64(wg)) + (dh * (np.abs(av) + ea)) @ np.abs(f64(wu))
    within(dx[tail], f64(alone), 2 * 2 * f * 2.0 ** -23 * 1.01 * m)


# ---------------------------------------------------------------- nothing else is written

class Guarded:
    """Tensors inside buffers that are checked behind them (and in front)."""
    PAD = 512

    def __init__(self):
        self.buffers = []

    def __call__(self, t):
        nbytes = t.numel() * t.element_size()
        buf = torch.full((self.PAD + nbytes + self.PAD,), 0xA5, dtype=U8, device=dev())
        self.buffers.append((buf, nbytes))
        v = buf[self.PAD:self.PAD + nbytes].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    def mx8(self, q):
        return mo.Mx8Tensor(q.rows, q.k, codes=self(q.codes), scales=self(q.scales))

    def check(self):
        for buf, nbytes in self.buffers:
            assert (buf[:self.PAD] == 0xA5).all() and (buf[self.PAD + nbytes:] == 0xA5).all()


@pytest.mark.parametrize("t,d,f", [(1, 33, 47), (1, 512, 520), (2, 40, 72), (3, 40, 72), (130, 200, 301), (777, 515, 1003), (2300, 520, 1153), (2311, 1096, 1160)])
def test_buffers_end_where_the_call_ends(t, d, f):
    g = Guarded()
    bf = lambda *s: g(torch.zeros(s, dtype=BF16, device=dev()))   # noqa: E731
    fp = lambda *s: g(torch.zeros(s, device=dev()))   # noqa: E731
    ws = lambda n: g(torch.zeros(n, dtype=U8, device=dev()))   # noqa: E731
    x, wg, wu, wd = g(data(t, d)), g(data(f, d, seed=1)), g(data(f, d, seed=2)), g(data(d, f, seed=3))
    n8, s8, g8, u8 = (g.mx8(empty8(t, k)) for k in (d, d, f, f))
    s = bf(t, d)
    mo.mx8_quantize(x, s8)
    mo.mx8_dequantize(s8, fp(t, d))
    mo.mx8_dequantize(s8, s)
    mo.rms_norm(x, bf(t, d), residual=s, sum_out=bf(t, d), out8=n8, weight=fp(d))
    mo.rms_norm_grad(x, n8, bf(t, d), dweight=fp(d), workspace=ws(mo.mo_rms_norm_grad_workspace_bytes(t, d)))
    small, big = ws(mo.mo_linear_workspace_bytes(t, d, f)), ws(mo.mo_linear_workspace_bytes(t, d, f, grad=True))
    for out in (bf(t, f), fp(t, f)):
        mo.linear(x, wg, out, bias=fp(f), activation="silu", residual=out, pre=bf(t, f), workspace=small)
        mo.linear(n8, wg, out, bias=fp(f), activation="gelu", pre=u8, workspace=small)
        mo.linear(x, wg, out, workspace=small)
    dout = bf(t, f)
    mo.linear_grad(dout, n8, wg, dx=bf(t, d), dw=fp(f, d), dbias=fp(f), activation="silu", pre=u8, workspace=big)
    mo.linear_grad(dout, x, wg, dx=fp(t, d), dw=bf(f, d), dbias=fp(f), workspace=big)
    small, big = ws(mo.mo_gated_ffn_workspace_bytes(t, d, f)), ws(mo.mo_gated_ffn_workspace_bytes(t, d, f, grad=True))
    mo.gated_ffn(n8, wg, wu, wd, s, residual=s, gate=g8, up=u8, workspace=small)
    mo.gated_ffn(x, wg, wu, wd, fp(t, d), workspace=small)
    gate, up = bf(t, f), bf(t, f)
    mo.gated_ffn(x, wg, wu, wd, fp(t, d), gate=gate, up=up, workspace=small)
    for pair in ((g8, u8), (gate, up)):
        mo.gated_ffn_grad(s, n8, *pair, wg, wu, wd, dx=bf(t, d), dw_gate=fp(f, d), dw_up=fp(f, d), dw_down=fp(d, f), workspace=big)
        mo.gated_ffn_grad(s, x, *pair, wg, wu, wd, dx=fp(t, d), dw_gate=bf(f, d), dw_up=bf(f, d), dw_down=bf(d, f), workspace=big)
    clean()
    g.check()


# ---------------------------------------------------------------- values that are not numbers

@pytest.mark.parametrize("t,d,f", [(6, 40, 72), (700, 64, 2000), (300, 2112, 264)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_token_that_is_no_number_stays_alone(t, d, f, bad):
    """The bad token's rows are not finite, the others are what they are without it."""
    x, wg, wu, wd = data(t, d), data(f, d, seed=1, std=d ** -0.5), data(f, d, seed=2, std=d ** -0.5), data(d, f, seed=3, std=f ** -0.5)
    y = x.clone()
    y[3, 5] = bad
    keep = [i for i in range(t) if i != 3]
    ws = mo.gated_ffn_workspace(t, d, f, grad=True)
    ls = mo.linear_workspace(t, d, f, grad=True)
    got = []
    for v in (x, y):
        norm, n8 = torch.empty_like(x), empty8(t, d)
        g8, u8, z8 = empty8(t, f), empty8(t, f), empty8(t, f)
        out, lin, dx, dl = torch.empty_like(x), torch.empty(t, f, dtype=BF16, device=dev()), torch.empty_like(x), torch.empty_like(x)
        mo.rms_norm(v, norm, out8=n8)
        mo.gated_ffn(v, wg, wu, wd, out, residual=v, gate=g8, up=u8, workspace=ws)
        mo.gated_ffn_grad(x, None, g8, u8, wg, wu, wd, dx=dx, workspace=ws)
        mo.linear(v, wg, lin, activation="gelu_tanh", pre=z8, workspace=ls)
        mo.linear_grad(torch.ones_like(lin), None, wg, dx=dl, activation="gelu_tanh", pre=z8, workspace=ls)
        deq = torch.empty_like(x)
        mo.mx8_dequantize(n8, deq)
        got.append((norm, deq, out, lin, dx, dl))
    clean()
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a[keep], b[keep]), i
        assert torch.isfinite(a).all() and not torch.isfinite(b[3]).all(), i
    # a token's infinity divided by itself, or summed with both signs, is no number in every column
    assert torch.isnan(got[1][2][3]).all() and torch.isnan(got[1][4][3]).all()


@pytest.mark.parametrize("t,d,f", [(6, 40, 72), (2400, 64, 2300)])
def test_padding_is_zeros_beside_values_that_are_no_numbers(t, d, f):
    x = data(t, d)
    x[3, 5] = float("inf")
    w, z8, out = data(f, d, seed=1), empty8(t, f), torch.empty(t, f, dtype=BF16, device=dev())
    mo.linear(x, w, out, activation="silu", pre=z8, workspace=mo.linear_workspace(t, d, f))
    g8, u8, y = empty8(t, f), empty8(t, f), torch.empty(t, d, dtype=BF16, device=dev())
    mo.gated_ffn(x, w, w, data(d, f, seed=2), y, gate=g8, up=u8, workspace=mo.gated_ffn_workspace(t, d, f))
    n8 = empty8(t, d)
    mo.rms_norm(x, out8=n8)
    clean()
    for q in (z8, g8, u8, n8):
        assert (q.codes[:, q.k:] == 0).all() and (q.scales[3] == 255).any()
        assert (q.scales[[i for i in range(t) if i != 3]] != 255).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_block_that_is_no_number_stays_alone(bad):
    x = data(4, 100)
    x[2, 40] = bad
    q, out = empty8(4, 100), torch.empty(4, 100, device=dev())
    mo.mx8_quantize(x, q)
    mo.mx8_dequantize(q, out)
    clean()
    nan = torch.isnan(out)
    assert nan[2, 32:64].all() and int(nan.sum()) == 32


def test_large_arguments_of_activations():
    """act and act' at both ends: 0 and the argument, 0 and 1, and none of them NaN."""
    z = torch.tensor([[-3e38, -1e30, -1e4, -200.0, -60.0, 0.0, 60.0, 200.0, 1e4, 1e30, 3e38, -0.0] + [0.0] * 52], device=dev()).to(BF16)
    eye = torch.eye(64, dtype=BF16, device=dev())
    ws = mo.linear_workspace(1, 64, 64, grad=True)
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        out, dx = torch.empty(1, 64, device=dev()), torch.empty(1, 64, device=dev())
        mo.linear(z, eye, out, activation=name, workspace=ws)
        mo.linear_grad(torch.ones_like(z), None, eye, dx=dx, activation=name, pre=z, workspace=ws)
        clean()
        o, s, v = out[0], dx[0], z[0].float()
        assert torch.equal(o[6:11], v[6:11]) and (s[6:11] == 1).all(), name
        assert (o[:5].abs() <= 1e-20).all() and (s[:5].abs() <= 1e-20).all(), name


# ---------------------------------------------------------------- streams, graphs, repeats

class Step:
    """A gated block with its norm, forward and backward, in buffers of its own but for the workspaces."""

    def __init__(self, t, d, f, ws, norm_ws, seed):
        self.ws, self.norm_ws = ws, norm_ws
        self.x, self.s, self.ds = data(t, d, seed=seed), data(t, d, seed=seed + 1), data(t, d, seed=seed + 2)
        self.w, self.b = data(d, dtype=F32, seed=seed + 3), data(f, dtype=F32, seed=seed + 7)
        self.mats = [data(f, d, seed=seed + 4, std=d ** -0.5), data(f, d, seed=seed + 5, std=d ** -0.5), data(d, f, seed=seed + 6, std=f ** -0.5)]
        self.n8, self.s8, self.g8, self.u8 = empty8(t, d), empty8(t, d), empty8(t, f), empty8(t, f)
        e = torch.empty_like
        self.sum, self.out, self.dn, self.dx, self.dw = e(self.s), e(self.s), e(self.s), e(self.s), e(self.w)
        self.h, self.z8, self.y, self.db = torch.empty(t, f, dtype=BF16, device=dev()), empty8(t, f), e(self.s), torch.empty(f, device=dev())
        self.grads = [e(m) for m in self.mats]
        self.g1, self.served, self.logits = e(self.mats[0]), e(self.s), e(self.h)

    def run(self, stream=None):
        k = dict(stream=stream)
        mo.rms_norm(self.x, weight=self.w, residual=self.s, sum_out=self.sum, out8=self.n8, **k)
        mo.mx8_quantize(self.sum, self.s8, **k)
        mo.gated_ffn(self.n8, *self.mats, self.out, residual=self.sum, gate=self.g8, up=self.u8, workspace=self.ws, **k)
        mo.gated_ffn(self.x, *self.mats, self.served, workspace=self.ws, **k)
        mo.linear(self.served, self.mats[0], self.logits, workspace=self.ws, **k)
        mo.linear(self.out, self.mats[0], self.h, bias=self.b, activation="gelu", pre=self.z8, workspace=self.ws, **k)
        mo.linear_grad(self.h, self.out, self.mats[0], dx=self.y, dw=self.g1, dbias=self.db, activation="gelu", pre=self.z8, workspace=self.ws, **k)
        mo.gated_ffn_grad(self.ds, self.n8, self.g8, self.u8, *self.mats, dx=self.dn, dw_gate=self.grads[0], dw_up=self.grads[1],
                          dw_down=self.grads[2], workspace=self.ws, **k)
        mo.rms_norm_grad(self.dn, self.s8, self.dx, weight=self.w, dresidual=self.ds, dweight=self.dw, workspace=self.norm_ws, **k)

    def results(self):
        return [self.sum, self.out, self.h, self.y, self.g1, self.db, self.dn, self.dx, self.dw, self.served, self.logits, *self.grads,
                *(v for q in (self.n8, self.s8, self.g8, self.u8, self.z8) for v in (q.codes, q.scales))]

    def spoil(self):
        for v in self.results():
            v.view(U8).fill_(0x77)

    def take(self):
        return [v.clone() for v in self.results()]


def workspaces(t, d, f):
    n = max(mo.mo_gated_ffn_workspace_bytes(t, d, f, grad=True), mo.mo_linear_workspace_bytes(t, d, f, grad=True))
    return torch.empty(n, dtype=U8, device=dev()), mo.rms_norm_grad_workspace(t, d)


def same(a, b):
    return all(torch.equal(x.view(U8), y.view(U8)) for x, y in zip(a, b))


SIZES = [(1, 64, 96), (2, 520, 1000), (37, 200, 301), (513, 256, 704), (2304, 1032, 1160)]


@pytest.mark.parametrize("t,d,f", SIZES)
def test_two_graphs_share_a_workspace(t, d, f):
    ws = workspaces(t, d, f)
    steps, want, graphs = [Step(t, d, f, *ws, seed=s) for s in (0, 50)], [], []
    for s in steps:
        s.run()
        want.append(s.take())
    clean()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for order in ((0, 1, 0), (1, 1, 0)):
        for i in order:
            steps[i].spoil()
            ws[0].fill_(0xFF)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(steps[i].take(), want[i]), (order, i)
        # one behind the other, and an eager run between them
        for s in steps:
            s.spoil()
        graphs[0].replay()
        steps[1].run()
        graphs[0].replay()
        clean()
        assert same(steps[0].take(), want[0]) and same(steps[1].take(), want[1])
    # new inputs in the same places
    steps[0].x.copy_(steps[1].x)
    steps[0].run()
    fresh = steps[0].take()
    steps[0].spoil()
    graphs[0].replay()
    clean()
    assert same(steps[0].take(), fresh) and not same(fresh, want[0])


@pytest.mark.parametrize("t,d,f", SIZES)
def test_another_stream_and_two_at_once(t, d, f):
    a, b = Step(t, d, f, *workspaces(t, d, f), seed=0), Step(t, d, f, *workspaces(t, d, f), seed=50)
    want = []
    for s in (a, b):
        s.run()
        want.append(s.take())
        s.spoil()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    a.run(stream=streams[0])                 # given
    with torch.cuda.stream(streams[1]):      # current
        b.run()
    for s in streams:
        s.synchronize()
    clean()
    assert same(a.take(), want[0]) and same(b.take(), want[1])


@pytest.mark.parametrize("t,d,f", SIZES + [(40000, 40, 72)])
def test_repeats_bit_for_bit(t, d, f):
    s = Step(t, d, f, *workspaces(t, d, f), seed=0)
    s.run()
    first = s.take()
    for fill in (0x00, 0xFF, 0x5A):
        s.spoil()
        s.ws.fill_(fill)
        s.norm_ws.fill_(fill)
        s.run()
        clean()
        assert same(s.take(), first)


def test_no_tokens():
    d, f = 40, 72
    s = Step(0, d, f, *(mo.gated_ffn_workspace(0, d, f, grad=True), mo.rms_norm_grad_workspace(0, d)), seed=0)
    kept = [g.clone() for g in (s.grads[0], s.g1)]
    s.run()
    clean()
    assert all(not g.any() for g in (*s.grads, s.g1, s.db, s.dw))   # sums over nothing
    s.grads[0].copy_(kept[0].nan_to_num())
    mo.gated_ffn_grad(s.ds, s.n8, s.g8, s.u8, *s.mats, dw_gate=s.grads[0], workspace=s.ws, accumulate=True)
    clean()
    assert torch.equal(s.grads[0], kept[0].nan_to_num())


def test_addresses_at_odd_multiples_of_16_bytes():
    """Inputs and outputs that are aligned to 16 bytes and no more give the same bits."""
    t, d, f = 300, 264, 520
    ws = workspaces(t, d, f)
    a, b = Step(t, d, f, *ws, seed=0), Step(t, d, f, *ws, seed=0)

    def moved(v):
        buf = torch.empty(v.numel() * v.element_size() + 16 + 240, dtype=U8, device=dev())
        at = (16 - buf.data_ptr() % 32) % 32
        o = buf[at:at + v.numel() * v.element_size()].view(v.dtype).view(v.shape)
        assert o.data_ptr() % 32 == 16
        return o.copy_(v)

    for k, v in list(vars(b).items()):
        if torch.is_tensor(v) and k not in ("ws", "norm_ws"):
            setattr(b, k, moved(v))
        elif isinstance(v, mo.Mx8Tensor):
            setattr(b, k, mo.Mx8Tensor(v.rows, v.k, codes=moved(v.codes), scales=moved(v.scales)))
        elif isinstance(v, list):
            setattr(b, k, [moved(x) for x in v])
    a.run()
    b.run()
    clean()
    assert same(a.take(), b.take())


# ---------------------------------------------------------------- the example

def test_example_runs_and_repeats():
    m = example()
    losses = m.train(steps=4)
    assert all(math.isfinite(x) for x in losses)
    assert m.train(steps=4) == losses


def test_example_gradients():
    """Each operator of a forward and a backward pass of the example against the formula of what it was given."""
    model = example().Model(vocab=264, dim=136, inner=200, seq=32, batch=5)
    n = model.n
    tokens = torch.randint(0, model.vocab, (n,), device=dev(), generator=torch.Generator(dev()).manual_seed(3))
    gated, plain = model.blocks
    model.forward(tokens)
    clean()
    s0 = f64(model.table.w)[tokens.cpu().numpy()]
    s = f64(torch.from_numpy(s0).to(BF16))     # the stream as the lookup stored it
    R, eps = ROUND[BF16], 2.0 ** -23

    def product(a, w):
        return a.shape[1] * eps * (np.abs(a) @ np.abs(w).T)

    # gated block: norm and its 8-bit result, gate and up, the stream
    assert np.array_equal(values(gated.s8), ol.mx8_quantize(s)[2])
    want = ol.rms_norm(s, f64(gated.norm.w))[0]
    within8(gated.n8, want, norm_tol(want), "n8")
    n8, wg, wu, wd = values(gated.n8), f64(gated.gate.b), f64(gated.up.b), f64(gated.down.b)
    g, u = n8 @ wg.T, n8 @ wu.T
    eg, eu = product(n8, wg) + eps * np.abs(g), product(n8, wu) + eps * np.abs(u)
    within8(gated.g8, g, eg, "gate")
    within8(gated.u8, u, eu, "up")
    a = ol.act(g, "silu")[0]
    ea = 1.13 * eg + act_error(g, "silu")
    eh = ea * np.abs(u) + (np.abs(a) + ea) * eu
    eh = eh + (R + eps) * (np.abs(a * u) + eh)
    s1 = s + (a * u) @ wd.T
    e1 = eh @ np.abs(wd).T + wd.shape[1] * eps * ((np.abs(a * u) + eh) @ np.abs(wd).T) + eps * np.abs(s1)
    # (the second block's checkpoint is of the stream as the first stored it)
    within8(plain.s8, s1, e1 + R * (np.abs(s1) + e1), "s8")
    # plain block, from what is still there: n, z and h are stored
    z = f64(plain.n) @ f64(plain.w1.b).T + f64(plain.b1.w)
    ez = product(f64(plain.n), f64(plain.w1.b)) + eps * np.abs(z)
    within8(plain.z8, z, ez, "z8")
    h = ol.act(z, "gelu_tanh")[0]
    e = 1.13 * ez + act_error(z, "gelu_tanh") + eps * np.abs(h)
    within(plain.h, h, e + R * (np.abs(h) + e), "h")
    want = ol.rms_norm(f64(model.s), f64(model.norm.w))[0]
    within(model.z, want, norm_tol(want) + R * 1.01 * np.abs(want), "z")
    want = f64(model.z) @ f64(model.head.b).T
    within(model.logits, want, product(f64(model.z), f64(model.head.b)) + eps * np.abs(want), "logits")

    # backward, a gradient at a time
    dlogits = data(n, model.vocab, seed=9, std=1e-3)
    mo.linear_grad(dlogits, model.z, model.head.b, dx=model.dz, dw=model.head.grad, workspace=model.ws)
    dl, zv, wh = f64(dlogits), f64(model.z), f64(model.head.b)
    for got, want, e in ((model.dz, dl @ wh, product(dl, wh.T)), (model.head.grad, dl.T @ zv, product(dl.T, zv.T))):
        within(got, want, e + (R + eps) * (np.abs(want) + e), "head")
    mo.rms_norm_grad(model.dz, model.s, model.ds, weight=model.norm.w, dweight=model.norm.grad, workspace=model.norm_ws)

    def norm_grad(dy, x, w, dres, dx, dw):
        want, want_w = ol.rms_norm_grad(dy, x, w, 1e-6, dres)
        r = 1 / np.sqrt(np.mean(x * x, 1, keepdims=True) + 1e-6)
        m = np.abs(dy * w)
        mag = r * (m + np.abs(x * r) * np.mean(m * np.abs(x * r), 1, keepdims=True)) + (0 if dres is None else np.abs(dres))
        tol = 240 * 2.0 ** -24 * mag
        within(dx, want, tol + R * (np.abs(want) + tol), "norm dx")
        within(dw, want_w, (n + 80) * 2.0 ** -24 * np.abs(dy * x * r).sum(0) + eps * np.abs(want_w), "norm dweight")

    norm_grad(f64(model.dz), f64(model.s), f64(model.norm.w), None, model.ds, model.norm.grad)
    ds = f64(model.ds)
    plain.backward(model.ds, model.ws, model.norm_ws)
    clean()
    w1, w2, h, nv = f64(plain.w1.b), f64(plain.w2.b), f64(plain.h), f64(plain.n)
    for got, want, e in ((plain.dh, ds @ w2, product(ds, w2.T)), (plain.w2.grad, ds.T @ h, product(ds.T, h.T))):
        within(got, want, e + (R + eps) * (np.abs(want) + e), "w2")
    within(plain.b2.grad, ds.sum(0), n * 2.0 ** -24 * np.abs(ds).sum(0) + eps * np.abs(ds).sum(0), "b2")
    dh, zv = f64(plain.dh), values(plain.z8)
    dz = dh * ol.act(zv, "gelu_tanh")[1]
    ed = np.abs(dh) * act_error(zv, "gelu_tanh")
    within(plain.b1.grad, dz.sum(0), ed.sum(0) + n * 2.0 ** -24 * (np.abs(dz) + ed).sum(0) + eps * np.abs(dz).sum(0), "b1")
    ed = ed + R * (np.abs(dz) + ed)
    m = np.abs(dz) + ed
    for got, want, e in ((plain.dn, dz @ w1, ed @ np.abs(w1) + dz.shape[1] * eps * (m @ np.abs(w1))),
                         (plain.w1.grad, dz.T @ nv, ed.T @ np.abs(nv) + n * eps * (m.T @ np.abs(nv)))):
        within(got, want, e + (R + eps) * (np.abs(want) + e), "w1")
    norm_grad(f64(plain.dn), values(plain.s8), f64(plain.norm.w), ds, model.ds, plain.norm.grad)
    ds = f64(model.ds)
    gated.backward(model.ds, model.ws, model.norm_ws)
    clean()
    gv, uv = values(gated.g8), values(gated.u8)
    a, slope = ol.act(gv, "silu")
    ea, dh, edh = act_error(gv, "silu"), np.abs(ds @ wd), product(ds, wd.T)
    mg, mu, mh = dh * np.abs(uv * slope), dh * np.abs(a), np.abs(a * uv)
    eg, eu, eh = np.abs(uv) * (edh * (np.abs(slope) + ea) + dh * ea), edh * (np.abs(a) + ea) + dh * ea, ea * np.abs(uv)
    r4 = R + 4 * 2.0 ** -24
    eg, eu, eh = eg + r4 * (mg + eg), eu + r4 * (mu + eu), eh + r4 * (mh + eh)
    want = ol.gated_ffn_grad(ds, n8, gv, uv, wg, wu, wd, "silu")
    f = wg.shape[0]
    e = eg @ np.abs(wg) + eu @ np.abs(wu) + 2 * f * eps * ((mg + eg) @ np.abs(wg) + (mu + eu) @ np.abs(wu))
    within(gated.dn, want[0], e + R * (np.abs(want[0]) + e), "dn")
    for got, v, m, em in ((gated.gate.grad, want[1], mg, eg), (gated.up.grad, want[2], mu, eu)):
        e = em.T @ np.abs(n8) + n * eps * ((m + em).T @ np.abs(n8))
        within(got, v, e + (R + eps) * (np.abs(v) + e), "gate, up")
    e = np.abs(ds).T @ eh + n * eps * (np.abs(ds).T @ (mh + eh))
    within(gated.down.grad, want[3], e + (R + eps) * (np.abs(want[3]) + e), "down")
    norm_grad(f64(gated.dn), values(gated.s8), f64(gated.norm.w), ds, model.ds, gated.norm.grad)
    mo.embed_grad(model.ds, tokens, model.table.grad, model.embed_ws)
    clean()
    want = np.zeros((model.vocab, model.ds.shape[1]))
    np.add.at(want, tokens.cpu().numpy(), f64(model.ds))
    mags = np.zeros_like(want)
    np.add.at(mags, tokens.cpu().numpy(), np.abs(f64(model.ds)))
    within(model.table.grad, want, n * 2.0 ** -24 * mags, "table")
