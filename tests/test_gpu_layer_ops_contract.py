"""Feed-forward operators on the GPU: calls that the documentation allows beside
the usual ones, at both ends of the numbers' range and of the sizes."""
import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
import test_gpu_layer_ops as base
from gpu_util import f64
from oracle import layer_ops as ol
from test_gpu_layer_ops import BF16, clean, dev, empty8

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
