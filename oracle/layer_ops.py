"""Float64 oracle of the feed-forward operators: 8-bit tensors, residual
root-mean-square norm, products with epilogues, the gated block, and their
gradients. NumPy, plain formulas; shares no code with the library."""
import math

import numpy as np

SQRT_2_PI = math.sqrt(2.0 / math.pi)


# ---------------------------------------------------------------- 8-bit tensors

def _e4m3_table():
    v = np.empty(128)
    for c in range(127):
        e, f = c >> 3, c & 7
        v[c] = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    return v


E4M3 = _e4m3_table()
MIDPOINTS = (E4M3[:126] + E4M3[1:127]) / 2


def mx8_quantize(x):
    """(codes [rows, 32 nb], scales [rows, nb], values [rows, k]) of x."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    nb = -(-k // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :k] = x
    v = v.reshape(rows, nb, 32)
    codes = np.zeros(v.shape, dtype=np.uint8)
    scales = np.zeros((rows, nb), dtype=np.uint8)
    values = np.zeros(v.shape)
    for r in range(rows):
        for b in range(nb):
            block = v[r, b]
            top = np.abs(block).max() if not np.isnan(block).any() else np.nan
            if not np.isfinite(top):
                scales[r, b] = 255
                values[r, b] = np.nan
                continue
            e = -127
            while 448.0 * 2.0 ** e < top:
                e += 1 if top <= 448.0 * 2.0 ** (e + 40) else 40
            scales[r, b] = e + 127
            y = np.abs(block) * 2.0 ** -e
            c = np.searchsorted(MIDPOINTS, y)                       # the first code whose upper midpoint is >= y
            tie = (c < 126) & (y == MIDPOINTS[np.minimum(c, 125)]) & (c % 2 == 1)
            c = np.where(tie, c + 1, c)                             # ties to the even code
            codes[r, b] = c + 128 * np.signbit(block)
            values[r, b] = np.where(np.signbit(block), -E4M3[c], E4M3[c]) * 2.0 ** e
    return codes.reshape(rows, -1), scales, values.reshape(rows, -1)[:, :k]


def mx8_values(codes, scales, k):
    c = np.asarray(codes).astype(np.int64)
    s = np.where(np.asarray(scales) == 255, np.nan, np.exp2(np.asarray(scales).astype(np.float64) - 127))
    v = np.where(c >= 128, -E4M3[c % 128], E4M3[c % 128])
    return (v * np.repeat(s, 32, axis=1))[:, :k]


# ---------------------------------------------------------------- norm

def rms_norm(x, weight=None, eps=1e-6, residual=None):
    """(y, s)"""
    s = x if residual is None else x + residual
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return s * r * (1.0 if weight is None else weight), s


def rms_norm_grad(dy, s, weight=None, eps=1e-6, dresidual=None):
    """(dx, dweight)"""
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    n = s * r
    g = dy if weight is None else dy * weight
    dx = r * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return dx if dresidual is None else dx + dresidual, (dy * n).sum(axis=0)


# ---------------------------------------------------------------- activations

def _erfc(x):
    return np.vectorize(math.erfc, otypes=[float])(x)


def act(z, name):
    """(value, slope)"""
    if name is None:
        return z, np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, z, 0.0), np.where(z > 0, 1.0, 0.0)
    if name == "silu":
        s = 0.5 * (1 + np.tanh(z / 2))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        p = 0.5 * _erfc(-z / math.sqrt(2))
        return z * p, p + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    assert name == "gelu_tanh"
    t = np.tanh(SQRT_2_PI * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * SQRT_2_PI * (1 + 3 * 0.044715 * z * z)


# ---------------------------------------------------------------- products

def linear(x, w, bias=None, activation=None, residual=None):
    """(out, z)"""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, activation)[0]
    return (y if residual is None else y + residual), z


def linear_grad(dout, x, w, activation=None, pre=None):
    """(dx, dw, dbias)"""
    dz = dout if activation is None else dout * act(pre, activation)[1]
    return dz @ w, dz.T @ x, dz.sum(axis=0)


def gated_ffn(x, wg, wu, wd, activation="silu", residual=None):
    """(out, gate, up)"""
    g, u = x @ wg.T, x @ wu.T
    y = (act(g, activation)[0] * u) @ wd.T
    return (y if residual is None else y + residual), g, u


def gated_ffn_grad(dout, x, gate, up, wg, wu, wd, activation="silu"):
    """(dx, dw_gate, dw_up, dw_down)"""
    a, slope = act(gate, activation)
    dh = dout @ wd
    dg, du = dh * up * slope, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dout.T @ (a * up)
