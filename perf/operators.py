"""Workloads of the training-step operators around the optimizer: embedding
lookup and its gradient, counter-based dropout, and microscaled 4-bit
quantisation with its product.

`run` computes a case either with the library's operators (`own` true) or in
plain form: elementary torch operations in 32 bits, rounded once at the end.
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = {"mx": 32, "nv": 16}            # elements that share a scale
MAX_CODE, MAX_NV_SCALE = 6.0, 448.0     # largest 4-bit value, largest e4m3 scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token: a row of a GPT-2-width table and its position's row, where latency is all
        {"name": "lookup one token", "op": "lookup", "n": 1, "vocab": 50257, "dim": 1280, "table": "f32", "out": "bf16",
         "scale": 1.0, "positions": 1024, "p": 0.0},
        # a training batch into the Llama-style 8B table, scaled by sqrt(dim), with embedding dropout
        {"name": "lookup 8B batch", "op": "lookup", "n": 16384, "vocab": 128256, "dim": 4096, "table": "f32", "out": "bf16",
         "scale": 64.0, "positions": 0, "p": 0.1},
        # the embedding gradient of eight 1024-token sequences, under the embedding dropout
        {"name": "grad GPT-2 batch", "op": "grad", "n": 8192, "vocab": 50257, "dim": 1280, "dout": "bf16", "scale": 1.0,
         "p": 0.1, "padding": 0.0, "accumulate": False},
        # the gradient of the 8B table: 2.1 GB written for the AdamW tail
        {"name": "grad 8B batch", "op": "grad", "n": 16384, "vocab": 128256, "dim": 4096, "dout": "bf16", "scale": 64.0,
         "p": 0.0, "padding": 0.0, "accumulate": False},
        # gradient accumulation with padded sequences, few rows that many tokens share, an odd width
        {"name": "grad accumulated odd", "op": "grad", "n": 3001, "vocab": 1003, "dim": 257, "dout": "f32", "scale": 1.0,
         "p": 0.25, "padding": 0.3, "accumulate": True},
        # residual dropout of an 8B-width activation
        {"name": "dropout residual", "op": "dropout", "n": 16384 * 4096, "dtype": "bf16", "residual": True, "p": 0.1},
        # the backward pass of a small odd tensor
        {"name": "dropout odd", "op": "dropout", "n": 1023 * 257, "dtype": "f32", "residual": False, "p": 0.5},
        # an 8B feed-forward weight after its update, in the orientations of the forward and the backward product
        {"name": "quantize weight mx", "op": "quantize", "rows": 14336, "cols": 4096, "dtype": "f32", "format": "mx",
         "stochastic": False},
        # an output gradient, rounded stochastically
        {"name": "quantize gradient nv", "op": "quantize", "rows": 4096, "cols": 5120, "dtype": "bf16", "format": "nv",
         "stochastic": True},
        # one token through an 8B feed-forward weight
        {"name": "product one token nv", "op": "product", "m": 1, "n": 14336, "k": 4096, "format": "nv"},
        # a batch through the same
        {"name": "product 8B batch mx", "op": "product", "m": 8192, "n": 14336, "k": 4096, "format": "mx"},
        # forward and backward of a GPT-2 Large feed-forward weight: the output, and the gradients of input and weight
        {"name": "linear GPT-2 step nv", "op": "linear", "tokens": 8192, "cols": 1280, "rows": 5120, "format": "nv"},
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):   # most widths are multiples of 8 to 64, some are odd
        w = between(lo, hi)
        step = rng.choice([1, 8, 32, 64])
        return max(step, w // step * step)

    op = rng.choice(["lookup", "grad", "dropout", "quantize", "product", "linear"])
    if op == "lookup":
        return {"op": op, "n": between(1, 16384), "vocab": between(256, 128256), "dim": width(16, 4096),
                "table": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "scale": rng.choice([1.0, 0.5, 8.0]),
                "positions": rng.choice([0, 128, 1024]), "p": rng.choice([0.0, 0.1, 0.3])}
    if op == "grad":
        return {"op": op, "n": between(1, 16384), "vocab": between(256, 128256), "dim": width(16, 4096),
                "dout": rng.choice(["f32", "bf16"]), "scale": rng.choice([1.0, 0.5, 8.0]), "p": rng.choice([0.0, 0.1, 0.3]),
                "padding": rng.choice([0.0, 0.0, 0.2, 0.6]), "accumulate": rng.choice([False, True])}
    if op == "dropout":
        return {"op": op, "n": between(1000, 16384 * 4096), "dtype": rng.choice(["f32", "bf16"]),
                "residual": rng.choice([False, True]), "p": rng.choice([0.05, 0.1, 0.3, 0.5])}
    if op == "quantize":
        return {"op": op, "rows": between(1, 14336), "cols": width(16, 4096), "dtype": rng.choice(["f32", "bf16"]),
                "format": rng.choice(["mx", "nv"]), "stochastic": rng.choice([False, True])}
    if op == "product":
        return {"op": op, "m": between(1, 8192), "n": width(64, 14336), "k": width(32, 4096), "format": rng.choice(["mx", "nv"])}
    return {"op": op, "tokens": between(16, 8192), "cols": width(64, 2560), "rows": width(64, 5120),
            "format": rng.choice(["mx", "nv"])}


# ------------------------------------------------------------------ inputs

def _token_shares(vocab):
    """Token frequencies of natural text, near enough: 1 / (rank + 2.7)."""
    w = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return w / w.sum()


def _tokens(g, n, vocab):
    cdf = torch.from_numpy(np.cumsum(_token_shares(vocab)).astype(np.float32)).cuda()
    rank = torch.searchsorted(cdf, torch.rand(n, generator=g, device="cuda")).clamp_(max=vocab - 1)
    return torch.randperm(vocab, generator=g, device="cuda")[rank]


def _normal(g, shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DTYPES[dtype])


def _activation(g, rows, cols, dtype="bf16", std=1.0):
    """Values whose rows and columns differ in size, as those of activations and gradients do."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    x *= torch.exp(torch.randn((1, cols), generator=g, device="cuda"))
    return (x * std).to(DTYPES[dtype])


def _packed(x, fmt):
    """A 4-bit tensor as a program keeps it: codes (two a byte, the even one low), scales in
    tiles of 128 rows by 4 blocks, and the magnitude that fixes the tensor's own scale."""
    rows, k = x.shape
    amax = x.float().abs().amax().reshape(1) if fmt == "nv" else None
    value, scale, code, sbits = _quantize(x.float(), fmt, None, 0, amax)
    kp = -(-k // 32) * 32
    c = torch.zeros((rows, kp), dtype=torch.uint8, device=x.device)
    c[:, :k] = code
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    nb = sbits.shape[1]
    tiles = -(-nb // 4)
    s = torch.zeros((-(-rows // 128) * 128, tiles * 4), dtype=torch.uint8, device=x.device)
    s[:rows, :nb] = sbits
    scales = s.reshape(-1, 4, 32, tiles, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return {"codes": codes.contiguous(), "scales": scales, "amax": amax, "rows": rows, "k": k, "format": fmt}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c["seed"] = 1000003 * seed + 17      # of the counter-based generator
    op = c["op"]
    if op == "lookup":
        c["table_t"] = _normal(g, (c["vocab"], c["dim"]), c["table"], 0.02)
        c["tokens_t"] = _tokens(g, c["n"], c["vocab"])
        c["add_t"] = _normal(g, (c["positions"], c["dim"]), c["table"], 0.02) if c["positions"] else None
        c["out_t"] = torch.empty((c["n"], c["dim"]), dtype=DTYPES[c["out"]], device="cuda")
    elif op == "grad":
        c["tokens_t"] = _tokens(g, c["n"], c["vocab"])
        c["padding_idx"] = -1
        if c["padding"]:
            c["padding_idx"] = 0
            c["tokens_t"][torch.rand(c["n"], generator=g, device="cuda") < c["padding"]] = 0
        c["dout_t"] = _normal(g, (c["n"], c["dim"]), c["dout"], 1e-3)
        c["grad_t"] = _normal(g, (c["vocab"], c["dim"]), "f32", 1e-3)   # the gradient so far, where it is added to
    elif op == "dropout":
        c["x_t"] = _normal(g, (c["n"],), c["dtype"])
        c["residual_t"] = _normal(g, (c["n"],), c["dtype"]) if c["residual"] else None
        c["out_t"] = torch.empty_like(c["x_t"])
    elif op == "quantize":
        c["x_t"] = _activation(g, c["rows"], c["cols"], c["dtype"], 1e-3 if c["stochastic"] else 0.02)
        c["row_t"] = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device="cuda")
        c["col_t"] = torch.empty((c["cols"], c["rows"]), dtype=torch.bfloat16, device="cuda")
    elif op == "product":
        c["a_t"] = _packed(_activation(g, c["m"], c["k"]), c["format"])
        c["b_t"] = _packed(_activation(g, c["n"], c["k"], "f32", 0.02), c["format"])
        c["out_t"] = torch.empty((c["m"], c["n"]), dtype=torch.bfloat16, device="cuda")
    else:
        c["x_t"] = _activation(g, c["tokens"], c["cols"])
        c["w_t"] = _normal(g, (c["rows"], c["cols"]), "f32", 0.02)
        c["dy_t"] = _activation(g, c["tokens"], c["rows"], "bf16", 1e-3)
        c["y_t"] = torch.empty((c["tokens"], c["rows"]), dtype=torch.bfloat16, device="cuda")
        c["dx_t"] = torch.empty((c["tokens"], c["cols"]), dtype=torch.bfloat16, device="cuda")
        c["dw_t"] = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device="cuda")
    if own:   # what the library's users keep from step to step: workspaces and the storage of 4-bit tensors
        import matrix_optimizers_zero_gb300 as mo
        f = c.get("format")
        if op == "grad":
            c["ws"] = mo.embed_grad_workspace(c["n"], c["vocab"], c["dim"])
        elif op == "quantize":
            c["q"] = mo.Fp4Tensor(c["rows"], c["cols"], f), mo.Fp4Tensor(c["cols"], c["rows"], f)
        elif op == "product":
            c["q"] = tuple(mo.Fp4Tensor(t["rows"], t["k"], f, codes=t["codes"], scales=t["scales"], amax=t["amax"])
                           for t in (c["a_t"], c["b_t"]))
        elif op == "linear":
            t, r, k = c["tokens"], c["rows"], c["cols"]
            c["q"] = tuple(mo.Fp4Tensor(*s, f) for s in ((t, k), (k, t), (r, k), (k, r), (t, r), (r, t)))
    return c


# ------------------------------------------------------------------ the library's operators

def _run_own(c):
    import matrix_optimizers_zero_gb300 as mo
    op = c["op"]
    if op == "lookup":
        drop = mo.Dropout(c["p"], c["seed"]) if c["p"] else None
        mo.embed_lookup(c["table_t"], c["tokens_t"], c["out_t"], scale=c["scale"], add=c["add_t"], dropout=drop)
        return c["out_t"]
    if op == "grad":
        drop = mo.Dropout(c["p"], c["seed"]) if c["p"] else None
        mo.embed_grad(c["dout_t"], c["tokens_t"], c["grad_t"], c["ws"], scale=c["scale"], padding_idx=c["padding_idx"],
                      accumulate=c["accumulate"], dropout=drop)
        return c["grad_t"]
    if op == "dropout":
        mo.dropout_apply(c["x_t"], c["out_t"], mo.Dropout(c["p"], c["seed"]), residual=c["residual_t"])
        return c["out_t"]
    if op == "quantize":
        rnd = mo.Random(c["seed"]) if c["stochastic"] else None
        row, col = c["q"]
        mo.fp4_quantize(c["x_t"], row, col, stochastic=rnd)
        mo.fp4_dequantize(row, c["row_t"])
        mo.fp4_dequantize(col, c["col_t"])
        return {"row": c["row_t"], "col": c["col_t"]}
    if op == "product":
        mo.fp4_product(*c["q"], c["out_t"])
        return c["out_t"]
    x, xt, w, wt, dy, dyt = c["q"]
    mo.fp4_quantize(c["x_t"], x, xt)
    mo.fp4_quantize(c["w_t"], w, wt)
    mo.fp4_quantize(c["dy_t"], dy, dyt, stochastic=mo.Random(c["seed"]))
    mo.fp4_product(x, w, c["y_t"])
    mo.fp4_product(dy, wt, c["dx_t"])
    mo.fp4_product(dyt, xt, c["dw_t"])
    return {"y": c["y_t"], "dx": c["dx_t"], "dw": c["dw_t"]}


# ------------------------------------------------------------------ plain form

def _philox16(groups, seed, offset):
    """Philox4x32-10 (Salmon et al., 2011) for counters 0..groups-1: eight 16-bit numbers each."""
    m32 = 0xFFFFFFFF
    j = torch.arange(groups, dtype=torch.int64, device="cuda")
    a, b, c, d = j & m32, j >> 32, torch.full_like(j, offset & m32), torch.full_like(j, (offset >> 32) & m32)
    k0, k1 = seed & m32, (seed >> 32) & m32
    for _ in range(10):   # the generator's rounds
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((q >> 32) & m32) ^ b ^ k0, q & m32, ((p >> 32) & m32) ^ d ^ k1, p & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return torch.stack([a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16], 1).reshape(-1)


def _keep(n, p, seed):
    """(mask, factor): an element is kept where its 16-bit number is at least round(65536 p)."""
    t = round(65536 * p)
    return _philox16(-(-n // 8), seed, 0)[:n] >= t, 65536.0 / (65536 - t)


def _block_view(x, block):
    rows, k = x.shape
    pad = -k % block
    return (torch.nn.functional.pad(x, (0, pad)) if pad else x).reshape(rows, -1, block)


def _pow2(e):
    """2^e in 32 bits for whole -127 <= e <= 127, from its bit pattern (2^-127 is subnormal)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _tensor_scale(amax):
    """The smallest power of two g with amax <= 6 * 448 g; 1 for a tensor of zeros."""
    m, e = torch.frexp(amax)      # m in [0.5, 1); 2688 = 0.65625 * 2^12
    g = _pow2(torch.where(m <= 0.65625, e - 12, e - 11).clamp(min=-126))
    return torch.where(amax > 0, g, torch.ones_like(g))


def _e4m3_values(like):
    i = torch.arange(127, device=like.device)
    e, f = i >> 3, (i & 7).float()
    return torch.where(e == 0, f / 512, (1 + f / 8) * _pow2(e - 7))


def _quantize(x, fmt, seed, offset, amax):
    """(values, scale of each block, codes, bits of the scales) of x, blocks along its rows. Each
    block's scale is the smallest of its type with which no element exceeds 6."""
    v = _block_view(x, BLOCK[fmt])
    top = v.abs().amax(2)
    if fmt == "mx":
        m, e = torch.frexp(top)      # 6 = 0.75 * 2^3
        e = torch.where(top > 0, torch.where(m <= 0.75, e - 3, e - 2), torch.full_like(e, -127)).clamp(min=-127)
        bits, s = (e + 127).to(torch.uint8), _pow2(e)
    else:
        g = _tensor_scale(amax)
        levels = _e4m3_values(x)
        i = torch.searchsorted(6 * levels, top / g).clamp(max=126)
        bits, s = i.to(torch.uint8), levels[i] * g
    y = torch.where(s[..., None] > 0, v.abs() / s[..., None], torch.zeros_like(v)).clamp(max=MAX_CODE)
    if seed is None:   # to the nearest, ties to the even code
        code = (y > 0.25).to(torch.int32) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5)
    else:              # up with the probability of the remainder, from 16-bit numbers
        rows, k = x.shape
        kp = -(-k // 32) * 32
        u = _philox16(rows * kp // 8, seed, offset).reshape(rows, kp)[:, :v.shape[1] * v.shape[2]].reshape(v.shape)
        f = (y * 131072).to(torch.int64)
        code = torch.where(y < 2, (f + u) >> 16, torch.where(y < 4, ((f + 2 * u) >> 17) + 2, ((f + 4 * u) >> 18) + 4))
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    mag = levels[code.long()] * s[..., None]
    rows, k = x.shape
    value = torch.where(v < 0, -mag, mag).reshape(rows, -1)[:, :k]
    code = (code + 8 * (v < 0)).to(torch.uint8).reshape(rows, -1)[:, :k]
    return value, s, code, bits


def _fake(x, fmt, seed=None, offset=0):
    """x in 32 bits as its 4-bit form stands for it."""
    return _quantize(x, fmt, seed, offset, x.abs().amax().reshape(1) if fmt == "nv" else None)[0]


def _unpacked(t):
    """The values of a packed 4-bit tensor, in 32 bits."""
    rows, k, fmt = t["rows"], t["k"], t["format"]
    c = torch.stack([t["codes"] & 15, t["codes"] >> 4], 2).reshape(rows, -1)
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=c.device)
    nb = -(-k // BLOCK[fmt])
    s = t["scales"].reshape(-(-rows // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)[:rows, :nb]
    if fmt == "mx":
        s = _pow2(s.to(torch.int32) - 127)
    else:
        s = _e4m3_values(c)[s.long()] * _tensor_scale(t["amax"])
    return (levels[c.long()][:, :k].contiguous() * s.repeat_interleave(BLOCK[fmt], 1)[:, :k])


def _run_plain(c):
    op = c["op"]
    if op == "lookup":
        v = c["table_t"][c["tokens_t"]].float() * c["scale"]
        if c["add_t"] is not None:
            v = v + c["add_t"].float()[torch.arange(c["n"], device="cuda") % c["positions"]]
        if c["p"]:
            keep, f = _keep(v.numel(), c["p"], c["seed"])
            v = torch.where(keep.reshape(v.shape), v * f, torch.zeros_like(v))
        c["out_t"].copy_(v)
        return c["out_t"]
    if op == "grad":
        d = c["dout_t"].float()
        if c["p"]:
            keep, f = _keep(d.numel(), c["p"], c["seed"])
            d = torch.where(keep.reshape(d.shape), d * f, torch.zeros_like(d))
        d = d * c["scale"]
        if c["padding_idx"] >= 0:
            d = torch.where((c["tokens_t"] == c["padding_idx"])[:, None], torch.zeros_like(d), d)
        if not c["accumulate"]:
            c["grad_t"].zero_()
        c["grad_t"].index_add_(0, c["tokens_t"], d)
        return c["grad_t"]
    if op == "dropout":
        keep, f = _keep(c["n"], c["p"], c["seed"])
        x = c["x_t"].float()
        v = torch.where(keep, x * f, torch.zeros_like(x))
        c["out_t"].copy_(v + c["residual_t"].float() if c["residual"] else v)
        return c["out_t"]
    if op == "quantize":
        seed = c["seed"] if c["stochastic"] else None
        x = c["x_t"].float()
        c["row_t"].copy_(_fake(x, c["format"], seed, 0))
        c["col_t"].copy_(_fake(x.T.contiguous(), c["format"], seed, 1))
        return {"row": c["row_t"], "col": c["col_t"]}
    if op == "product":
        c["out_t"].copy_(_unpacked(c["a_t"]) @ _unpacked(c["b_t"]).T)
        return c["out_t"]
    f, x, w, dy = c["format"], c["x_t"].float(), c["w_t"], c["dy_t"].float()
    c["y_t"].copy_(_fake(x, f) @ _fake(w, f).T)
    c["dx_t"].copy_(_fake(dy, f, c["seed"], 0) @ _fake(w.T.contiguous(), f).T)
    c["dw_t"].copy_(_fake(dy.T.contiguous(), f, c["seed"], 1) @ _fake(x.T.contiguous(), f).T)
    return {"y": c["y_t"], "dx": c["dx_t"], "dw": c["dw_t"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ bytes and operations

def _fp4_bytes(rows, k, fmt):
    return rows * k * (0.5 + 1.0 / BLOCK[fmt])


def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op in ("lookup", "grad"):
        # a row is read (written) once however many tokens name it: the expected number of distinct tokens
        share = _token_shares(case["vocab"])
        n = case["n"] * (1 - case.get("padding", 0.0))
        rows = float((1 - np.exp(n * np.log1p(-share))).sum())
        if op == "lookup":
            b = rows * case["dim"] * size[case["table"]] + case["n"] * (case["dim"] * size[case["out"]] + 8)
            b += min(case["positions"], case["n"]) * case["dim"] * size[case["table"]]
            return {"bytes": b, "flops": 2.0 * case["n"] * case["dim"]}
        written = rows * 2 if case["accumulate"] else case["vocab"]
        return {"bytes": n * case["dim"] * size[case["dout"]] + case["n"] * 8 + written * case["dim"] * 4,
                "flops": 2.0 * n * case["dim"]}
    if op == "dropout":
        return {"bytes": case["n"] * size[case["dtype"]] * (3 if case["residual"] else 2), "flops": 2.0 * case["n"]}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        # the input, then codes and scales and the values they stand for, in both orientations
        return {"bytes": n * (size[case["dtype"]] + 2 * 2) + 2 * _fp4_bytes(case["rows"], case["cols"], case["format"]),
                "flops": 4.0 * n}
    if op == "product":
        m, n, k, f = case["m"], case["n"], case["k"], case["format"]
        return {"bytes": _fp4_bytes(m, k, f) + _fp4_bytes(n, k, f) + 2 * m * n, "flops": 2.0 * m * n * k}
    t, r, k, f = case["tokens"], case["rows"], case["cols"], case["format"]
    # x, w, dy in, y, dx, dw out; each 4-bit operand is written by its quantisation and read by its product
    b = 2 * t * k + 4 * r * k + 2 * t * r + 2 * t * r + 2 * t * k + 2 * r * k
    b += 4 * (_fp4_bytes(t, k, f) + _fp4_bytes(r, k, f) + _fp4_bytes(t, r, f))
    return {"bytes": b, "flops": 6.0 * t * r * k}


# ------------------------------------------------------------------ 64 bits

def _mulhilo16(a, const):
    """High and low words of a 32 x 32-bit product, from 16-bit limbs."""
    a0, a1, c0, c1 = a % 65536, a // 65536, const % 65536, const // 65536
    mid = a1 * c0 + (a0 * c0) // 65536
    mid2 = a0 * c1 + mid % 65536
    return a1 * c1 + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (a0 * c0) % 65536


def _exact_random(index, seed, offset):
    """The 16-bit number of each element index."""
    block, lane = torch.div(index, 8, rounding_mode="floor"), index % 8
    x = [block % 2**32, torch.div(block, 2**32, rounding_mode="floor"), torch.full_like(block, offset % 2**32),
         torch.full_like(block, offset // 2**32)]
    for r in range(10):
        k0, k1 = (seed % 2**32 + r * 0x9E3779B9) % 2**32, (seed // 2**32 + r * 0xBB67AE85) % 2**32
        h0, l0 = _mulhilo16(x[0], 0xD2511F53)
        h1, l1 = _mulhilo16(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
    word = torch.where(lane < 4, torch.where(lane < 2, x[0], x[1]), torch.where(lane < 6, x[2], x[3]))
    return torch.where(lane % 2 == 0, word % 65536, torch.div(word, 65536, rounding_mode="floor"))


def _exact_drop(v, p, seed):
    """Dropout of v in 64 bits, a slice at a time."""
    t = round(65536 * p)
    out, flat, part = torch.empty_like(v).reshape(-1), v.reshape(-1), 1 << 24
    for at in range(0, flat.numel(), part):
        x = flat[at:at + part]
        u = _exact_random(torch.arange(at, at + x.numel(), device="cuda"), seed, 0)
        out[at:at + part] = torch.where(u < t, torch.zeros_like(x), x / (1 - t / 65536))
    return out.reshape(v.shape)


def _exact_scales(fmt):
    """The value of each scale's bits, in increasing order."""
    if fmt == "mx":
        return torch.from_numpy(np.ldexp(1.0, np.arange(-127, 128)))
    i = np.arange(127)
    return torch.from_numpy(np.where(i < 8, i / 512.0, np.ldexp(8.0 + i % 8, i // 8 - 10)))


def _exact_values(x, fmt, seed=None, offset=0):
    """The values that the 4-bit form of x (64 bits) stands for, blocks along its rows."""
    rows, k = x.shape
    block = BLOCK[fmt]
    out = torch.zeros_like(x)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    if fmt == "nv":
        top = float(x.abs().max())
        g = 2.0 ** math.ceil(math.log2(top / 2688)) if top > 0 else 1.0
        while g * 2688 < top:
            g *= 2
        while g * 1344 >= top > 0:
            g /= 2
        scales = _exact_scales(fmt).to(x.device) * g
    else:
        scales = _exact_scales(fmt).to(x.device)
    step = max(1, (1 << 23) // max(1, k))
    kp = -(-k // 32) * 32
    for r in range(0, rows, step):
        part = torch.zeros((min(step, rows - r), kp), dtype=torch.float64, device=x.device)
        part[:, :k] = x[r:r + step]
        v = part.reshape(part.shape[0], -1, block)
        top = v.abs().amax(2, keepdim=True)
        s = scales[torch.searchsorted(scales, top / 6).clamp(max=scales.numel() - 1)]
        y = torch.where(s > 0, v.abs() / s, torch.zeros_like(v)).clamp(max=6.0)
        hi = torch.searchsorted(grid, y).clamp(max=7)           # grid[lo] <= y <= grid[hi]
        lo = torch.where(grid[hi] > y, hi - 1, hi).clamp(min=0)
        gap = grid[(lo + 1).clamp(max=7)] - grid[lo]
        part_up = torch.where(gap > 0, (y - grid[lo]) / gap, torch.zeros_like(y))
        if seed is None:
            up = (part_up > 0.5) | ((part_up == 0.5) & (lo % 2 == 1))
        else:
            at = torch.arange(r, r + part.shape[0], device=x.device)[:, None] * kp + torch.arange(kp, device=x.device)
            u = _exact_random(at, seed, offset).reshape(v.shape)
            fixed = torch.where(y < 2, torch.floor((y - grid[lo]) * 131072),
                                torch.where(y < 4, torch.floor((y - grid[lo]) * 131072) / 2, torch.floor((y - grid[lo]) * 131072) / 4))
            up = fixed + u >= 65536
        q = grid[torch.where(up, lo + 1, lo).clamp(max=7)] * s
        out[r:r + step] = torch.where(v < 0, -q, q).reshape(part.shape)[:, :k]
    return out


def _exact_unpacked(t):
    rows, k, fmt = t["rows"], t["k"], t["format"]
    r = torch.arange(rows, device="cuda")[:, None]
    e = torch.arange(k, device="cuda")[None]
    byte = t["codes"].long()[r, e // 2]
    code = torch.where(e % 2 == 0, byte % 16, byte // 16)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.where(code >= 8, -grid[code % 8], grid[code % 8])
    nb = -(-k // BLOCK[fmt])
    b = torch.arange(nb, device="cuda")[None]
    at = ((r // 128) * (-(-nb // 4)) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    s = t["scales"].long()[at]
    s = _exact_scales(fmt).to(s.device)[s]
    if fmt == "nv":
        top = float(t["amax"])
        g = 1.0
        while g * 2688 < top:
            g *= 2
        while g * 1344 >= top > 0:
            g /= 2
        s = s * g
    return v * s[:, torch.arange(k, device="cuda") // BLOCK[fmt]]


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "lookup":
        v = c["table_t"].double()[c["tokens_t"]] * c["scale"]
        if c["positions"]:
            v += c["add_t"].double()[torch.arange(c["n"], device="cuda") % c["positions"]]
        return _exact_drop(v, c["p"], c["seed"]) if c["p"] else v
    if op == "grad":
        d = c["dout_t"].double()
        d = (_exact_drop(d, c["p"], c["seed"]) if c["p"] else d) * c["scale"]
        live = c["tokens_t"] != c["padding_idx"]
        out = c["grad_t"].double() if c["accumulate"] else torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device="cuda")
        return out.index_put_((c["tokens_t"][live],), d[live], accumulate=True)
    if op == "dropout":
        v = _exact_drop(c["x_t"].double(), c["p"], c["seed"])
        return v + c["residual_t"].double() if c["residual"] else v
    if op == "quantize":
        seed = c["seed"] if c["stochastic"] else None
        x = c["x_t"].double()
        return {"row": _exact_values(x, c["format"], seed, 0), "col": _exact_values(x.T.contiguous(), c["format"], seed, 1)}
    if op == "product":
        return _exact_unpacked(c["a_t"]) @ _exact_unpacked(c["b_t"]).T
    f, x, w, dy = c["format"], c["x_t"].double(), c["w_t"].double(), c["dy_t"].double()
    y = _exact_values(x, f) @ _exact_values(w, f).T
    dx = _exact_values(dy, f, c["seed"], 0) @ _exact_values(w.T.contiguous(), f).T
    dw = _exact_values(dy.T.contiguous(), f, c["seed"], 1) @ _exact_values(x.T.contiguous(), f).T
    return {"y": y, "dx": dx, "dw": dw}
