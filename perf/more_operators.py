"""Workloads of the feed-forward half of a transformer layer: root-mean-square
norm with the residual's addition and an 8-bit output, matrix products with
bias, activation and residual in their epilogue, the gated feed-forward block,
and the 8-bit activation checkpoints that their backward passes read.

`run` computes a case either with the library's operators (`own` true) or in
plain form: elementary torch operations in 32 bits, rounded once at the end.
`exact` gives the same outputs from the definitions in 64 bits.

8-bit tensors: e4m3 codes [rows, 32 ceil(k / 32)] and for each block of 32
elements of a row the exponent + 127 of its scale, the smallest power of two
with which no element exceeds 448. They are returned as the values they stand
for, which bf16 holds exactly.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token between two layers of the Llama-style 8B table, where latency is all
        {"name": "norm one token", "op": "norm", "rows": 1, "dim": 4096, "dtype": "bf16", "residual": True, "out": "bf16", "mx8": False},
        # a training batch: the residual stream's sum, and the normalised values in 8 bits alone, both the
        # feed-forward block's input and its checkpoint
        {"name": "norm 8B batch", "op": "norm", "rows": 16384, "dim": 4096, "dtype": "bf16", "residual": True, "out": "", "mx8": True},
        # its backward pass from an 8-bit checkpoint of the sum, with the gradient that passes the block by
        {"name": "norm grad 8B batch", "op": "norm_grad", "rows": 16384, "dim": 4096, "dtype": "bf16", "mx8": True, "residual": True,
         "accumulate": False},
        # a feed-forward activation of GPT-2 Large put into 8 bits and taken out again
        {"name": "checkpoint GPT-2 batch", "op": "checkpoint", "rows": 8192, "cols": 5120, "dtype": "bf16"},
        # a small odd tensor
        {"name": "checkpoint odd", "op": "checkpoint", "rows": 1023, "cols": 1283, "dtype": "f32"},
        # one token through a GPT-2 Large feed-forward weight
        {"name": "linear one token", "op": "linear", "tokens": 1, "cols": 1280, "rows": 5120, "bias": True, "act": "gelu_tanh",
         "residual": False, "x": "bf16", "pre": "", "out": "bf16"},
        # eight 1024-token sequences through the same, with the pre-activation kept in 8 bits
        {"name": "linear GPT-2 batch", "op": "linear", "tokens": 8192, "cols": 1280, "rows": 5120, "bias": True, "act": "gelu_tanh",
         "residual": False, "x": "bf16", "pre": "mx8", "out": "bf16"},
        # their backward pass from 8-bit checkpoints of the input and the pre-activation
        {"name": "linear grad GPT-2 batch", "op": "linear_grad", "tokens": 8192, "cols": 1280, "rows": 5120, "bias": True,
         "act": "gelu_tanh", "x": "mx8", "pre": "mx8", "accumulate": False},
        # odd everything, added to a residual in fp32
        {"name": "linear odd residual", "op": "linear", "tokens": 777, "cols": 1003, "rows": 515, "bias": False, "act": "",
         "residual": True, "x": "bf16", "pre": "", "out": "f32"},
        # one token through the gated block of the 8B table: 352 MB of weights
        {"name": "ffn one token", "op": "ffn", "tokens": 1, "dim": 4096, "inner": 14336, "act": "silu", "residual": True, "x": "bf16",
         "save": ""},
        # a batch forward, from the norm's 8-bit output, with 8-bit checkpoints
        {"name": "ffn 8B batch", "op": "ffn", "tokens": 8192, "dim": 4096, "inner": 14336, "act": "silu", "residual": True, "x": "mx8",
         "save": "mx8"},
        # forward and backward, all gradients
        {"name": "ffn 8B step", "op": "ffn_step", "tokens": 4096, "dim": 4096, "inner": 14336, "act": "silu", "residual": True,
         "x": "mx8", "save": "mx8"},
    ]


def draw(rng):
    def between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):   # most widths are multiples of 8 to 64, some are odd
        w = between(lo, hi)
        step = rng.choice([1, 8, 32, 64])
        return max(step, w // step * step)

    op = rng.choice(["norm", "norm_grad", "checkpoint", "linear", "linear_grad", "ffn", "ffn_step"])
    if op == "norm":
        mx8 = rng.choice([False, True])
        return {"op": op, "rows": between(1, 16384), "dim": width(16, 8192), "dtype": rng.choice(["f32", "bf16"]),
                "residual": rng.choice([False, True]), "out": rng.choice(["f32", "bf16", ""] if mx8 else ["f32", "bf16"]), "mx8": mx8}
    if op == "norm_grad":
        return {"op": op, "rows": between(1, 16384), "dim": width(16, 8192), "dtype": rng.choice(["f32", "bf16"]),
                "mx8": rng.choice([False, True]), "residual": rng.choice([False, True]), "accumulate": rng.choice([False, True])}
    if op == "checkpoint":
        return {"op": op, "rows": between(1, 16384), "cols": width(16, 5120), "dtype": rng.choice(["f32", "bf16"])}
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
    kind = rng.choice(["bf16", "mx8"])
    if op == "linear":
        act = rng.choice(["", act])
        return {"op": op, "tokens": between(1, 8192), "cols": width(32, 5120), "rows": width(32, 5120), "bias": rng.choice([False, True]),
                "act": act, "residual": rng.choice([False, True]), "x": kind, "pre": rng.choice(["", "bf16", "mx8"]) if act else "",
                "out": rng.choice(["f32", "bf16"])}
    if op == "linear_grad":
        act = rng.choice(["", act])
        return {"op": op, "tokens": between(1, 8192), "cols": width(32, 5120), "rows": width(32, 5120), "bias": rng.choice([False, True]),
                "act": act, "x": kind, "pre": rng.choice(["bf16", "mx8"]) if act else "", "accumulate": rng.choice([False, True])}
    if op == "ffn":
        return {"op": op, "tokens": between(1, 8192), "dim": width(32, 4096), "inner": width(64, 14336), "act": act,
                "residual": rng.choice([False, True]), "x": kind, "save": rng.choice(["", "bf16", "mx8"])}
    return {"op": op, "tokens": between(1, 4096), "dim": width(32, 4096), "inner": width(64, 14336), "act": act,
            "residual": rng.choice([False, True]), "x": kind, "save": rng.choice(["bf16", "mx8"])}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DTYPES[dtype])


def _stream(g, rows, dim, dtype="bf16", std=1.0):
    """Values whose rows and columns differ in size, as those of a residual stream and of gradients do."""
    x = torch.randn((rows, dim), generator=g, device="cuda")
    x *= torch.exp(torch.randn((rows, 1), generator=g, device="cuda") * 0.5)
    x *= torch.exp(torch.randn((1, dim), generator=g, device="cuda") * 0.5)
    return (x * std).to(DTYPES[dtype])


def _normed(g, rows, dim):
    """Values as a norm leaves them: rows of one size, columns that differ."""
    x = torch.randn((rows, dim), generator=g, device="cuda") * torch.exp(torch.randn((1, dim), generator=g, device="cuda") * 0.5)
    return (x / x.square().mean(1, keepdim=True).sqrt()).to(torch.bfloat16)


def _storage(rows, k):
    nb = -(-k // 32)
    return {"codes": torch.zeros((rows, 32 * nb), dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros((rows, nb), dtype=torch.uint8, device="cuda"), "k": k}


def _packed(x):
    """An 8-bit tensor as a program keeps it."""
    t = _storage(*x.shape)
    code, bits = _mx8(x.float())
    t["codes"].copy_(code)
    t["scales"].copy_(bits)
    return t


def _kept(x, kind):
    return _packed(x) if kind == "mx8" else x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = c["op"]
    if op == "norm":
        n, d = c["rows"], c["dim"]
        c["x_t"] = _stream(g, n, d, c["dtype"])
        c["residual_t"] = _stream(g, n, d, c["dtype"]) if c["residual"] else None
        c["weight_t"] = _normal(g, (d,), std=0.3) + 1
        c["sum_t"] = torch.empty_like(c["x_t"]) if c["residual"] else None
        c["out_t"] = torch.empty((n, d), dtype=DTYPES[c["out"]], device="cuda") if c["out"] else None
        c["out8_t"] = _storage(n, d) if c["mx8"] else None
        c["back_t"] = torch.empty((n, d), dtype=torch.bfloat16, device="cuda") if c["mx8"] else None
    elif op == "norm_grad":
        n, d = c["rows"], c["dim"]
        c["x_t"] = _kept(_stream(g, n, d, c["dtype"]), "mx8" if c["mx8"] else "")
        c["dy_t"] = _stream(g, n, d, c["dtype"], 1e-3)
        c["dres_t"] = _stream(g, n, d, c["dtype"], 1e-3) if c["residual"] else None
        c["weight_t"] = _normal(g, (d,), std=0.3) + 1
        c["dx_t"] = torch.empty_like(c["dy_t"])
        c["dweight0_t"] = _normal(g, (d,), std=1e-2)   # the gradient so far, where it is added to
        c["dweight_t"] = torch.empty_like(c["dweight0_t"])
    elif op == "checkpoint":
        c["x_t"] = _stream(g, c["rows"], c["cols"], c["dtype"])
        c["q_t"] = _storage(c["rows"], c["cols"])
        c["back_t"] = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device="cuda")
    elif op in ("linear", "linear_grad"):
        t, k, n = c["tokens"], c["cols"], c["rows"]
        c["x_t"] = _kept(_normed(g, t, k), c["x"])
        c["w_t"] = _normal(g, (n, k), "bf16", 1 / math.sqrt(k))
        c["bias_t"] = _normal(g, (n,), std=0.1) if c["bias"] else None
        if op == "linear":
            c["residual_t"] = _stream(g, t, n, c["out"]) if c["residual"] else None
            c["pre_t"] = {"": lambda: None, "bf16": lambda: torch.empty((t, n), dtype=torch.bfloat16, device="cuda"),
                          "mx8": lambda: _storage(t, n)}[c["pre"]]()
            c["back_t"] = torch.empty((t, n), dtype=torch.bfloat16, device="cuda") if c["pre"] == "mx8" else None
            c["out_t"] = torch.empty((t, n), dtype=DTYPES[c["out"]], device="cuda")
        else:
            c["dout_t"] = _stream(g, t, n, "bf16", 1e-3)
            c["pre_t"] = _kept(_normal(g, (t, n), "bf16", 1.2), c["pre"]) if c["pre"] else None
            c["dx_t"] = torch.empty((t, k), dtype=torch.bfloat16, device="cuda")
            c["dw0_t"] = _normal(g, (n, k), "bf16", 1e-2)
            c["db0_t"] = _normal(g, (n,), std=1e-2)
            c["dw_t"], c["db_t"] = torch.empty_like(c["dw0_t"]), torch.empty_like(c["db0_t"]) if c["bias"] else None
    else:
        t, d, f = c["tokens"], c["dim"], c["inner"]
        c["x_t"] = _kept(_normed(g, t, d), c["x"])
        c["gate_w"] = _normal(g, (f, d), "bf16", 1.2 / math.sqrt(d))
        c["up_w"] = _normal(g, (f, d), "bf16", 1.2 / math.sqrt(d))
        c["down_w"] = _normal(g, (d, f), "bf16", 1 / math.sqrt(f))
        c["residual_t"] = _stream(g, t, d) if c["residual"] else None
        keep = {"": lambda: None, "bf16": lambda: torch.empty((t, f), dtype=torch.bfloat16, device="cuda"),
                "mx8": lambda: _storage(t, f)}[c["save"]]
        c["gate_t"], c["up_t"] = keep(), keep()
        c["out_t"] = torch.empty((t, d), dtype=torch.bfloat16, device="cuda")
        if op == "ffn_step":
            c["dout_t"] = _stream(g, t, d, "bf16", 1e-3)
            c["dx_t"] = torch.empty((t, d), dtype=torch.bfloat16, device="cuda")
            for name in ("gate", "up", "down"):
                c["d" + name] = torch.empty_like(c[name + "_w"])
        elif c["save"] == "mx8":
            c["gate_back"], c["up_back"] = (torch.empty((t, f), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:   # what the library's users keep from step to step: workspaces and the handles of 8-bit tensors
        import matrix_optimizers_zero_gb300 as mo
        for name, v in list(c.items()):
            if isinstance(v, dict):
                c[name] = mo.Mx8Tensor(v["codes"].shape[0], v["k"], codes=v["codes"], scales=v["scales"])
        if op == "norm_grad":
            c["ws"] = mo.rms_norm_grad_workspace(c["rows"], c["dim"])
        elif op in ("linear", "linear_grad"):
            c["ws"] = mo.linear_workspace(c["tokens"], c["cols"], c["rows"], grad=op == "linear_grad")
        elif op in ("ffn", "ffn_step"):
            c["ws"] = mo.gated_ffn_workspace(c["tokens"], c["dim"], c["inner"], grad=op == "ffn_step")
    return c


# ------------------------------------------------------------------ the library's operators

def _run_own(c):
    import matrix_optimizers_zero_gb300 as mo
    op = c["op"]
    if op == "norm":
        mo.rms_norm(c["x_t"], c["out_t"], weight=c["weight_t"], eps=EPS, residual=c["residual_t"], sum_out=c["sum_t"], out8=c["out8_t"])
        if c["mx8"]:
            mo.mx8_dequantize(c["out8_t"], c["back_t"])
        return {"out": c["out_t"], "out8": c["back_t"], "sum": c["sum_t"]}
    if op == "norm_grad":
        if c["accumulate"]:
            c["dweight_t"].copy_(c["dweight0_t"])
        mo.rms_norm_grad(c["dy_t"], c["x_t"], c["dx_t"], weight=c["weight_t"], eps=EPS, dresidual=c["dres_t"], dweight=c["dweight_t"],
                         workspace=c["ws"], accumulate=c["accumulate"])
        return {"dx": c["dx_t"], "dweight": c["dweight_t"]}
    if op == "checkpoint":
        mo.mx8_quantize(c["x_t"], c["q_t"])
        mo.mx8_dequantize(c["q_t"], c["back_t"])
        return c["back_t"]
    act = c["act"] or None
    if op == "linear":
        mo.linear(c["x_t"], c["w_t"], c["out_t"], bias=c["bias_t"], activation=act, residual=c["residual_t"], pre=c["pre_t"],
                  workspace=c["ws"])
        if c["pre"] == "mx8":
            mo.mx8_dequantize(c["pre_t"], c["back_t"])
        return {"out": c["out_t"], "pre": c["back_t"] if c["pre"] == "mx8" else c["pre_t"]}
    if op == "linear_grad":
        if c["accumulate"]:
            c["dw_t"].copy_(c["dw0_t"])
            if c["bias"]:
                c["db_t"].copy_(c["db0_t"])
        mo.linear_grad(c["dout_t"], c["x_t"], c["w_t"], dx=c["dx_t"], dw=c["dw_t"], dbias=c["db_t"], activation=act, pre=c["pre_t"],
                       workspace=c["ws"], accumulate=c["accumulate"])
        return {"dx": c["dx_t"], "dw": c["dw_t"], "dbias": c["db_t"]}
    mo.gated_ffn(c["x_t"], c["gate_w"], c["up_w"], c["down_w"], c["out_t"], activation=act, residual=c["residual_t"], gate=c["gate_t"],
                 up=c["up_t"], workspace=c["ws"])
    if op == "ffn":
        if c["save"] == "mx8":
            mo.mx8_dequantize(c["gate_t"], c["gate_back"])
            mo.mx8_dequantize(c["up_t"], c["up_back"])
            return {"out": c["out_t"], "gate": c["gate_back"], "up": c["up_back"]}
        return {"out": c["out_t"], "gate": c["gate_t"], "up": c["up_t"]}
    mo.gated_ffn_grad(c["dout_t"], c["x_t"], c["gate_t"], c["up_t"], c["gate_w"], c["up_w"], c["down_w"], activation=act, dx=c["dx_t"],
                      dw_gate=c["dgate"], dw_up=c["dup"], dw_down=c["ddown"], workspace=c["ws"])
    return {"out": c["out_t"], "dx": c["dx_t"], "dgate": c["dgate"], "dup": c["dup"], "ddown": c["ddown"]}


# ------------------------------------------------------------------ plain form

def _pow2(e):
    """2^e in 32 bits for whole -126 <= e <= 127, from its bit pattern."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _mx8(x):
    """(codes, bits of the scales) of x, rows padded with zeros to whole blocks of 32."""
    rows, k = x.shape
    v = torch.nn.functional.pad(x, (0, -k % 32)).reshape(rows, -1, 32)
    top = v.abs().amax(2)
    m, e = torch.frexp(top)      # 448 = 0.875 * 2^9
    e = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.full_like(e, -127)).clamp(min=-127)
    code = (v * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return code.reshape(rows, -1), (e + 127).to(torch.uint8)


def _values(t, x=None):
    """What an 8-bit tensor stands for, in 32 bits; a plain tensor as it is."""
    if not isinstance(t, dict):
        return t.float()
    v = t["codes"].view(torch.float8_e4m3fn).float().reshape(t["codes"].shape[0], -1, 32)
    e = t["scales"].to(torch.int32) - 127
    half = torch.div(e, 2, rounding_mode="floor")   # in two steps: 2^-127 is no normal number
    v = v * _pow2(half)[..., None] * _pow2(e - half)[..., None]
    return v.reshape(v.shape[0], -1)[:, :t["k"]]


def _put(t, x):
    """x kept in t, in 8 bits or in t's own type; the values that are kept."""
    if isinstance(t, dict):
        code, bits = _mx8(x)
        t["codes"].copy_(code)
        t["scales"].copy_(bits)
    else:
        t.copy_(x)
    return _values(t)


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-a * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(c):
    op = c["op"]
    if op == "norm":
        s = c["x_t"].float()
        if c["residual"]:
            s = s + c["residual_t"].float()
            c["sum_t"].copy_(s)
        y = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * c["weight_t"]
        if c["out"]:
            c["out_t"].copy_(y)
        if c["mx8"]:
            c["back_t"].copy_(_put(c["out8_t"], y))
        return {"out": c["out_t"], "out8": c["back_t"], "sum": c["sum_t"]}
    if op == "norm_grad":
        s, dy = _values(c["x_t"]), c["dy_t"].float()
        r = 1 / torch.sqrt(s.square().mean(1, keepdim=True) + EPS)
        n = s * r
        g = dy * c["weight_t"]
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        c["dx_t"].copy_(dx + c["dres_t"].float() if c["residual"] else dx)
        dw = (dy * n).sum(0)
        c["dweight_t"].copy_(dw + c["dweight0_t"] if c["accumulate"] else dw)
        return {"dx": c["dx_t"], "dweight": c["dweight_t"]}
    if op == "checkpoint":
        c["back_t"].copy_(_put(c["q_t"], c["x_t"].float()))
        return c["back_t"]
    x = _values(c["x_t"])
    if op == "linear":
        z = x @ c["w_t"].float().T
        if c["bias"]:
            z = z + c["bias_t"]
        if c["pre"]:
            kept = _put(c["pre_t"], z)
            if c["pre"] == "mx8":
                c["back_t"].copy_(kept)
        y = _act(z, c["act"])
        c["out_t"].copy_(y + c["residual_t"].float() if c["residual"] else y)
        return {"out": c["out_t"], "pre": c["back_t"] if c["pre"] == "mx8" else c["pre_t"]}
    if op == "linear_grad":
        dz = c["dout_t"].float()
        if c["act"]:
            dz = dz * _act_slope(_values(c["pre_t"]), c["act"])
        c["dx_t"].copy_(dz @ c["w_t"].float())
        dw = dz.T @ x
        c["dw_t"].copy_(dw + c["dw0_t"].float() if c["accumulate"] else dw)
        if c["bias"]:
            c["db_t"].copy_(dz.sum(0) + c["db0_t"] if c["accumulate"] else dz.sum(0))
        return {"dx": c["dx_t"], "dw": c["dw_t"], "dbias": c["db_t"]}
    wg, wu, wd = c["gate_w"].float(), c["up_w"].float(), c["down_w"].float()
    gate, up = x @ wg.T, x @ wu.T
    y = (_act(gate, c["act"]) * up) @ wd.T
    c["out_t"].copy_(y + c["residual_t"].float() if c["residual"] else y)
    if c["save"]:
        gate, up = _put(c["gate_t"], gate), _put(c["up_t"], up)
    if op == "ffn":
        if c["save"] == "mx8":
            c["gate_back"].copy_(gate)
            c["up_back"].copy_(up)
            return {"out": c["out_t"], "gate": c["gate_back"], "up": c["up_back"]}
        return {"out": c["out_t"], "gate": c["gate_t"], "up": c["up_t"]}
    dy = c["dout_t"].float()
    dh = dy @ wd
    a = _act(gate, c["act"])
    dgate, dup = dh * up * _act_slope(gate, c["act"]), dh * a
    c["ddown"].copy_(dy.T @ (a * up))
    c["dgate"].copy_(dgate.T @ x)
    c["dup"].copy_(dup.T @ x)
    c["dx_t"].copy_(dgate @ wg + dup @ wu)
    return {"out": c["out_t"], "dx": c["dx_t"], "dgate": c["dgate"], "dup": c["dup"], "ddown": c["ddown"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    size = {"f32": 4, "bf16": 2, "mx8": 33 / 32, "": 0}
    c, op = case, case["op"]
    if op == "norm":
        n = c["rows"] * c["dim"]
        # the values that an 8-bit output stands for are written too (and read from it)
        b = size[c["dtype"]] * (3 if c["residual"] else 1) + size[c["out"]] + ((size["mx8"] + 2) if c["mx8"] else 0)
        return {"bytes": n * b + 4 * c["dim"], "flops": 6.0 * n}
    if op == "norm_grad":
        n = c["rows"] * c["dim"]
        b = size[c["dtype"]] * (3 if c["residual"] else 2) + (size["mx8"] if c["mx8"] else size[c["dtype"]])
        return {"bytes": n * b + 4 * c["dim"] * (3 if c["accumulate"] else 2), "flops": 12.0 * n}
    if op == "checkpoint":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (size[c["dtype"]] + size["mx8"] + 2), "flops": 3.0 * n}
    if op == "linear":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        b = t * k * size[c["x"]] + 2 * n * k + 4 * n * c["bias"]
        b += t * n * (size[c["out"]] * (2 if c["residual"] else 1) + size[c["pre"]] + (2 if c["pre"] == "mx8" else 0))
        return {"bytes": b, "flops": 2.0 * t * k * n}
    if op == "linear_grad":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        b = t * n * (2 + size[c["pre"]]) + t * k * (size[c["x"]] + 2) + 2 * n * k * (3 if c["accumulate"] else 2)
        return {"bytes": b + 4 * n * c["bias"] * (2 if c["accumulate"] else 1), "flops": 4.0 * t * k * n}
    t, d, f = c["tokens"], c["dim"], c["inner"]
    b = t * d * (size[c["x"]] + 2 * (2 if c["residual"] else 1)) + 6 * d * f + 2 * t * f * size[c["save"]]
    if op == "ffn":
        return {"bytes": b + (2 * t * f * 2 if c["save"] == "mx8" else 0), "flops": 6.0 * t * d * f}
    # the backward pass: dout, the checkpoints, the input and the weights again; dx and three gradients
    b += t * d * (2 + size[c["x"]] + 2) + 2 * t * f * size[c["save"]] + 12 * d * f
    return {"bytes": b, "flops": 18.0 * t * d * f}


# ------------------------------------------------------------------ 64 bits

def _exact_kept(x):
    """The values that the 8-bit form of x (64 bits) stands for."""
    rows, k = x.shape
    out = torch.empty_like(x)
    part = max(1, (1 << 25) // max(1, k))
    for r in range(0, rows, part):
        v = x[r:r + part]
        whole = torch.zeros((v.shape[0], -(-k // 32) * 32), dtype=torch.float64, device=x.device)
        whole[:, :k] = v
        blocks = whole.view(v.shape[0], -1, 32)
        top = blocks.abs().amax(2, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top / 448, torch.full_like(top, 2.0 ** -127))))
        e = torch.where(448 * torch.exp2(e) < top, e + 1, e)             # where the logarithm was rounded
        e = torch.where((448 * torch.exp2(e - 1) >= top), e - 1, e).clamp(min=-127)
        s = torch.exp2(e)
        y = blocks.abs() / s
        at = torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))
        at = torch.where(torch.exp2(at) > y.clamp(min=2.0 ** -6), at - 1, at)
        step = torch.exp2(at.clamp(min=-6.0) - 3)                         # of e4m3 around y
        q = torch.round(y / step) * step * s                              # ties to the even multiple
        out[r:r + part] = torch.where(blocks < 0, -q, q).reshape(v.shape[0], -1)[:, :k]
    return out


def _exact_values(t):
    if not isinstance(t, dict):
        return t.double()
    code = t["codes"].to(torch.int64)[:, :t["k"]]
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(8 + m, e - 10))
    v = torch.where(code >= 128, -v, v)
    s = torch.exp2(t["scales"].double() - 127)
    return v * s.repeat_interleave(32, 1)[:, :t["k"]]


def _exact_act(z, name):
    """(value, slope) of an activation."""
    if name == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(z / 2 ** 0.5))
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if name == "gelu_tanh":
        b = (2 / math.pi) ** 0.5
        t = torch.tanh(b * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * b * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def exact(case, seed):
    global own
    was, own = own, False
    c = prepare(case, seed)
    own = was
    op = c["op"]
    if op == "norm":
        s = c["x_t"].double()
        if c["residual"]:
            s += c["residual_t"].double()
        y = s * torch.rsqrt((s * s).sum(1, keepdim=True) / s.shape[1] + EPS) * c["weight_t"].double()
        return {"out": y if c["out"] else None, "out8": _exact_kept(y) if c["mx8"] else None, "sum": s if c["residual"] else None}
    if op == "norm_grad":
        s, dy = _exact_values(c["x_t"]), c["dy_t"].double()
        d = s.shape[1]
        r = torch.rsqrt((s * s).sum(1, keepdim=True) / d + EPS)
        g = dy * c["weight_t"].double()
        dx = r * g - s * (r ** 3 * (g * s).sum(1, keepdim=True) / d)
        dw = torch.einsum("td,td->d", dy, s * r)
        return {"dx": dx + c["dres_t"].double() if c["residual"] else dx, "dweight": dw + c["dweight0_t"].double() if c["accumulate"] else dw}
    if op == "checkpoint":
        return _exact_kept(c["x_t"].double())
    x = _exact_values(c["x_t"])
    if op == "linear":
        z = torch.einsum("tk,nk->tn", x, c["w_t"].double())
        if c["bias"]:
            z += c["bias_t"].double()
        y = _exact_act(z, c["act"])[0]
        return {"out": y + c["residual_t"].double() if c["residual"] else y,
                "pre": {"": lambda: None, "bf16": lambda: z, "mx8": lambda: _exact_kept(z)}[c["pre"]]()}
    if op == "linear_grad":
        dz = c["dout_t"].double()
        if c["act"]:
            dz = dz * _exact_act(_exact_values(c["pre_t"]), c["act"])[1]
        dw, db = torch.einsum("tn,tk->nk", dz, x), dz.sum(0)
        if c["accumulate"]:
            dw, db = dw + c["dw0_t"].double(), db + c["db0_t"].double()
        return {"dx": torch.einsum("tn,nk->tk", dz, c["w_t"].double()), "dw": dw, "dbias": db if c["bias"] else None}
    wg, wu, wd = c["gate_w"].double(), c["up_w"].double(), c["down_w"].double()
    gate, up = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
    out = torch.einsum("tf,df->td", _exact_act(gate, c["act"])[0] * up, wd)
    if c["residual"]:
        out += c["residual_t"].double()
    if c["save"]:
        # bf16 checkpoints are rounded as torch rounds 64 bits to them
        gate, up = (_exact_kept(v) if c["save"] == "mx8" else v.to(torch.bfloat16).double() for v in (gate, up))
    if op == "ffn":
        return {"out": out, "gate": gate if c["save"] else None, "up": up if c["save"] else None}
    dy = c["dout_t"].double()
    a, slope = _exact_act(gate, c["act"])
    dh = torch.einsum("td,df->tf", dy, wd)
    dgate, dup = dh * up * slope, dh * a
    return {"out": out, "dx": torch.einsum("tf,fd->td", dgate, wg) + torch.einsum("tf,fd->td", dup, wu),
            "dgate": torch.einsum("tf,td->fd", dgate, x), "dup": torch.einsum("tf,td->fd", dup, x),
            "ddown": torch.einsum("td,tf->df", dy, a * up)}
