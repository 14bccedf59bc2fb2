"""Microscaled 4-bit quantisation and product on the GPU against the float64
oracle.

Quantisation is an exact function of its input (mx; nv from bf16 input, whose
quotients lie no nearer than 2^-16 to a rounding boundary unless exactly on
it), so codes and scale bytes have to be equal. A stochastic nv code may differ
where the fp32 rounding of the quotient moves its 2^-17 fixed-point digit:
at most 1 element in 2^10 is allowed.

Product: the products of codes are exact; each of the K additions in fp32 is
off by at most 2^-23 of the terms' magnitudes so far (truncation counted),
then one rounding to the output's type."""
import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from gpu_util import f64
from oracle import train_ops as ot

pytestmark = pytest.mark.gpu
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def dev():
    return torch.device("cuda")


def data(rows, cols, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(1.5 * torch.randn((rows, 1), generator=g))
    return (x * std).to(dtype).to(dev())


def storage(rows, k, fmt, fill=0xA5):
    q = mo.Fp4Tensor(rows, k, fmt)
    q.codes.fill_(fill)      # whatever was there before
    q.scales.fill_(fill)
    return q


def check_storage(q, x, fmt, stochastic=None, amax=None):
    codes, bits, values = ot.fp4_quantize(x, fmt, stochastic, amax)
    want_c, want_s = ot.fp4_pack(codes, bits, fmt)
    got_c, got_s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(got_s, want_s)
    nan = np.isnan(values)
    if stochastic is not None and fmt == "nv":
        assert np.mean(got_c != want_c) <= 2.0 ** -9   # two elements a byte
    elif not nan.any():
        assert np.array_equal(got_c, want_c)
    return values


SHAPES = [(1, 1), (1, 32), (3, 33), (128, 128), (130, 257), (127, 64), (64, 1000), (257, 40), (300, 16), (31, 4096)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_both_orientations(fmt, dtype, rows, cols):
    x = data(rows, cols, dtype, rows * 7 + cols)
    if fmt == "nv" and dtype == torch.float32:
        x = x.bfloat16().float()
    row, col = storage(rows, cols, fmt), storage(cols, rows, fmt)
    mo.fp4_quantize(x, row, col)
    values = check_storage(row, f64(x), fmt)
    check_storage(col, f64(x).T, fmt)
    if fmt == "nv":
        assert float(row.amax) == float(col.amax) == float(x.float().abs().max())
    for odt in (torch.float32, torch.bfloat16):
        out = torch.full((rows, cols), 3.0, dtype=odt, device=dev())
        mo.fp4_dequantize(row, out)
        assert np.array_equal(f64(out), values)
    # one orientation alone is the same
    alone = storage(rows, cols, fmt, 0x5A)
    mo.fp4_quantize(x, alone)
    assert torch.equal(alone.codes, row.codes) and torch.equal(alone.scales, row.scales)
    alone = storage(cols, rows, fmt, 0x5A)
    mo.fp4_quantize(x, None, alone)
    assert torch.equal(alone.codes, col.codes) and torch.equal(alone.scales, col.scales)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 7), (130, 257), (64, 100), (256, 512)])
def test_quantize_stochastic(fmt, dtype, rows, cols):
    x = data(rows, cols, dtype, rows + cols, 1e-3)
    row, col = storage(rows, cols, fmt), storage(cols, rows, fmt)
    seed, offset = 2 ** 60 + 5, 2 ** 35 + 1
    mo.fp4_quantize(x, row, col, stochastic=mo.Random(seed, offset))
    check_storage(row, f64(x), fmt, (seed, offset))
    check_storage(col, f64(x).T, fmt, (seed, offset + 1))
    again = storage(rows, cols, fmt, 1)
    off = torch.tensor([offset], dtype=torch.int64, device=dev())
    mo.fp4_quantize(x, again, stochastic=mo.Random(seed, 0, off))
    assert torch.equal(again.codes, row.codes)


def test_quantize_ties_and_signs():
    x = torch.zeros((2, 32), device=dev())
    x[0, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    for fmt in ("mx", "nv"):
        q = storage(2, 32, fmt)
        # nv: amax 2688 makes g = 1, and the block's scale 1
        mo.fp4_quantize(x, q, amax=torch.tensor([2688.0], device=dev()) if fmt == "nv" else None)
        out = torch.empty((2, 32), device=dev())
        mo.fp4_dequantize(q, out)
        pos = [6, 0, 1, 1, 2, 2, 4, 4]
        assert out[0, :16].tolist() == pos + [-v for v in pos]
        assert not out[1].any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_zeros_extremes_and_bad_values(fmt):
    rows, cols = 140, 96
    x = torch.zeros((rows, cols), device=dev())
    x[1] = 1e-42                               # subnormal
    x[2] = 2.0 ** 100
    x[3, 5], x[4, 40], x[5, 95] = float("nan"), float("inf"), -float("inf")
    x[6] = 1.0
    row, col = storage(rows, cols, fmt), storage(cols, rows, fmt)
    mo.fp4_quantize(x, row, col)
    v = check_storage(row, f64(x), fmt)
    check_storage(col, f64(x).T, fmt)
    out = torch.empty((rows, cols), device=dev())
    mo.fp4_dequantize(row, out)
    assert np.array_equal(f64(out), v, equal_nan=True)
    B = ot.FP4_BLOCK[fmt]
    assert np.isnan(f64(out)).sum() == 3 * B


def test_quantize_caller_amax_too_small_saturates():
    x = torch.full((1, 32), -1e6, device=dev())
    x[0, 1], x[0, 20:] = 3e38, 5.0
    q = storage(1, 32, "nv")
    mo.fp4_quantize(x, q, amax=torch.tensor([2688.0], device=dev()))
    out = torch.empty((1, 32), device=dev())
    mo.fp4_dequantize(q, out)
    assert out[0, 0] == -2688 and out[0, 1] == 2688


def test_quantize_caller_amax():
    x = data(70, 90, torch.bfloat16, 3)
    amax = torch.tensor([1000.0], device=dev())
    q = storage(70, 90, "nv")
    mo.fp4_quantize(x, q, amax=amax)
    check_storage(q, f64(x), "nv", amax=1000.0)
    assert float(q.amax) == 1000.0


# ---------------------------------------------------------------- product

def packed(x, fmt, seed):
    codes, bits, values = ot.fp4_quantize(x, fmt)
    c, s = ot.fp4_pack(codes, bits, fmt)
    amax = torch.tensor([np.abs(x).max()], dtype=torch.float32, device=dev())
    q = mo.Fp4Tensor(x.shape[0], x.shape[1], fmt, codes=torch.from_numpy(c).to(dev()), scales=torch.from_numpy(s).to(dev()),
                     amax=amax if fmt == "nv" else None)
    return q, torch.from_numpy(values).to(dev())


def operand(rows, k, fmt, seed):
    return packed(f64(data(rows, k, torch.bfloat16, seed)), fmt, seed)


def check_product(q, v, out):
    ref = v[0] @ v[1].T
    mag = v[0].abs() @ v[1].abs().T
    k = v[0].shape[1]
    err = (out.double() - ref).abs()
    bound = k * 2.0 ** -23 * mag + ROUND[out.dtype] * ref.abs() * 1.01
    assert bool((err <= bound).all()), f"worst excess {(err - bound).max().item():.3e} of {mag.max().item():.3e}"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 128, 64), (1, 300, 4096), (5, 77, 33), (16, 128, 256), (17, 129, 1000), (33, 260, 96), (64, 5, 64),
    (100, 1000, 512), (128, 64, 2048), (129, 100, 160),            # few rows, or few tiles
    (300, 5120, 64), (257, 5128, 96), (260, 5001, 1000), (2051, 2600, 320),   # pairs: whole, 16-byte, odd rows; several tiles
])
def test_product(fmt, odt, m, n, k):
    a, va = operand(m, k, fmt, m + k)
    b, vb = operand(n, k, fmt, n + k + 1)
    out = torch.full((m, n), 9.0, dtype=odt, device=dev())
    mo.fp4_product(a, b, out)
    assert mo.mo_last_device_error() == 0
    check_product((a, b), (va, vb), out)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,n,k", [(2048, 8192, 1280), (1000, 7000, 4000), (5000, 2500, 2304)])
def test_product_many_tiles_and_stages(fmt, m, n, k):
    # every CTA pair takes several tiles of many stages: all rings go round
    a, b = mo.Fp4Tensor(m, k, fmt), mo.Fp4Tensor(n, k, fmt)
    mo.fp4_quantize(data(m, k, torch.bfloat16, 1), a)
    mo.fp4_quantize(data(n, k, torch.bfloat16, 2), b)
    va, vb = torch.empty((m, k), device=dev()), torch.empty((n, k), device=dev())
    mo.fp4_dequantize(a, va)
    mo.fp4_dequantize(b, vb)
    for odt in (torch.float32, torch.bfloat16):
        out = torch.full((m, n), 9.0, dtype=odt, device=dev())
        mo.fp4_product(a, b, out)
        assert mo.mo_last_device_error() == 0
        check_product((a, b), (va.double(), vb.double()), out)


@pytest.mark.parametrize("m,n,k", [(40, 200, 2048), (300, 5120, 512)])
def test_product_repeats_bit_for_bit_and_on_a_side_stream(m, n, k):
    a, _ = operand(m, k, "nv", 1)
    b, _ = operand(n, k, "nv", 2)
    outs = [torch.zeros((m, n), device=dev()) for _ in range(4)]
    for o in outs[:3]:
        mo.fp4_product(a, b, o)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    mo.fp4_product(a, b, outs[3], stream=s)
    s.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("m,n", [(20, 200), (300, 5120)])
def test_product_keeps_bad_values_to_their_rows_and_columns(m, n):
    k = 256
    x = f64(data(m, k, torch.bfloat16, 1))
    w = f64(data(n, k, torch.bfloat16, 2))
    x[7, 100], w[50, 3] = np.nan, np.inf
    for fmt in ("mx", "nv"):
        cx, bx, _ = ot.fp4_quantize(x, fmt)
        cw, bw, _ = ot.fp4_quantize(w, fmt)
        qs = []
        for c, b_ in ((cx, bx), (cw, bw)):
            p, s = ot.fp4_pack(c, b_, fmt)
            qs.append(mo.Fp4Tensor(c.shape[0], k, fmt, codes=torch.from_numpy(p).to(dev()), scales=torch.from_numpy(s).to(dev())))
        out = torch.zeros((m, n), device=dev())
        mo.fp4_product(*qs, out)
        bad = torch.isnan(out)
        want = torch.zeros((m, n), dtype=torch.bool, device=dev())
        want[7], want[:, 50] = True, True
        assert torch.equal(bad, want)


def test_product_of_nothing_is_zero():
    a, b = mo.Fp4Tensor(5, 0, "mx"), mo.Fp4Tensor(7, 0, "mx")
    out = torch.full((5, 7), 2.0, device=dev())
    mo.fp4_product(a, b, out)
    assert not out.any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_layer_gradients_against_the_formula(fmt):
    # y = x w^T; dx = dy w; dw = dy^T x, each of its own 4-bit operands
    t, r, c = 200, 160, 288
    x, w, dy = data(t, c, torch.bfloat16, 1), data(r, c, torch.float32, 2, 0.05).bfloat16().float(), data(t, r, torch.bfloat16, 3, 1e-3)
    q = {n: storage(*s, fmt) for n, s in dict(x=(t, c), xt=(c, t), w=(r, c), wt=(c, r), dy=(t, r), dyt=(r, t)).items()}
    mo.fp4_quantize(x, q["x"], q["xt"])
    mo.fp4_quantize(w, q["w"], q["wt"])
    mo.fp4_quantize(dy, q["dy"], q["dyt"])
    val = {}
    for n, t_ in q.items():
        val[n] = torch.empty((t_.rows, t_.k), device=dev())
        mo.fp4_dequantize(t_, val[n])
        val[n] = val[n].double()
    for a, b in (("x", "w"), ("dy", "wt"), ("dyt", "xt")):
        for odt in (torch.float32, torch.bfloat16):
            out = torch.empty((q[a].rows, q[b].rows), dtype=odt, device=dev())
            mo.fp4_product(q[a], q[b], out)
            check_product((q[a], q[b]), (val[a], val[b]), out)


def test_input_gradient_against_differences():
    # x moves by whole code steps that keep its scales: the output's difference is the products' with the gradient
    k, n = 64, 48
    x = torch.zeros((1, k), device=dev())
    x[0, 0], x[0, 32] = 6.0, 6.0
    w = data(n, k, torch.bfloat16, 5)
    step = torch.zeros_like(x)
    step[0, 1:32], step[0, 33:] = 1.0, -2.0
    qx, qx2, qw, qwt = storage(1, k, "mx"), storage(1, k, "mx"), storage(n, k, "mx"), storage(k, n, "mx")
    mo.fp4_quantize(w, qw)
    values = torch.empty((n, k), device=dev())
    mo.fp4_dequantize(qw, values)
    y, y2 = torch.empty((1, n), device=dev()), torch.empty((1, n), device=dev())
    mo.fp4_quantize(x, qx)
    mo.fp4_quantize(x + step, qx2)
    mo.fp4_product(qx, qw, y)
    mo.fp4_product(qx2, qw, y2)
    want = step.double() @ values.double().T      # <step, dx> for dy = each unit vector
    mag = (x.abs() + step.abs()).double() @ values.double().abs().T
    assert bool(((y2.double() - y.double() - want).abs() <= 2 * k * 2.0 ** -23 * mag).all())


# ---------------------------------------------------------------- past 32 bits, graphs

def test_quantize_past_32_bit_elements():
    rows, cols = 2 ** 20 + 3, 4160              # 4.4 G elements
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev())
    spots = torch.tensor([0, 2 ** 19 + 1, 2 ** 20 - 200, rows - 1], device=dev())
    x[spots] = data(len(spots), cols, torch.bfloat16, 1)
    row, col = mo.Fp4Tensor(rows, cols, "mx"), mo.Fp4Tensor(cols, rows, "mx")
    mo.fp4_quantize(x, row, col)
    _, _, values = ot.fp4_quantize(f64(x[spots]), "mx")
    del x
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev())
    mo.fp4_dequantize(row, out)
    assert np.array_equal(f64(out[spots]), values)
    out[spots] = 0
    assert not any(bool(part.any()) for part in out.split(2 ** 16))


@pytest.mark.parametrize("n", [40000, 39999])
def test_product_past_32_bit_outputs(n):
    m, k = 120000, 64                            # 4.8 G outputs
    a, b = mo.Fp4Tensor(m, k, "mx"), mo.Fp4Tensor(n, k, "mx")
    mo.fp4_quantize(data(m, k, torch.bfloat16, 1), a)
    mo.fp4_quantize(data(n, k, torch.bfloat16, 2), b)
    va, vb = torch.empty((m, k), device=dev()), torch.empty((n, k), device=dev())
    mo.fp4_dequantize(a, va)
    mo.fp4_dequantize(b, vb)
    out = torch.empty((m, n), dtype=torch.bfloat16, device=dev())
    mo.fp4_product(a, b, out)
    assert mo.mo_last_device_error() == 0
    for r0 in (0, 53500, 53687, 107374, m - 300):   # around 2^31 and 2^32 outputs
        part = slice(r0, r0 + 300)
        check_product((a, b), (va[part].double(), vb.double()), out[part])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_captured_in_a_graph(fmt):
    t, r, c = 300, 5120, 288
    x, w = data(t, c, torch.bfloat16, 1), data(r, c, torch.float32, 2)
    xq, xt, wq = mo.Fp4Tensor(t, c, fmt), mo.Fp4Tensor(c, t, fmt), mo.Fp4Tensor(r, c, fmt)
    y, off = torch.empty((t, r), device=dev()), torch.zeros(1, dtype=torch.int64, device=dev())

    def step():
        mo.fp4_quantize(w, wq)
        mo.fp4_quantize(x, xq, xt, stochastic=mo.Random(3, 4, off))
        mo.fp4_product(xq, wq, y)
        off.add_(2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(data(t, c, torch.bfloat16, 7))
    off.fill_(40)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone(), xt.codes.clone()
    off.fill_(42)
    step()
    assert torch.equal(y, got[0]) and torch.equal(xt.codes, got[1])


@pytest.mark.parametrize("m,n,k", [(33, 131, 100), (300, 5113, 96)])
def test_nothing_outside_the_outputs_is_written(m, n, k):
    guard = 4096
    def guarded(count, dtype, value):
        whole = torch.full((count + 2 * guard,), value, dtype=dtype, device=dev())
        return whole, whole[guard:guard + count], value
    x, w = data(m, k, torch.float32, 1), data(n, k, torch.float32, 2)
    sizes = [(m, k), (k, m), (n, k)]
    keep, q = [], []
    for r, kk in sizes:
        c = guarded(mo.mo_fp4_codes_bytes(r, kk), torch.uint8, 0x5C)
        s = guarded(mo.mo_fp4_scales_bytes(r, kk, "nv"), torch.uint8, 0x5C)
        keep += [c, s]
        q.append(mo.Fp4Tensor(r, kk, "nv", codes=c[1], scales=s[1]))
    mo.fp4_quantize(x, q[0], q[1])
    mo.fp4_quantize(w, q[2])
    for dtype in (torch.float32, torch.bfloat16):
        y = guarded(m * n, dtype, 77.0)
        v = guarded(k * m, dtype, 77.0)
        keep += [y, v]
        mo.fp4_product(q[0], q[2], y[1].view(m, n))
        mo.fp4_dequantize(q[1], v[1].view(k, m))
    for whole, part, value in keep:
        assert bool((whole[:guard] == value).all()) and bool((whole[guard + part.numel():] == value).all())


@pytest.mark.parametrize("m,n,k", [(20, 200, 512), (100, 260, 6208), (300, 5120, 320)])   # few rows, split K, pairs
@pytest.mark.parametrize("sa,sb", [(90, 90), (115, 20), (30, 70), (-75, -75), (-75, -100), (-126, 110), (117, -126), (40, -30)])
def test_product_at_the_ends_of_the_tensor_scales(m, n, k, sa, sb):
    # the tensors' scales 2^sa and 2^sb; their product need not be a float where the result is one
    rng = np.random.default_rng(1000 + m + sa)
    qs, vs = [], []
    for rows, e, zero in ((m, sa, 3), (n, sb, 5)):
        v = rng.uniform(0.25, 1, size=(rows, k)) * 2688
        v[zero] = 0                              # a row of zeros stays 0
        v[zero + 1] *= 2.0 ** -12                # small sums
        v[0, 0] = 2688
        codes, bits, values = ot.fp4_quantize(v, "nv")
        c, s = ot.fp4_pack(codes, bits, "nv")
        amax = torch.tensor([min(2688 * 2.0 ** e, torch.finfo(torch.float32).max)], device=dev())
        qs.append(mo.Fp4Tensor(rows, k, "nv", codes=torch.from_numpy(c).to(dev()), scales=torch.from_numpy(s).to(dev()), amax=amax))
        vs.append(torch.from_numpy(values).to(dev()))
    sums = vs[0] @ vs[1].T
    for odt in (torch.float32, torch.bfloat16):
        out = torch.full((m, n), 9.0, dtype=odt, device=dev())
        mo.fp4_product(*qs, out)
        assert mo.mo_last_device_error() == 0
        assert not out[3].any() and not out[:, 5].any()
        # the roundings: k 2^-23 of the sum, one to the type, and its smallest step where the result is subnormal
        rel = k * 2.0 ** -23 + 1.01 * ROUND[odt]
        step = 2.0 ** (-149 if odt == torch.float32 else -133)
        most = torch.finfo(odt).max
        exact = sums * 2.0 ** sa * 2.0 ** sb
        lo, hi = exact * (1 - rel) - step, exact * (1 + rel) + step
        got = out.double()
        assert bool(((got >= lo) | (got == most)).all()) and bool(((got <= hi) | (hi >= most)).all())
        assert bool(torch.isinf(got)[lo > 1.01 * most].all()) and bool(torch.isfinite(got)[hi < most].all())
        if odt == torch.float32 and sa + sb == -150:
            assert bool((exact > 2.0 ** -126).any())   # results of full precision


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_product_of_many_tiles_repeats_bit_for_bit(fmt):
    # scales and accumulators change hands between the two CTAs of a pair in every stage and tile
    m, n, k = 2048, 8192, 1280
    a, b = mo.Fp4Tensor(m, k, fmt), mo.Fp4Tensor(n, k, fmt)
    mo.fp4_quantize(data(m, k, torch.bfloat16, 1), a)
    mo.fp4_quantize(data(n, k, torch.bfloat16, 2), b)
    first, out = torch.empty((m, n), device=dev()), torch.empty((m, n), device=dev())
    mo.fp4_product(a, b, first)
    for _ in range(30):
        out.fill_(float("nan"))
        mo.fp4_product(a, b, out)
        assert torch.equal(out, first)
    assert mo.mo_last_device_error() == 0


@pytest.mark.parametrize("rows,cols", [(1, 33), (130, 257), (257, 40), (64, 1000)])
def test_quantize_nv_of_full_mantissas(rows, cols):
    # fp32 weights. The quotient is rounded once to fp32: a value next to a tie differs from it by at least
    # 1 / 1.875 of the quotient's last place (the scale's mantissa is at most 1.875), so it is not rounded onto it
    x = data(rows, cols, torch.float32, rows + 3 * cols, 0.02)
    row, col = storage(rows, cols, "nv"), storage(cols, rows, "nv")
    mo.fp4_quantize(x, row, col)
    check_storage(row, f64(x), "nv")
    check_storage(col, f64(x).T, "nv")


@pytest.mark.parametrize("e", [0, 40, 116, -30, -101, -126])   # of the tensor's scale
def test_quantize_nv_beside_every_tie_of_every_scale(e):
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5])
    scales = ot.fp4_scale_values("nv")[1:]
    x = np.zeros((len(scales), 48), np.float32)
    for i, t in enumerate((ties * 2.0 ** e)[:, None] * scales[None, :]):
        t = t.astype(np.float32)
        for j, v in enumerate((np.nextafter(t, np.float32(0)), t, np.nextafter(t, np.float32(np.inf)))):
            x[:, 16 * j + 1 + i] = v
            x[:, 16 * j + 9 + i] = -v            # (columns 9 to 15)
    x[:, ::16] = (6 * scales * 2.0 ** e).astype(np.float32)[:, None]   # fixes the block's scale
    amax = 2688 * 2.0 ** e
    q = storage(*x.shape, "nv")
    mo.fp4_quantize(torch.from_numpy(x).to(dev()), q, amax=torch.tensor([amax], device=dev()))
    check_storage(q, x.astype(np.float64), "nv", amax=amax)
