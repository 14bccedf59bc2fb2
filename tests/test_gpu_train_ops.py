"""Embedding lookup, its gradient and dropout on the GPU against the float64
oracle.

Bounds: every output is a short chain of fp32 operations, each off by at most
u = 2^-24 of its result, rounded at the end to the output's type (fp32: u,
bf16 with its 8 significant bits: 2^-8). Dropout: product and factor (2 u), the residual's sum (u).
Lookup: scale, sum, factor (4 u). Gradient: a sum of k terms in any order is
off by at most (k - 1) u of the terms' magnitudes, the factor and the scale
add 3 u, the sum so far u. Each bound is taken per element."""
import numpy as np
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from gpu_util import f64
from oracle import train_ops as ot

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = 2.0 ** -8


def dev():
    return torch.device("cuda")


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(dev())


def rounding(dtype):
    return BF16 if dtype == torch.bfloat16 else U


def check(got, ref, bound):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), f"worst excess {(err - bound).max():.3e}"


# ---------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 1023, 8192, 8193, 100003])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(dtype, n, residual, p):
    x = randn((n,), dtype, n)
    r = randn((n,), dtype, n + 1) if residual else None
    y = torch.full_like(x, 7.0)
    mo.dropout_apply(x, y, mo.Dropout(p, seed=2 ** 63 + n, offset=2 ** 33 + 5), residual=r)
    ref = ot.dropout(f64(x), p, 2 ** 63 + n, 2 ** 33 + 5, f64(r) if residual else None)
    mag = np.abs(ot.dropout(f64(x), p, 2 ** 63 + n, 2 ** 33 + 5)) + (np.abs(f64(r)) if residual else 0)
    check(y, ref, 4 * U * mag + rounding(dtype) * np.abs(ref) * 1.01)
    if not residual:   # the mask itself
        f = ot.dropout_factors((n,), p, 2 ** 63 + n, 2 ** 33 + 5)
        assert np.array_equal((f64(y) != 0), (f > 0) & (f64(x) != 0))


def test_dropout_in_place_device_offset_and_backward():
    n = 5000
    x, r = randn((n,), torch.float32, 1), randn((n,), torch.float32, 2)
    want = torch.empty_like(x)
    mo.dropout_apply(x, want, mo.Dropout(0.25, seed=9, offset=12), residual=r)
    off = torch.tensor([5], dtype=torch.int64, device=dev())
    got = x.clone()
    mo.dropout_apply(got, got, mo.Dropout(0.25, seed=9, offset=7, offset_dev=off), residual=r)
    assert torch.equal(got, want)
    got = r.clone()
    mo.dropout_apply(x, got, mo.Dropout(0.25, seed=9, offset=12), residual=got)
    assert torch.equal(got, want)
    # the backward pass is the same map: <drop(a), b> = <a, drop(b)>
    b = randn((n,), torch.float32, 3)
    da, db = torch.empty_like(x), torch.empty_like(x)
    d = mo.Dropout(0.25, seed=9, offset=12)
    mo.dropout_apply(x, da, d)
    mo.dropout_apply(b, db, d)
    lhs, rhs = (f64(da) * f64(b)).sum(), (f64(x) * f64(db)).sum()
    assert abs(lhs - rhs) <= 4 * U * np.abs(f64(da) * f64(b)).sum()


def test_dropout_drops_nan_and_inf():
    n = 4096
    x = torch.full((n,), float("nan"), device=dev())
    x[::2] = float("inf")
    y = torch.empty_like(x)
    mo.dropout_apply(x, y, mo.Dropout(0.5, seed=3))
    f = ot.dropout_factors((n,), 0.5, 3)
    got = f64(y)
    assert np.all(got[f == 0] == 0)
    assert np.all(np.isnan(got[(f > 0) & (np.arange(n) % 2 == 1)])) and np.all(np.isposinf(got[(f > 0) & (np.arange(n) % 2 == 0)]))


def test_dropout_captured_in_a_graph_with_an_advancing_offset():
    n = 3001
    x = randn((n,), torch.float32, 4)
    y = torch.empty_like(x)
    off = torch.zeros(1, dtype=torch.int64, device=dev())
    d = mo.Dropout(0.3, seed=21, offset=100, offset_dev=off)
    mo.dropout_apply(x, y, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mo.dropout_apply(x, y, d)
        off.add_(1)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        f = ot.dropout_factors((n,), 0.3, 21, 100 + k)
        assert np.array_equal(f64(y) != 0, f > 0)


# ---------------------------------------------------------------- lookup

@pytest.mark.parametrize("tdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (1, 300, 1280), (37, 50, 8), (100, 1000, 257), (13, 7, 4096),
                                         (300, 999, 24), (5, 40, 2056), (64, 33, 130)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_lookup(tdt, odt, n, vocab, dim, p):
    table = randn((vocab, dim), tdt, dim)
    add = randn((6, dim), tdt, dim + 1) if n % 2 else None
    tokens = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int64)
    tokens = (tokens if dim % 3 else tokens.to(torch.int32)).to(dev())
    out = torch.full((n, dim), 9.0, dtype=odt, device=dev())
    mo.embed_lookup(table, tokens, out, scale=1.7, add=add, dropout=mo.Dropout(p, seed=77, offset=1) if p else None)
    scale = float(np.float32(1.7))
    a = None if add is None else f64(add)
    dr = (p, 77, 1) if p else None
    ref = ot.embed_lookup(f64(table), tokens.cpu().numpy(), scale, a, dr)
    mag = ot.embed_lookup(np.abs(f64(table)), tokens.cpu().numpy(), scale, None if a is None else np.abs(a), dr)
    check(out, ref, 5 * U * mag + rounding(odt) * np.abs(ref) * 1.01)
    assert mo.mo_last_device_error() == 0


@pytest.mark.parametrize("dim", [8, 24, 64])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_lookup_many_narrow_rows(dim, p):
    n, vocab = 2 ** 21 + 3, 5001                # more tokens than threads that take them
    table = randn((vocab, dim), torch.float32, 1)
    tokens = torch.randint(0, vocab, (n,), device=dev(), generator=torch.Generator(dev()).manual_seed(2))
    out = torch.full((n, dim), float("nan"), device=dev())
    mo.embed_lookup(table, tokens, out, dropout=mo.Dropout(p, seed=3, offset=7) if p else None)
    if p == 0:
        assert torch.equal(out, table[tokens])
        return
    for a in (0, n // 2 - 500, n - 1000):
        keep = (ot.random16(1000 * dim, 3, 7, a * dim) >= round(65536 * p)).reshape(1000, dim)
        ref = f64(table[tokens[a:a + 1000]]) * keep * (65536 / (65536 - round(65536 * p)))
        check(out[a:a + 1000], ref, 4 * U * np.abs(ref))


@pytest.mark.parametrize("dim", [16, 19])
def test_lookup_outside_the_table_reads_zeros_and_reports(dim):
    table = randn((10, dim), torch.float32, 0)
    tokens = torch.tensor([3, -1, 9, 10, 2 ** 40], dtype=torch.int64, device=dev())
    out = torch.full((5, dim), 5.0, device=dev())
    mo.embed_lookup(table, tokens, out)
    assert mo.mo_last_device_error() == -11
    assert mo.mo_last_device_error() == 0
    assert torch.equal(out[0], table[3]) and torch.equal(out[2], table[9])
    assert not out[[1, 3, 4]].any()


# ---------------------------------------------------------------- gradient

def run_grad(dout, tokens, vocab, scale=1.0, padding_idx=-1, drop=None, so_far=None, stream=None):
    n, dim = dout.shape
    grad = so_far.clone() if so_far is not None else torch.full((vocab, dim), float("nan"), device=dev())
    ws = mo.embed_grad_workspace(n, vocab, dim)
    ws.fill_(0xFF)   # whatever was there before
    mo.embed_grad(dout, tokens, grad, ws, scale=scale, padding_idx=padding_idx, accumulate=so_far is not None,
                  dropout=mo.Dropout(*drop) if drop else None, stream=stream)
    return grad


def check_grad(grad, dout, tokens, vocab, scale, padding_idx, drop, so_far):
    tk = tokens.cpu().numpy()
    s = float(np.float32(scale))
    base = None if so_far is None else f64(so_far)
    ref = ot.embed_grad(f64(dout), tk, vocab, s, padding_idx, drop, base)
    mag = ot.embed_grad(np.abs(f64(dout)), tk, vocab, abs(s), padding_idx, drop, None if base is None else np.abs(base))
    counts = np.bincount(tk[(tk >= 0) & (tk < vocab)], minlength=vocab)[:, None]
    check(grad, ref, (counts + 4) * U * mag)


def make_tokens(n, vocab, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        t = torch.randint(0, vocab, (n,), generator=g)
    elif kind == "one":                      # every token the same row
        t = torch.full((n,), vocab - 1)
    elif kind == "hot":                      # two rows take most of the batch, runs end inside chunks
        t = torch.randint(0, vocab, (n,), generator=g)
        r = torch.rand(n, generator=g)
        t[r < 0.45] = 0
        t[r > 0.6] = vocab // 2
    else:                                    # each row at most once
        t = torch.randperm(max(n, vocab), generator=g)[:n] % vocab
    return t.to(dev())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["uniform", "one", "hot", "distinct"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (2, 600, 8), (63, 511, 40), (64, 512, 33), (65, 513, 264), (1000, 100, 16),
                                         (4097, 3000, 24), (2500, 70000, 9)])
def test_grad(dtype, kind, n, vocab, dim):
    dout = randn((n, dim), dtype, n + dim)
    tokens = make_tokens(n, vocab, kind, n)
    grad = run_grad(dout, tokens, vocab, scale=-0.75)
    check_grad(grad, dout, tokens, vocab, -0.75, -1, None, None)
    assert mo.mo_last_device_error() == 0


@pytest.mark.parametrize("dim", [16, 21])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("drop", [None, (0.3, 5, 9)])
def test_grad_padding_accumulate_dropout(dim, accumulate, drop):
    n, vocab = 3000, 257
    dout = randn((n, dim), torch.float32, 1)
    tokens = make_tokens(n, vocab, "hot", 3).to(torch.int32)
    so_far = randn((vocab, dim), torch.float32, 2) if accumulate else None
    grad = run_grad(dout, tokens, vocab, 2.0, 0, drop, so_far)
    check_grad(grad, dout, tokens, vocab, 2.0, 0, drop, so_far)
    if accumulate:
        assert torch.equal(grad[0], so_far[0])   # the padding row is left alone
    else:
        assert not grad[0].any()


def test_grad_all_padding_and_no_tokens():
    vocab, dim = 30, 12
    tokens = torch.full((100,), 4, device=dev())
    dout = torch.full((100, dim), float("nan"), device=dev())
    assert not run_grad(dout, tokens, vocab, padding_idx=4).any()
    empty = torch.empty((0, dim), device=dev())
    none = torch.empty((0,), dtype=torch.int64, device=dev())
    assert not run_grad(empty, none, vocab).any()
    base = randn((vocab, dim), torch.float32, 0)
    assert torch.equal(run_grad(empty, none, vocab, so_far=base), base)


def test_grad_many_joined_chunks_and_repeatability():
    # one row over 80 chunks of 64 and more: both levels of the join
    n, vocab, dim = 70000, 20, 8
    tokens = torch.zeros(n, dtype=torch.int64, device=dev())
    tokens[:100] = 7
    tokens[-3000:] = 19
    tokens[::4001] = 3
    dout = randn((n, dim), torch.float32, 8)
    a = run_grad(dout, tokens, vocab)
    check_grad(a, dout, tokens, vocab, 1.0, -1, None, None)
    for _ in range(3):
        assert torch.equal(run_grad(dout, tokens, vocab), a)


def test_grad_bad_tokens_are_reported_and_ignored():
    n, vocab, dim = 200, 50, 16
    tokens = make_tokens(n, vocab, "uniform", 0)
    tokens[5], tokens[17], tokens[60] = -3, vocab, 2 ** 35
    dout = randn((n, dim), torch.float32, 1)
    grad = run_grad(dout, tokens, vocab)
    assert mo.mo_last_device_error() == -11
    check_grad(grad, dout, tokens, vocab, 1.0, -1, None, None)


def test_grad_keeps_nan_to_its_row():
    n, vocab, dim = 500, 20, 16
    tokens = make_tokens(n, vocab, "uniform", 0)
    dout = randn((n, dim), torch.float32, 1)
    dout[123] = float("nan")
    grad = run_grad(dout, tokens, vocab)
    bad = int(tokens[123])
    assert torch.isnan(grad[bad]).all()
    assert not torch.isnan(grad[torch.arange(vocab, device=dev()) != bad]).any()


def test_grad_wide_vocabulary_takes_three_passes():
    n, vocab, dim = 3000, 300000, 8
    dout = randn((n, dim), torch.float32, 1)
    tokens = make_tokens(n, vocab, "uniform", 5)
    tokens[::7] = vocab - 1
    grad = run_grad(dout, tokens, vocab)
    tk = tokens.cpu().numpy()
    rows = np.unique(tk)
    remap = np.searchsorted(rows, tk)
    small = torch.from_numpy(rows).to(dev())
    check_grad(grad[small], dout, torch.from_numpy(remap).to(dev()), len(rows), 1.0, -1, None, None)
    untouched = torch.ones(vocab, dtype=torch.bool, device=dev())
    untouched[small] = False
    assert not grad[untouched].any()


@pytest.mark.parametrize("n,vocab,dim", [(3000, 70001, 401), (20000, 300007, 96), (5, 2 ** 25 + 3, 1), (9000, 2 ** 23 + 1, 5),
                                         (700, 40000, 1024)])
def test_grad_tables_whose_zeros_both_launches_write(n, vocab, dim):
    dout = randn((n, dim), torch.float32, 1)
    tokens = make_tokens(n, vocab, "uniform", 5)
    tokens[::3] = vocab - 1 - tokens[::3] % 50          # touched rows beside each other at the end
    tokens[:4] = torch.tensor([0, vocab - 1, vocab // 2, 1], device=dev())
    grad = run_grad(dout, tokens, vocab)
    rows, remap = torch.unique(tokens, return_inverse=True)
    check_grad(grad[rows], dout, remap, len(rows), 1.0, -1, None, None)
    grad[rows] = 0
    assert not grad.any()


@pytest.mark.parametrize("n,vocab,dim,row", [(20000, 50257, 64, 50256), (20000, 50257, 65, 40000), (60000, 128256, 16, 128000),
                                             (5000, 40000, 1024, 39999)])
def test_grad_frequent_token_among_the_rows_zeroed_last(n, vocab, dim, row):
    dout = randn((n, dim), torch.float32, 1)
    tokens = torch.full((n,), row, device=dev())
    tokens[7::1000] = row - 1
    tokens[5::1001] = row - 77
    grad = run_grad(dout, tokens, vocab)
    rows, remap = torch.unique(tokens, return_inverse=True)
    check_grad(grad[rows], dout, remap, len(rows), 1.0, -1, None, None)
    grad[rows] = 0
    assert not grad.any()


@pytest.mark.parametrize("n", [65535, 65536, 65537, 200003])
@pytest.mark.parametrize("vocab,dim,kind", [(300, 16, "uniform"), (50257, 9, "hot"), (300007, 8, "uniform"), (130000, 8, "one"),
                                            (2 ** 18, 64, "distinct")])
def test_grad_many_tokens(n, vocab, dim, kind):
    dout = randn((n, dim), torch.bfloat16, 1)
    tokens = make_tokens(n, vocab, kind, 5)
    tokens[11] = vocab - 1
    grad = run_grad(dout, tokens, vocab)
    assert torch.equal(run_grad(dout, tokens, vocab), grad)
    rows, remap = torch.unique(tokens, return_inverse=True)
    check_grad(grad[rows], dout, remap, len(rows), 1.0, -1, None, None)
    grad[rows] = 0
    assert not grad.any()


@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_many_tokens_padding_dropout_bad_tokens(accumulate):
    n, vocab, dim = 90001, 2003, 24
    dout = randn((n, dim), torch.float32, 1)
    tokens = make_tokens(n, vocab, "hot", 3).to(torch.int32)
    tokens[5], tokens[70000] = -3, vocab
    so_far = randn((vocab, dim), torch.float32, 2) if accumulate else None
    grad = run_grad(dout, tokens, vocab, 2.0, 0, (0.3, 5, 9), so_far)
    assert mo.mo_last_device_error() == -11
    check_grad(grad, dout, tokens, vocab, 2.0, 0, (0.3, 5, 9), so_far)


def test_grad_many_tokens_captured_in_a_graph():
    n, vocab, dim = 70000, 3001, 16
    dout, tokens = randn((n, dim), torch.bfloat16, 1), make_tokens(n, vocab, "uniform", 2)
    grad, ws = torch.empty((vocab, dim), device=dev()), mo.embed_grad_workspace(n, vocab, dim)
    mo.embed_grad(dout, tokens, grad, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mo.embed_grad(dout, tokens, grad, ws)
    for seed in (3, 4):
        tokens.copy_(make_tokens(n, vocab, "uniform", seed))
        grad.fill_(float("nan"))
        graph.replay()
        check_grad(grad, dout, tokens, vocab, 1.0, -1, None, None)


def test_grad_against_differences_of_the_lookup():
    # the lookup is linear in its table: <lookup(E + D) - lookup(E), dout> = <grad, D>
    n, vocab, dim = 400, 60, 48
    E, D = randn((vocab, dim), torch.float32, 1), randn((vocab, dim), torch.float32, 2)
    tokens = make_tokens(n, vocab, "hot", 1)
    dout = randn((n, dim), torch.float32, 3)
    d = mo.Dropout(0.2, seed=4, offset=6)
    outs = []
    for t in (E + D, E):
        o = torch.empty((n, dim), device=dev())
        mo.embed_lookup(t, tokens, o, scale=3.0, dropout=d)
        outs.append(f64(o))
    g = run_grad(dout, tokens, vocab, 3.0, -1, (0.2, 4, 6))
    lhs, rhs = ((outs[0] - outs[1]) * f64(dout)).sum(), (f64(g) * f64(D)).sum()
    scale = ((np.abs(outs[0]) + np.abs(outs[1])) * np.abs(f64(dout))).sum()
    assert abs(lhs - rhs) <= 40 * U * scale


def test_grad_on_a_side_stream():
    n, vocab, dim = 2000, 100, 64
    dout, tokens = randn((n, dim), torch.bfloat16, 1), make_tokens(n, vocab, "uniform", 2)
    want = run_grad(dout, tokens, vocab)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run_grad(dout, tokens, vocab)
    s.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- past 32 bits, graphs

def test_dropout_past_32_bit_elements():
    n = 2 ** 32 + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device=dev())
    mo.dropout_apply(x, x, mo.Dropout(0.5, seed=17, offset=3))
    for first in (0, 2 ** 31 - 16, 2 ** 32 - 8, n - 4000):
        part = x[first:first + 4000].float().cpu().numpy()
        u = ot.random16(len(part), 17, 3, first)
        assert np.array_equal(part != 0, u >= 32768)


def test_lookup_and_grad_past_32_bit_offsets():
    vocab, dim = 2 ** 20 + 77, 4096            # 4.3 G elements
    table = torch.zeros((vocab, dim), dtype=torch.bfloat16, device=dev())
    rows = torch.tensor([0, 2 ** 19 - 1, 2 ** 19, 2 ** 20 - 1, 2 ** 20, vocab - 1], device=dev())
    table[rows] = randn((len(rows), dim), torch.bfloat16, 1)
    out = torch.empty((len(rows), dim), dtype=torch.bfloat16, device=dev())
    mo.embed_lookup(table, rows, out)
    assert torch.equal(out, table[rows])
    del table
    tokens = rows.repeat(40)
    dout = randn((len(tokens), dim), torch.float32, 2)
    grad = run_grad(dout, tokens, vocab)       # 17 GB
    want = dout.double().reshape(40, len(rows), dim).sum(0)
    mag = dout.double().abs().reshape(40, len(rows), dim).sum(0)
    assert bool(((grad[rows].double() - want).abs() <= 43 * U * mag).all())
    grad[rows] = 0
    assert not any(bool(part.any()) for part in grad.split(2 ** 18))


def test_lookup_and_grad_captured_in_a_graph():
    n, vocab, dim = 3000, 700, 264
    table, dout = randn((vocab, dim), torch.float32, 1), randn((n, dim), torch.bfloat16, 2)
    tokens = make_tokens(n, vocab, "hot", 3)
    out, grad = torch.empty((n, dim), device=dev()), torch.empty((vocab, dim), device=dev())
    ws = mo.embed_grad_workspace(n, vocab, dim)
    d = mo.Dropout(0.2, seed=5)

    def step():
        mo.embed_lookup(table, tokens, out, dropout=d)
        mo.embed_grad(dout, tokens, grad, ws, dropout=d)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    tokens.copy_(make_tokens(n, vocab, "uniform", 9))
    graph.replay()
    torch.cuda.synchronize()
    got_out, got_grad = out.clone(), grad.clone()
    step()
    assert torch.equal(out, got_out) and torch.equal(grad, got_grad)


@pytest.mark.parametrize("dim", [24, 25])
def test_nothing_outside_the_outputs_is_written(dim):
    n, vocab, guard = 1500, 333, 4096
    def guarded(count, dtype):
        t = torch.full((count + 2 * guard,), 77.0, dtype=dtype, device=dev())
        return t, t[guard:guard + count]
    dout, table = randn((n, dim), torch.float32, 1), randn((vocab, dim), torch.float32, 2)
    tokens = make_tokens(n, vocab, "hot", 3)
    whole_g, grad = guarded(vocab * dim, torch.float32)
    whole_o, out = guarded(n * dim, torch.bfloat16)
    whole_y, y = guarded(n * dim, torch.float32)
    ws_bytes = mo.mo_embed_grad_workspace_bytes(n, vocab, dim)
    whole_w = torch.full((ws_bytes + 2 * guard,), 0x5C, dtype=torch.uint8, device=dev())
    drop = mo.Dropout(0.3, seed=1)
    mo.embed_grad(dout, tokens, grad.view(vocab, dim), whole_w[guard:guard + ws_bytes], dropout=drop)
    mo.embed_lookup(table, tokens, out.view(n, dim), dropout=drop)
    mo.dropout_apply(dout.view(-1), y, drop)
    for whole, count in ((whole_g, vocab * dim), (whole_o, n * dim), (whole_y, n * dim)):
        assert bool((whole[:guard] == 77).all()) and bool((whole[guard + count:] == 77).all())
    assert bool((whole_w[:guard] == 0x5C).all()) and bool((whole_w[guard + ws_bytes:] == 0x5C).all())


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("n", [2 ** 21, 2 ** 21 + 1, 3 * 2 ** 20 + 5])
def test_grad_past_2_to_21_tokens_leaves_other_rows_alone(n, accumulate):
    # from 2^21 tokens on the launch's blocks no longer fit one row of its grid
    vocab, dim, padding = 50257, 8, 4000
    g = torch.Generator(dev()).manual_seed(n)
    tokens = 4000 + 3 * torch.randint(0, 500, (n,), generator=g, device=dev())   # 499 rows, and the padding
    dout = torch.randn((n, dim), generator=g, device=dev())
    so_far = torch.randn((vocab, dim), generator=g, device=dev()) if accumulate else None
    grad = run_grad(dout, tokens, vocab, 0.5, padding, None, so_far)
    named = torch.unique(tokens)
    named = named[named != padding]
    base = so_far.double() if accumulate else torch.zeros((vocab, dim), dtype=torch.float64, device=dev())
    keep = tokens != padding
    ref = base.index_add(0, tokens[keep], 0.5 * dout[keep].double())
    mag = base.abs().index_add(0, tokens[keep], 0.5 * dout[keep].double().abs())
    count = torch.bincount(tokens, minlength=vocab)[:, None]
    assert bool(((grad.double() - ref).abs() <= (count + 4) * U * mag)[named].all())
    others = torch.ones(vocab, dtype=torch.bool, device=dev())
    others[named] = False
    assert torch.equal(grad[others], so_far[others] if accumulate else torch.zeros_like(grad[others]))


@pytest.mark.parametrize("timeout_first", [True, False])
@pytest.mark.parametrize("call", ["lookup", "lookup odd", "grad", "grad many"])
def test_a_bad_token_does_not_hide_an_expired_wait(call, timeout_first):
    dim, n = (9 if call == "lookup odd" else 8), (70000 if call == "grad many" else 40)
    tokens = torch.zeros(n, dtype=torch.int64, device=dev())
    tokens[3] = 10
    x = torch.zeros((n, dim), device=dev())

    def bad_token():
        if call.startswith("lookup"):
            mo.embed_lookup(torch.zeros((10, dim), device=dev()), tokens, x)
        else:
            run_grad(x, tokens, 10)
    assert mo.mo_last_device_error() == 0
    if not timeout_first:
        bad_token()
    mo.mo_selftest_bounded_wait(20_000_000)    # 20 ms
    if timeout_first:
        bad_token()
    assert mo.mo_last_device_error() == -8
    assert mo.mo_last_device_error() == 0
    bad_token()
    assert mo.mo_last_device_error() == -11
