"""What callers of the feed-forward operators rely on beyond a single call's
values (no GPU needed)."""
import ctypes
import threading

import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
import test_layer_ops_binding as b
from matrix_optimizers_zero_gb300 import build as mo_build
from matrix_optimizers_zero_gb300 import layer_ops
from matrix_optimizers_zero_gb300.layer_ops import MoTensor
from test_layer_ops_binding import library  # noqa: F401  (a fixture)

NULL, SHAPE, ALIGN, PARAM, WS, OVERLAP = -1, -2, -3, -4, -5, -6
F32, BF16, MX8 = 0, 1, 2
A, B, C, D, E, F = (0x100000000 * k for k in range(1, 7))   # far apart, aligned, never read
BIG = 1 << 30


def ten(data):
    return MoTensor(data, None, BF16)


def ref(t):
    return ctypes.byref(t)


@pytest.fixture(scope="module")
def lib():
    mo_build.build()
    return mo.load_library()


# ---------------------------------------------------------------- workspaces

# Tokens around every size where a rule of the layout may change: parts of 8 tokens up to 608 of them (fewer
# where rows are wide), and slices of 32768.
TOKENS = sorted({t + o for t in (0, 8, 64, 512, 608, 1216, 2432, 4864, 9728, 14592, 32768, 65536, 100000, 1 << 20) for o in range(-9, 10) if t + o >= 0})


@pytest.mark.parametrize("cols,rows", [(64, 256), (1280, 5120), (8, 40), (33, 47), (40, 257), (65536, 24), (24, 70001), (4096, 100001)])
@pytest.mark.parametrize("grad", [False, True])
def test_a_linear_workspace_serves_smaller_batches(lib, cols, rows, grad):
    sizes = [mo.mo_linear_workspace_bytes(t, cols, rows, grad=grad) for t in TOKENS]
    assert all(sizes) and sizes == sorted(sizes)


@pytest.mark.parametrize("dim,inner", [(64, 256), (4096, 14336), (33, 47), (65536, 40), (40, 32768)])
@pytest.mark.parametrize("grad", [False, True])
def test_a_gated_workspace_serves_smaller_batches(lib, dim, inner, grad):
    sizes = [mo.mo_gated_ffn_workspace_bytes(t, dim, inner, grad=grad) for t in TOKENS]
    assert all(sizes) and sizes == sorted(sizes)


@pytest.mark.parametrize("dim", [1, 64, 300, 4096, 12288, 20001])
def test_a_norm_workspace_serves_smaller_batches(lib, dim):
    sizes = [mo.mo_rms_norm_grad_workspace_bytes(t, dim) for t in TOKENS]
    assert all(sizes) and sizes == sorted(sizes)


@pytest.mark.parametrize("tokens,cols,rows", [(8, 64, 256), (5000, 33, 47), (40000, 65536, 24), (9, 24, 70001)])
def test_a_gradient_workspace_serves_the_forward_pass(lib, tokens, cols, rows):
    assert mo.mo_linear_workspace_bytes(tokens, cols, rows, grad=True) >= mo.mo_linear_workspace_bytes(tokens, cols, rows)
    dim, inner = cols, min(rows, 32768)
    assert mo.mo_gated_ffn_workspace_bytes(tokens, dim, inner, grad=True) >= mo.mo_gated_ffn_workspace_bytes(tokens, dim, inner)


# ---------------------------------------------------------------- in place

@pytest.mark.parametrize("act", [0, 4])
@pytest.mark.parametrize("t,k,n,kw", [
    (8, 64, 64, dict(x=ten(A), res=A, out=A)),            # s += s w^T: other tiles read s
    (8, 63, 63, dict(x=ten(A), res=A, out=A)),
    (64, 64, 32, dict(w=A, res=A, out=A)),                # 64 tokens of 32 are as long as the weight
    (300, 1000, 1000, dict(x=ten(A), res=A, out=A)),
])
def test_a_product_does_not_replace_its_operands(lib, t, k, n, kw, act):
    a = dict(dict(x=ten(B), w=C, res=None, out=D), **kw)
    got = lib.linear_forward(ref(a["x"]), a["w"], t, k, n, None, act, a["res"], None, a["out"], BF16, E, BIG, None)
    assert got == OVERLAP


@pytest.mark.parametrize("w", ["wg", "wu", "wd"])
def test_a_gated_block_does_not_replace_its_weights(lib, w):
    a = dict(dict(wg=B, wu=C, wd=D), **{w: A})
    t, d, f = 96, 64, 96                                  # 96 tokens of 64 are as long as a weight
    assert lib.gated_ffn_forward(ref(ten(E)), a["wg"], a["wu"], a["wd"], t, d, f, 4, A, None, None, A, BF16, F, BIG, None) == OVERLAP


def test_a_norm_does_not_replace_its_weight(lib):
    """One row of fp32 is as long as the weight."""
    assert lib.rms_norm(A, None, F32, 1, 40, A, 1e-6, None, A, F32, None, None) == OVERLAP
    assert lib.rms_norm(A, B, F32, 1, 40, B, 1e-6, B, C, F32, None, None) == OVERLAP
    x = MoTensor(B, None, F32)
    assert lib.rms_norm_grad(A, F32, ref(x), 1, 40, A, 1e-6, None, A, None, 0, None, 0, None) == OVERLAP


def test_in_place_calls_pass_the_checks(lib):
    """What is read and written by the same threads, or by different launches, is no overlap: these calls go on
    to the device."""
    def passes(st):
        assert st not in (NULL, SHAPE, ALIGN, PARAM, WS, OVERLAP), st

    if torch.cuda.is_available():
        pytest.skip("addresses that nothing stands behind")
    passes(lib.linear_forward(ref(ten(A)), B, 8, 64, 32, None, 0, C, None, C, BF16, D, BIG, None))
    passes(lib.gated_ffn_forward(ref(ten(A)), B, C, D, 8, 64, 96, 4, E, None, None, E, BF16, F, BIG, None))
    passes(lib.gated_ffn_forward(ref(ten(A)), B, C, D, 8, 64, 96, 4, A, None, None, A, BF16, F, BIG, None))
    passes(lib.rms_norm(A, B, BF16, 4, 40, C, 1e-6, B, A, BF16, None, None))
    passes(lib.rms_norm_grad(A, BF16, ref(ten(B)), 4, 40, C, 1e-6, D, A, E, 0, F, BIG, None))
    passes(lib.rms_norm_grad(A, BF16, ref(ten(B)), 4, 40, C, 1e-6, D, D, E, 0, F, BIG, None))


# ---------------------------------------------------------------- threads

def test_a_second_thread_may_make_its_first_call_beside_the_first(monkeypatch):
    """What a call looks up once is complete for every thread that finds it: the second thread comes while the
    first one is looking up."""
    monkeypatch.setattr(layer_ops, "_dtypes", None)
    monkeypatch.setattr(layer_ops, "_current_device", None)
    seen, inside = [], []

    def lookup(obj, name, *default):
        if not inside:
            inside.append(True)
            t = threading.Thread(target=lambda: seen.append(layer_ops._here()))
            t.start()
            t.join()
        return lambda: 5

    monkeypatch.setattr(layer_ops, "getattr", lookup, raising=False)
    assert layer_ops._here() == 5 and seen == [5]


# ---------------------------------------------------------------- layouts

LAYOUTS = {   # argument -> its shape [rows, width], for every matrix that the binding checks by type and size
    "mx8_dequantize": {"out": (6, 40)}, "rms_norm": {"out": (6, 40), "residual": (6, 40), "sum_out": (6, 40)},
    "rms_norm_grad": {"dx": (6, 40), "dresidual": (6, 40)}, "linear": {"out": (6, 72), "residual": (6, 72)},
    "linear_grad": {"dx": (6, 40), "dw": (72, 40)}, "gated_ffn": {"out": (6, 40), "residual": (6, 40)},
    "gated_ffn_grad": {"dx": (6, 40), "dw_gate": (72, 40), "dw_up": (72, 40), "dw_down": (40, 72)}}
ARGS = [(name, arg) for name, args in LAYOUTS.items() for arg in args]


@pytest.mark.parametrize("name,arg", ARGS)
def test_refuses_matrices_that_lie_the_other_way(library, name, arg):
    f, kw = b.calls()[name]
    rows, width = LAYOUTS[name][arg]
    assert tuple(kw[arg].shape) == (rows, width)
    for shape in ((width, rows), (1, width, rows), (width, 2, rows // 2), (width // 2, 2, rows)):
        kw[arg] = b.Tensor(shape, kw[arg].dtype)
        with pytest.raises(ValueError, match="transpose"):
            f(**kw)
    assert not library.calls


@pytest.mark.parametrize("name,arg", ARGS)
def test_takes_views_of_the_same_rows(library, name, arg):
    f, kw = b.calls()[name]
    rows, width = LAYOUTS[name][arg]
    shapes = [(2, rows // 2, width), (1, rows, 1, width), (rows * width,), (1, rows * width), (rows, 4, width // 4), (2, rows // 2, 4, width // 4),
              (rows * 4, width // 4)]
    for shape in shapes:
        kw[arg] = b.Tensor(shape, kw[arg].dtype)
        f(**kw)
    assert len(library.calls) == len(shapes)


def test_square_and_single_rows_have_no_other_way(library):
    for t, d in ((40, 40), (1, 40), (40, 1)):
        mo.rms_norm(b.Tensor((t, d)), b.Tensor((t, d)), residual=b.Tensor((d, t) if t == d or t == 1 else (t, d)))
    assert len(library.calls) == 3


# ---------------------------------------------------------------- storage that moves

class At(b.Tensor):
    """A stand-in for a CUDA tensor at an address."""

    def __init__(self, shape, at, dtype=torch.uint8, device=0):
        super().__init__(shape, dtype, device)
        self.at = at

    def data_ptr(self):
        return self.at


def test_an_8_bit_tensor_is_where_its_storage_is(library):
    q = mo.Mx8Tensor(6, 40, codes=At((6, 64), 4096), scales=At((6, 2), 8192))
    x = b.Tensor((6, 40))

    def call():
        mo.mx8_quantize(x, q)
        got = library.calls[-1][1][4]._obj      # (what byref was given)
        return got.data, got.scales

    assert call() == (4096, 8192)
    q.codes.at = 1 << 20                        # t.data = another, or a resized storage
    assert call() == (1 << 20, 8192)
    q.scales = At((6, 2), 1 << 21)
    assert call() == (1 << 20, 1 << 21)
    n = len(library.calls)
    for bad in (At((6, 32), 1 << 22), At((6, 64), 1 << 22, torch.int8), At((6, 64), 1 << 22, device=1), At((6, 64), 1 << 22, device=-1)):
        q.codes = bad
        with pytest.raises(ValueError):
            mo.mx8_quantize(x, q)
    assert len(library.calls) == n
