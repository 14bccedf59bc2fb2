"""What callers of the feed-forward operators rely on beyond a single call's
values (no GPU needed)."""
import pytest

import matrix_optimizers_zero_gb300 as mo
from matrix_optimizers_zero_gb300 import build as mo_build


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
