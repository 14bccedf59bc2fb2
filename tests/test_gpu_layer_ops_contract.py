"""Feed-forward operators on the GPU: calls that the documentation allows beside
the usual ones, at both ends of the numbers' range and of the sizes."""
import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
import test_gpu_layer_ops as base
from test_gpu_layer_ops import BF16, clean, empty8

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
