"""The example that runs the training-step operators together with Muon and
AdamW: the loss of a task a table can learn has to fall."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_loss_falls(fmt):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=60, fmt=fmt)
    assert all(math.isfinite(x) for x in losses)
    assert losses[0] > 0.8 * math.log(512)
    assert sum(losses[-5:]) / 5 < 0.25 * losses[0]   # 512 successors, each seen about 240 times
    assert m.train(steps=3, fmt=fmt) == losses[:3]    # every operator repeats bit for bit
