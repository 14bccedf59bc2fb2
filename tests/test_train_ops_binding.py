"""The binding's own checks of its tensors (no GPU needed: stand-ins for CUDA
tensors, and a stand-in for the library that records its calls)."""
import os
import re

import pytest
import torch

import matrix_optimizers_zero_gb300 as mo
from matrix_optimizers_zero_gb300 import train_ops


class Tensor:
    def __init__(self, shape, dtype, cuda=True, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self._contiguous = torch.Size(shape), dtype, cuda, contiguous

    def is_contiguous(self):
        return self._contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(train_ops, "load_library", lambda: lib)
    monkeypatch.setattr(train_ops, "_stream_ptr", lambda stream, t: 0)
    return lib


def call_grad(workspace):
    mo.embed_grad(Tensor((5, 8), torch.float32), Tensor((5,), torch.int64), Tensor((9, 8), torch.float32), workspace)


def test_embed_grad_takes_a_device_workspace(library):
    call_grad(Tensor((1 << 16,), torch.uint8))
    (name, args), = library.calls
    assert name == "embed_grad" and (1 << 16) in args


@pytest.mark.parametrize("kw", [dict(cuda=False), dict(contiguous=False)])
def test_embed_grad_refuses_other_workspaces(library, kw):
    with pytest.raises(ValueError, match="workspace"):
        call_grad(Tensor((1 << 16,), torch.uint8, **kw))
    assert not library.calls


# ---------------------------------------------------------------- the documented use of the generator

def generator_streams(text, step):
    """(seed, offset) of every stream that the lines of a code sample draw from at a step."""
    used = []
    for line in text.splitlines():
        for cls, args in re.findall(r"mo\.(Dropout|Random)\(([^()]*)\)", line.split("#")[0]):
            made = eval(f"mo.{cls}({args})", {"mo": mo, "seed": 7, "step": step})
            r = made.random if cls == "Dropout" else made
            # a quantisation takes the next offset for the transposed tensor
            used += [(r.seed, r.offset + i) for i in range(2 if "fp4_quantize" in line else 1)]
    return used


@pytest.mark.parametrize("where", ["docstring", "README.md"])
def test_documented_offsets_never_repeat(where):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = train_ops.__doc__ if where == "docstring" else open(os.path.join(root, where), encoding="utf-8").read()
    assert len(generator_streams(text, 1)) == 3      # dropout, both orientations of a gradient
    used = [s for step in range(1, 9) for s in generator_streams(text, step)]
    assert len(set(used)) == len(used)
