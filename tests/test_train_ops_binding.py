"""The binding's own checks of its tensors (no GPU needed: stand-ins for CUDA
tensors, and a stand-in for the library that records its calls)."""
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
