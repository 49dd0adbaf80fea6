"""What the binding refuses in a tree call before the library sees it (no GPU:
the tensors are CPU tensors that say they are on a device)."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B


class OnCuda(torch.Tensor):
    """A CPU tensor that reports CUDA device 0."""
    is_cuda = property(lambda self: True)


class Recorder:
    """Stands for the library: notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return B.FKV_OK
        return call


def _cuda(t):
    return t.as_subclass(OnCuda)


@pytest.fixture
def ctx():
    c = object.__new__(B.Context)
    c.cfg = B.fkv_config(4, 2, 64, 4, 2, 64, B.FKV_BF16, 0, 0.0, 0)
    c.torch_dtype = torch.bfloat16
    c._keep = {}
    c.handle = None
    c._lib = Recorder()
    return c


def _tree(ctx, workspace):
    q = _cuda(torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16))
    seq = _cuda(torch.zeros(2, dtype=torch.int32))
    mask = _cuda(torch.zeros(2, 5, 1, dtype=torch.int64))
    ctx.fkv_tree_attn(q, 3, "fused", seq, mask, q, workspace, stream=0)


def test_a_workspace_on_the_device_passes(ctx):
    _tree(ctx, _cuda(torch.zeros(64, dtype=torch.uint8)))
    assert ctx._lib.calls == ["fkv_tree_attn"]


@pytest.mark.parametrize("what", ["cpu", "strided"])
def test_a_workspace_that_the_kernel_cannot_write_is_refused(ctx, what):
    big = torch.zeros(128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        _tree(ctx, big if what == "cpu" else _cuda(big)[::2])
    assert ctx._lib.calls == []
