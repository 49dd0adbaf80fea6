"""What the binding refuses in a tree call before the library sees it (no GPU:
the tensors are CPU tensors that say they are on a device)."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B


class OnCuda(torch.Tensor):
    """A CPU tensor that reports a CUDA device."""
    index = 0

    def get_device(self):
        return self.index


class Recorder:
    """Stands for the library: notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return B.FKV_OK
        return call


def _cuda(t, index=0):
    t = t.as_subclass(OnCuda)
    t.index = index
    return t


@pytest.fixture
def ctx():
    c = object.__new__(B.Context)
    c._device = 0
    c.cfg = B.fkv_config(4, 2, 64, 4, 2, 64, B.FKV_BF16, 0, 0.0, 0)
    c.torch_dtype = torch.bfloat16
    c._keep = {}
    c.handle = None
    c._lib = Recorder()
    return c


def _tree(ctx, workspace, **other):
    """A tree call, with `other` tensors in the place of the right ones."""
    q = _cuda(torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16))
    t = dict(q=q, out=q, seq_lens=_cuda(torch.zeros(2, dtype=torch.int32)),
             tree_mask=_cuda(torch.zeros(2, 5, 1, dtype=torch.int64)), node_counts=None)
    t.update(other)
    ctx.fkv_tree_attn(t["q"], 3, "fused", t["seq_lens"], t["tree_mask"], t["out"], workspace,
                      node_counts=t["node_counts"], stream=0)


def test_a_workspace_on_the_device_passes(ctx):
    _tree(ctx, _cuda(torch.zeros(64, dtype=torch.uint8)))
    assert ctx._lib.calls == ["fkv_tree_attn"]


@pytest.mark.parametrize("what", ["cpu", "strided"])
def test_a_workspace_that_the_kernel_cannot_write_is_refused(ctx, what):
    big = torch.zeros(128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        _tree(ctx, big if what == "cpu" else _cuda(big)[::2])
    assert ctx._lib.calls == []


@pytest.mark.parametrize("name,shape,dtype", [
    ("q", (2, 4, 5, 64), torch.bfloat16), ("out", (2, 4, 5, 64), torch.bfloat16),
    ("seq_lens", (2,), torch.int32), ("tree_mask", (2, 5, 1), torch.int64),
    ("node_counts", (2,), torch.int32), ("workspace", (64,), torch.uint8)])
def test_tensors_of_another_device_are_refused(ctx, name, shape, dtype):
    """The kernels run on the context's device, which need not reach their memory."""
    other = _cuda(torch.zeros(shape, dtype=dtype), index=1)
    ws = _cuda(torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="%s.*context's device" % name):
        if name == "workspace":
            _tree(ctx, other)
        else:
            _tree(ctx, ws, **{name: other})
    i, j = (_cuda(torch.zeros(2, dtype=torch.int32), index=k) for k in (0, 1))
    idx = _cuda(torch.zeros(2, 3, dtype=torch.int32))
    for a, b in ((i, j), (j, i)):
        with pytest.raises(ValueError, match="context's device"):
            ctx.fkv_reorder_seqs(a, b, stream=0)
        with pytest.raises(ValueError, match="context's device"):
            ctx.fkv_compact_rows(a, idx, b, stream=0)
    assert ctx._lib.calls == []
