"""What the binding refuses in calls on 8-bit caches, and in read-back, before the library sees
them (no GPU: the tensors are CPU tensors that say they are on a device)."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B

BATCH, ROWS, HEADS, D = 2, 200, 2, 64
COLS = 8                                     # 200 rows are 7 blocks of 32, in whole fours


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
            return COLS if name == "fkv_q8_scale_cols" else B.FKV_OK
        return call

    def made(self):
        return [c for c in self.calls if c != "fkv_q8_scale_cols"]


def _cuda(t, index=0):
    t = t.as_subclass(OnCuda)
    t.index = index
    return t


@pytest.fixture
def ctx():
    c = object.__new__(B.Context)
    c._device = 0
    c.cfg = B.fkv_config(4, BATCH, ROWS, 4, HEADS, D, B.FKV_BF16, 0, 0.0, 0)
    c.torch_dtype = torch.bfloat16
    c._keep = {}
    c._ring = {}
    c.handle = None
    c._lib = Recorder()
    return c


def _codes(dtype=torch.float8_e4m3fn, shape=(BATCH, HEADS, ROWS, D)):
    return torch.zeros(shape, dtype=torch.uint8).view(dtype) if dtype == torch.float8_e4m3fn else \
        torch.zeros(shape, dtype=dtype)


def _scales(shape=(BATCH, HEADS, COLS), dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _bind(ctx, **other):
    t = dict(kc=_cuda(_codes()), vc=_cuda(_codes()), ks=_cuda(_scales()), vs=_cuda(_scales()))
    t.update(other)
    ctx.fkv_bind_layer_cache_q8(1, t["kc"], t["vc"], t["ks"], t["vs"])


def test_codes_of_either_type_are_bound_and_kept(ctx):
    _bind(ctx)
    _bind(ctx, kc=_cuda(_codes(torch.uint8)))
    assert ctx._lib.made() == ["fkv_bind_layer_cache_q8"] * 2
    assert len(ctx._keep[("kv", 1)]) == 4


@pytest.mark.parametrize("name,bad", [
    ("kc", _codes(torch.int8)), ("vc", _codes(torch.bfloat16)), ("kc", _codes(shape=(BATCH, HEADS, ROWS - 1, D))),
    ("vc", _codes(shape=(BATCH, ROWS, HEADS, D))), ("ks", _scales(dtype=torch.float64)),
    ("vs", _scales((BATCH, HEADS, COLS - 1))), ("ks", _scales((BATCH, HEADS, ROWS)))])
def test_planes_of_another_shape_or_type_are_refused(ctx, name, bad):
    with pytest.raises((ValueError, TypeError)):
        _bind(ctx, **{name: _cuda(bad)})
    assert ctx._lib.made() == []


@pytest.mark.parametrize("name", ["kc", "vc", "ks", "vs"])
@pytest.mark.parametrize("what", ["cpu", "other device", "strided"])
def test_planes_that_the_kernels_cannot_reach_are_refused(ctx, name, what):
    t = _codes() if name[1] == "c" else _scales()
    if what == "other device":
        t = _cuda(t, index=1)
    elif what == "strided":
        t = _cuda(t.transpose(0, 1))
    with pytest.raises((ValueError, TypeError)):
        _bind(ctx, **{name: t})
    assert ctx._lib.made() == []


def test_a_ring_has_the_rings_rows(ctx):
    ctx._ring[1] = 64
    with pytest.raises((ValueError, TypeError)):
        _bind(ctx)
    short = lambda: _cuda(_codes(shape=(BATCH, HEADS, 64, D)))
    _bind(ctx, kc=short(), vc=short())
    assert ctx._lib.made() == ["fkv_bind_layer_cache_q8"]


def _read(ctx, T=None, **other):
    rows = torch.zeros(BATCH, HEADS, 5, D, dtype=torch.bfloat16)
    t = dict(pos=_cuda(torch.zeros(BATCH, dtype=torch.int32)), k=_cuda(rows), v=_cuda(rows.clone()))
    t.update(other)
    ctx.fkv_read_kv(3, "fused", t["pos"], t["k"], t["v"], T=T, stream=0)


def test_read_passes(ctx):
    _read(ctx)
    _read(ctx, T=5)
    assert ctx._lib.made() == ["fkv_read_kv"] * 2


@pytest.mark.parametrize("name,bad", [
    ("pos", torch.zeros(BATCH, dtype=torch.int64)), ("pos", torch.zeros(BATCH + 1, dtype=torch.int32)),
    ("k", torch.zeros(BATCH, HEADS, 5, D)), ("v", torch.zeros(BATCH, HEADS, 4, D, dtype=torch.bfloat16)),
    ("k", torch.zeros(BATCH, 5, HEADS, D, dtype=torch.bfloat16).transpose(1, 2))])
def test_read_refuses_other_shapes_types_and_strides(ctx, name, bad):
    with pytest.raises((ValueError, TypeError)):
        _read(ctx, **{name: _cuda(bad)})
    assert ctx._lib.made() == []


@pytest.mark.parametrize("name,shape,dtype", [("pos", (BATCH,), torch.int32),
                                             ("k", (BATCH, HEADS, 5, D), torch.bfloat16),
                                             ("v", (BATCH, HEADS, 5, D), torch.bfloat16)])
@pytest.mark.parametrize("device", ["cpu", "other"])
def test_read_refuses_tensors_of_another_device(ctx, name, shape, dtype, device):
    t = torch.zeros(shape, dtype=dtype)
    with pytest.raises((ValueError, TypeError)):
        _read(ctx, **{name: t if device == "cpu" else _cuda(t, index=1)})
    assert ctx._lib.made() == []


def test_read_refuses_more_rows_than_the_outputs_have(ctx):
    with pytest.raises((ValueError, TypeError)):
        _read(ctx, T=6)
    assert ctx._lib.made() == []
