"""fkv_tree_attn where it gives up, meets rows that are not finite, or reads
caches that were bound anew, on the GPU."""

import numpy as np
import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from parity import f64
from tree_parity import TreeSetup

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


# columns of query rows a CTA: 2 T
@pytest.mark.parametrize("fmt,mode,T,kw", [
    ("bf16", "lite", 4, {}), ("bf16", "fused", 16, {}), ("bf16", "fused", 64, {}), ("bf16", "lite", 33, dict(D=128)),
    ("q4", "lite", 4, {}), ("q4", "fused", 16, {}), ("q4", "scaled", 32, dict(D=96)), ("q4", "fused", 64, dict(D=128)),
    ("bf16", "lite", 12, dict(window=100, ring=896)), ("q4", "lite", 12, dict(window=100, ring=896))])
def test_a_wait_that_runs_out_is_reported(fmt, mode, T, kw):
    """With a limit of 0 every wait of the tensor-core kernel gives up without a look at
    its barrier: the call ends with a status, and the next one is whole."""
    s = TreeSetup(fmt=fmt, mode=mode, T=T, Bt=3, lens=(700, 1300, 90), S=1400, **kw)
    s.ctx.fkv_set_wait_limit(0)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    assert s.ctx.fkv_get_device_status() == B.FKV_OK       # reported once
    s.ctx.fkv_set_wait_limit(10 ** 9)
    s.out.fill_(-77)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check("after a timeout")


def test_fp32_calls_wait_for_nothing():
    s = TreeSetup(fmt="f32", T=16, lens=(700, 1300, 90), S=1400)
    s.ctx.fkv_set_wait_limit(0)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check("limit 0")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_a_replay_after_one_that_gave_up(fmt):
    """As documented: once the workspace is zeroed."""
    s = TreeSetup(fmt=fmt, T=12, Bt=3, lens=(700, 1300, 90), S=1400)
    s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        s.run(stream=side)
    s.ctx.fkv_set_wait_limit(0)
    g.replay()
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    s.ctx.fkv_set_wait_limit(10 ** 9)
    s.ws.zero_()
    for _ in range(2):
        s.out.fill_(-77)
        g.replay()
        assert s.ctx.fkv_get_device_status() == B.FKV_OK
        s.check("replay")


def _params(s, x):
    """The (scale, min) pairs of 4-bit records as bf16."""
    return x.view(torch.bfloat16)[..., s.D // 4:s.D // 4 + s.D // 8]


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_records_not_seen_may_hold_anything(mode, bad):
    """Scales and minima that are not finite behind the last row and in rows no node sees."""
    T = 12
    masks = [[(1 << i) | 1 for i in range(T)] for _ in range(3)]
    for m in masks:
        m[3] = 1            # node 3 is seen by nobody, itself included
    s = TreeSetup(fmt="q4", T=T, mode=mode, masks=masks, lens=(0, 120, 200), S=320)
    s.run()
    clean = s.out.clone()
    for b, P in enumerate(s.lens):
        for l in (1, 2):
            for x in (s.k[l], s.v[l]):
                _params(s, x)[b, :, P + T:] = bad
                _params(s, x)[b, :, P + 3, 0::2] = bad      # scales
                _params(s, x)[b, :, P + 3, 5] = bad         # one group's minimum
    s.out.fill_(-77)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert torch.equal(s.out, clean)


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_a_bad_row_stays_with_the_nodes_that_see_it(fmt, bad, what, mode):
    """A drafted key or value row (its 4-bit parameters) that is not finite."""
    T = 6
    masks = [[1, 2, 1 | 4, 2 | 8, 1 | 16, 2 | 32]] * 2
    s = TreeSetup(fmt=fmt, mode=mode, T=T, Bt=2, masks=masks, lens=(40, 127), S=256)
    s.run()
    clean = s.out.clone()
    for l in (1, 2):
        x = getattr(s, what)[l]
        for b, P in enumerate(s.lens):
            (_params(s, x) if fmt == "q4" else x)[b, :, P + 1] = bad
    s.run()
    even, odd = [0, 2, 4], [1, 3, 5]
    assert torch.equal(s.out[:, :, even], clean[:, :, even])
    assert not torch.isfinite(s.out[:, :, odd].float()).any()


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("window,ring,T", [(100, 111, 12), (128, 257, 7), (64, 128, 65)])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_rings_with_ragged_trees(fmt, window, ring, T, mode):
    lens = (0, ring - 1, ring, 5 * ring // 2, 1200 - T)
    s = TreeSetup(fmt=fmt, mode=mode, window=window, ring=ring, T=T, Bt=5, S=1200, lens=lens,
                  counts=[T, 1, 0, T // 2, T - 1])
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check("R=%d" % ring)


def test_one_node_over_4_bit_caches_is_near_decode():
    """fkv_decode_attn keeps the dequantised values in fp32, this call rounds them to bf16:
    both are within this call's bound of the oracle."""
    s = TreeSetup(fmt="q4", T=1, masks=[[1]] * 3, lens=(0, 127, 200))
    s.run()
    s.check("T=1")
    dec = torch.empty_like(s.q[:, :, 0]).contiguous()
    s.ctx.fkv_decode_attn(s.q[:, :, 0].contiguous(), s.layer, s.mode, s.seq + 1, dec, s.ctx.workspace())
    ref, bound = s.reference()
    assert (np.abs(f64(s.out[:, :, 0]) - f64(dec)) <= 2 * bound[:, :, 0]).all()


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_buffers_bound_anew(fmt):
    """Each call reads the buffers, and the ring rows, of the last bind."""
    s = TreeSetup(fmt=fmt, mode="lite", T=9, window=100, lens=(0, 127, 200), S=320)
    s.run()
    s.check("first buffers")
    t = TreeSetup(fmt=fmt, mode="lite", T=9, window=100, lens=(0, 127, 200), S=320, seed=1)
    for l in (1, 2):
        s.ctx.fkv_bind_layer_cache(l, t.k[l], t.v[l])
    s.k, s.v = t.k, t.v
    s.run()
    s.check("other buffers")
    r = TreeSetup(fmt=fmt, mode="lite", T=9, window=100, ring=120, lens=(0, 127, 200), S=320, seed=2)
    for l in (1, 2):
        s.ctx.fkv_set_ring_rows(l, 120)
        s.ctx.fkv_bind_layer_cache(l, r.k[l], r.v[l])
    s.k, s.v, s.ring, s.rows = r.k, r.v, 120, 120
    s.run()
    s.check("rings")
    for l in (1, 2):
        s.ctx.fkv_set_ring_rows(l, 0)
        s.ctx.fkv_bind_layer_cache(l, t.k[l], t.v[l])
    s.k, s.v, s.ring, s.rows = t.k, t.v, 0, 320
    s.run()
    s.check("full length again")
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
