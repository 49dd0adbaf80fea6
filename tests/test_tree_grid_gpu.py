"""The grids and workspaces that fkv_tree_attn plans, on the GPU."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from tree_parity import TreeSetup

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [16, 33, 40, 48, 65, 100, 128])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
def test_fp32_calls_are_one_wave(D, T):
    """Every CTA has two partial records in the workspace, so its size tells how many
    there are: no more than the device holds at once.  Two of 256 threads an SM at
    most; over 128 channels one, since three tiles of 64 rows of 132 floats are 101 KB
    of the SM's 228 KB, and the probabilities and masks another 18 KB."""
    H, G, rows = 2, 4, 64
    ctx = B.Context(4, 1, 4096, H * G, H, D, "f32")
    tiles = -(-G * T // rows)
    places = torch.cuda.get_device_properties(0).multi_processor_count * (1 if D == 128 else 2)
    assert ctx.fkv_tree_workspace_bytes(T) <= places * 2 * rows * (D + 2) * 4 + H * tiles * 8


@pytest.mark.parametrize("D,T,mode", [(64, 40, "lite"), (80, 48, "fused"), (128, 33, "scaled")])
def test_fp32_three_row_tiles(D, T, mode):
    s = TreeSetup(D=D, T=T, G=4, fmt="f32", mode=mode, lens=(0, 700, 1300), S=1400)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check("three row tiles")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,Bt", [(64, 1, 1), (64, 4, 3), (80, 2, 3), (96, 4, 300), (128, 4, 3), (128, 2, 1024)])
def test_workspaces_grow_with_the_nodes(dtype, D, G, Bt):
    """A workspace for T nodes serves every call with fewer."""
    ctx = B.Context(4, Bt, 4096, 2 * G, 2, D, dtype)
    sizes = [ctx.fkv_tree_workspace_bytes(T) for T in range(1, 129)]
    assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("fmt,D,G,T,fewer", [("bf16", 64, 4, 80, (64, 33, 8)), ("f32", 64, 4, 112, (64, 16, 4)),
                                             ("q4", 128, 2, 112, (96, 64, 16)), ("f32", 128, 4, 33, (32, 4))])
def test_the_largest_tree_s_workspace_serves_smaller_ones(fmt, D, G, T, fewer):
    big = TreeSetup(D=D, G=G, T=T, fmt=fmt, mode="lite", lens=(100, 700, 1200), S=1400)
    for t in fewer:
        s = TreeSetup(D=D, G=G, T=t, fmt=fmt, mode="lite", lens=(100, 700, 1200), S=1400)
        want = s.run().clone()
        s.ws = big.ws
        s.out.fill_(-77)
        assert torch.equal(s.run(), want)
        assert s.ctx.fkv_get_device_status() == B.FKV_OK
