"""8-bit caches whose scales are zero: appends against the oracle."""

import pytest
import torch

from q8_parity import BLOCK
from test_q8_gpu import Cache, u8

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("T", [1, 40])
def test_append_joins_a_block_of_scale_zero(T, D, dtype):
    """Scale 0 says that a block's values are zeros, whatever its codes: the rows before the new ones
    stay zeros (and codes that are no numbers stay none)."""
    c = Cache(3, 2, 200, D, dtype, seed=D + T)
    pos = [5, 37, 159 - T]
    for codes, scales in (c.k, c.v):
        for b, p in enumerate(pos):
            scales[b, :, p // BLOCK] = 0
        codes.view(torch.uint8)[1, :, 33, 7] = 0xFF
    c.check(c.new(T), c.new(T, 0.01), pos)
    k, v = (torch.full((3, 2, 5, D), 7.0, dtype=c.dt, device="cuda") for _ in range(2))
    c.ctx.fkv_read_kv(1, "vanilla", i32([p // BLOCK * BLOCK for p in pos]), k, v)
    for x in (k, v):
        assert bool((x[::2] == 0).all())
        seen = x[1].isnan()
        assert bool(seen[:, 1, 7].all()) and int(seen.sum()) == 2 and bool((x[1][~seen] == 0).all())
    c.ctx.close()


def test_append_joins_a_block_of_scale_zero_on_a_ring():
    c = Cache(2, 2, 1000, 64, ring=96, seed=3)
    for codes, scales in (c.k, c.v):
        scales[:, :, 1] = 0
    c.check(c.new(3), c.new(3, 20.0), [96 + 40, 3 * 96 + 63])
    assert not u8(c.k[0])[:, :, 32:40].view("int8").__and__(0x7F).any()
    c.ctx.close()
