"""Calls at the last positions that a context can have, 2^31 - 2 and before: over rings, which make
such contexts fit.  A call's rows, tiles and masks are those of the same call any whole number of
rings (and tiles) earlier, so its results are too, bit for bit."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from q8_parity import Setup, check_prefill

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1                  # positions of a context


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("mode", ["lite", "scaled", "fused"])
@pytest.mark.parametrize("D,G", [(64, 2), (80, 1), (96, 2), (96, 1), (128, 1), (128, 4)])
@pytest.mark.parametrize("end,C,window", [(LAST, 1, 33), (LAST, 100, 200), (LAST, 300, 40), (LAST - 50, 257, 300),
                                          (LAST - 127, 16, 500), (LAST - 129, 129, 1)])
def test_prefill_over_8_bit_rings(end, C, window, D, G, mode):
    ring = 896
    s = Setup(mode, 1, LAST, 1, G, D, window=window, ring=ring, seed=C)
    q = s.query(1, G, C, D)
    out, _ = check_prefill(s, end - C, C, q)
    before = torch.empty_like(q)
    s.ctx.fkv_prefill_attn_chunk(q, s.layer, s.mode, end - C - 2 ** 20 * ring, C, before)
    assert torch.equal(out, before)
    s.close()


@pytest.mark.parametrize("G", [1, 2])
def test_prefill_over_8_bit_rings_of_rows_that_are_no_numbers(G):
    C, window, ring = 300, 100, 512
    s = Setup("lite", 1, LAST, 1, G, 64, window=window, ring=ring, seed=1)
    q = s.query(1, G, C, 64)
    clean, _ = check_prefill(s, LAST - C, C, q)
    codes = s.v[0][0].view(torch.uint8)
    m = torch.arange(LAST - C, LAST, device="cuda")
    for t in (LAST - 1, LAST - 2, LAST - 40, LAST - C, LAST - C - 1, LAST - C - 99):
        old = int(codes[0, 0, t % ring, 5])
        codes[0, 0, t % ring, 5] = 0x7F
        out = torch.empty_like(q)
        s.ctx.fkv_prefill_attn_chunk(q, s.layer, s.mode, LAST - C, C, out)
        codes[0, 0, t % ring, 5] = old
        sees = (m >= t) & (m < t + window)
        assert bool(out[:, :, sees].isnan().all()), LAST - t
        assert torch.equal(out[:, :, ~sees], clean[:, :, ~sees]), LAST - t
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.close()


@pytest.mark.parametrize("mode", ["lite", "scaled", "fused"])
@pytest.mark.parametrize("D,G", [(64, 2), (80, 1), (96, 2), (96, 1), (128, 1), (128, 2)])
@pytest.mark.parametrize("end,C,window", [(LAST, 1, 33), (LAST, 100, 200), (LAST, 300, 40), (LAST - 50, 257, 300),
                                          (LAST - 127, 16, 500), (LAST - 129, 129, 1)])
def test_prefill_over_bf16_rings(end, C, window, D, G, mode):
    ring = 896                      # whole tiles of 64, 112 and 128 keys
    g = torch.Generator(device="cuda").manual_seed(C)
    ctx = B.Context(4, 1, LAST, G, 1, D, "bf16")
    for layer in (1, 2):
        k, v = (torch.randn(1, 1, ring, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        ctx.fkv_set_ring_rows(layer, ring)
        ctx.fkv_bind_layer_cache(layer, k, v)
    ctx.fkv_set_window(4, window)
    ctx.fkv_set_fusion_weights(4, *(torch.randn(1, D, generator=g, device="cuda") * 0.3 + 0.5 for _ in range(4)))
    q = torch.randn(1, G, C, D, generator=g, device="cuda").to(torch.bfloat16)
    out, before = torch.full_like(q, float("nan")), torch.empty_like(q)
    ctx.fkv_prefill_attn_chunk(q, 4, mode, end - C, C, out)
    # the same rows and tiles, at positions that test_ring_gpu.py checks
    ctx.fkv_prefill_attn_chunk(q, 4, mode, (end - C) % ring + 2 * ring, C, before)
    assert ctx.fkv_get_device_status() == B.FKV_OK
    assert bool(out.isfinite().all()) and torch.equal(out, before)
    ctx.close()
