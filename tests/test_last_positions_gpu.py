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


def test_decode_and_read_back_of_a_full_length_of_2_31_rows():
    """One sequence of every position there is (planes of 137 GB: keys and values share their codes).
    Queries of zeros weigh all keys alike, and the last block alone holds values."""
    free, _ = torch.cuda.mem_get_info()
    if free < 150 << 30:
        pytest.skip("needs 150 GiB of device memory")
    D = 64
    ctx = B.Context(2, 1, LAST, 1, 1, D, "f32")
    codes = torch.zeros(1, 1, LAST, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 1, ctx.fkv_q8_scale_cols(), device="cuda")
    last = LAST - LAST // 32 * 32                               # rows of the last block
    codes[0, 0, -last:] = 0x78                                  # 256
    scales[0, 0, LAST // 32] = 2.0 ** 20
    ctx.fkv_bind_layer_cache_q8(1, codes, codes, scales, scales)
    q = torch.zeros(1, 1, D, device="cuda")
    out = torch.empty_like(q)
    ctx.fkv_decode_attn(q, 1, "vanilla", i32([LAST]), out, ctx.workspace())
    assert ctx.fkv_get_device_status() == B.FKV_OK
    # a lane adds one sum of four weights a group of 16 rows: as many fp32 roundings as its warp
    # (of 12 a CTA) has groups
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ref = last * 2.0 ** 28 / LAST
    assert float((out - ref).abs().max()) <= ref * (LAST / 16 / (12 * sms) + 128) * 2.0 ** -24
    k, v = (torch.empty(1, 1, 40, D, device="cuda") for _ in range(2))
    ctx.fkv_read_kv(1, "vanilla", i32([LAST - 40]), k, v)
    want = torch.where(torch.arange(40, device="cuda") >= 40 - last, 2.0 ** 28, 0.0)[:, None].expand(40, D)
    assert torch.equal(k[0, 0], want) and torch.equal(v[0, 0], want)
    ctx.close()
    del codes, scales
    torch.cuda.empty_cache()
