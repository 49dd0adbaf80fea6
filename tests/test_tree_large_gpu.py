"""Tree attention, compaction and reordering on caches whose last sequence lies
behind 2^31 elements and 2^32 bytes: an offset kept in 32 bits would reach
another sequence's rows, which hold NaN (or bytes that are no copy)."""

import numpy as np
import pytest
import torch

import oracle as O
from cross_layer_kv_gb300 import fusedkv as B
from tree_parity import ULP, mask_words

pytestmark = pytest.mark.gpu

S, D, T, H = 65536, 64, 6, 64
# sequences: H * S rows of 64 values (records of 48 bytes) each
BATCH = {"bf16": 10, "f32": 10, "q4": 23}


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _caches(fmt, seed):
    """A context of one storage layer and its K and V, 0xff in every byte (NaN)."""
    Bt = BATCH[fmt]
    ctx = B.Context(2, Bt, S, H, H, D, "f32" if fmt == "f32" else "bf16")
    size = ctx.fkv_q4_row_bytes() if fmt == "q4" else D * (4 if fmt == "f32" else 2)
    kv = [torch.full((Bt, H, S, size), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    before = (Bt - 1) * H * S                 # rows before the last sequence's
    assert before * size > 1 << 32
    assert fmt == "q4" or before * D > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fmt == "q4":
        ctx.fkv_bind_layer_cache_q4(1, *kv)
    else:
        ctx.fkv_bind_layer_cache(1, *(x.view(ctx.torch_dtype) for x in kv))
    return ctx, kv, g


def _fill_unit(ctx, fmt, x, b, h, g):
    """Random rows of one (sequence, head); returned in float64."""
    new = torch.randn(S, D, generator=g, device="cuda").to(ctx.torch_dtype)
    if fmt != "q4":
        x[b, h].view(ctx.torch_dtype).copy_(new)
        return new.double()
    rec = O.q4_pack(*O.q4_quantize(new.float().cpu().numpy()[None, None]))
    x[b, h].copy_(torch.from_numpy(rec[0, 0]))
    return torch.from_numpy(np.asarray(O.q4_dequantize_records(rec, D)[0, 0], dtype=np.float64)).cuda()


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_tree_attention(fmt):
    """The bound is that of tree_parity.TreeSetup.reference."""
    ctx, kv, g = _caches(fmt, 5)
    Bt = BATCH[fmt]
    unit = {h: [_fill_unit(ctx, fmt, x, Bt - 1, h, g) for x in kv] for h in (0, H - 1)}
    q = torch.randn(Bt, H, T, D, generator=g, device="cuda").to(ctx.torch_dtype)
    out = torch.full_like(q, -77)
    seq = torch.tensor([0] * (Bt - 1) + [S - T], dtype=torch.int32, device="cuda")
    counts = torch.tensor([0] * (Bt - 1) + [T], dtype=torch.int32, device="cuda")
    masks = [[(2 << i) - 1 for i in range(T)]] * Bt
    ctx.fkv_tree_attn(q, 1, "vanilla", seq, mask_words(masks, T), out, ctx.tree_workspace(T), node_counts=counts)
    assert ctx.fkv_get_device_status() == B.FKV_OK
    assert (out[:-1] == -77).all()
    u16, u32 = ULP["bf16"], ULP["f32"]
    u_o, u_p = (4 * u32, 0.0) if fmt == "f32" else (u16, u16)
    u_kv = u16 if fmt == "q4" else 0.0
    see = torch.ones(T, S, dtype=torch.bool, device="cuda")
    see[:, S - T:] = torch.tril(torch.ones(T, T, dtype=torch.bool, device="cuda"))
    for h, (k, v) in unit.items():
        qq = q[-1, h].double()
        p = torch.softmax((qq @ k.T / 8.0).masked_fill(~see, -float("inf")), -1)
        ref = p @ v
        ds = (u_kv + (2 * D + 16) * u32) * (qq.abs() @ k.abs().T / 8.0).masked_fill(~see, 0.0).amax(1, keepdim=True)
        bound = u_o * ref.abs() + (p * (u_p + u_kv + 2 * ds + 1040 * u32)) @ v.abs()
        err = (out[-1, h].double() - ref).abs()
        assert (err <= bound).all(), "head %d: %.3g of the bound" % (h, float((err / bound).max()))


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_moves(fmt):
    """The last sequence takes rows of the one before it, then closes up a path."""
    ctx, kv, g = _caches(fmt, 6)
    Bt, n = BATCH[fmt], 300
    for x in kv:
        x[-2, :, :n].random_(0, 256, generator=g)
        x[-1, :, n - 40:n].random_(0, 256, generator=g)
    old = [x[-2:].clone() for x in kv]
    src = torch.tensor([-1] * (Bt - 1) + [Bt - 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0] * (Bt - 1) + [n - 20], dtype=torch.int32, device="cuda")
    ctx.fkv_reorder_seqs(src, lens)
    pos = torch.tensor([0] * (Bt - 1) + [n - 30], dtype=torch.int32, device="cuda")
    path = [2, 7, 15, 29]
    idx = torch.tensor([[0] * 4] * (Bt - 1) + [path], dtype=torch.int32, device="cuda")
    counts = torch.tensor([0] * (Bt - 1) + [4], dtype=torch.int32, device="cuda")
    ctx.fkv_compact_rows(pos, idx, counts)
    assert ctx.fkv_get_device_status() == B.FKV_OK
    for x, o in zip(kv, old):
        want = o[1].clone()
        want[:, :n - 20] = o[0][:, :n - 20]
        want[:, n - 30:n - 26] = want[:, [n - 30 + j for j in path]].clone()
        assert torch.equal(x[-1], want)
        assert torch.equal(x[-2], o[0])
        assert (x[:-2].view(torch.int64) == -1).all()
