"""8-bit caches whose scales are zero, no powers of two, or far apart between the two sources of a
fused layer: appends against the oracle, attention against float64 with derived bounds."""

import math

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from q8_parity import BLOCK, Setup, check_decode, check_prefill, reconstruct, values
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


@pytest.mark.parametrize("mode", ["vanilla", "scaled", "fused"])
def test_fp32_decode_of_scales_that_are_no_powers_of_two(mode):
    """One key: the output is its value, off by P's two halves (2^-22), two sums of a matrix product
    (2^-23 each, should it truncate) and about six more fp32 roundings (2^-24 each): below 2^-20 of
    the magnitudes that are added up, for any scale of the range that is promised."""
    n = 64
    s = Setup(mode, n, 40, 2, 2, 64, dtype="f32", seed=12)
    g = s.gen
    e = torch.randint(-63, 38, (n, 2, 1), generator=g, device="cuda").double()
    e[:8], e[8:16] = -63, 37
    for planes in s.planes.values():
        for _, scales in planes:
            m = torch.rand(n, 2, 1, generator=g, device="cuda").double() + 1
            scales[:] = (torch.exp2(e) * m).float()
    q = s.query(n, 4, 64)
    out = torch.empty_like(q)
    s.ctx.fkv_decode_attn(q, s.layer, mode, i32([1] * n), out, s.ctx.workspace())
    v = [values(x)[:, :, 0] for x in s.v]
    w = [s.w[2].double(), s.w[3].double()] if mode != "vanilla" else [torch.ones(2, 64, device="cuda").double()]
    ref, size = sum(a * b for a, b in zip(w, v)), sum((a * b).abs() for a, b in zip(w, v))
    err = (out.view(n, 2, 2, 64).double() - ref[:, :, None]).abs()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert bool((err <= 2.0 ** -20 * size[:, :, None]).all()), float((err / size[:, :, None].clamp(min=1e-300)).max())
    s.close()


def test_fp32_decode_of_equal_scores_under_other_scales():
    """Keys of zeros: every weight is 1 / n, whatever its block's value scale (n + 64 sums, decode_bound)."""
    n = 200
    s = Setup("vanilla", 4, n, 2, 2, 64, dtype="f32", seed=13)
    s.k[0][0].view(torch.uint8).zero_()
    scales = s.v[0][1]
    scales[:] = torch.exp2(torch.tensor([-60.0, -31.0, 0.0, 30.0], device="cuda"))[:, None, None] * \
        (torch.rand(scales.shape, generator=s.gen, device="cuda") + 1)
    s.v[0][0].view(torch.uint8).bitwise_and_(0x7F)      # no cancellation
    q = s.query(4, 4, 64)
    out = torch.empty_like(q)
    s.ctx.fkv_decode_attn(q, s.layer, "vanilla", i32([n] * 4), out, s.ctx.workspace())
    ref = values(s.v[0]).mean(2)
    err = (out.view(4, 2, 2, 64).double() - ref[:, :, None]).abs() / ref[:, :, None]
    assert float(err.max()) <= 2.0 ** -20 + (n + 64) * 2.0 ** -24, float(err.max())
    s.close()


def _apart(s, gap, how):
    """The blocks of one source get scales 2^gap times the other's.  `weights`: and weights 2^-gap
    times; `zero weights`: its weights are 0; `zeros`: its codes are (and its scales still count)."""
    first, last = min(s.planes), max(s.planes)
    big = last if gap > 0 else first
    for codes, scales in s.planes[big]:
        scales *= 2.0 ** abs(gap)
        if how == "zeros":
            codes.view(torch.uint8).zero_()
    mine = (1, 3) if big == last else (0, 2)
    for i in mine:
        if how == "weights":
            s.w[i] *= 2.0 ** -abs(gap)
        elif how == "zero weights":
            s.w[i].zero_()


APART = [(28, "weights"), (-28, "weights"), (20, "weights"), (28, "zero weights"), (-28, "zero weights")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("gap,how", APART)
def test_decode_of_sources_whose_scales_are_far_apart(gap, how, D, dtype):
    s = Setup("fused", 2, 300, 2, 2, D, dtype=dtype, seed=D + gap)
    _apart(s, gap, how)
    check_decode(s, [300, 77], what="%s 2^%d" % (how, gap))
    s.close()


def _by_head(batch, seed):
    """Gaps of other sizes and signs in heads beside each other."""
    s = Setup("fused", batch, 130, 4, 2, 96, seed=seed)
    first, last = min(s.planes), max(s.planes)
    for h, gap in enumerate((0, 26, -26, 12)):
        for _, scales in s.planes[last if gap > 0 else first]:
            scales[:, h] *= 2.0 ** abs(gap)
        for i in ((1, 3) if gap > 0 else (0, 2)):
            s.w[i][h] *= 2.0 ** -abs(gap)
    return s


def test_decode_of_heads_whose_sources_lie_apart_each_in_its_way():
    s = _by_head(3, 5)
    check_decode(s, [130, 1, 66])
    s.close()


@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("gap,how", APART)
def test_prefill_of_sources_whose_scales_are_far_apart(gap, how, D):
    """What a source brings counts by its scales times its weights."""
    s = Setup("fused", 1, 300, 2, 2, D, seed=D + gap)
    _apart(s, gap, how)
    check_prefill(s, 0, 300, what="%s 2^%d" % (how, gap))
    s.close()


def test_prefill_of_heads_whose_sources_lie_apart_each_in_its_way():
    s = _by_head(1, 6)
    check_prefill(s, 0, 130)
    s.close()


@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("gap", [18, -18])
def test_prefill_beside_a_source_of_zeros_whose_scales_are_larger(gap, D):
    """The other source's rows keep what fp16 has below the frame of their block.  With S the larger of
    the sources' scales times the powers of two above their heads' largest weights, elements are held
    in units of S / 64; a ratio of scales (a power of two) is exact; a code times it is off by 2^-25
    below fp16's normal range, times a weight of up to 2^4; the product and the sum by 2^-25 each; and a
    weight by 2^-25 / 2^4 of that power of two, below the normal range, times its own scale and code."""
    s = Setup("fused", 1, 300, 2, 2, D, seed=D + gap)
    _apart(s, gap, "zeros")
    C, h = 300, 2.0 ** -11
    q = s.query(1, 4, C, D)
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_prefill_attn(q, s.layer, "fused", C, out)
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    K, V = s.rows()
    w = [x.double().abs() for x in s.w]
    Ka, Va = reconstruct("fused", w, [values(x).abs() for x in s.k], [values(x).abs() for x in s.v])
    top = [torch.exp2(torch.floor(torch.log2(x.amax(-1))) + 1)[None, :, None] for x in w]
    rows = torch.arange(C, device="cuda") // BLOCK
    off = []
    for p, i in ((s.k, 0), (s.v, 2)):
        a, b = p[0][1].double() * top[i], p[1][1].double() * top[i + 1]
        off.append((torch.maximum(a, b) * (18 * 2.0 ** -25 / 64) + (a + b) * 448 * 2.0 ** -29)[:, :, rows])
    see = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    for g in range(4):
        kh, qq = g // 2, q[0, g].double()
        p = torch.softmax((qq @ K[0, kh].T * s.scale).masked_fill(~see, -math.inf), -1)
        size = (qq.abs() @ Ka[0, kh].T * s.scale).masked_fill(~see, 0.0).amax(-1, keepdim=True)
        keys = (off[0][0, kh][None].expand(C, C).masked_fill(~see, 0.0)).amax(-1, keepdim=True)
        score = (4 * h + (2 * D + 8) * 2.0 ** -23) * size + 2.0 ** -21 + qq.abs().sum(-1, keepdim=True) * s.scale * keys
        pv, ref = p @ Va[0, kh], p @ V[0, kh]
        bound = (2 * score + 5 * h + (C + 64) * 2.0 ** -23) * pv + (p @ off[1][0, kh])[:, None] \
            + C * 2.0 ** -31 * Va[0, kh].max() + 2.0 ** -8 * ref.abs()
        err = (out[0, g].double() - ref).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
    s.close()
