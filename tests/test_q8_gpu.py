"""8-bit caches on the GPU through the C ABI: the quantising append against the oracle (codes and
scales exactly), reading rows back, and decode attention against float64 with derived bounds."""

import numpy as np
import pytest
import torch

import oracle as O
from cross_layer_kv_gb300 import fusedkv as B
from q8_parity import BLOCK, Setup, attend, check_decode, cols, decode_bound, make_plane, reconstruct, values

pytestmark = pytest.mark.gpu
DIMS = [64, 80, 96, 128]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

class Cache:
    """One bound 8-bit layer of a context."""

    def __init__(self, batch, heads, seq, D, dtype="bf16", ring=0, seed=0, spread=1.0, powers=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx = B.Context(4, batch, seq, heads, heads, D, dtype)
        rows = ring or seq
        if ring:
            self.ctx.fkv_set_ring_rows(1, ring)
        self.k, self.v = (make_plane(g, batch, heads, rows, D, spread, powers=powers) for _ in range(2))
        self.ctx.fkv_bind_layer_cache_q8(1, self.k[0], self.v[0], self.k[1], self.v[1])
        self.gen, self.dt = g, torch.float32 if dtype == "f32" else torch.bfloat16

    def new(self, T, size=1.0):
        c = self.ctx.cfg
        shape = (c.batch, c.num_kv_heads, T, c.head_dim)
        k = torch.exp2(torch.randn(c.batch, c.num_kv_heads, 1, 1, generator=self.gen, device="cuda") * 3)
        return (torch.randn(shape, generator=self.gen, device="cuda") * k * size).to(self.dt)

    def check(self, kn, vn, pos):
        """Append and compare codes and scales with the oracle; rows that the format gives up are skipped."""
        before = [(u8(x[0]), x[1].cpu().numpy()) for x in (self.k, self.v)]
        self.ctx.fkv_append_kv(1, kn, vn, i32(pos))
        assert self.ctx.fkv_get_device_status() == B.FKV_OK
        for (c0, s0), x, new in zip(before, (self.k, self.v), (kn, vn)):
            codes, scales, kept = O.q8_append(c0, s0, new.double().cpu().numpy(), pos)
            np.testing.assert_array_equal(x[1].cpu().numpy(), scales)
            got = u8(x[0])
            for b in range(got.shape[0]):
                np.testing.assert_array_equal(got[b][:, kept[b]], codes[b][:, kept[b]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 100])
def test_append_matches_oracle(D, T, dtype):
    c = Cache(4, 3, 200, D, dtype, seed=D + T)
    c.check(c.new(T), c.new(T, 0.01), [0, 33, 64, 200 - T])
    c.check(c.new(T, 50.0), c.new(T), [5, 31, 63, 199 - T])


@pytest.mark.parametrize("T", [1, 40, 65])
def test_append_over_a_ring(T):
    c = Cache(3, 2, 1000, 64, ring=96, seed=T)
    for pos in ([0, 95, 96], [97, 500, 1000 - T], [31, 64, 191]):
        c.check(c.new(T), c.new(T, 20.0), pos)


def test_append_scales_of_a_caller():
    """Scales that are not powers of two, on the cache before the append."""
    c = Cache(2, 2, 128, 96, seed=5, powers=False)
    c.check(c.new(3, 100.0), c.new(3, 1e-3), [10, 77])


def test_append_token_by_token():
    c = Cache(2, 2, 70, 64, seed=9)
    kn, vn = c.new(70), c.new(70)
    grow = torch.exp2(torch.arange(70, device="cuda") % 32 / 4)[:, None]
    kn = (kn * grow).to(torch.bfloat16)
    for t in range(70):
        c.check(kn[:, :, t:t + 1].contiguous(), vn[:, :, t:t + 1].contiguous(), [t, t])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_extremes(dtype):
    """Zeros, infinities, NaN, the largest and the smallest values, stale scales that are not numbers."""
    c = Cache(1, 1, 160, 64, dtype, seed=3)
    top = torch.finfo(c.dt).max
    x = c.new(8)
    x[0, 0, 0] = 0
    x[0, 0, 1, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
    v = c.new(8)
    v[0, 0, 2, 0] = top
    v[0, 0, 3, 0] = -top
    c.check(x, v, [0])
    tiny = torch.full_like(x, 1e-38)
    c.check(tiny, torch.zeros_like(x), [32])
    c.check(torch.full_like(x, float("nan")), torch.full_like(x, float("inf")), [64])
    for s in (c.k[1], c.v[1]):
        s[0, 0, 3:] = float("nan")
    c.check(c.new(8), c.new(8), [96])            # a block's first row: its old scale is not read
    got = u8(c.k[0])[0, 0, 1, :4]
    assert list(got[:3]) == [0x7F, 0x7F, 0x7F]


def test_append_joins_a_block_whose_scale_is_no_number():
    """A scale that no append made (uninitialised memory): the new rows are right all the same."""
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        c = Cache(1, 1, 64, 64, seed=4)
        c.k[1][0, 0, 0] = bad
        kn, vn = c.new(2), c.new(2)
        c.ctx.fkv_append_kv(1, kn, vn, i32([3]))
        s = O.q8_need(float(kn.abs().max()))
        assert float(c.k[1][0, 0, 0]) == s
        np.testing.assert_array_equal(u8(c.k[0])[0, 0, 3:5], O.e4m3_encode(kn[0, 0].double().cpu().numpy() / s))


def test_append_out_of_range_skipped_and_flagged():
    c = Cache(4, 2, 64, 64, seed=6)
    before = [x.clone() for p in (c.k, c.v) for x in (p[0].view(torch.uint8), p[1])]
    kn, vn = c.new(3), c.new(3)
    c.ctx.fkv_append_kv(1, kn, vn, i32([-1, 62, 1 << 30, 2147483647]))
    assert c.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    after = [c.k[0].view(torch.uint8), c.k[1], c.v[0].view(torch.uint8), c.v[1]]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    c.ctx.fkv_append_kv(1, kn[:, :, :0].contiguous(), vn[:, :, :0].contiguous(), i32([0] * 4))
    assert c.ctx.fkv_get_device_status() == B.FKV_OK


def test_append_leaves_other_rows_alone():
    """Blocks that the call does not touch, and the padding scales, keep their bytes."""
    c = Cache(2, 2, 200, 80, seed=7)
    k0, s0 = u8(c.k[0]).copy(), c.k[1].cpu().numpy().copy()
    c.ctx.fkv_append_kv(1, c.new(40), c.new(40), i32([70, 64]))     # blocks 2 and 3
    got, s = u8(c.k[0]), c.k[1].cpu().numpy()
    for rows in (slice(0, 64), slice(128, 200)):
        np.testing.assert_array_equal(got[:, :, rows], k0[:, :, rows])
    np.testing.assert_array_equal(s[:, :, [0, 1, 4, 5, 6, 7]], s0[:, :, [0, 1, 4, 5, 6, 7]])


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------

def _read(s, pos, T):
    shape = (s.batch, s.H, T, s.D)
    k, v = (torch.full(shape, 7.0, dtype=s.torch_dtype, device="cuda") for _ in range(2))
    s.ctx.fkv_read_kv(s.layer, s.mode, i32(pos), k, v)
    return k, v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["vanilla", "lite", "scaled", "fused"])
@pytest.mark.parametrize("D", DIMS)
def test_read_matches_definition(D, mode, dtype):
    s = Setup(mode, 3, 150, 2, 1, D, dtype, seed=D, powers=D != 80)
    K, V = s.rows()
    Ks = sum(values(x).abs() for x in s.k) * 2       # weights below 2 in magnitude
    Vs = sum(values(x).abs() for x in s.v) * 2
    for pos, T in (([0, 1, 149], 1), ([0, 33, 50], 100), ([0, 0, 0], 150)):
        for got, ref, size in zip(_read(s, pos, T), (K, V), (Ks, Vs)):
            u = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
            for b, p in enumerate(pos):
                # value * scale, its product and the sum round once each in fp32; then the output
                bound = u * ref[b, :, p:p + T].abs() + 3 * 2.0 ** -24 * size[b, :, p:p + T] * 2
                assert bool(((got[b].double() - ref[b, :, p:p + T]).abs() <= bound).all()), (pos, T, b)
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.close()


def test_read_out_of_range_and_empty():
    s = Setup("lite", 3, 64, 2, 2, 64)
    k, v = _read(s, [-1, 62, 61], 3)
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    assert bool((k[:2] == 7).all()) and bool((v[:2] == 7).all()) and not bool((k[2] == 7).all())
    s.ctx.fkv_read_kv(s.layer, s.mode, i32([0] * 3), k[:, :, :0].contiguous(), v[:, :, :0].contiguous())
    for T in (65,):
        with pytest.raises(B.FkvError) as e:
            _read(s, [0] * 3, T)
        assert e.value.status == B.FKV_ERR_INVALID_ARG
    s.close()


def test_read_over_a_ring():
    s = Setup("fused", 2, 500, 2, 1, 96, ring=64, window=30)
    K, V = s.rows()
    k, v = _read(s, [70, 436], 64)
    for b, p in enumerate((70, 436)):
        at = torch.arange(p, p + 64, device="cuda") % 64
        assert float((k[b].double() - K[b][:, at]).abs().max()) <= 2.0 ** -8 * float(K.abs().max())
        assert float((v[b].double() - V[b][:, at]).abs().max()) <= 2.0 ** -8 * float(V.abs().max())
    s.close()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_read_other_formats(fmt, D):
    """Plain rows come back as they are; 4-bit rows as their codes say; fused over both."""
    batch, heads, seq = 2, 2, 40
    g = torch.Generator(device="cuda").manual_seed(D)
    ctx = B.Context(4, batch, seq, heads, heads, D, "f32" if fmt == "f32" else "bf16")
    dt = ctx.torch_dtype
    vals = {}
    for l in (1, 2):
        x = [torch.randn(batch, heads, seq, D, generator=g, device="cuda").to(dt) for _ in range(2)]
        if fmt == "q4":
            recs = [torch.from_numpy(O.q4_pack(*O.q4_quantize(t.float().cpu().numpy()))).cuda() for t in x]
            ctx.fkv_bind_layer_cache_q4(l, *recs)
            vals[l] = [torch.from_numpy(O.q4_dequantize_records(r.cpu().numpy(), D)).cuda() for r in recs]
            vals[l, "keep"] = recs
        else:
            ctx.fkv_bind_layer_cache(l, *x)
            vals[l] = [t.double() for t in x]
            vals[l, "keep"] = x
    w = [torch.randn(heads, D, generator=g, device="cuda") for _ in range(4)]
    ctx.fkv_set_fusion_weights(4, *w)
    k, v = (torch.empty(batch, heads, 9, D, dtype=dt, device="cuda") for _ in range(2))
    u = 2.0 ** -24 if fmt == "f32" else 2.0 ** -8
    for layer, mode in ((1, "vanilla"), (4, "lite"), (4, "scaled"), (4, "fused")):
        ctx.fkv_read_kv(layer, mode, i32([0, 31]), k, v)
        src = {"vanilla": ([1], [1]), "lite": ([2], [1]), "scaled": ([2], [1]), "fused": ([1, 2], [1, 2])}[mode]
        K, V = reconstruct(mode, w, [vals[l][0] for l in src[0]], [vals[l][1] for l in src[1]])
        size = (sum(vals[l][i].abs() for l in (1, 2) for i in (0, 1)) + 1) * max(1.0, float(max(x.abs().max() for x in w)))
        for got, ref in ((k, K), (v, V)):
            for b, p in enumerate((0, 31)):
                r = ref[b, :, p:p + 9]
                if mode in ("vanilla", "lite") and fmt != "q4":
                    assert torch.equal(got[b].double(), r)
                bound = u * r.abs() + 4 * 2.0 ** -24 * size[b, :, p:p + 9]
                assert bool(((got[b].double() - r).abs() <= bound).all())
    ctx.close()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("mode", ["vanilla", "lite", "scaled", "fused"])
def test_decode_matches_reference(mode, D, G, dtype):
    s = Setup(mode, 5, 300, 2, G, D, dtype, seed=D + G)
    check_decode(s, [1, 33, 127, 300, 2], what="%s D=%d G=%d %s" % (mode, D, G, dtype))
    s.close()


@pytest.mark.parametrize("mode,D,G,seq,heads,batch", [
    ("lite", 64, 2, 8192, 8, 3), ("fused", 80, 2, 20000, 3, 2), ("vanilla", 128, 4, 5001, 4, 3),
    ("fused", 96, 4, 3000, 5, 4), ("scaled", 96, 1, 9999, 1, 1), ("fused", 64, 1, 70000, 1, 1)])
def test_decode_long_and_ragged(mode, D, G, seq, heads, batch):
    s = Setup(mode, batch, seq, heads, G, D, seed=seq, spread=2.0)
    lens = [seq] + [(seq * (i + 1)) // (batch + 1) + i for i in range(batch - 1)]
    check_decode(s, lens, what="long")
    s.close()


@pytest.mark.parametrize("ctas", [1, 2, 7, 152, 400])
def test_decode_grids(ctas):
    s = Setup("fused", 3, 700, 3, 2, 80, seed=ctas, decode_ctas=ctas)
    check_decode(s, [700, 5, 351])
    s.close()


@pytest.mark.parametrize("mode", ["vanilla", "fused"])
@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("window,ring", [(1, 0), (100, 0), (600, 0), (1, 32), (33, 64), (97, 128), (300, 352), (500, 896)])
def test_decode_windows_and_rings(window, ring, D, mode):
    s = Setup(mode, 4, 2000, 2, 2, D, window=window, ring=ring, seed=window)
    check_decode(s, [1, 50, 1031, 2000], what="window %d ring %d" % (window, ring))
    s.close()


def test_decode_scales_of_a_caller():
    s = Setup("fused", 2, 200, 2, 2, 64, powers=False, seed=8)
    check_decode(s, [200, 77])
    s.close()


def test_decode_softmax_scale_and_large_scores():
    s = Setup("lite", 2, 200, 2, 2, 64, seed=8, softmax_scale=3.0)
    check_decode(s, [200, 77])
    s.close()


def test_decode_empty_and_bad_lengths():
    s = Setup("fused", 4, 100, 2, 2, 64, seed=1)
    q = s.query(4, 4, 64)
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, "fused", i32([0, -3, 100, 101]), out, s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    assert bool((out[:2] == 0).all()) and bool(out[2:].isfinite().all())
    s.close()


def test_decode_does_not_use_what_lies_behind_the_length():
    """Codes and scales that are not numbers behind the last row, or before a window, change nothing."""
    for window in (0, 40):
        s = Setup("fused", 2, 256, 2, 2, 80, seed=2, window=window)
        lens = [130, 97]
        q = s.query(2, 4, 80)
        a, _ = check_decode(s, lens, q)
        for k, v in s.planes.values():
            for codes, scales in (k, v):
                for b, L in enumerate(lens):
                    codes.view(torch.uint8)[b, :, L:] = 0x7F
                    scales[b, :, (L + BLOCK - 1) // BLOCK:] = float("nan")
                    if window:
                        codes.view(torch.uint8)[b, :, :L - window] = 0x7F
                        scales[b, :, :(L - window) // BLOCK] = float("inf")
        out = torch.empty_like(q)
        s.ctx.fkv_decode_attn(q, s.layer, s.mode, i32(lens), out, s.ctx.workspace())
        assert torch.equal(a, out)
        s.close()


def test_decode_rows_that_are_not_finite():
    s = Setup("vanilla", 2, 100, 2, 2, 64, seed=2)
    s.k[0][0].view(torch.uint8)[0, 0, 50, 3] = 0x7F
    s.v[0][0].view(torch.uint8)[0, 1, 60, 5] = 0xFF
    q = s.query(2, 4, 64)
    out = torch.empty_like(q)
    s.ctx.fkv_decode_attn(q, s.layer, s.mode, i32([100, 100]), out, s.ctx.workspace())
    assert bool(out[0, :2].isnan().all())
    assert bool(out[0, 2:, 5].isnan().all()) and bool(out[0, 2:, :5].isfinite().all())
    assert bool(out[1].isfinite().all())
    s.close()


def test_decode_noalloc_and_graph():
    s = Setup("fused", 3, 500, 2, 2, 96, seed=3)
    lens = i32([500, 77, 250])
    q = s.query(3, 4, 96)
    ws = s.ctx.workspace()
    a, b = torch.empty_like(q), torch.empty_like(q)
    s.ctx.fkv_decode_attn(q, s.layer, "fused", lens, a, ws)
    s.ctx.fkv_decode_attn_noalloc(q, s.layer, "fused", lens, b)
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            s.ctx.fkv_decode_attn(q, s.layer, "fused", lens, out, ws)
    for seed in range(3):
        q.copy_(s.query(3, 4, 96))
        graph.replay()
        torch.cuda.synchronize()
        s.ctx.fkv_decode_attn(q, s.layer, "fused", lens, a, ws)
        torch.cuda.synchronize()
        assert torch.equal(a, out)
    s.close()


def test_a_captured_decode_step_appends_and_attends():
    """Append, read-back and attention of a step, captured once and replayed as the sequences grow."""
    D, H, batch, seq = 64, 2, 2, 96
    s = Setup("lite", batch, seq, H, 2, D, seed=11, layers=2)      # one storage layer
    lens, pos = i32([40, 62]), i32([39, 61])
    kn, vn = s.query(batch, H, 1, D), s.query(batch, H, 1, D)
    q, ws = s.query(batch, H * 2, D), s.ctx.workspace()
    out, k1, v1 = torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
    planes = s.planes[1]
    host = [(u8(c), x.cpu().numpy().astype(np.float64)) for c, x in planes]

    def step():
        s.ctx.fkv_append_kv(1, kn, vn, pos)
        s.ctx.fkv_read_kv(2, "lite", pos, k1, v1)
        s.ctx.fkv_decode_attn(q, 2, "lite", lens, out, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(6):
        kn.copy_(s.query(batch, H, 1, D) * 2.0 ** t)
        vn.copy_(s.query(batch, H, 1, D))
        q.copy_(s.query(batch, H * 2, D))
        graph.replay()
        at = pos.tolist()
        host = [O.q8_append(c, x, n.double().cpu().numpy(), at)[:2] for (c, x), n in zip(host, (kn, vn))]
        K, V = (torch.from_numpy(O.q8_values(c, x)).cuda() for c, x in host)
        for b, p in enumerate(at):
            assert torch.equal(k1[b, :, 0].double(), K[b, :, p]) and torch.equal(v1[b, :, 0].double(), V[b, :, p])
            for h in range(H):
                see = torch.ones(2, p + 1, dtype=torch.bool, device="cuda")
                ref, size, pv = attend(q[b, 2 * h:2 * h + 2].double(), K[b, h, :p + 1], V[b, h, :p + 1], s.scale, see)
                bound = decode_bound(ref, size, pv, D, p + 1, "bf16")
                assert bool(((out[b, 2 * h:2 * h + 2].double() - ref).abs() <= bound).all())
        pos += 1
        lens += 1
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.close()


def test_offsets_past_32_bits():
    """The last sequence of planes of more than 2^32 codes."""
    batch, H, seq, D = 40, 8, 131072, 128
    ctx = B.Context(2, batch, seq, H, H, D, "bf16")
    planes = [(torch.empty(batch, H, seq, D, dtype=torch.uint8, device="cuda"),
               torch.empty(batch, H, cols(seq), device="cuda")) for _ in range(2)]
    assert planes[0][0].numel() > 2 ** 32
    ctx.fkv_bind_layer_cache_q8(1, planes[0][0], planes[1][0], planes[0][1], planes[1][1])
    T = 300
    g = torch.Generator(device="cuda").manual_seed(0)
    kn, vn = (torch.randn(batch, H, T, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = [0] * (batch - 1) + [seq - T]
    start = (seq - T) // BLOCK * BLOCK
    for codes, scales in planes:
        codes[-1, :, start:] = 0
        scales[-1, :, start // BLOCK:] = 2.0 ** -9
    ctx.fkv_append_kv(1, kn, vn, i32(pos))
    k, v = torch.empty_like(kn), torch.empty_like(vn)
    ctx.fkv_read_kv(1, "vanilla", i32(pos), k, v)
    # appended values keep 4 significant bits
    assert bool(((k - kn).abs().float() <= kn.abs().float() * 2.0 ** -4 + 2.0 ** -16).all())
    assert bool(((v - vn).abs().float() <= vn.abs().float() * 2.0 ** -4 + 2.0 ** -16).all())
    ctx.fkv_set_window(1, T)
    q = torch.randn(batch, H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    lens = [T] * (batch - 1) + [seq]
    ctx.fkv_decode_attn(q, 1, "vanilla", i32(lens), out, ctx.workspace())
    assert ctx.fkv_get_device_status() == B.FKV_OK
    for b in (0, batch - 2, batch - 1):
        for h in (0, H - 1):
            see = torch.ones(1, T, dtype=torch.bool, device="cuda")
            ref, size, pv = attend(q[b, h:h + 1].double(), k[b, h].double(), v[b, h].double(), D ** -0.5, see)
            assert bool(((out[b, h:h + 1].double() - ref).abs() <= decode_bound(ref, size, pv, D, T, "bf16")).all())
    ctx.close()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _status(call):
    with pytest.raises(B.FkvError) as e:
        call()
    return e.value.status


def test_refusals():
    s = Setup("fused", 2, 128, 2, 2, 64)
    ctx, D = s.ctx, 64
    lib, h = ctx._lib, ctx.handle
    bind = lib.fkv_bind_layer_cache_q8
    assert bind(h, 0, 16, 16, 16, 16) == bind(h, 7, 16, 16, 16, 16) == B.FKV_ERR_INVALID_ARG
    assert bind(h, 4, 16, 16, 16, 16) == B.FKV_ERR_UNSUPPORTED            # upper layers store nothing
    for bad in ((None, 16, 16, 16), (16, None, 16, 16), (16, 16, None, 16), (16, 16, 16, None), (8, 16, 16, 16),
                (16, 24, 16, 16), (16, 16, 4, 16), (16, 16, 16, 8)):
        assert bind(h, 1, *bad) == B.FKV_ERR_INVALID_ARG
    assert [lib.fkv_q8_scale_cols(r) for r in (-1, 0, 1, 32, 128, 129, 8192)] == [0, 0, 4, 4, 4, 8, 256]
    q = s.query(2, 4, 3, D)
    lens = i32([3, 3])
    mask = torch.ones(2, 3, 1, dtype=torch.int64, device="cuda")
    tree = lambda: ctx.fkv_tree_attn(q, 6, "fused", lens, mask, torch.empty_like(q), ctx.tree_workspace(3))
    assert _status(tree) == B.FKV_ERR_UNSUPPORTED
    assert _status(lambda: ctx.fkv_compact_rows(lens, i32([[0], [0]]), lens)) == B.FKV_ERR_UNSUPPORTED
    assert _status(lambda: ctx.fkv_reorder_seqs(i32([0, 0]), lens)) == B.FKV_ERR_UNSUPPORTED
    # a mix of formats
    plain = torch.zeros(2, 2, 128, D, dtype=torch.bfloat16, device="cuda")
    ctx.fkv_bind_layer_cache(1, plain, plain)
    q1 = s.query(2, 4, D)
    decode = lambda: ctx.fkv_decode_attn(q1, 6, "fused", lens, torch.empty_like(q1), ctx.workspace())
    assert _status(decode) == B.FKV_ERR_UNSUPPORTED
    out = torch.empty(2, 2, 3, D, dtype=torch.bfloat16, device="cuda")
    assert _status(lambda: ctx.fkv_read_kv(6, "fused", lens, out, out.clone())) == B.FKV_ERR_UNSUPPORTED
    read = lib.fkv_read_kv
    a = out.data_ptr()
    for bad in ((None, 1, a, a), (a, -1, a, a), (a, 1, None, a), (a, 1, a, None), (a, 1, a + 8, a), (a + 2, 1, a, a),
                (a, 129, a, a)):
        assert read(h, 3, 0, bad[0], bad[1], bad[2], bad[3], None) == B.FKV_ERR_INVALID_ARG
    assert read(h, 9, 0, a, 1, a, a, None) == B.FKV_ERR_INVALID_ARG
    assert read(None, 1, 0, a, 1, a, a, None) == B.FKV_ERR_INVALID_ARG
    assert read(h, 6, 0, a, 1, a, a, None) == B.FKV_ERR_UNSUPPORTED        # an upper layer's own rows
    s.close()


def test_ring_refusals():
    s = Setup("vanilla", 1, 500, 2, 1, 64, window=33, ring=64)
    q = s.query(1, 2, 64)
    decode = lambda: s.ctx.fkv_decode_attn(q, 2, "vanilla", i32([100]), torch.empty_like(q), s.ctx.workspace())
    decode()
    s.ctx.fkv_set_window(2, 34)                     # a row that the newest block may have taken with it
    assert _status(decode) == B.FKV_ERR_UNSUPPORTED
    s.ctx.fkv_set_window(2, 0)
    assert _status(decode) == B.FKV_ERR_INVALID_ARG
    new = s.query(1, 2, 34, 64)
    assert _status(lambda: s.ctx.fkv_append_kv(2, new, new, i32([0]))) == B.FKV_ERR_INVALID_ARG
    new = s.query(1, 2, 33, 64)
    s.ctx.fkv_append_kv(2, new, new, i32([3]))
    s.ctx.fkv_set_ring_rows(2, 48)                  # not whole blocks
    s.ctx.fkv_set_window(2, 3)
    assert _status(decode) == B.FKV_ERR_UNSUPPORTED
    new = s.query(1, 2, 1, 64)
    assert _status(lambda: s.ctx.fkv_append_kv(2, new, new, i32([0]))) == B.FKV_ERR_UNSUPPORTED
    s.close()
