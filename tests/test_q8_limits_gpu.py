"""Calls on 8-bit caches at the ends of their ranges: the largest batches, prefill chunks that few
CTAs share, calls at once on several streams, graphs that share a workspace."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from q8_parity import Setup, attend, check_decode, check_prefill, decode_bound, reconstruct, values

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("mode,D,G,heads,dtype", [("lite", 128, 4, 1, "bf16"), ("fused", 128, 4, 1, "f32"),
                                                  ("fused", 96, 4, 1, "bf16"), ("vanilla", 80, 4, 3, "f32"),
                                                  ("scaled", 64, 1, 2, "bf16")])
def test_decode_of_the_largest_batches(mode, D, G, heads, dtype):
    s = Setup(mode, 1024, 70, heads, G, D, dtype=dtype, seed=D)
    lens = [(37 * b) % 71 for b in range(1024)]
    lens = [x or 70 for x in lens]
    check_decode(s, lens)
    s.close()


def test_decode_of_a_large_batch_with_empty_sequences():
    """Most sequences are empty (and noted): their outputs are zero, the others' are right."""
    s = Setup("lite", 1000, 300, 1, 2, 64, seed=2)
    q = s.query(1000, 2, 64)
    full, _ = check_decode(s, [300] * 1000, q)
    lens = [300 if b % 97 == 5 else 0 for b in range(1000)]
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, "lite", i32(lens), out, s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    there = torch.tensor(lens, device="cuda") > 0
    assert bool((out[~there] == 0).all())
    # the same rows, split over other warps: two calls' roundings, 2^-8 of the output and 2^-11 of
    # sum p |V| <= max |V| each (decode_bound), and half as much again for the sums in fp32
    top = float(s.rows()[1].abs().max())
    d = (out[there].double() - full[there].double()).abs()
    assert bool((d <= 2 * (2.0 ** -8 * full[there].double().abs() + 1.5 * 2.0 ** -11 * top)).all())
    s.close()


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("batch,q_start,C", [(1, 3980, 16), (1, 4090, 1), (3, 2040, 50), (1, 1000, 300)])
def test_prefill_chunks_of_few_rows(mode, D, batch, q_start, C):
    """Few units and rows behind many keys: several CTAs take a share of the keys each."""
    s = Setup(mode, batch, 4096, 1, 2, D, seed=D + C)
    check_prefill(s, q_start, C, what="%s %d" % (mode, D))
    s.close()


@pytest.mark.parametrize("window,ring", [(1, 0), (33, 0), (900, 0), (2000, 0), (40, 128), (1500, 2048)])
def test_prefill_chunks_of_few_rows_in_windows(window, ring):
    s = Setup("fused", 1, 4096, 1, 1, 64, window=window, ring=ring, seed=7)
    check_prefill(s, 3500, 30, what="window %d ring %d" % (window, ring))
    s.close()


@pytest.mark.parametrize("which", ["k", "v"])
def test_prefill_chunks_of_few_rows_with_rows_that_are_no_numbers(which):
    s = Setup("fused", 1, 4096, 1, 1, 64, seed=8)
    q = s.query(1, 1, 16, 64)
    clean, _ = check_prefill(s, 4000, 16, q)
    plane = getattr(s, which)[0][0].view(torch.uint8)
    for t in (0, 600, 3999, 4007, 4015, 4016):
        old = int(plane[0, 0, t, 3])
        plane[0, 0, t, 3] = 0x7F
        out = torch.empty_like(q)
        s.ctx.fkv_prefill_attn_chunk(q, s.layer, "fused", 4000, 16, out)
        plane[0, 0, t, 3] = old
        sees = torch.arange(4000, 4016, device="cuda") >= t
        assert bool(out[:, :, sees].isnan().all()), t
        assert torch.equal(out[:, :, ~sees], clean[:, :, ~sees]), t
    s.close()


@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_shared_chunks_whose_waits_run_out(mode):
    s = Setup(mode, 1, 4096, 1, 1, 64, seed=9)
    q = s.query(1, 1, 16, 64)
    s.ctx.fkv_set_wait_limit(0)
    s.ctx.fkv_prefill_attn_chunk(q, s.layer, mode, 4000, 16, torch.empty_like(q))
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    s.ctx.fkv_set_wait_limit(1000000000)
    check_prefill(s, 4000, 16, q)
    s.close()


def test_calls_at_once_on_two_streams():
    """Decode with a workspace each, prefill and read-back of one context on two streams: as alone."""
    s = Setup("fused", 4, 3000, 2, 2, 64, seed=10)
    lens = i32([3000, 1, 77, 2048])
    pos = i32([0, 5, 100, 2000])
    qs = [(s.query(4, 4, 64), s.query(4, 4, 200, 64)) for _ in range(2)]

    def calls(q1, q2, ws):
        out = torch.empty_like(q1), torch.empty_like(q2), s.query(4, 2, 300, 64), s.query(4, 2, 300, 64)
        s.ctx.fkv_decode_attn(q1, s.layer, "fused", lens, out[0], ws)
        s.ctx.fkv_prefill_attn_chunk(q2, s.layer, "fused", 2500, 200, out[1])
        s.ctx.fkv_read_kv(s.layer, "fused", pos, out[2], out[3])
        return out

    spaces = [s.ctx.workspace() for _ in range(2)]
    alone = [calls(*q, ws) for q, ws in zip(qs, spaces)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for q, ws, st in zip(qs, spaces, streams):
            with torch.cuda.stream(st):
                got.append(calls(*q, ws))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.close()


def test_graphs_that_share_a_workspace():
    """Two captured decode steps of other lengths, replayed in turn on one stream."""
    s = Setup("lite", 2, 3000, 2, 2, 128, seed=12)
    ws = s.ctx.workspace()
    qs = [s.query(2, 4, 128) for _ in range(2)]
    lens = [i32([3000, 17]), i32([1, 2900])]
    want, outs, graphs = [], [], []
    for q, L in zip(qs, lens):
        want.append(torch.empty_like(q))
        s.ctx.fkv_decode_attn(q, s.layer, "lite", L, want[-1], ws)
    for q, L in zip(qs, lens):
        outs.append(torch.empty_like(q))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.ctx.fkv_decode_attn(q, s.layer, "lite", L, outs[-1], ws)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    s.close()


def test_planes_that_start_inside_an_allocation():
    """Codes, scales, queries and outputs at the smallest alignment that a call takes, with canaries
    around the outputs."""
    D, H, batch, seq = 80, 1, 2, 100
    s = Setup("vanilla", batch, seq, H, 1, D, seed=13)
    (kc, ks), (vc, vs) = s.planes[2]

    def move(t):
        raw = torch.full((t.numel() * t.element_size() + 48,), 0x55, dtype=torch.uint8, device="cuda")
        new = raw[16:16 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        new.view(torch.uint8).copy_(t.view(torch.uint8))
        return new, raw

    whole = [move(t) for t in (kc, vc, ks, vs)]
    s.ctx.fkv_bind_layer_cache_q8(2, *[t for t, _ in whole])
    q, qp = s.query(batch, H, D), s.query(batch, H, 20, D)
    a, b = torch.empty_like(q), torch.empty_like(qp)
    (qm, _), (am, ra), (qpm, _), (bm, rb) = move(q), move(a), move(qp), move(b)
    lens = i32([100, 33])
    ws = s.ctx.workspace()
    s.ctx.fkv_decode_attn(q, 2, "vanilla", lens, a, ws)
    s.ctx.fkv_prefill_attn_chunk(qp, 2, "vanilla", 80, 20, b)
    s.ctx.fkv_decode_attn(qm, 2, "vanilla", lens, am, ws)
    s.ctx.fkv_prefill_attn_chunk(qpm, 2, "vanilla", 80, 20, bm)
    new, pos = s.query(batch, H, 7, D), i32([50, 60])
    s.ctx.fkv_append_kv(2, new, new, pos)
    back = [move(torch.zeros_like(new)) for _ in range(2)]
    s.ctx.fkv_read_kv(2, "vanilla", pos, back[0][0], back[1][0])
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert torch.equal(a, am) and torch.equal(b, bm) and torch.equal(back[0][0], back[1][0])
    for _, raw in whole + [(am, ra), (bm, rb)] + back:
        assert bool((raw[:16] == 0x55).all()) and bool((raw[-32:] == 0x55).all())
    s.close()


def _far_apart(s):
    """Values of about 2^30, beside a block of zeros with the scale that appended zeros have, one
    with codes but no scale (never written), and keys without a scale."""
    for l, ((kc, ks), (vc, vs)) in s.planes.items():
        vs *= 2.0 ** 30
        vc.view(torch.uint8)[:, :, 64:96] = 0
        vs[:, :, 2] = 2.0 ** -100
        vs[:, :, 4] = ks[:, :, 4] = ks[:, :, 1] = 0


@pytest.mark.parametrize("mode,dtype", [("vanilla", "bf16"), ("lite", "f32"), ("scaled", "bf16"), ("fused", "bf16"),
                                        ("fused", "f32")])
def test_decode_blocks_of_zeros_beside_large_values(mode, dtype):
    s = Setup(mode, 2, 300, 2, 2, 96, dtype=dtype, seed=14)
    _far_apart(s)
    check_decode(s, [300, 100])
    s.close()


@pytest.mark.parametrize("mode", ["vanilla", "scaled", "fused"])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_prefill_blocks_of_zeros_beside_large_values(mode, D):
    s = Setup(mode, 1, 300, 2, 2, D, seed=14)
    _far_apart(s)
    check_prefill(s, 20, 280)
    s.close()


@pytest.mark.parametrize("mode", ["vanilla", "fused"])
def test_caches_that_were_never_written_read_as_zeros(mode):
    s = Setup(mode, 2, 300, 2, 2, 64, seed=15)
    for planes in s.planes.values():
        for codes, scales in planes:
            codes.view(torch.uint8).zero_()
            scales.zero_()
    q, qp = s.query(2, 4, 64), s.query(2, 4, 300, 64)
    out, outp = torch.full_like(q, float("nan")), torch.full_like(qp, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, mode, i32([300, 33]), out, s.ctx.workspace())
    s.ctx.fkv_prefill_attn(qp, s.layer, mode, 300, outp)
    assert bool((out == 0).all()) and bool((outp == 0).all())
    # and one written block counts beside them
    new, pos = s.query(2, 2, 1, 64), i32([200, 32])
    for l in s.planes:
        s.ctx.fkv_append_kv(l, new, new, pos)
    check_decode(s, [300, 33], q)
    check_prefill(s, 0, 300, qp)
    s.close()


@pytest.mark.parametrize("mode", ["vanilla", "fused"])
def test_values_of_tiny_scales(mode):
    """Smaller than attention keeps: no more than the values themselves, and numbers."""
    s = Setup(mode, 1, 300, 2, 2, 64, seed=16)
    for _, (vc, vs) in s.planes.values():
        vs *= 2.0 ** -80
    top = float(s.rows()[1].abs().max()) * 1.01
    q, qp = s.query(1, 4, 64), s.query(1, 4, 300, 64)
    out, outp = torch.full_like(q, float("nan")), torch.full_like(qp, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, mode, i32([300]), out, s.ctx.workspace())
    s.ctx.fkv_prefill_attn(qp, s.layer, mode, 300, outp)
    assert bool((out.abs() <= top).all()) and bool((outp.abs() <= top).all())
    s.close()


def test_decode_of_no_rows_at_all():
    s = Setup("lite", 3, 300, 2, 2, 64, seed=17)
    q = s.query(3, 4, 64)
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, "lite", i32([0, 0, 0]), out, s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    assert bool((out == 0).all())
    s.close()


@pytest.mark.parametrize("mode,D,window,ring", [("fused", 80, 0, 0), ("fused", 128, 300, 352), ("scaled", 96, 0, 0),
                                                ("vanilla", 64, 500, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_any_scales_and_steep_scores(mode, D, window, ring, dtype):
    """Scales that are no powers of two, up to 2^18 apart, and scores of hundreds.  Two sources
    round P each for itself then, so a rounding is relative to the sums of both sources' magnitudes
    (of scores and of values), which may cancel; and what falls below 2^-31 of the largest weight
    times value scale may vanish: at most 2^-31 of the largest value for each of n keys."""
    s = Setup(mode, 3, 1500, 2, 2, D, dtype=dtype, window=window, ring=ring, seed=18, spread=3.0, powers=False,
              softmax_scale=0.5)
    lens = [1500, 700, 33]
    q = s.query(3, 4, D)
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, mode, i32(lens), out, s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    K, V = s.rows()
    Ka, Va = reconstruct(mode, [x.abs() for x in s.w], [values(x).abs() for x in s.k], [values(x).abs() for x in s.v])
    for b, L in enumerate(lens):
        pos = torch.arange(max(0, L - window) if window else 0, L, device="cuda")
        at = pos % ring if ring else pos
        for h in range(2):
            qq = q[b, 2 * h:2 * h + 2].double()
            see = torch.ones(2, len(pos), dtype=torch.bool, device="cuda")
            ref, _, _ = attend(qq, K[b, h, at], V[b, h, at], s.scale, see)
            p = torch.softmax(qq @ K[b, h, at].T * s.scale, -1)
            size = (qq.abs() @ Ka[b, h, at].T * s.scale).amax(-1, keepdim=True)
            bound = decode_bound(ref, size, p @ Va[b, h, at], D, len(pos), dtype)
            bound = bound + len(pos) * 2.0 ** -31 * Va[b, h, at].max()
            assert bool(((out[b, 2 * h:2 * h + 2].double() - ref).abs() <= bound).all()), (b, h)
    s.close()
