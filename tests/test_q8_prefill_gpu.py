"""Prefill over 8-bit caches on the GPU through the C ABI, against float64 with derived bounds."""

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from q8_parity import BLOCK, Setup, check_decode, check_prefill, values

pytestmark = pytest.mark.gpu
DIMS = [64, 80, 96, 128]
MODES = ["vanilla", "lite", "scaled", "fused"]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("mode", MODES)
def test_prefill_matches_reference(mode, D, G):
    s = Setup(mode, 2, 400, 2, G, D, seed=D + G)
    check_prefill(s, 0, 400, what="%s D=%d G=%d" % (mode, D, G))
    check_prefill(s, 151, 249, what="chunk %s D=%d G=%d" % (mode, D, G))
    s.close()


@pytest.mark.parametrize("mode,D", [("lite", 64), ("fused", 96), ("fused", 128)])
@pytest.mark.parametrize("q_start,C", [(0, 1), (0, 15), (0, 129), (1, 1), (15, 2), (111, 1), (112, 1), (500, 12), (63, 65),
                                       (127, 257), (639, 1)])
def test_prefill_sizes(q_start, C, mode, D):
    s = Setup(mode, 1, 640, 1, 2, D, seed=C)
    check_prefill(s, q_start, C, what="%d+%d" % (q_start, C))
    s.close()


@pytest.mark.parametrize("mode,D,G,seq", [("lite", 96, 2, 3000), ("fused", 80, 1, 2500), ("fused", 128, 2, 2100),
                                          ("scaled", 128, 4, 1700), ("vanilla", 64, 2, 4096)])
def test_prefill_long(mode, D, G, seq):
    s = Setup(mode, 1, seq, 2, G, D, seed=seq, spread=2.0)
    check_prefill(s, 0, seq, rows=[0, 1, 127, 128, seq // 2, seq - 130, seq - 1])
    s.close()


def test_prefill_scales_far_apart():
    """Blocks whose value and key scales differ by up to 2^30, and a block of zeros."""
    s = Setup("vanilla", 1, 300, 2, 2, 64, seed=5)
    for codes, scales in (s.k[0], s.v[0]):
        scales[:, :, 2] = 2.0 ** -100
        codes.view(torch.uint8)[:, :, 64:96] = 0
    s.v[0][1][:, :, 4] = 2.0 ** -30
    s.v[0][1][:, :, 6] = 2.0 ** 4
    s.k[0][1][:, :, 5] = 2.0 ** -20
    check_prefill(s, 0, 300)
    s.close()


def test_prefill_scales_of_a_caller():
    for mode in ("vanilla", "fused"):
        s = Setup(mode, 1, 300, 2, 2, 80, powers=False, seed=8)
        check_prefill(s, 0, 300)
        s.close()


@pytest.mark.parametrize("size", [1e-30, 1e-4, 1e4, 1e30])
def test_prefill_queries_and_weights_of_any_size(size):
    """Queries of any magnitude (and key weights or scales that bring the scores back)."""
    s = Setup("scaled", 1, 200, 1, 2, 64, seed=8)
    s.w[0] /= size
    s.ctx.fkv_set_fusion_weights(s.layer, *s.w)
    q = (s.query(1, 2, 200, 64).float() * size).to(torch.bfloat16)
    check_prefill(s, 0, 200, q)
    s.close()
    f = Setup("fused", 1, 200, 1, 2, 64, seed=9)
    for i in (0, 1):
        f.w[i] /= size
    for i in (2, 3):
        f.w[i] *= min(size, 1e20)
    f.ctx.fkv_set_fusion_weights(f.layer, *f.w)
    check_prefill(f, 0, 200, (f.query(1, 2, 200, 64).float() * size).to(torch.bfloat16))
    f.close()


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,q_start,C", [(1, 0, 300), (40, 0, 300), (128, 130, 300), (500, 100, 700), (7, 799, 1)])
def test_prefill_windows(window, q_start, C, D, mode):
    s = Setup(mode, 1, 800, 2, 2, D, window=window, seed=window)
    check_prefill(s, q_start, C, what="window %d" % window)
    s.close()


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("D,G", [(64, 2), (80, 1), (128, 2)])
@pytest.mark.parametrize("window,ring,q_start,C", [
    (10, 64, 1000, 20), (10, 64, 20, 24), (10, 64, 30, 24), (33, 96, 555, 33), (200, 512, 1400, 250), (500, 896, 700, 300),
    (100, 160, 1900, 30), (64, 896, 0, 896)])
def test_prefill_over_rings(window, ring, q_start, C, D, G, mode):
    s = Setup(mode, 2, 2000, 2, G, D, window=window, ring=ring, seed=ring)
    check_prefill(s, q_start, C, what="window %d ring %d" % (window, ring))
    s.close()


def test_prefill_does_not_use_what_it_may_not_see():
    """Codes and scales that are not numbers behind the chunk, and before a window."""
    for mode in ("vanilla", "fused"):
        for window in (0, 37):
            s = Setup(mode, 1, 500, 2, 2, 80, window=window, seed=3)
            q = s.query(1, 4, 100, 80)
            a, _ = check_prefill(s, 150, 100, q)
            for plane in s.planes.values():
                for codes, scales in plane:
                    codes.view(torch.uint8)[:, :, 250:] = 0x7F
                    scales[:, :, 8:] = float("nan")
                    if window:
                        codes.view(torch.uint8)[:, :, :114] = 0x7F
                        scales[:, :, :3] = float("nan")
            out = torch.empty_like(q)
            s.ctx.fkv_prefill_attn_chunk(q, s.layer, mode, 150, 100, out)
            assert torch.equal(a, out)
            s.close()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("mode", ["vanilla", "fused"])
@pytest.mark.parametrize("window", [0, 30, 200])
def test_prefill_rows_that_are_not_finite(window, mode, which):
    """A row that is not a number reaches the queries that see it, and no others."""
    s = Setup(mode, 1, 700, 1, 2, 64, window=window, seed=3)
    q_start, C = 100, 600
    q = s.query(1, 2, C, 64)
    clean, _ = check_prefill(s, q_start, C, q)
    for t in (50, 99, 100, 101, 227, 228, 355, 356, 690, 699):
        plane = getattr(s, which)[-1][0].view(torch.uint8)
        old = int(plane[0, 0, t, 5])
        plane[0, 0, t, 5] = 0xFF
        out = torch.empty_like(q)
        s.ctx.fkv_prefill_attn_chunk(q, s.layer, mode, q_start, C, out)
        plane[0, 0, t, 5] = old
        m = torch.arange(q_start, q_start + C, device="cuda")
        sees = (m >= t) & ((m < t + window) if window else True)
        assert bool(out[:, :, sees].isnan().all()), t
        assert torch.equal(out[:, :, ~sees], clean[:, :, ~sees]), t
    s.close()


def test_prefill_then_decode_after_appends():
    """A prompt in three chunks, appended and attended over as it grows, then a token."""
    D, H, G, seq = 96, 2, 2, 500
    s = Setup("fused", 2, seq, H, G, D, seed=21)
    at = 0
    for C in (130, 1, 250):
        for l in (1, 3):
            s.ctx.fkv_append_kv(l, s.query(2, H, C, D), s.query(2, H, C, D), i32([at, at]))
        check_prefill(s, at, C, what="chunk at %d" % at)
        at += C
    for l in (1, 3):
        s.ctx.fkv_append_kv(l, s.query(2, H, 1, D), s.query(2, H, 1, D), i32([at, at]))
    check_decode(s, [at + 1, at + 1])
    s.close()


def test_prefill_captured():
    s = Setup("fused", 1, 300, 2, 2, 64, seed=4)
    q = s.query(1, 4, 200, 64)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    s.ctx.fkv_prefill_attn_chunk(q, s.layer, "fused", 100, 200, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.ctx.fkv_prefill_attn_chunk(q, s.layer, "fused", 100, 200, out)
    for _ in range(2):
        q.copy_(s.query(1, 4, 200, 64))
        graph.replay()
        s.ctx.fkv_prefill_attn_chunk(q, s.layer, "fused", 100, 200, ref)
        assert torch.equal(out, ref)
    s.close()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_waits_that_run_out(mode, D):
    """Decode and prefill calls whose waits give up at once say so, and later calls are right."""
    s = Setup(mode, 2, 600, 2, 2, D, seed=6)
    q1, q2 = s.query(2, 4, D), s.query(2, 4, 600, D)
    s.ctx.fkv_set_wait_limit(0)
    s.ctx.fkv_decode_attn(q1, s.layer, mode, i32([600, 5]), torch.empty_like(q1), s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    s.ctx.fkv_prefill_attn(q2, s.layer, mode, 600, torch.empty_like(q2))
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    s.ctx.fkv_set_wait_limit(1000000000)
    check_decode(s, [600, 5], q1)
    check_prefill(s, 0, 600, q2, rows=[0, 300, 599])
    s.close()


def test_prefill_refusals():
    def status(call):
        with pytest.raises(B.FkvError) as e:
            call()
        return e.value.status

    f = Setup("vanilla", 1, 100, 1, 2, 64, dtype="f32")
    q = f.query(1, 2, 10, 64)
    assert status(lambda: f.ctx.fkv_prefill_attn(q, 2, "vanilla", 10, torch.empty_like(q))) == B.FKV_ERR_UNSUPPORTED
    f.close()
    s = Setup("vanilla", 1, 1000, 1, 2, 64, window=40, ring=128)
    call = lambda q_start, C: s.ctx.fkv_prefill_attn_chunk(s.query(1, 2, C, 64), 2, "vanilla", q_start, C,
                                                           s.query(1, 2, C, 64))
    call(28, 100)                                   # not yet wrapped
    call(200, 58)
    assert status(lambda: call(200, 59)) == B.FKV_ERR_UNSUPPORTED
    assert status(lambda: call(990, 11)) == B.FKV_ERR_INVALID_ARG
    s.ctx.fkv_set_window(2, 0)
    assert status(lambda: call(200, 10)) == B.FKV_ERR_INVALID_ARG
    s.close()
