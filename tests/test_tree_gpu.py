"""fkv_tree_attn on the GPU, through the C ABI, against the float64 oracle
(error bounds: tree_parity.TreeSetup.reference)."""

import numpy as np
import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from parity import f64
from tree_parity import TreeSetup, mask_words

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def _run(what, **kw):
    s = TreeSetup(**kw)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check(what)
    s.ctx.close()


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("mode", ["vanilla", "lite", "scaled", "fused"])
def test_modes_and_dims(fmt, D, mode):
    _run("%s %d %s" % (fmt, D, mode), D=D, mode=mode, fmt=fmt, T=9)


@pytest.mark.parametrize("fmt,G", [("bf16", 1), ("bf16", 4), ("f32", 1), ("f32", 4), ("q4", 1)])
def test_group_sizes(fmt, G):
    _run("G=%d" % G, fmt=fmt, G=G, T=11, H=3)


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 33, 63, 64, 65, 127, 128])
def test_node_numbers(fmt, T):
    _run("T=%d" % T, fmt=fmt, T=T, S=400, lens=(0, 130, 271), D=64, G=2, H=1)


@pytest.mark.parametrize("fmt,T,G", [("bf16", 128, 4), ("bf16", 96, 4), ("bf16", 70, 2), ("f32", 70, 4),
                                     ("q4", 128, 2), ("q4", 40, 2)])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_many_rows(fmt, T, G, mode):
    _run("T=%d G=%d" % (T, G), fmt=fmt, T=T, G=G, mode=mode, S=420, lens=(3, 128, 290), D=128, H=2)


@pytest.mark.parametrize("fmt,Bt", [("bf16", 300), ("f32", 300), ("q4", 300), ("bf16", 1024), ("q4", 1024)])
def test_large_batches(fmt, Bt):
    """The lengths of the batch take shared memory from the tiles."""
    T = 3
    lens = [(7 * b) % 61 for b in range(Bt)]
    counts = [b % (T + 1) for b in range(Bt)]
    _run("B=%d" % Bt, fmt=fmt, Bt=Bt, T=T, S=64, lens=lens, counts=counts, H=1, G=1, D=128)


@pytest.mark.parametrize("P", [0, 1, 15, 16, 31, 63, 64, 65, 112, 119, 120, 121, 127, 128, 129, 255, 256, 1000])
def test_prefix_lengths_around_tiles(P):
    for mode in ("lite", "fused"):
        _run("P=%d" % P, mode=mode, T=8, S=1024, lens=(P,), Bt=1, D=80)


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_any_mask_and_empty_rows(fmt):
    """Masks that are no tree: rows without a bit, without their own bit, full rows."""
    T = 5
    masks = [[0, 0b00010, 0b11111, 0b00001, 0], [0b11111] * T, [0] * T]
    s = TreeSetup(fmt=fmt, T=T, masks=masks, lens=(0, 0, 0))
    s.run()
    s.check("no prefix")
    got = f64(s.out)
    assert (got[0, :, 0] == 0).all() and (got[0, :, 4] == 0).all() and (got[2] == 0).all()
    _run("with a prefix", fmt=fmt, T=T, masks=masks, lens=(1, 130, 64))


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_ragged_node_counts(fmt):
    """Nodes behind the count keep their output, and bits of missing nodes are ignored."""
    T = 20
    masks = [[2 ** T - 1] * T for _ in range(5)]
    _run("counts", fmt=fmt, T=T, Bt=5, masks=masks, lens=(0, 128, 299, 17, 0), counts=[20, 0, 20, 1, 0], S=320)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_rows_not_seen_may_hold_anything(fmt, mode):
    """NaN and infinities behind the last row and in rows no node sees."""
    T = 12
    masks = [[(1 << i) | 1 for i in range(T)] for _ in range(3)]
    for m in masks:
        m[3] = 1            # node 3 is seen by nobody, itself included
    s = TreeSetup(fmt=fmt, T=T, mode=mode, masks=masks, lens=(0, 120, 200), S=320)
    s.run()
    clean = s.out.clone()
    for b, P in enumerate(s.lens):
        for l in (1, 2):
            s.k[l][b, :, P + T:] = float("nan")
            s.v[l][b, :, P + T:] = float("inf")
            s.v[l][b, :, P + T + 1:] = float("nan")
            s.k[l][b, :, P + 3] = float("inf")
            s.v[l][b, :, P + 3] = float("nan")
    s.out.fill_(-77)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert torch.equal(s.out, clean)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_node_stays_with_those_that_see_it(fmt, bad):
    """A drafted row that is not finite does not reach nodes that do not see it."""
    T = 6
    masks = [[1, 2, 1 | 4, 2 | 8, 1 | 16, 2 | 32]] * 2
    s = TreeSetup(fmt=fmt, T=T, Bt=2, masks=masks, lens=(40, 127), S=256)
    s.run()
    clean = s.out.clone()
    for l in (1, 2):
        for b, P in enumerate(s.lens):
            s.v[l][b, :, P + 1] = bad
    s.run()
    even, odd = [0, 2, 4], [1, 3, 5]
    assert torch.equal(s.out[:, :, even], clean[:, :, even])
    assert not torch.isfinite(s.out[:, :, odd].float()).any()


def test_bad_lengths_are_flagged():
    s = TreeSetup(Bt=4, T=9, lens=(-1, 312, 100, 20), counts=[9, 9, 10, 9], S=320)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
    assert (s.out[:3] == 0).all()
    # the sequence beside them is right
    good = TreeSetup(Bt=4, T=9, lens=(1, 1, 1, 20), S=320)
    good.run()
    assert torch.equal(s.out[3], good.out[3])
    assert s.ctx.fkv_get_device_status() == B.FKV_OK


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("window", [1, 2, 5, 64, 130, 300])
def test_windows(fmt, window):
    _run("W=%d" % window, fmt=fmt, window=window, T=14, lens=(0, 77, 290), S=320, mode="lite")
    if fmt != "q4":
        _run("W=%d" % window, fmt=fmt, window=window, T=33, lens=(3, 128, 270), S=320, G=1)


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("window,ring,T", [(100, 111, 12), (128, 257, 7), (1, 8, 8), (64, 128, 65), (250, 300, 40)])
def test_rings(fmt, window, ring, T):
    _run("R=%d" % ring, fmt=fmt, window=window, ring=ring, T=T, Bt=5, S=1200,
         lens=(0, ring - 1, ring, 5 * ring // 2, 1200 - T if ring > 64 else 3 * ring + 5))
    _run("R=%d" % ring, fmt=fmt, window=window, ring=ring, T=T, Bt=2, S=1200, mode="vanilla", D=96,
         lens=(ring // 2, 2 * ring - 3))


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 61, 500])
@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_every_split(fmt, splits):
    _run("splits=%d" % splits, fmt=fmt, splits=splits, T=10, Bt=4, lens=(900, 0, 1500, 133), S=1600,
         H=2, G=1, D=128 if fmt == "bf16" else 64)


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_one_node_matches_decode(fmt):
    s = TreeSetup(fmt=fmt, T=1, masks=[[1]] * 3, lens=(0, 127, 200))
    s.run()
    s.check("T=1")
    dec = torch.empty_like(s.q[:, :, 0]).contiguous()
    s.ctx.fkv_decode_attn(s.q[:, :, 0].contiguous(), s.layer, s.mode, s.seq + 1, dec, s.ctx.workspace())
    ref, bound = s.reference()
    assert (np.abs(f64(s.out[:, :, 0]) - f64(dec)) <= 2 * bound[:, :, 0]).all()


def test_large_scores_and_weights():
    """Scores of hundreds, so that the running maximum moves far, and weights of any sign."""
    w = torch.randn(4, 2, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 2
    for mode in ("scaled", "fused"):
        s = TreeSetup(mode=mode, T=16, lens=(300, 511, 700), S=800, weights=w)
        s.run()
        s.check("weights")
    s = TreeSetup(mode="lite", T=16, lens=(300, 511, 700), S=800, scale=20.0)
    s.run()
    s.check("scale")
    # keys that grow along the cache: every tile raises the maximum
    s = TreeSetup(mode="lite", T=16, lens=(300, 511, 700), S=800)
    ramp = torch.linspace(0.1, 12, 800, device="cuda")[None, None, :, None]
    for l in (1, 2):
        s.k[l].copy_((s.k[l].float().abs() * ramp).to(s.dt))
    s.q.copy_(s.q.abs())
    s.run()
    s.check("ramp")


def test_same_inputs_same_bits():
    s = TreeSetup(T=21, Bt=3, lens=(700, 1300, 90), S=1400)
    a = s.run().clone()
    for _ in range(5):
        assert torch.equal(s.run(), a)


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_graphs_that_share_a_workspace(fmt):
    """Two captured calls with one workspace, replayed in turn with new inputs, between eager calls."""
    s = TreeSetup(fmt=fmt, T=13, Bt=3, lens=(700, 1300, 90), S=1400, seed=1)
    t = torch.empty_like(s.out)
    graphs = []
    side = torch.cuda.Stream()
    s.run()
    torch.cuda.synchronize()
    for mode, out in (("fused", s.out), ("lite", t)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                s.ctx.fkv_tree_attn(s.q, 3, mode, s.seq, s.mask, out, s.ws, stream=side)
        graphs.append(g)
    for k in range(3):
        s.q.copy_(torch.randn(s.q.shape, device="cuda").to(s.dt))
        s.seq.copy_(torch.tensor([600 - 50 * k, 1100 + 60 * k, 17 * k], dtype=torch.int32))
        s.lens = s.seq.tolist()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        s.mode = "fused"
        s.check("replay %d" % k)
        e = torch.empty_like(t)
        s.ctx.fkv_tree_attn(s.q, 3, "lite", s.seq, s.mask, e, s.ws)
        assert torch.equal(e, t)


def test_other_stream_is_ordered():
    s = TreeSetup(T=16, Bt=3, lens=(700, 1300, 90), S=1400)
    ref = s.run().clone()
    side = torch.cuda.Stream()
    q = s.q.clone()
    s.q.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        s.q.copy_(q)
        s.run()                 # on torch's current stream
        got = s.out.clone()
    side.synchronize()
    assert torch.equal(got, ref)


def test_two_calls_at_once():
    """Unordered streams, a workspace each, bf16 beside fp32 and 4-bit calls."""
    sets = [TreeSetup(fmt=f, T=t, Bt=3, lens=(700, 1300, 90), S=1400, seed=i)
            for i, (f, t) in enumerate([("bf16", 16), ("f32", 9), ("q4", 16), ("bf16", 64)])]
    want = [s.run().clone() for s in sets]
    for s in sets:
        s.out.fill_(-77)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, st in zip(sets, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert s.ctx.fkv_get_device_status() == B.FKV_OK
        assert torch.equal(s.out, w)


def test_workspace_of_more_nodes_serves_fewer():
    s = TreeSetup(T=9, Bt=3, lens=(700, 1300, 90), S=1400)
    ref = s.run().clone()
    s.ws = s.ctx.tree_workspace(128)
    assert torch.equal(s.run(), ref)


def test_host_refusals():
    s = TreeSetup(T=8, fmt="bf16")
    lib, c, p = s.ctx._lib, s.ctx, lambda t: t.data_ptr()
    n = s.ws.numel()

    def call(layer=3, mode=B.FKV_FUSED, q=p(s.q), seq=p(s.seq), cnt=None, mask=p(s.mask), T=8,
             out=p(s.out), ws=p(s.ws), size=n):
        return lib.fkv_tree_attn(c.handle, q, layer, mode, seq, cnt, mask, T, out, ws, size, None)

    inv = B.FKV_ERR_INVALID_ARG
    assert call(T=0) == inv and call(T=129) == inv and call(T=-3) == inv
    assert call(layer=0) == inv and call(layer=5) == inv and call(mode=4) == inv
    assert call(q=None) == inv and call(q=p(s.q) + 8) == inv and call(out=None) == inv
    assert call(seq=None) == inv and call(seq=p(s.seq) + 2) == inv
    assert call(cnt=p(s.seq) + 1) == inv and call(mask=None) == inv and call(mask=p(s.mask) + 4) == inv
    assert call(mode=B.FKV_VANILLA) == B.FKV_ERR_UNSUPPORTED        # upper layers store nothing
    assert call(ws=None) == B.FKV_ERR_WORKSPACE and call(size=16) == B.FKV_ERR_WORKSPACE
    assert call(ws=p(s.ws) + 8) == B.FKV_ERR_WORKSPACE
    assert c.fkv_tree_workspace_bytes(0) == 0 and c.fkv_tree_workspace_bytes(129) == 0
    with pytest.raises(ValueError):
        c.tree_workspace(0)
    r = TreeSetup(T=8, window=100, ring=107, lens=(0, 20, 300))
    r.run()
    r.ctx.fkv_set_window(3, 101)                                    # 101 + 8 - 1 > 107
    with pytest.raises(B.FkvError) as e:
        r.run()
    assert e.value.status == B.FKV_ERR_UNSUPPORTED
    for w in (0, 108):
        r.ctx.fkv_set_window(3, w)
        with pytest.raises(B.FkvError) as e:
            r.run()
        assert e.value.status == inv
    short = B.Context(4, 1, 4, 2, 2, 64, "bf16")                    # S_max below T
    assert short.fkv_tree_workspace_bytes(8) == 0 and short.fkv_tree_workspace_bytes(4) > 0
    assert lib.fkv_tree_attn(short.handle, p(s.q), 1, 0, p(s.seq), None, p(s.mask), 8, p(s.out), p(s.ws),
                             n, None) == inv
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert (s.out == -77).all()


def test_timeout_path():
    """Every wait reports a timeout at once; the next call is whole again."""
    s = TreeSetup(T=16, Bt=3, lens=(700, 1300, 90), S=1400)
    s.ctx.fkv_set_wait_limit(0)
    s.run()
    st = s.ctx.fkv_get_device_status()
    s.ctx.fkv_set_wait_limit(10 ** 9)
    assert st in (B.FKV_OK, B.FKV_ERR_TIMEOUT)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    s.check("after a timeout")


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last unit against a double-precision product."""
    Bt, H, S, D, T = 5, 16, 65536, 64, 6
    ctx = B.Context(2, Bt, S, H, H, D, "f32")
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.empty(Bt, H, S, D, device="cuda")
    k.normal_(generator=g)
    assert k.numel() * 4 > 1 << 32 or k.numel() * 8 > 1 << 31
    ctx.fkv_bind_layer_cache(1, k, k)
    q = torch.randn(Bt, H, T, D, generator=g, device="cuda")
    lens = [4, 4, 4, 4, S - T]
    masks = [[(2 << i) - 1 for i in range(T)]] * Bt
    out = torch.empty_like(q)
    ctx.fkv_tree_attn(q, 1, "vanilla", torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      mask_words(masks, T), out, ctx.tree_workspace(T))
    assert ctx.fkv_get_device_status() == B.FKV_OK
    kk = k[-1, -1].double()
    s = q[-1, -1].double() @ kk.T / 8.0
    see = torch.ones(T, S, dtype=torch.bool, device="cuda")
    see[:, S - T:] = torch.tril(torch.ones(T, T, dtype=torch.bool, device="cuda"))
    ref = torch.softmax(s.masked_fill(~see, -float("inf")), -1) @ kk
    assert (out[-1, -1].double() - ref).abs().max() < 1e-5
