"""Tree attention over 4-bit caches on the GPU: no less exact than its output's
rounding, over the range of fp16 (bounds: q4_bounds.py)."""

import numpy as np
import pytest
import torch

import oracle as O
import q4_bounds
from cross_layer_kv_gb300 import fusedkv as B
from parity import f64
from tree_parity import TreeSetup

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def _run(s, what=""):
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    return q4_bounds.check(s, what)


@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("T", [1, 9, 16, 40])
@pytest.mark.parametrize("mode", ["lite", "scaled", "fused"])
def test_the_error_is_the_output_s_rounding(D, T, mode):
    """Rounding a bf16 output alone is off by r in L2.  Each of the four operands (query times
    weight, keys, probabilities, values) is off by at most 2^-11 / sqrt(3) of itself in the mean
    square, an eighth of the output's 2^-8 / sqrt(3); a score's error of 2 * 2^-11 / sqrt(3) of
    scores of order 1 counts once in the output.  Together sqrt(1 + 4 / 64) r = 1.03 r; 1.25 r
    leaves room for scores above 1 and for the chance in few outputs."""
    s = TreeSetup(fmt="q4", D=D, T=T, mode=mode, lens=(60, 700, 1300), S=1400)
    _run(s)
    ref, _ = s.reference()
    err = np.linalg.norm(f64(s.out) - ref)
    alone = np.linalg.norm(f64(torch.from_numpy(ref).to(torch.bfloat16)) - ref)
    assert err <= 1.25 * alone, "%.3g times the rounding" % (err / alone)


@pytest.mark.parametrize("mode", ["lite", "scaled", "fused"])
@pytest.mark.parametrize("kv_scale", [1e-4, 1e-3, 0.02, 50.0, 700.0, 3e3])
def test_caches_of_any_size(mode, kv_scale):
    """Scores of order 1 at every size of the keys."""
    s = TreeSetup(fmt="q4", D=64, T=14, mode=mode, lens=(3, 200, 700), S=800, kv_scale=kv_scale,
                  scale=0.125 / kv_scale)
    _run(s, "kv %g" % kv_scale)


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("D", [64, 96])
def test_rows_of_different_sizes(mode, what, D):
    """Single rows at the ends of the range, and tiny ones, among usual ones."""
    s = TreeSetup(fmt="q4", D=D, T=20, mode=mode, lens=(0, 130, 700), S=800, window=0)
    g = np.random.default_rng(4)
    for l in (1, 2):
        x = getattr(s, what)[l]
        codes, sc, lo = O.q4_unpack(x.cpu().numpy(), s.D)
        powers = g.choice([0, 0, 0, -13, -30, 8, 11] if what == "v" else [0, 0, 0, -30, -90, -12], sc.shape[:-1])
        f = (2.0 ** powers.astype(np.float64))[..., None]
        rec = O.q4_pack(codes, (sc * f).astype(np.float32), (lo * f).astype(np.float32))
        x.copy_(torch.from_numpy(rec))
    _run(s, what)


def test_large_keys_and_scales():
    """Keys of 10^2 to 10^4 in single rows: scores that decide the softmax alone."""
    s = TreeSetup(fmt="q4", D=64, T=9, mode="lite", lens=(100, 300, 700), S=800)
    codes, sc, lo = O.q4_unpack(s.k[2].cpu().numpy(), s.D)
    for row, f in ((3, 2.0 ** 7), (40, 2.0 ** 9), (77, 2.0 ** 11)):
        sc[1:, :, row] *= np.float32(f)
        lo[1:, :, row] *= np.float32(f)
    s.k[2].copy_(torch.from_numpy(O.q4_pack(codes, sc, lo)))
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    got = f64(s.out)
    k = O.q4_dequantize_records(s.k[2].cpu().numpy(), s.D)
    v = O.q4_dequantize_records(s.v[1].cpu().numpy(), s.D)
    ref = O.tree_attention(f64(s.q), k, v, s.lens, s.masks)
    # the largest key's score is positive and wins, or negative and gives way to the next one:
    # gaps of 10^2 and more (scores off by 2^-10 of 10^4 and less) leave one row, whose value's error
    # is 2^-8 + 2^-11 of it and 3 * 2^-25
    for b in (1, 2):
        qq = f64(s.q)[b].reshape(s.H, s.G, s.T, s.D)
        sc = np.einsum("hgtd,hsd->hgts", qq, k[b, :, :s.lens[b]]) * s.scale
        best = np.sort(sc, -1)
        sure = (best[..., -1] - best[..., -2] > 100).reshape(s.H * s.G, s.T)
        assert sure.mean() > 0.5      # all three scores are negative for one query in eight
        err = np.abs(got[b] - ref[b])[sure]
        assert (err <= (2.0 ** -8 + 2.0 ** -11) * 1.01 * np.abs(ref[b][sure]) + 3 * 2.0 ** -25).all()
    np.testing.assert_array_less(np.abs(got[0] - ref[0]), 0.05)   # the sequence beside them


@pytest.mark.parametrize("mode", ["lite", "scaled", "fused"])
def test_queries_of_different_sizes(mode):
    """Query rows (and weights) outside fp16's range, tiny ones and large ones, node by node."""
    w = torch.rand(4, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) + 0.5
    w[0:2] *= 1e-5
    s = TreeSetup(fmt="q4", T=12, mode=mode, lens=(60, 200, 700), S=800, weights=w,
                  scale=0.125 if mode == "lite" else 1e4)
    s.q.mul_((2.0 ** torch.arange(-9, 3, device="cuda", dtype=torch.float32)).to(s.q.dtype)[None, None, :, None])
    s.q[:, :, 5] *= 2.0 ** -30
    _run(s, "queries")
    s.q[:, :, 7] *= 2.0 ** 20       # one row far above the others
    _run(s, "a large row")


@pytest.mark.parametrize("mode", ["lite", "fused"])
@pytest.mark.parametrize("size", [1e-30, 1e-9, 1e5, 1e30])
def test_rows_not_seen_of_any_size_change_nothing(mode, size):
    T = 12
    masks = [[(1 << i) | 1 for i in range(T)] for _ in range(3)]
    for m in masks:
        m[3] = 1            # node 3 is seen by nobody, itself included
    s = TreeSetup(fmt="q4", T=T, mode=mode, masks=masks, lens=(0, 120, 200), S=320)
    s.run()
    clean = s.out.clone()
    for b, P in enumerate(s.lens):
        for l in (1, 2):
            for x in (s.k[l], s.v[l]):
                q4_bounds.params(s, x)[b, :, P + T:] = size
                q4_bounds.params(s, x)[b, :, P + 3] = size
    s.out.fill_(-77)
    s.run()
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    assert torch.equal(s.out, clean)


@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_missing_nodes_queries_are_not_used(mode):
    s = TreeSetup(fmt="q4", T=12, mode=mode, lens=(60, 200, 700), counts=[5, 12, 0], S=800)
    s.run()
    clean = s.out.clone()
    for b, n in enumerate(s.counts):
        s.q[b, :, n:] = float("nan")
        s.q[b, :, n + 1::2] = 1e38
    s.run()
    assert torch.equal(s.out, clean)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_a_row_out_of_range_stays_with_the_nodes_that_see_it(mode, what):
    """Keys and values above 2^14 may count as not finite, for the nodes that see them alone."""
    T = 6
    masks = [[1, 2, 1 | 4, 2 | 8, 1 | 16, 2 | 32]] * 2
    s = TreeSetup(fmt="q4", T=T, mode=mode, Bt=2, masks=masks, lens=(40, 127), S=256)
    s.run()
    clean = s.out.clone()
    for l in (1, 2):
        for b, P in enumerate(s.lens):
            q4_bounds.params(s, (s.k if what == "k" else s.v)[l])[b, :, P + 1] = 1e30
    s.run()
    assert torch.equal(s.out[:, :, [0, 2, 4]], clean[:, :, [0, 2, 4]])
