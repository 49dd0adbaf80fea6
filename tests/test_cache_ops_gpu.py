"""fkv_compact_rows and fkv_reorder_seqs on the GPU: moves are exact, so every
byte of every cache is compared with the oracle's."""

import random

import numpy as np
import pytest
import torch

import oracle as O
from cross_layer_kv_gb300 import fusedkv as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """Contexts whose layers hold different formats and ring sizes, caches as raw bytes."""

    def __init__(self, Bt=4, H=2, S=96, D=64, layers=6, dtype="bf16", rings=None, q4=(), only=None, seed=0):
        self.ctx = B.Context(layers, Bt, S, H, H, D, dtype)
        self.rings, self.caches = rings or {}, {}
        g = torch.Generator(device="cuda").manual_seed(seed)
        for l in range(1, layers // 2 + 1):
            if only and l not in only:
                continue
            rows = self.rings.get(l, 0) or S
            if l in self.rings:
                self.ctx.fkv_set_ring_rows(l, self.rings[l])
            nb = self.ctx.fkv_q4_row_bytes() if l in q4 else D * (4 if dtype == "f32" else 2)
            kv = [torch.randint(0, 256, (Bt, H, rows, nb), generator=g, device="cuda", dtype=torch.uint8)
                  for _ in range(2)]
            if l in q4:
                self.ctx.fkv_bind_layer_cache_q4(l, *kv)
            else:
                self.ctx.fkv_bind_layer_cache(l, *(x.view(self.ctx.torch_dtype) for x in kv))
            self.caches[l] = kv

    def snapshot(self):
        return {l: [x.cpu().numpy() for x in kv] for l, kv in self.caches.items()}

    def expect(self, old, fn):
        for l, kv in self.caches.items():
            for i, x in enumerate(kv):
                np.testing.assert_array_equal(x.cpu().numpy(), fn(old[l][i], self.rings.get(l, 0)),
                                              err_msg="layer %d %s" % (l, "KV"[i]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
@pytest.mark.parametrize("A", [1, 5, 17, 64, 128])
def test_compact(dtype, D, A):
    S, Bt = 200, 4
    m = Model(Bt=Bt, S=S, D=D, dtype=dtype, H=3)
    rng = random.Random(A * D)
    pos = [0, 13, S - max(A, 1), 50]
    counts = [A, 0, A, rng.randint(1, A)]
    idx = [[rng.randrange(0, min(S - p, 140)) for _ in range(A)] for p in pos]   # any order, repeats
    old = m.snapshot()
    m.ctx.fkv_compact_rows(_i32(pos), _i32(idx), _i32(counts))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.compact_rows(x, pos, idx, counts, ring))


def test_compact_mixed_formats_and_rings():
    m = Model(layers=10, S=300, rings={2: 70, 4: 131}, q4=(3, 4), only=(1, 2, 3, 4))
    pos, counts = [0, 65, 130, 250], [3, 4, 6, 2]
    idx = [[0, 2, 5, 0, 0, 0], [1, 4, 5, 9, 0, 0], [0, 1, 2, 3, 60, 69], [40, 0, 0, 0, 0, 0]]
    old = m.snapshot()
    m.ctx.fkv_compact_rows(_i32(pos), _i32(idx), _i32(counts))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.compact_rows(x, pos, idx, counts, ring))


def test_compact_bad_sequences_are_left_and_flagged():
    S = 96
    good = dict(pos=10, idx=[0, 3], count=2)
    for bad in (dict(pos=-1), dict(pos=S), dict(pos=S - 1), dict(count=3), dict(count=-1),
                dict(idx=[0, -1]), dict(idx=[0, S - 10]), dict(idx=[0, 40])):
        m = Model(rings={2: 40}, S=S)
        rows = [dict(good) for _ in range(4)]
        rows[1].update(bad)
        pos, idx, counts = ([r[k] for r in rows] for k in ("pos", "idx", "count"))
        old = m.snapshot()
        m.ctx.fkv_compact_rows(_i32(pos), _i32(idx), _i32(counts))
        assert m.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG, bad
        counts[1], pos[1], idx[1] = 0, 0, [0, 0]
        m.expect(old, lambda x, ring: O.compact_rows(x, pos, idx, counts, ring))
    # an entry behind the count is not read
    m = Model(S=S)
    m.ctx.fkv_compact_rows(_i32([0] * 4), _i32([[1, -5]] * 4), _i32([1] * 4))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 80), ("f32", 96), ("bf16", 128)])
@pytest.mark.parametrize("src", [[0, 0, 0, 0], [1, 2, 3, 0], [3, -1, 2, 0], [0, 1, 2, 3], [2, 2, 1, 1]])
def test_reorder(dtype, D, src):
    S = 333
    m = Model(S=S, D=D, dtype=dtype, H=3)
    lens = [S, 17, 0, 130]
    old = m.snapshot()
    m.ctx.fkv_reorder_seqs(_i32(src), _i32(lens))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.reorder_seqs(x, src, lens))


@pytest.mark.parametrize("Bt,S,H", [(1, 50, 1), (2, 4000, 2), (33, 257, 1), (64, 700, 2), (300, 60, 1), (1024, 9, 1)])
def test_reorder_batches(Bt, S, H):
    rng = random.Random(Bt)
    for kind in ("permutation", "any", "fork"):
        m = Model(Bt=Bt, S=S, H=H, layers=4)
        src = list(range(Bt))
        if kind == "permutation":
            rng.shuffle(src)
        elif kind == "any":
            src = [rng.randrange(-1, Bt) for _ in src]
        else:
            src = [0] * Bt
        lens = [rng.randint(0, S) for _ in src]
        old = m.snapshot()
        m.ctx.fkv_reorder_seqs(_i32(src), _i32(lens))
        assert m.ctx.fkv_get_device_status() == B.FKV_OK
        m.expect(old, lambda x, ring: O.reorder_seqs(x, src, lens))


def test_reorder_mixed_formats_rings_and_many_layers():
    m = Model(Bt=5, layers=140, S=150, rings={2: 70, 4: 131}, q4=(3, 4), H=1)
    src, lens = [4, 0, 2, 1, 1], [150, 100, 7, 69, 1]
    old = m.snapshot()
    m.ctx.fkv_reorder_seqs(_i32(src), _i32(lens))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.reorder_seqs(x, src, lens))
    old = m.snapshot()
    pos, idx, counts = [3, 60, 100, 0, 140], [[2, 5], [0, 1], [7, 3], [1, 0], [9, 8]], [2, 2, 2, 2, 2]
    m.ctx.fkv_compact_rows(_i32(pos), _i32(idx), _i32(counts))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.compact_rows(x, pos, idx, counts, ring))


def test_reorder_bad_sequences_are_left_and_flagged():
    for s, n in ((4, 10), (-2, 10), (2, -1), (2, 97)):
        m = Model(S=96)
        src, lens = [2, s, 3, 0], [50, n, 96, 20]
        old = m.snapshot()
        m.ctx.fkv_reorder_seqs(_i32(src), _i32(lens))
        assert m.ctx.fkv_get_device_status() == B.FKV_ERR_DEVICE_ARG
        src[1], lens[1] = -1, 0
        m.expect(old, lambda x, ring: O.reorder_seqs(x, src, lens))


def test_a_buffer_of_several_layers_moves_once():
    ctx = B.Context(6, 3, 40, 1, 1, 64, "bf16")
    kv = torch.randn(3, 1, 40, 64, device="cuda").to(torch.bfloat16)
    other = torch.randn(3, 1, 40, 64, device="cuda").to(torch.bfloat16)
    ctx.fkv_bind_layer_cache(1, kv, kv)
    ctx.fkv_bind_layer_cache(2, other, kv)
    ctx.fkv_bind_layer_cache(3, kv, other)
    a, b = kv.view(torch.int16).cpu().numpy(), other.view(torch.int16).cpu().numpy()
    src, lens = [1, 2, 0], [40, 40, 40]
    ctx.fkv_reorder_seqs(_i32(src), _i32(lens))
    pos, idx, counts = [0, 5, 9], [[1, 0], [3, 2], [4, 9]], [2, 2, 2]
    ctx.fkv_compact_rows(_i32(pos), _i32(idx), _i32(counts))
    for x, t in ((a, kv), (b, other)):
        ref = O.compact_rows(O.reorder_seqs(x, src, lens), pos, idx, counts)
        np.testing.assert_array_equal(t.view(torch.int16).cpu().numpy(), ref)


def test_replayed_moves():
    """Captured moves, replayed with other contents of the same index tensors."""
    m = Model(S=300, D=128)
    src, lens = _i32([1, 2, 3, 0]), _i32([300, 10, 77, 200])
    pos, idx, counts = _i32([0] * 4), _i32([[3, 1]] * 4), _i32([2] * 4)
    side = torch.cuda.Stream()
    m.ctx.fkv_reorder_seqs(_i32([-1] * 4), lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        m.ctx.fkv_reorder_seqs(src, lens, stream=side)
        m.ctx.fkv_compact_rows(pos, idx, counts, stream=side)
    for k in range(3):
        s, p = [[1, 2, 3, 0], [0, 0, 3, 3], [2, -1, 2, 1]][k], [0, 20 * k, 7, 100]
        src.copy_(_i32(s))
        pos.copy_(_i32(p))
        old = m.snapshot()
        g.replay()
        torch.cuda.synchronize()
        m.expect(old, lambda x, ring: O.compact_rows(O.reorder_seqs(x, s, lens.tolist()), p,
                                                     idx.tolist(), [2] * 4))


def test_host_refusals():
    m = Model()
    lib, h, p = m.ctx._lib, m.ctx.handle, lambda t: t.data_ptr()
    t, i = _i32([0] * 4), _i32([[0]] * 4)
    inv = B.FKV_ERR_INVALID_ARG
    assert lib.fkv_compact_rows(h, p(t), p(i), p(t), 0, None) == B.FKV_OK
    assert lib.fkv_compact_rows(h, p(t), p(i), p(t), -1, None) == inv
    assert lib.fkv_compact_rows(h, p(t), p(i), p(t), 129, None) == inv
    assert lib.fkv_compact_rows(h, p(t), p(i), p(t), 97, None) == inv     # above S_max = 96
    assert lib.fkv_compact_rows(h, None, p(i), p(t), 1, None) == inv
    assert lib.fkv_compact_rows(h, p(t), None, p(t), 1, None) == inv
    assert lib.fkv_compact_rows(h, p(t), p(i), p(t) + 2, 1, None) == inv
    assert lib.fkv_reorder_seqs(h, None, p(t), None) == inv
    assert lib.fkv_reorder_seqs(h, p(t), p(t) + 1, None) == inv
    empty = B.Context(4, 4, 96, 2, 2, 64, "bf16")
    assert lib.fkv_reorder_seqs(empty.handle, p(t), p(t), None) == inv
    assert lib.fkv_compact_rows(empty.handle, p(t), p(i), p(t), 1, None) == inv


def test_reorder_timeout_path():
    m = Model(S=300)
    m.ctx.fkv_set_wait_limit(0)
    m.ctx.fkv_reorder_seqs(_i32([1, 0, 3, 2]), _i32([300] * 4))
    assert m.ctx.fkv_get_device_status() == B.FKV_ERR_TIMEOUT
    m.ctx.fkv_set_wait_limit(10 ** 9)
    old = m.snapshot()
    m.ctx.fkv_reorder_seqs(_i32([1, 0, 3, 2]), _i32([300] * 4))
    assert m.ctx.fkv_get_device_status() == B.FKV_OK
    m.expect(old, lambda x, ring: O.reorder_seqs(x, [1, 0, 3, 2], [300] * 4))
