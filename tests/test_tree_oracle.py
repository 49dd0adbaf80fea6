"""CPU pins of the oracle's tree attention, row compaction and sequence
reordering, and the host checks of their entry points that need no GPU."""

import numpy as np
import pytest

import cross_layer_kv_gb300 as fkv
import oracle as O
from cross_layer_kv_gb300 import fusedkv as B


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def _chain(T):
    return [(1 << (i + 1)) - 1 for i in range(T)]


def test_chain_is_chunked_prefill():
    q, k, v = _rand(2, 4, 5, 8), _rand(2, 2, 20, 8, seed=1), _rand(2, 2, 20, 8, seed=2)
    for window in (0, 3, 9):
        got = O.tree_attention(q, k, v, [11, 11], [_chain(5)] * 2, window=window)
        ref = O.chunk_prefill_attention(q, 11, k, v, window=window)
        np.testing.assert_allclose(got, ref, atol=1e-13)


def test_one_node_is_decode():
    q, k, v = _rand(3, 2, 1, 8), _rand(3, 1, 12, 8, seed=1), _rand(3, 1, 12, 8, seed=2)
    for window in (0, 4):
        got = O.tree_attention(q, k, v, [0, 5, 11], [[1]] * 3, window=window)
        ref = O.decode_attention(q[:, :, 0], k, v, [1, 6, 12], window=window)
        np.testing.assert_allclose(got[:, :, 0], ref, atol=1e-13)


def test_a_path_of_a_tree_is_decode_over_its_rows():
    # nodes 0 and 1 attach to the prefix, 2 to 0, 3 to 1, 4 to 2
    masks = [[1, 2, 1 | 4, 2 | 8, 1 | 4 | 16]]
    q, k, v = _rand(1, 1, 5, 8), _rand(1, 1, 12, 8, seed=1), _rand(1, 1, 12, 8, seed=2)
    got = O.tree_attention(q, k, v, [7], masks)
    for node, path in ((4, [0, 2, 4]), (3, [1, 3])):
        rows = list(range(7)) + [7 + j for j in path]
        ref = O.decode_attention(q[:, :, node], k[:, :, rows], v[:, :, rows], [len(rows)])
        np.testing.assert_allclose(got[:, :, node], ref, atol=1e-13)


def test_nothing_visible_and_missing_nodes():
    q, k, v = _rand(2, 1, 3, 8), _rand(2, 1, 6, 8, seed=1), _rand(2, 1, 6, 8, seed=2)
    got = O.tree_attention(q, k, v, [0, 2], [[0, 2, 7], [0, 0, 0]], counts=[2, 1])
    assert (got[0, 0, 0] == 0).all()                     # no row seen: zeros
    np.testing.assert_allclose(got[0, 0, 1], v[0, 0, 1])  # one row seen: its value
    assert np.isnan(got[0, 0, 2]).all() and np.isnan(got[1, 0, 1:]).all()
    assert np.isfinite(got[1, 0, 0]).all()


def test_compact_rows_by_hand():
    c = np.arange(2 * 1 * 8 * 1, dtype=float).reshape(2, 1, 8, 1)
    new = O.compact_rows(c, [2, 0], [[0, 3, 1], [4, 4, 9]], [3, 2])
    np.testing.assert_array_equal(new[0, 0, :, 0], [0, 1, 2, 5, 3, 5, 6, 7])
    np.testing.assert_array_equal(new[1, 0, :, 0], [12, 12, 10, 11, 12, 13, 14, 15])
    ring = O.compact_rows(c, [13, 8], [[1, 2], [0, 0]], [2, 0], ring=8)
    np.testing.assert_array_equal(ring[0, 0, :, 0], [0, 1, 2, 3, 4, 6, 7, 7])


def test_reorder_seqs_by_hand():
    c = np.arange(3 * 1 * 4 * 1, dtype=float).reshape(3, 1, 4, 1)
    new = O.reorder_seqs(c, [1, 2, 0], [4, 2, 9])     # a cycle, ragged
    np.testing.assert_array_equal(new[:, 0, :, 0], [[4, 5, 6, 7], [8, 9, 6, 7], [0, 1, 2, 3]])
    np.testing.assert_array_equal(O.reorder_seqs(c, [-1, 1, 2], [4, 4, 4]), c)


def test_null_context_is_rejected():
    lib = fkv.load()
    assert lib.fkv_tree_workspace_bytes(None, 8) == 0
    assert lib.fkv_tree_attn(None, 16, 3, 2, 16, None, 16, 8, 16, 16, 1 << 20, None) == \
        B.FKV_ERR_INVALID_ARG
    assert lib.fkv_compact_rows(None, 16, 16, 16, 4, None) == B.FKV_ERR_INVALID_ARG
    assert lib.fkv_reorder_seqs(None, 16, 16, None) == B.FKV_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", ["cpu", "shape", "dtype", "stride"])
def test_binding_refuses_wrong_tensors(bad):
    """The binding's own checks come before the library is called."""
    import torch
    ctx = object.__new__(B.Context)
    ctx.cfg = B.fkv_config(4, 2, 64, 4, 2, 64, B.FKV_BF16, 0, 0.0, 0)
    ctx.torch_dtype = torch.bfloat16
    ctx.handle = None
    ctx._lib = None
    t = dict(cpu=torch.zeros(2, dtype=torch.int32), shape=torch.zeros(3, dtype=torch.int32),
             dtype=torch.zeros(2, dtype=torch.int64), stride=torch.zeros(4, dtype=torch.int32)[::2])[bad]
    with pytest.raises(ValueError):
        ctx.fkv_reorder_seqs(t, t)
    with pytest.raises(ValueError):
        ctx.fkv_compact_rows(t, torch.zeros(2, 3, dtype=torch.int32), t)
    q = torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ctx.fkv_tree_attn(q, 3, "fused", t, torch.zeros(2, 5, 1, dtype=torch.int64), q, q)
