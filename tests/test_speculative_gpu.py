"""Rounds of speculative decoding and a beam fork over one context, as a user
makes them: append drafts, attend in every layer, keep a path, reorder."""

import random

import numpy as np
import pytest
import torch

import oracle as O
from cross_layer_kv_gb300 import fusedkv as B
from parity import f64
from tree_parity import mask_words, random_masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("mode", ["lite", "fused"])
def test_rounds(fmt, mode):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L, Bt, S, H, G, D, T = 6, 3, 400, 2, 2, 64, 11
    n = L // 2
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    ctx = B.Context(L, Bt, S, H * G, H, D, "f32" if fmt == "f32" else "bf16")
    g = torch.Generator(device="cuda").manual_seed(7)
    rng = random.Random(7)
    caches = {}
    for l in range(1, n + 1):
        if fmt == "q4":
            caches[l] = (ctx.q4_cache(), ctx.q4_cache())
            ctx.fkv_bind_layer_cache_q4(l, *caches[l])
        else:
            caches[l] = tuple(torch.zeros(Bt, H, S, D, dtype=dt, device="cuda") for _ in range(2))
            ctx.fkv_bind_layer_cache(l, *caches[l])
    weights = {}
    for l in range(n + 1, L + 1):
        weights[l] = [torch.randn(H, D, generator=g, device="cuda") * 0.3 + 0.5 for _ in range(4)]
        ctx.fkv_set_fusion_weights(l, *weights[l])
    mirror = {l: [np.zeros((Bt, H, S, D)) for _ in range(2)] for l in range(1, n + 1)}

    def stored(x):                      # what the cache holds of appended rows
        x = f64(x)
        return O.q4_dequantize(*O.q4_quantize(x)) if fmt == "q4" else x

    lens = [150, 1, 260]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = ctx.tree_workspace(T)
    zero = torch.zeros(Bt, dtype=torch.int32, device="cuda")
    for l in range(1, n + 1):           # prompts (rows behind a length are never read)
        kv = [torch.randn(Bt, H, 260, D, generator=g, device="cuda").to(dt) for _ in range(2)]
        ctx.fkv_append_kv(l, *kv, zero)
        for i in range(2):
            mirror[l][i][:, :, :260] = stored(kv[i])
    bar = 1e-5 if fmt == "f32" else 5e-3
    for step in range(4):
        masks = random_masks(rng, Bt, T)
        for l in range(1, n + 1):
            kv = [torch.randn(Bt, H, T, D, generator=g, device="cuda").to(dt) for _ in range(2)]
            ctx.fkv_append_kv(l, *kv, seq)
            for i in range(2):
                for b in range(Bt):
                    mirror[l][i][b, :, lens[b]:lens[b] + T] = stored(kv[i])[b]
        for l in range(1, L + 1):
            q = torch.randn(Bt, H * G, T, D, generator=g, device="cuda").to(dt)
            out = torch.empty_like(q)
            ctx.fkv_tree_attn(q, l, mode, seq, mask_words(masks, T), out, ws)
            k, v = O.reconstruct_kv(l, L, mode, {x: c[0] for x, c in mirror.items()},
                                    {x: c[1] for x, c in mirror.items()},
                                    {x: tuple(f64(y) for y in w) for x, w in weights.items()})
            ref = O.tree_attention(f64(q), k, v, lens, masks)
            rel = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
            assert rel <= bar, "round %d layer %d: rel-L2 %.3g" % (step, l, rel)
        paths = []
        for b in range(Bt):             # accept the path to a random node
            node = rng.randrange(T)
            paths.append([j for j in range(T) if masks[b][node] >> j & 1])
        A = max(len(x) for x in paths)
        idx = [x + [0] * (A - len(x)) for x in paths]
        counts = [len(x) for x in paths]
        ctx.fkv_compact_rows(seq, torch.tensor(idx, dtype=torch.int32, device="cuda"),
                             torch.tensor(counts, dtype=torch.int32, device="cuda"))
        for l in mirror:
            mirror[l] = [O.compact_rows(x, lens, idx, counts) for x in mirror[l]]
        lens = [p + c for p, c in zip(lens, counts)]
        if step == 1:                   # the first sequence ends: its slot continues the last one
            src = [2, 0, -1]
            lens = [lens[2], lens[0], lens[2]]
            seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
            ctx.fkv_reorder_seqs(torch.tensor(src, dtype=torch.int32, device="cuda"), seq)
            for l in mirror:
                mirror[l] = [O.reorder_seqs(x, src, lens) for x in mirror[l]]
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert ctx.fkv_get_device_status() == B.FKV_OK
