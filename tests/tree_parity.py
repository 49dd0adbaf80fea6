"""Set-up, oracle and error bounds of the tree attention tests."""

from __future__ import annotations

import math
import random

import numpy as np
import torch

import oracle as O
from cross_layer_kv_gb300 import fusedkv as B
from parity import BF16_REL_L2, f64

ULP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative


def random_masks(rng, B_, T):
    """Ancestor masks of random trees, one per sequence."""
    out = []
    for _ in range(B_):
        m = []
        for i in range(T):
            parent = rng.randint(-1, i - 1) if rng.random() < 0.4 else max(-1, i - rng.randint(1, 3))
            m.append((m[parent] if parent >= 0 else 0) | (1 << i))
        out.append(m)
    return out


def mask_words(masks, T, device="cuda"):
    n = (T + 63) // 64
    rows = [[[(x >> (64 * w) & (2 ** 64 - 1)) - (2 ** 64 if x >> (64 * w + 63) & 1 else 0)
              for w in range(n)] for x in m] for m in masks]
    return torch.tensor(rows, dtype=torch.int64, device=device)


class TreeSetup:
    """Caches of layers 1 and n, weights, drafted queries of one call."""

    def __init__(self, D=64, H=2, G=2, Bt=3, S=320, T=7, mode="fused", fmt="bf16", lens=(0, 127, 200),
                 masks=None, counts=None, window=0, ring=0, seed=0, splits=0, scale=0.0, weights=None,
                 kv_scale=1.0):
        rng = random.Random(seed + 17)
        self.__dict__.update(D=D, H=H, G=G, Bt=Bt, S=S, T=T, mode=mode, fmt=fmt, window=window,
                             ring=ring, lens=list(lens), counts=counts)
        self.masks = random_masks(rng, Bt, T) if masks is None else masks
        self.dt = torch.float32 if fmt == "f32" else torch.bfloat16
        self.ctx = B.Context(4, Bt, S, H * G, H, D, "f32" if fmt == "f32" else "bf16",
                             softmax_scale=scale, decode_ctas=splits)
        self.scale = scale or 1.0 / math.sqrt(D)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layer = 2 if mode == "vanilla" else 3
        rows = ring or S
        self.rows = rows
        self.k, self.v = {}, {}
        for l in (1, 2):
            if ring:
                self.ctx.fkv_set_ring_rows(l, ring)
            kv = [(torch.randn(Bt, H, rows, D, generator=g, device="cuda") * kv_scale).to(self.dt)
                  for _ in range(2)]
            if fmt == "q4":
                kv = [torch.from_numpy(O.q4_pack(*O.q4_quantize(x.cpu().float().numpy()))).cuda()
                      for x in kv]
                self.ctx.fkv_bind_layer_cache_q4(l, *kv)
            else:
                self.ctx.fkv_bind_layer_cache(l, *kv)
            self.k[l], self.v[l] = kv
        w = torch.randn(4, H, D, generator=g, device="cuda") * 0.3 + 0.5
        self.w = [x.contiguous() for x in (w if weights is None else weights).unbind(0)]
        self.ctx.fkv_set_fusion_weights(3, *self.w)
        if window:
            self.ctx.fkv_set_window(self.layer, window)
        self.q = torch.randn(Bt, H * G, T, D, generator=g, device="cuda").to(self.dt)
        self.out = torch.full_like(self.q, -77.0)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        self.mask = mask_words(self.masks, T)
        self.ws = self.ctx.tree_workspace(T)
        self.ws.random_(0, 256)                      # its contents need no initialisation

    def run(self, stream=None):
        self.ctx.fkv_tree_attn(self.q, self.layer, self.mode, self.seq, self.mask, self.out, self.ws,
                               node_counts=self.cnt, stream=stream)
        return self.out

    # -- the oracle ------------------------------------------------------
    def plain_caches(self):
        """{layer: (K, V)} in float64, rows in order of position."""
        out = {}
        for l in (1, 2):
            kv = []
            for x in (self.k[l], self.v[l]):
                x = O.q4_dequantize_records(x.cpu().numpy(), self.D) if self.fmt == "q4" else f64(x)
                if self.ring:
                    y = np.zeros((self.Bt, self.H, self.S, self.D))
                    for b in range(self.Bt):
                        end = self.lens[b] + self.T
                        for p in range(max(0, end - self.ring), end):
                            y[b, :, p] = x[b, :, p % self.ring]
                    x = y
                kv.append(np.asarray(x, dtype=np.float64))
            out[l] = tuple(kv)
        return out

    def reference(self):
        """(output, bound): the oracle's output and how far the library's may be off.

        With u half a step of the type (2^-8 bf16, 2^-24 fp32), an output differs by at most
          u |o|                             its own rounding,
          (u_p + 2 ds) sum_t p_t |v_t|      probabilities rounded to bf16 (u_p), scores off by ds,
          u_v sum_t p_t |v_t|               4-bit values dequantised to bf16,
        to first order, where ds = scale * sum_d (u_q |q a k| + u_k |q a k|): the query times the
        key weights is held in two bf16 halves (u_q = 2^-16, weighted modes; over 4-bit caches in one,
        2^-8), 4-bit keys in one (u_k).  fp32 sums
        of n terms add n 2^-24 of the sum of their magnitudes (D terms a score, the rows a value;
        rows above 1024 add in random order and are counted as 1024).
        """
        caches = self.plain_caches()
        kc, vc = {l: c[0] for l, c in caches.items()}, {l: c[1] for l, c in caches.items()}
        ws = {3: tuple(f64(x) for x in self.w)}
        k, v = O.reconstruct_kv(self.layer, 4, self.mode, kc, vc, ws)
        q = f64(self.q)
        ref = O.tree_attention(q, k, v, self.lens, self.masks, self.counts, self.scale, self.window)
        # magnitudes, with every product's absolute value
        aw = {3: tuple(np.abs(x) for x in ws[3])}
        ka, va = O.reconstruct_kv(self.layer, 4, self.mode, {l: np.abs(x) for l, x in kc.items()},
                                  {l: np.abs(x) for l, x in vc.items()}, aw)
        u16, u32 = ULP["bf16"], ULP["f32"]
        f32 = self.fmt == "f32"
        weighted = self.mode in ("fused", "scaled")
        u_o = u32 * 4 if f32 else u16
        u_p = 0.0 if f32 else u16
        u_q = (u16 if self.fmt == "q4" else u16 * u16) if weighted and not f32 else 0.0
        u_k = u_v = u16 if self.fmt == "q4" else 0.0
        bound = np.full(ref.shape, np.inf)
        for b in range(self.Bt):
            P, N = self.lens[b], self.T if self.counts is None else self.counts[b]
            if N <= 0:
                continue
            bits = np.array([[(self.masks[b][i] >> j) & 1 for j in range(N)] for i in range(N)], bool)
            depth = np.maximum(bits.sum(1) - 1, 0)
            see = np.concatenate([np.ones((N, P), bool), bits], 1)
            if self.window:
                key = np.concatenate([np.arange(P), P + depth])
                see &= key[None, :] > (P + depth)[:, None] - self.window
            for h in range(self.H * self.G):
                kk, vv = k[b, h // self.G, :P + N], v[b, h // self.G, :P + N]
                qq = q[b, h, :N]
                s = np.where(see, self.scale * qq @ kk.T, -np.inf)
                top = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
                mag = self.scale * np.abs(qq) @ ka[b, h // self.G, :P + N].T
                ds = (u_q + u_k + (2 * self.D + 16) * u32) * mag
                terms = min(P + N, 1024) + 16
                w = p * (u_p + u_v + 2 * np.where(see, ds, 0.0).max(1, keepdims=True) + terms * u32)
                bound[b, h, :N] = u_o * np.abs(ref[b, h, :N]) + w @ va[b, h // self.G, :P + N]
        return ref, bound + 1e-30

    def check(self, what=""):
        ref, bound = self.reference()
        got = f64(self.out)
        left = np.isnan(ref)                        # nodes that do not exist
        assert (got[left] == -77.0).all(), "%s: rows of missing nodes were written" % what
        got, ref, bound = got[~left], ref[~left], bound[~left]
        assert np.isfinite(got).all(), "%s: non-finite output" % what
        err = np.abs(got - ref)
        worst = float((err / bound).max()) if err.size else 0.0
        assert worst <= 1.0, "%s: error %.3g of its bound (max-abs %.3g)" % (what, worst, err.max())
        den = float(np.linalg.norm(ref))
        rel = float(np.linalg.norm(got - ref)) / den if den else 0.0
        bar = 1e-5 if self.fmt == "f32" else BF16_REL_L2
        assert rel <= bar, "%s: rel-L2 %.3g" % (what, rel)
        return worst, rel
