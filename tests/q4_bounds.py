"""How far a tree call over 4-bit caches may be from the oracle: its operands are
fp16 (half a step is 2^-11 of a value, 2^-25 below 2^-14), with a power of two
per query row where the row leaves fp16's range."""

from __future__ import annotations

import numpy as np
import torch

import oracle as O
from parity import f64

U11, U25, U16, U32 = 2.0 ** -11, 2.0 ** -25, 2.0 ** -8, 2.0 ** -24


def params(s, x):
    """The (scale, minimum) pairs of records as bf16 [..., 2 * D / 16], a view."""
    return x.view(torch.bfloat16)[..., s.D // 4:s.D // 4 + s.D // 8]


# absolute error of a key or value beside 2^-11 of it: three roundings (scale,
# minimum, value) below 2^-14
FLOOR = 3 * U25


def reference(s):
    """(output, bound) of a TreeSetup over 4-bit full-length caches.

    The output's own rounding (2^-8); probabilities: 2^-11 of them, 2^-25 in units where the
    reference is 2^4 (2^-29 of a column's sum); values and keys as above; query times weight 2^-11
    (exact without weights) and 2^-25 of its row's largest (or of 1); fp32 sums as in
    TreeSetup.reference."""
    n = 2
    two = s.mode == "fused"
    ks, vs = ([1, n], [1, n]) if two else ([n], [1])
    assert s.mode in ("lite", "scaled", "fused") and not s.ring
    kf = {l: O.q4_dequantize_records(s.k[l].cpu().numpy(), s.D) for l in (1, 2)}
    vf = {l: O.q4_dequantize_records(s.v[l].cpu().numpy(), s.D) for l in (1, 2)}
    w = [f64(x) for x in s.w]
    weighted = s.mode != "lite"
    aw = [w[0], w[1]] if two else [w[0] if weighted else np.ones_like(w[0])]
    bw = [w[2], w[3]] if two else [w[2] if weighted else np.ones_like(w[2])]
    q = f64(s.q)
    k = sum(a[None, :, None] * kf[l] for a, l in zip(aw, ks))
    v = sum(b[None, :, None] * vf[l] for b, l in zip(bw, vs))
    ref = O.tree_attention(q, k, v, s.lens, s.masks, s.counts, s.scale, s.window)
    bound = np.full(ref.shape, np.inf)
    for b in range(s.Bt):
        P, N = s.lens[b], s.T if s.counts is None else s.counts[b]
        if N <= 0:
            continue
        bits = np.array([[(s.masks[b][i] >> j) & 1 for j in range(N)] for i in range(N)], bool)
        depth = np.maximum(bits.sum(1) - 1, 0)
        see = np.concatenate([np.ones((N, P), bool), bits], 1)
        if s.window:
            key = np.concatenate([np.arange(P), P + depth])
            see &= key[None, :] > (P + depth)[:, None] - s.window
        for h in range(s.H * s.G):
            hk = h // s.G
            rows = slice(0, P + N)
            qq = q[b, h, :N]
            sc = np.where(see, s.scale * qq @ k[b, hk, rows].T, -np.inf)
            top = sc.max(1, keepdims=True)
            p = np.exp(sc - np.where(np.isfinite(top), top, 0.0))
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
            mag, ds = 0.0, 0.0
            qa = [qq * a[hk][None] for a in aw]
            qtop = np.maximum(np.max([np.abs(x).max(1) for x in qa], axis=0), 1.0)[:, None]
            for x, l in zip(qa, ks):
                kk = np.abs(kf[l][b, hk, rows])
                x = np.abs(x)
                mag = mag + x @ kk.T
                ds = ds + x @ (U11 * kk + FLOOR).T
                ds = ds + ((U11 if weighted else 0.0) * x + U25 * qtop) @ kk.T
            ds = s.scale * (ds + (2 * s.D + 16) * U32 * mag)
            ds = np.where(see, ds, 0.0).max(1, keepdims=True)
            va = sum(np.abs(bb[hk])[None] * np.abs(vf[l][b, hk, rows]) for bb, l in zip(bw, vs))
            vfl = sum(np.abs(bb[hk])[None] for bb in bw) * FLOOR
            terms = min(P + N, 1024) + 16
            lost = ds[:, 0] > 10                    # scores of thousands: no bound
            grow = np.expm1(2 * np.minimum(ds, 10))   # scores off by ds either way
            bound[b, h, :N] = (U16 * np.abs(ref[b, h, :N]) +
                               (p * (2 * U11 + grow + terms * U32)) @ va +
                               (see * U25 / 16) @ va + (1 + grow) * p.sum(1, keepdims=True) * vfl)
            bound[b, h, :N][lost] = np.inf
    return ref, bound * 1.01 + 1e-30              # second-order terms


def check(s, what=""):
    ref, bound = reference(s)
    got = f64(s.out)
    live = ~np.isnan(ref)
    assert np.isfinite(got[live]).all(), "%s: non-finite output" % what
    err = np.abs(got - ref)[live]
    worst = float((err / bound[live]).max())
    assert worst <= 1.0, "%s: %.3g of the bound" % (what, worst)
    return worst
