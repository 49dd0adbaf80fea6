"""Shared helpers of the 8-bit cache tests: caches, a float64 reference, and error bounds
derived from the arithmetic.  Test infrastructure only."""

from __future__ import annotations

import math

import torch

from cross_layer_kv_gb300 import fusedkv as B

BLOCK = 32


def cols(rows):
    return (rows + 127) // 128 * 4


def make_plane(gen, batch, heads, rows, D, spread=1.0, device="cuda", powers=True):
    """Random codes and scales of one plane: values of about unit size, times a
    factor 2^k, |k| <= 3 * spread, that changes from block to block."""
    x = torch.randn(batch, heads, rows, D, generator=gen, device=device) * 64
    codes = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    k = torch.randn(batch, heads, cols(rows), generator=gen, device=device).clamp(-3, 3) * spread
    if powers:
        k = k.round()
    return codes, torch.exp2(k - 6)


def values(plane):
    """A plane in float64."""
    codes, scales = plane
    rows = codes.shape[2]
    at = torch.arange(rows, device=codes.device) // BLOCK
    return codes.double() * scales[:, :, at, None].double()


def reconstruct(mode, w, k, v):
    """K^i, V^i in float64 of the sources' values (lists of one or two)."""
    if mode in ("vanilla", "lite"):
        return k[0], v[0]
    w = [x.double()[None, :, None, :] for x in w]
    if mode == "scaled":
        return w[0] * k[0], w[2] * v[0]
    return w[0] * k[0] + w[1] * k[1], w[2] * v[0] + w[3] * v[1]


def attend(q, K, V, scale, see):
    """softmax(scale q K^T) V in float64 with the visible keys `see` [T, S]; q [T, D].  Also the
    largest sum of absolute products of a score, and sum p |V|."""
    s = (q @ K.T) * scale
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top == -math.inf, 0.0, top)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    size = (q.abs() @ K.abs().T * abs(scale)).masked_fill(~see, 0.0).amax(-1, keepdim=True)
    return p @ V, size, p @ V.abs()


def decode_bound(ref, size, pv, D, n, dtype):
    """How far fp32 arithmetic may be off: a score is a sum of 2 D products with prescaled queries
    (three roundings each) and their scales, the exponential and its base add 2^-21, a softmax
    weight is off by twice a score's error, and n weighted values are added up in fp32; then one
    rounding of the output.  bf16 contexts round each weight to fp16 for its product with a value
    (the softmax's sum takes it unrounded): a factor 1 + d, |d| <= 2^-11, on each term of sum p V,
    so at most 2^-11 sum p |V|."""
    u, w = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 0.0)
    score = (2 * D + 8) * 2.0 ** -24 * size + 2.0 ** -21
    return (2 * score + w + (n + 64) * 2.0 ** -24) * pv + u * ref.abs()


class Setup:
    """A context over 8-bit caches: the storage layers that a layer's mode reads."""

    def __init__(self, mode, batch, seq, heads, group, D, dtype="bf16", layers=6, window=0, ring=0, seed=0,
                 spread=1.0, powers=True, decode_ctas=0, softmax_scale=0.0):
        self.mode, self.D, self.G, self.H, self.batch, self.seq = mode, D, group, heads, batch, seq
        self.window, self.ring, self.dtype = window, ring, dtype
        self.scale = softmax_scale or 1.0 / math.sqrt(D)
        n = layers // 2
        rows = ring or seq
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx = B.Context(layers, batch, seq, heads * group, heads, D, dtype, decode_ctas=decode_ctas,
                             softmax_scale=softmax_scale)
        two = mode == "fused"
        self.layer = 2 if mode == "vanilla" else layers
        read = [2] if mode == "vanilla" else [1, n]
        self.planes = {l: tuple(make_plane(g, batch, heads, rows, D, spread, powers=powers) for _ in range(2))
                       for l in read}
        for l, (k, v) in self.planes.items():
            if ring:
                self.ctx.fkv_set_ring_rows(l, ring)
            self.ctx.fkv_bind_layer_cache_q8(l, k[0], v[0], k[1], v[1])
        if window:
            self.ctx.fkv_set_window(self.layer, window)
        self.w = [(torch.randn(heads, D, generator=g, device="cuda") * 0.3 + 0.5) for _ in range(4)]
        if mode in ("scaled", "fused"):
            self.ctx.fkv_set_fusion_weights(self.layer, *self.w)
        if mode == "vanilla":
            self.k, self.v = [self.planes[2][0]], [self.planes[2][1]]
        elif two:
            self.k, self.v = [self.planes[1][0], self.planes[n][0]], [self.planes[1][1], self.planes[n][1]]
        else:
            self.k, self.v = [self.planes[n][0]], [self.planes[1][1]]
        self.torch_dtype = torch.float32 if dtype == "f32" else torch.bfloat16

    def rows(self):
        return reconstruct(self.mode, self.w, [values(x) for x in self.k], [values(x) for x in self.v])

    def query(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(self.torch_dtype)

    def close(self):
        self.ctx.close()


def check_decode(s, lens, q=None, what=""):
    """One decode call against the reference, element by element."""
    q = s.query(s.batch, s.H * s.G, s.D) if q is None else q
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_decode_attn(q, s.layer, s.mode, torch.tensor(lens, dtype=torch.int32, device="cuda"), out,
                          s.ctx.workspace())
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    K, V = s.rows()
    worst = 0.0
    for b, L in enumerate(lens):
        pos = torch.arange(max(0, L - s.window) if s.window else 0, L, device="cuda")
        at = pos % s.ring if s.ring else pos
        for h in range(s.H):
            see = torch.ones(s.G, len(pos), dtype=torch.bool, device="cuda")
            ref, size, pv = attend(q[b, h * s.G:(h + 1) * s.G].double(), K[b, h, at], V[b, h, at], s.scale, see)
            err = (out[b, h * s.G:(h + 1) * s.G].double() - ref).abs()
            bound = decode_bound(ref, size, pv, s.D, len(pos), s.dtype)
            worst = max(worst, float((err / bound).max()))
            assert bool((err <= bound).all()), "%s b=%d h=%d: %.2f of the bound" % (what, b, h, worst)
    return out, worst


def check_prefill(s, q_start, C, q=None, what="", rows=None):
    """One chunk against the reference, element by element (`rows`: of these chunk rows only)."""
    q = s.query(s.batch, s.H * s.G, C, s.D) if q is None else q
    out = torch.full_like(q, float("nan"))
    s.ctx.fkv_prefill_attn_chunk(q, s.layer, s.mode, q_start, C, out)
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    K, V = s.rows()
    w = [x.abs() for x in s.w]
    Ka, Va = reconstruct(s.mode, w, [values(x).abs() for x in s.k], [values(x).abs() for x in s.v])
    lo = max(0, q_start - s.window + 1) if s.window else 0
    pos = torch.arange(lo, q_start + C, device="cuda")
    at = pos % s.ring if s.ring else pos
    sel = torch.arange(C, device="cuda") if rows is None else torch.tensor(rows, device="cuda")
    mine = (q_start + sel)[:, None]
    see = pos <= mine
    if s.window:
        see = see & (pos > mine - s.window)
    # fp16 operands, 2^-11 a rounding.  Two sources: a weight, a ratio of scales and a product
    # each round once, and their sum; a scaled query once.  P rounds once.
    h = 2.0 ** -11
    k_round = {"fused": 4, "scaled": 1}.get(s.mode, 0) * h
    v_round = (1 + (4 if s.mode == "fused" else 0)) * h
    n, worst = len(pos), 0.0
    for b in range(s.batch):
        for kh in range(s.H):
            for g in range(kh * s.G, (kh + 1) * s.G):
                qq = q[b, g, sel].double()
                ref, _, _ = attend(qq, K[b, kh, at], V[b, kh, at], s.scale, see)
                sc = (qq @ K[b, kh, at].T * s.scale).masked_fill(~see, -math.inf)
                p = torch.softmax(sc, -1)
                size = (qq.abs() @ Ka[b, kh, at].T * s.scale).masked_fill(~see, 0.0).amax(-1, keepdim=True)
                pv = p @ Va[b, kh, at]
                score = (k_round + (2 * s.D + 8) * 2.0 ** -23) * size + 2.0 ** -21
                top = Va[b, kh, at].max()
                # P below 2^-32 of its frame may vanish
                bound = (2 * score + v_round + (n + 64) * 2.0 ** -23) * pv + n * 2.0 ** -31 * top + 2.0 ** -8 * ref.abs()
                err = (out[b, g, sel].double() - ref).abs()
                worst = max(worst, float((err / bound).max()))
                assert bool((err <= bound).all()), "%s b=%d h=%d: %.2f of the bound" % (what, b, g, worst)
    return out, worst
