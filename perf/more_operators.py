"""8-bit KV caches with a scale for each block of tokens and head: what is measured.

A layer's K or V cache holds e4m3 codes ``[B, H_kv, rows, D]`` and fp32 scales
``[B, H_kv, cols]``, one for every 32 rows of a KV head (``cols`` is a multiple of 4); a value is
its code times its block's scale.  Four operators:

* ``write``: new keys and values quantised into the cache as they are appended, then read back as
  the layer's attention sees them (a row that starts a block starts its scale, a row that joins
  one may raise the scale of the rows before it);
* ``read``: rows of a layer read back in every mode (its own, Lite, scaled, fused from two
  layers);
* ``decode``: attention of one token per sequence over 8-bit caches;
* ``prefill``: causal attention of a prompt, or of a chunk of one behind cached rows.

A case is a dict of plain values; sizes are those of the repository's workloads (332M, 650M, 1.5B
and 4B shapes) or generic.
"""

import math
import random

import torch

own = False

_DEV = "cuda"
_BLOCK = 32          # rows that share a scale
_TOP = 448.0         # the largest e4m3 value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name, layers, batch, seq, q_heads, kv_heads, head_dim, mode, rows, dtype="bf16", ragged=True,
          window=0, ring=0):
    """`rows`: new rows (write), rows read (read), chunk length (prefill); `seq`: capacity of a sequence."""
    c = dict(op=op, layers=layers, batch=batch, seq=seq, q_heads=q_heads, kv_heads=kv_heads,
             head_dim=head_dim, mode=mode, rows=rows, dtype=dtype, ragged=ragged, window=window, ring=ring)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one fp32 token of one user joins a block: latency
        _case("write", "write-tiny-f32", 4, 1, 256, 4, 2, 64, "vanilla", 1, dtype="f32"),
        # a decode step's token of a batch of users
        _case("write", "write-332M-token", 12, 32, 8192, 16, 8, 64, "vanilla", 1),
        # prompts of a batch, odd length, starting inside blocks
        _case("write", "write-1.5B-prompt", 24, 16, 4096, 16, 8, 128, "vanilla", 2001),
        # a few recent rows of a reconstruction layer
        _case("read", "read-332M-fused", 12, 32, 8192, 16, 8, 64, "fused", 77),
        # a long prefix handed on in bf16
        _case("read", "read-4B-lite", 36, 4, 32768, 32, 16, 80, "lite", 16384),
        # one small fp32 model: latency
        _case("decode", "decode-tiny-f32", 4, 1, 256, 4, 2, 64, "fused", 1, dtype="f32", ragged=False),
        # a hybrid model's window layer over ring caches
        _case("decode", "decode-650M-ring", 16, 16, 8192, 16, 8, 96, "vanilla", 1, window=512, ring=896),
        # a batch of users at long contexts
        _case("decode", "decode-332M-lite", 12, 32, 8192, 16, 8, 64, "lite", 1, ragged=False),
        # few users at very long contexts
        _case("decode", "decode-4B-fused", 36, 4, 131072, 32, 16, 80, "fused", 1),
        # a chunk of a prompt over wrapped ring caches
        _case("prefill", "prefill-650M-ring", 16, 2, 8192, 16, 8, 96, "lite", 300, window=512, ring=896),
        # a whole prompt
        _case("prefill", "prefill-650M-lite", 16, 4, 8192, 16, 8, 96, "lite", 8192),
        # a chunk of a long prompt in a reconstruction layer, odd length
        _case("prefill", "prefill-1.5B-fused", 24, 4, 8192, 16, 8, 128, "fused", 1023),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode", "prefill", "prefill"))
    layers = 2 * rng.randint(2, 18)
    head_dim = rng.choice((64, 80, 96, 128))
    kv_heads = rng.randint(1, 16)
    group = rng.choice((1, 2, 2, 4))
    dtype = "bf16" if op == "prefill" else rng.choice(("bf16", "bf16", "bf16", "f32"))
    mode = rng.choice(("vanilla", "lite", "fused", "fused", "scaled"))
    row = head_dim * kv_heads * (8 if mode == "fused" and op != "write" else 4)   # about a position's bytes
    window, ring = 0, 0
    if op == "write":
        batch = _log_int(rng, 1, 48)
        rows = _log_int(rng, 1, max(1, min(4096, int(1e8 / (row * batch)))))
        seq = rows + rng.randint(100, 1000)
        if rng.random() < 0.25:
            ring = _BLOCK * ((rows + 63) // _BLOCK + rng.randint(1, 8))
            seq = ring + rng.randint(rows + 70, 3 * ring + rows + 70)
        return _case(op, "", layers, batch, seq, kv_heads * group, kv_heads, head_dim, "vanilla", rows,
                     dtype=dtype, ring=ring)
    if op == "read":
        batch = _log_int(rng, 1, 48)
        rows = _log_int(rng, 1, max(1, min(20000, int(2e8 / (row * batch)))))
        return _case(op, "", layers, batch, rows + rng.randint(0, 500), kv_heads * group, kv_heads, head_dim,
                     mode, rows, dtype=dtype)
    if op == "decode":
        batch = _log_int(rng, 1, 48)
        most = (1e8 if dtype == "f32" else 1e9) / (row * batch)
        seq = _log_int(rng, 160, max(161, min(131072, int(most))))
        if rng.random() < 0.25:
            window = rng.randint(1, max(1, seq - 64))
            ring = rng.choice((0, _BLOCK * ((window + 2 * _BLOCK) // _BLOCK + rng.randint(0, 3))))
            ring = ring if ring < seq else 0
        return _case(op, "", layers, batch, seq, kv_heads * group, kv_heads, head_dim, mode, 1, dtype=dtype,
                     ragged=rng.random() < 0.8, window=window, ring=ring)
    # at most about half of the largest listed call's products
    batch = _log_int(rng, 1, 8)
    rows = _log_int(rng, 1, 4096)
    most = int(4e11 / (4.0 * batch * kv_heads * group * head_dim * rows))
    seq = rows + (0 if rng.random() < 0.4 else _log_int(rng, 1, max(1, min(16384, most))))
    if rng.random() < 0.25:
        window = rng.randint(1, 1000)
        ring = rng.choice((0, _BLOCK * ((rows + window + 2 * _BLOCK) // _BLOCK + rng.randint(0, 3))))
        ring = ring if ring < seq else 0
    return _case(op, "", layers, batch, seq, kv_heads * group, kv_heads, head_dim, mode, rows, window=window,
                 ring=ring)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, salt):
    return torch.Generator(device=_DEV).manual_seed(seed * 1000 + salt)


def _dt(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _cols(rows):
    return (rows + 127) // 128 * 4


def _need(amax):
    """The smallest power of two whose 448-fold reaches amax (frexp: amax = m * 2^x, 1/2 <= m < 1),
    made from its exponent's bits."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(-100, 119)
    return ((torch.where(amax > 0, e, -100) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Whole rows [B, H, rows, D] -> codes, scales."""
    B, H, R, D = x.shape
    nb = (R + _BLOCK - 1) // _BLOCK
    pad = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * _BLOCK - R)).view(B, H, nb, _BLOCK, D)
    s = _need(pad.abs().amax((-1, -2)))
    codes = (pad / s[..., None, None]).view(B, H, nb * _BLOCK, D)[:, :, :R].to(torch.float8_e4m3fn)
    scales = torch.zeros(B, H, _cols(R), device=_DEV)
    scales[..., :nb] = s
    return codes.contiguous(), scales


def _cache(c, seed, salt):
    """One layer's K or V cache of keys or values that differ in size from head to head, as
    (codes, scales); a batch row at a time, so that the wide values stay few."""
    R, H, D = c["ring"] or c["seq"], c["kv_heads"], c["head_dim"]
    gen = _gen(seed, salt)
    codes = torch.empty(c["batch"], H, R, D, dtype=torch.float8_e4m3fn, device=_DEV)
    scales = torch.empty(c["batch"], H, _cols(R), device=_DEV)
    size = torch.exp(0.3 * torch.randn(H, 1, 1, generator=gen, device=_DEV))
    for b in range(c["batch"]):
        x = torch.randn(1, H, R, D, generator=gen, device=_DEV) * size
        q, s = _quantise(x)
        codes[b:b + 1].view(torch.uint8).copy_(q.view(torch.uint8))
        scales[b:b + 1] = s
    return codes, scales


def _lens(c, seed):
    r = random.Random(seed * 7919 + 1)
    hi = c["seq"]
    return [r.randint(max(1, hi // 2), hi) if c["ragged"] else hi for _ in range(c["batch"])]


def _starts(c, seed):
    """First position written or read of each sequence."""
    r = random.Random(seed * 104729 + 2)
    if c["op"] == "write":
        hi = c["seq"] - c["rows"] - 64
        lo = min(hi, c["ring"]) if c["ring"] else _BLOCK - 1
        return [r.randint(lo, hi) for _ in range(c["batch"])]
    return [r.randint(0, c["seq"] - c["rows"]) for _ in range(c["batch"])]


def prepare(case, seed):
    c = case
    n, D, op = c["layers"] // 2, c["head_dim"], c["op"]
    two = c["mode"] == "fused"
    layer = 1 if c["mode"] == "vanilla" else n + 1
    w = torch.randn(4, c["kv_heads"], D, generator=_gen(seed, 9), device=_DEV) * 0.3 + 0.5
    w[:2, :, D // 2:] = w[:2, :, : D // 2]      # key weights are tied across rotation pairs
    st = dict(c=c, layer=layer, w=[x.contiguous() for x in w.unbind(0)],
              k=[_cache(c, seed, 1)] + ([_cache(c, seed, 2)] if two else []),
              v=[_cache(c, seed, 3)] + ([_cache(c, seed, 4)] if two else []))
    shape = (c["batch"], c["kv_heads"], c["rows"], D)
    if op == "write":
        # some heads' new rows are larger than all before them and raise their blocks' scales
        size = torch.exp(torch.randn(c["kv_heads"], 1, 1, generator=_gen(seed, 10), device=_DEV))
        st["k_new"], st["v_new"] = ((torch.randn(shape, generator=_gen(seed, s), device=_DEV) * size).to(_dt(c))
                                    for s in (5, 6))
        at = _starts(c, seed)
        back = _BLOCK - 1                        # rows before the new ones, whose codes may have changed
        back = min(back, c["ring"] - c["rows"] - _BLOCK) if c["ring"] else back
        st.update(pos=torch.tensor(at, dtype=torch.int32, device=_DEV), at=at, back=back, total=c["rows"] + back,
                  first=torch.tensor([p - back for p in at], dtype=torch.int32, device=_DEV))
    elif op == "read":
        st.update(total=c["rows"], first=torch.tensor(_starts(c, seed), dtype=torch.int32, device=_DEV))
    if op in ("write", "read"):
        out = (c["batch"], c["kv_heads"], st["total"], D)
        st["k_out"], st["v_out"] = (torch.empty(out, dtype=_dt(c), device=_DEV) for _ in range(2))
    else:
        q = (c["batch"], c["q_heads"], D) if op == "decode" else (c["batch"], c["q_heads"], c["rows"], D)
        st["q"] = torch.randn(q, generator=_gen(seed, 5), device=_DEV, dtype=_dt(c))
        st["out"] = torch.empty_like(st["q"])
        lens = _lens(c, seed)
        st.update(lens=torch.tensor(lens, dtype=torch.int32, device=_DEV), longest=max(lens),
                  start=c["seq"] - c["rows"])
    if own:
        from cross_layer_kv_gb300 import Context
        ctx = Context(c["layers"], c["batch"], c["seq"], c["q_heads"], c["kv_heads"], D, c["dtype"])
        # fused: K^1, K^n, V^1, V^n; lite and scaled: K^n and V^1, here one layer's pair
        for l, i in ((1, 0), (n, 1)) if two else ((1, 0),):
            if c["ring"]:
                ctx.fkv_set_ring_rows(l, c["ring"])
            ctx.fkv_bind_layer_cache_q8(l, st["k"][i][0], st["v"][i][0], st["k"][i][1], st["v"][i][1])
        if layer > n:
            if not two:
                ctx.fkv_set_sources(layer, c["mode"], 1, 0, 1, 0)
            ctx.fkv_set_fusion_weights(layer, *st["w"])
        if c["window"]:
            ctx.fkv_set_window(layer, c["window"])
        st["ctx"] = ctx
        if op == "decode":
            st["workspace"] = ctx.workspace()
    return st


# ---------------------------------------------------------------------------
# one pass, plain form
# ---------------------------------------------------------------------------

def _values(cache, first=0, last=None):
    """Cache rows [first, last) in 32 bits."""
    codes, scales = cache
    last = codes.shape[2] if last is None else last
    block = torch.arange(first, last, device=_DEV) // _BLOCK
    return codes[:, :, first:last].float() * scales[:, :, block, None]


def _fuse(c, w, x, which):
    w0, w1 = (w[0], w[1]) if which == "k" else (w[2], w[3])
    if c["mode"] == "fused":
        return w0[None, :, None] * x[0] + w1[None, :, None] * x[1]
    return w0[None, :, None] * x[0] if c["mode"] == "scaled" else x[0]


def _plain_append(c, cache, new, pos):
    codes, scales = cache
    raw = codes.view(torch.uint8)
    T, B, H, D = c["rows"], c["batch"], c["kv_heads"], c["head_dim"]
    nb = (T + _BLOCK - 2) // _BLOCK + 1
    pos = pos.long()
    block = pos[:, None] // _BLOCK + torch.arange(nb, device=_DEV)                      # [B, nb]
    at = block[..., None] * _BLOCK + torch.arange(_BLOCK, device=_DEV)                  # [B, nb, 32]
    t = at - pos[:, None, None]
    fresh_row = (t >= 0) & (t < T)
    slot = block % (c["ring"] // _BLOCK) if c["ring"] else block
    row = (slot[..., None] * _BLOCK + torch.arange(_BLOCK, device=_DEV)).view(B, -1)
    b = torch.arange(B, device=_DEV)[:, None]
    old = raw[b, :, row].view(B, nb, _BLOCK, H, D)
    x = new[b, :, t.clamp(0, T - 1).view(B, -1)].view(B, nb, _BLOCK, H, D).float()
    finite = torch.isfinite(x) & fresh_row[..., None, None]
    need = _need(torch.where(finite, x.abs(), 0.0).amax((2, 4)))                        # [B, nb, H]
    s_old = scales[b, :, slot]
    s = torch.where((block * _BLOCK >= pos[:, None])[..., None], need, torch.maximum(s_old, need))
    s = torch.where(fresh_row.any(-1)[..., None], s, s_old)
    step = s[:, :, None, :, None]
    moved = old.view(torch.float8_e4m3fn).float() * (s_old / s)[:, :, None, :, None]
    y = torch.where(fresh_row[..., None, None], x / step, moved).clamp(-_TOP, _TOP)
    y = y.to(torch.float8_e4m3fn).view(torch.uint8)
    raw[b, :, row] = y.view(B, -1, H, D)
    scales[b, :, slot] = s


def _plain_rows(st, which):
    """Rows first .. first + total - 1 of every sequence as the layer sees them."""
    c = st["c"]
    at = st["first"].long()[:, None] + torch.arange(st["total"], device=_DEV)
    row = at % c["ring"] if c["ring"] else at
    b = torch.arange(c["batch"], device=_DEV)[:, None]
    xs = [(codes.view(torch.uint8)[b, :, row].view(torch.float8_e4m3fn).float()
           * scales[b, :, row // _BLOCK][..., None]).transpose(1, 2) for codes, scales in st[which]]
    return _fuse(c, st["w"], xs, which).to(_dt(c)).contiguous()


def _plain_decode(st):
    c = st["c"]
    B, H, D = c["batch"], c["kv_heads"], c["head_dim"]
    rows = c["ring"] or st["longest"]
    out = torch.empty_like(st["q"])
    step = max(1, int(1.5e9 // (H * rows * D)))
    at = torch.arange(rows, device=_DEV)
    lens = st["lens"].long()[:, None]
    if c["ring"]:
        at = lens - 1 - (lens - 1 - at) % c["ring"]       # row r holds the last position of its residue
    see = (at < lens) & (at >= 0)
    if c["window"]:
        see = see & (at > lens - 1 - c["window"])
    for b in range(0, B, step):
        e = min(B, b + step)
        k = _fuse(c, st["w"], [_values((x[b:e], s[b:e]), 0, rows) for x, s in st["k"]], "k")
        q = st["q"][b:e].float().view(e - b, H, -1, D)
        s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
        del k
        s = s.masked_fill(~see[b:e, None, None], -math.inf)
        p = (s - s.amax(-1, keepdim=True)).exp()
        v = _fuse(c, st["w"], [_values((x[b:e], s_[b:e]), 0, rows) for x, s_ in st["v"]], "v")
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[b:e] = o.view(e - b, -1, D).to(out.dtype)
    return out


def _plain_prefill(st):
    c, start, T = st["c"], st["start"], st["c"]["rows"]
    H, D, G = c["kv_heads"], c["head_dim"], c["q_heads"] // c["kv_heads"]
    S = c["seq"]
    first = max(0, start - c["window"] + 1) if c["window"] else 0
    pos = torch.arange(first, S, device=_DEV)
    row = pos % c["ring"] if c["ring"] else pos
    mine = torch.arange(start, S, device=_DEV)[:, None]
    hidden = pos > mine
    if c["window"]:
        hidden = hidden | (pos <= mine - c["window"])
    out = torch.empty_like(st["q"])
    for b in range(c["batch"]):
        k, v = (_fuse(c, st["w"], [_values((x[b:b + 1], s[b:b + 1]))[:, :, row] for x, s in st[n]], n)[0]
                for n in ("k", "v"))
        for h in range(H):
            q = st["q"][b, h * G:(h + 1) * G].float()
            s = torch.matmul(q, k[h].T).mul_(1.0 / math.sqrt(D)).masked_fill_(hidden, -math.inf)
            p = s.sub_(s.amax(-1, keepdim=True)).exp_()
            out[b, h * G:(h + 1) * G] = (torch.matmul(p, v[h]) / p.sum(-1, keepdim=True)).to(out.dtype)
    return out


def run(state):
    st, c = state, state["c"]
    op = c["op"]
    if op in ("write", "read"):
        if own:
            if op == "write":
                st["ctx"].fkv_append_kv(st["layer"], st["k_new"], st["v_new"], st["pos"])
            st["ctx"].fkv_read_kv(st["layer"], c["mode"], st["first"], st["k_out"], st["v_out"])
            k, v = st["k_out"], st["v_out"]
        else:
            if op == "write":
                _plain_append(c, st["k"][0], st["k_new"], st["pos"])
                _plain_append(c, st["v"][0], st["v_new"], st["pos"])
            k, v = _plain_rows(st, "k"), _plain_rows(st, "v")
        return (k, v, st["k"][0][1], st["v"][0][1]) if op == "write" else (k, v)
    if op == "decode":
        if own:
            return st["ctx"].fkv_decode_attn(st["q"], st["layer"], c["mode"], st["lens"], st["out"],
                                             st["workspace"])
        return _plain_decode(st)
    if own:
        return st["ctx"].fkv_prefill_attn_chunk(st["q"], st["layer"], c["mode"], st["start"], c["rows"], st["out"])
    return _plain_prefill(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    D, H, B, T = c["head_dim"], c["kv_heads"], c["batch"], c["rows"]
    elem = 4 if c["dtype"] == "f32" else 2
    planes = 4 if c["mode"] == "fused" else 2
    code = D + 4.0 / _BLOCK                        # bytes of a row of one plane
    if c["op"] == "write":
        # new rows in, codes out; the codes back in, values out
        return {"bytes": 2.0 * B * H * (T * (D * elem + code) + (T + _BLOCK / 2) * (code + D * elem)), "flops": 0.0}
    if c["op"] == "read":
        return {"bytes": B * H * T * (planes * code + 2.0 * D * elem), "flops": 0.0}
    if c["op"] == "decode":
        rows = c["seq"] * (0.75 if c["ragged"] else 1.0)
        rows = min(rows, c["window"]) if c["window"] else rows
        return {"bytes": planes * code * H * B * rows + 2.0 * B * c["q_heads"] * D * elem,
                "flops": 4.0 * B * c["q_heads"] * D * rows}
    start = c["seq"] - T
    if c["window"]:
        seen = sum(min(c["window"], start + i + 1) for i in range(T))
    else:
        seen = T * start + T * (T + 1) / 2
    keys = min(c["seq"], T + c["window"] - 1) if c["window"] else c["seq"]
    return {"bytes": planes * code * H * B * keys + 2.0 * B * c["q_heads"] * T * D * elem,
            "flops": 4.0 * B * c["q_heads"] * D * seen}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _wide(cache, b, h, at):
    """Rows `at` of one head in 64 bits."""
    codes, scales = cache
    return codes[b, h].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * scales[b, h][at // _BLOCK].double()[:, None]


def _power(e):
    """2^e in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(y):
    """To the nearest value with 3 fraction bits and exponents from -6, ties to even."""
    _, x = torch.frexp(y)
    unit = _power((x - 1).clamp(min=-6) - 3)
    return (torch.round(y / unit) * unit).clamp(-_TOP, _TOP)


def _exact_write(c, st, seed):
    at, T, D, B, H = st["at"], c["rows"], c["head_dim"], c["batch"], c["kv_heads"]
    outs, scales = [], []
    for which in ("k", "v"):
        codes, sc = st[which][0]
        new, sc = st[which + "_new"].double(), sc.double().clone()
        out = torch.zeros(B, H, st["total"], D, dtype=torch.float64, device=_DEV)
        for b, p in enumerate(at):
            lo = p - st["back"]
            pos = torch.arange(lo, p + T, device=_DEV)
            rows = pos % c["ring"] if c["ring"] else pos
            x = torch.stack([_wide(st[which][0], b, h, rows) for h in range(H)])
            x[:, st["back"]:] = new[b]
            for g in range(p // _BLOCK, (p + T - 1) // _BLOCK + 1):
                i, e = max(g * _BLOCK, lo) - lo, min(g * _BLOCK + _BLOCK, p + T) - lo
                n = max(g * _BLOCK, p) - lo
                slot = g % (c["ring"] // _BLOCK) if c["ring"] else g
                amax = x[:, n:e].abs().amax((1, 2))
                m, ex = torch.frexp(amax)
                s = _power(torch.where(amax > 0, (ex - 9 + (m > 0.875)).clamp(-100, 119), -100))
                if g * _BLOCK < p:
                    s = torch.maximum(s, sc[b, :, slot])
                sc[b, :, slot] = s
                x[:, i:e] = _round_e4m3(x[:, i:e] / s[:, None, None]) * s[:, None, None]
            out[b] = x
        outs.append(out)
        scales.append(sc)
    return (*outs, *scales)


def exact(case, seed):
    global own
    c = case
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if c["op"] == "write":
        if c["batch"] * c["rows"] > 60000:
            return None
        return _exact_write(c, st, seed)
    B, H, D, T = c["batch"], c["kv_heads"], c["head_dim"], c["rows"]
    wt = [x.double() for x in st["w"]]

    def rows_of(b, h, at):
        ks, vs = ([_wide(x, b, h, at) for x in st[n]] for n in ("k", "v"))
        if c["mode"] == "fused":
            return wt[0][h] * ks[0] + wt[1][h] * ks[1], wt[2][h] * vs[0] + wt[3][h] * vs[1]
        if c["mode"] == "scaled":
            return wt[0][h] * ks[0], wt[2][h] * vs[0]
        return ks[0], vs[0]

    if c["op"] == "read":
        k, v = (torch.zeros(B, H, T, D, dtype=torch.float64, device=_DEV) for _ in range(2))
        for b, f in enumerate(st["first"].tolist()):
            for h in range(H):
                k[b, h], v[b, h] = rows_of(b, h, torch.arange(f, f + T, device=_DEV))
        return k, v
    G = c["q_heads"] // H
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    lens = st["lens"].tolist()
    for b in range(B):
        end = lens[b] if c["op"] == "decode" else c["seq"]
        start = end - 1 if c["op"] == "decode" else st["start"]
        lo = max(0, start - c["window"] + 1) if c["window"] else 0
        pos = torch.arange(lo, end, device=_DEV)
        mine = torch.arange(start, end, device=_DEV)[:, None]
        see = pos <= mine
        if c["window"]:
            see &= mine - pos < c["window"]
        for h in range(H):
            k, v = rows_of(b, h, pos % c["ring"] if c["ring"] else pos)
            for g in range(h * G, (h + 1) * G):
                q = st["q"][b, g].double().view(-1, D)
                s = (q @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf)
                out[b, g] = (torch.softmax(s, -1) @ v).view(out[b, g].shape)
    return out
