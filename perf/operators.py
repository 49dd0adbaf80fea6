"""Speculative and beam decoding over cross-layer KV caches: what is measured.

Three operators over the caches of a context (``[B, H_kv, S, D]`` per stored layer):

* ``tree``: attention of a tree of drafted tokens over a cached prefix, in every mode of the
  framework (vanilla, lite, fused, scaled), on full-length, ring and 4-bit caches;
* ``compact``: after verification, the accepted nodes' rows of every layer move to the end of the
  committed prefix;
* ``reorder``: sequences of the batch become copies of others (beams that fork, prompts that are
  shared), in every layer.

A case is a dict of plain values; sizes are those of the repository's workloads (332M, 650M, 1.5B
and 4B shapes) or generic.
"""

import math

import torch

own = False

_DEV = "cuda"
_GROUP = 16          # channels per 4-bit group


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tree(name, layers, batch, seq, q_heads, kv_heads, head_dim, mode, nodes, dtype="bf16",
          ragged=True, window=0, ring=0):
    c = dict(op="tree", layers=layers, batch=batch, seq=seq, q_heads=q_heads, kv_heads=kv_heads,
             head_dim=head_dim, mode=mode, nodes=nodes, dtype=dtype, ragged=ragged, window=window,
             ring=ring)
    return dict(name=name, **c) if name else c


def _compact(name, layers, batch, seq, kv_heads, head_dim, nodes, accept, dtype="bf16"):
    c = dict(op="compact", layers=layers, batch=batch, seq=seq, kv_heads=kv_heads,
             head_dim=head_dim, nodes=nodes, accept=accept, dtype=dtype)
    return dict(name=name, **c) if name else c


def _reorder(name, layers, batch, seq, kv_heads, head_dim, beams, dtype="bf16"):
    c = dict(op="reorder", layers=layers, batch=batch, seq=seq, kv_heads=kv_heads,
             head_dim=head_dim, beams=beams, dtype=dtype)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one small fp32 model drafting for one user: latency
        _tree("tree-tiny-f32", 4, 1, 256, 4, 2, 64, "fused", 7, dtype="f32", ragged=False),
        # a batch of users, a short chain of drafts: the smallest trees served at scale
        _tree("tree-332M-lite-8", 12, 32, 8192, 16, 8, 64, "lite", 8),
        # the same model with a wide tree
        _tree("tree-332M-fused-64", 12, 32, 8192, 16, 8, 64, "fused", 64),
        # 4-bit caches, a mid-size tree
        _tree("tree-332M-q4-16", 12, 32, 8192, 16, 8, 64, "fused", 16, dtype="q4"),
        # a storage layer of a hybrid model: sliding window, ring cache, few rows: latency
        _tree("tree-650M-ring-12", 16, 4, 8192, 16, 8, 96, "vanilla", 12, window=512, ring=896),
        # long ragged contexts, a usual tree, odd size
        _tree("tree-1.5B-fused-26", 24, 16, 32768, 16, 8, 128, "fused", 26),
        # very long contexts, few users
        _tree("tree-4B-lite-16", 36, 4, 131072, 32, 16, 80, "lite", 16),
        # a step of verification in a small and in a deep model
        _compact("compact-332M", 12, 32, 2048, 8, 64, 64, 5),
        _compact("compact-4B", 36, 8, 2048, 16, 80, 48, 12),
        # one prompt forked into a few beams of a small model: latency
        _reorder("reorder-tiny-f32", 4, 4, 256, 2, 64, 4, dtype="f32"),
        # beam search over a batch of prompts, some beams die and fork from survivors
        _reorder("reorder-332M", 12, 32, 2048, 8, 64, 4),
        # a long shared prompt forked for parallel samples
        _reorder("reorder-4B", 36, 4, 8192, 16, 80, 4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "compact", "reorder"))
    layers = 2 * rng.randint(2, 18)
    head_dim = rng.choice((64, 80, 96, 128))
    kv_heads = rng.randint(1, 16)
    if op == "tree":
        dtype = rng.choice(("bf16", "bf16", "bf16", "bf16", "q4", "f32"))
        group = rng.choice((1, 2) if dtype == "q4" else (1, 2, 4))
        mode = rng.choice(("vanilla", "lite", "fused", "fused", "scaled"))
        nodes = rng.randint(1, 64)
        window, ring = 0, 0
        batch = _log_int(rng, 1, 48)
        # at most about 1.5 GB of cache a call, and for fp32 a smaller model's share of that
        row = (8 if mode == "fused" else 4) * head_dim * (2 if dtype == "f32" else 1)
        most = (6e7 if dtype == "f32" else 1.5e9) / (row * batch * kv_heads)
        seq = _log_int(rng, 160, max(161, min(65536, int(most))))
        if rng.random() < 0.25:
            window = rng.randint(1, max(1, seq - 130))
            ring = rng.choice((0, min(seq, window + nodes + rng.randint(0, 40))))
        return _tree("", layers, batch, seq, kv_heads * group, kv_heads, head_dim, mode, nodes,
                     dtype=dtype, ragged=rng.random() < 0.8, window=window, ring=ring)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "compact":
        nodes = rng.randint(16, 64)
        return _compact("", layers, _log_int(rng, 1, 32), rng.randint(512, 1500), kv_heads, head_dim,
                        nodes, rng.randint(1, 15), dtype=dtype)
    beams = rng.randint(2, 8)
    batch = beams * rng.randint(1, 4)
    row = layers * head_dim * (4 if dtype == "f32" else 2) * kv_heads * batch
    return _reorder("", layers, batch, _log_int(rng, 64, max(65, min(8192, int(1.5e9 / row)))), kv_heads,
                    head_dim, beams, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, salt):
    return torch.Generator(device=_DEV).manual_seed(seed * 1000 + salt)


def _lens(c, seed, room):
    """Committed rows of each sequence, with `room` rows left behind them."""
    import random
    r = random.Random(seed * 7919 + 1)
    hi = c["seq"] - room
    lo = max(1, hi // 2)
    return [r.randint(lo, hi) if c.get("ragged", True) else hi for _ in range(c["batch"])]


def _random_trees(c, seed):
    """Per sequence: the nodes' ancestor masks (self included) of a random tree whose nodes attach
    to the prefix or to one of the nodes before them."""
    import random
    r = random.Random(seed * 104729 + 2)
    rows = []
    for _ in range(c["batch"]):
        m = []
        for i in range(c["nodes"]):
            parent = r.randint(-1, i - 1) if r.random() < 0.5 else max(-1, i - r.randint(1, 4))
            m.append((m[parent] if parent >= 0 else 0) | (1 << i))
        rows.append(m)
    return rows


def _sources(c):
    """Number of stored layers that the attending layer reads for keys, and for values."""
    return 2 if c["mode"] == "fused" else 1


def _quantise(x):
    """Rows of D channels as 4-bit records: D/2 bytes of codes, (scale, min) in bf16 for every 16
    channels, padded to 16 bytes."""
    shape, D = x.shape[:-1], x.shape[-1]
    g = x.float().reshape(*shape, D // _GROUP, _GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo) / 15).to(torch.bfloat16)
    s = scale.float().unsqueeze(-1)
    code = torch.where(s > 0, torch.round((g - lo.unsqueeze(-1)) / torch.where(s > 0, s, 1.0)), 0.0)
    code = code.clamp(0, 15).to(torch.uint8).reshape(*shape, D)
    rec = torch.zeros(*shape, (D // 2 + D // 4 + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
    rec[..., : D // 2] = code[..., 0::2] | (code[..., 1::2] << 4)
    prm = torch.stack((scale, lo.to(torch.bfloat16)), -1).contiguous().view(torch.uint8)
    rec[..., D // 2: D // 2 + D // 4] = prm.reshape(*shape, D // 4)
    return rec


def _cache(c, seed, salt):
    """One layer's K or V cache: post-RoPE keys and values of unit variance."""
    rows = c.get("ring") or c["seq"]
    shape = (c["batch"], c["kv_heads"], rows, c["head_dim"])
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    x = torch.randn(shape, generator=_gen(seed, salt), device=_DEV, dtype=dt)
    return _quantise(x) if c["dtype"] == "q4" else x


def _prepare_tree(c, seed):
    n, T, D = c["layers"] // 2, c["nodes"], c["head_dim"]
    lens = _lens(c, seed, T)
    trees = _random_trees(c, seed)
    words = [[(m & (2 ** 63 - 1)) - (m & 2 ** 63) for m in t] for t in trees]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    two = _sources(c) == 2
    w = torch.randn(4, c["kv_heads"], D, generator=_gen(seed, 9), device=_DEV) * 0.3 + 0.5
    w[:2, :, D // 2:] = w[:2, :, : D // 2]      # key weights are tied across rotation pairs
    st = dict(
        c=c, k=[_cache(c, seed, 1)] + ([_cache(c, seed, 2)] if two else []),
        v=[_cache(c, seed, 3)] + ([_cache(c, seed, 4)] if two else []),
        w=[x.contiguous() for x in w.unbind(0)],
        q=torch.randn(c["batch"], c["q_heads"], T, D, generator=_gen(seed, 5), device=_DEV, dtype=dt),
        lens=torch.tensor(lens, dtype=torch.int32, device=_DEV),
        tree=torch.tensor(words, dtype=torch.int64, device=_DEV).unsqueeze(-1).contiguous(),
        longest=max(lens) + T, layer=n + 1)
    st["out"] = torch.empty_like(st["q"])
    if own:
        from cross_layer_kv_gb300 import Context
        layer = 1 if c["mode"] == "vanilla" else n + 1
        ctx = Context(c["layers"], c["batch"], c["seq"], c["q_heads"], c["kv_heads"], D,
                      "f32" if c["dtype"] == "f32" else "bf16")
        bind = ctx.fkv_bind_layer_cache_q4 if c["dtype"] == "q4" else ctx.fkv_bind_layer_cache
        if c["ring"]:
            for l in sorted({1, n}):
                ctx.fkv_set_ring_rows(l, c["ring"])
        if c["mode"] == "vanilla":
            bind(1, st["k"][0], st["v"][0])
        else:
            # fused: K^1, K^n, V^1, V^n; lite and scaled: K^n and V^1, here one layer's pair
            bind(1, st["k"][0], st["v"][0])
            if two:
                bind(n, st["k"][1], st["v"][1])
            else:
                ctx.fkv_set_sources(layer, c["mode"], 1, 0, 1, 0)
            ctx.fkv_set_fusion_weights(layer, *st["w"])
        if c["window"]:
            ctx.fkv_set_window(layer, c["window"])
        st.update(ctx=ctx, layer=layer, workspace=ctx.tree_workspace(T))
    return st


def _layers_cache(c, seed):
    """K and V of every stored layer, [n, 2, B, H_kv, S, D]."""
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    shape = (c["layers"] // 2, 2, c["batch"], c["kv_heads"], c["seq"], c["head_dim"])
    return torch.randn(shape, generator=_gen(seed, 1), device=_DEV, dtype=dt)


def _context(c, big):
    from cross_layer_kv_gb300 import Context
    ctx = Context(c["layers"], c["batch"], c["seq"], c["kv_heads"], c["kv_heads"], c["head_dim"], c["dtype"])
    for l in range(1, c["layers"] // 2 + 1):
        ctx.fkv_bind_layer_cache(l, big[l - 1, 0], big[l - 1, 1])
    return ctx


def _paths(c, seed):
    """Accepted nodes of each sequence, root first.  Nodes are numbered level by level; the first
    level is the widest, so the nodes below it lie behind the accepted path's end."""
    import random
    r = random.Random(seed * 31337 + 3)
    paths = []
    for _ in range(c["batch"]):
        most = min(c["accept"], c["nodes"])
        count = r.randint(min(1, most), most)
        first = r.choice([0] + list(range(count, min(c["nodes"], count + 8))))
        rest = sorted(r.sample(range(max(first + 1, count), c["nodes"]),
                               min(count - 1, c["nodes"] - max(first + 1, count))))
        paths.append([first] + rest)
    return paths


def _prepare_compact(c, seed):
    big = _layers_cache(c, seed)
    lens, paths = _lens(c, seed, c["nodes"]), _paths(c, seed)
    A = max(len(p) for p in paths)
    st = dict(c=c, big=big, A=A, where=lens,
              pos=torch.tensor(lens, dtype=torch.int32, device=_DEV),
              idx=torch.tensor([p + [0] * (A - len(p)) for p in paths], dtype=torch.int32, device=_DEV),
              counts=torch.tensor([len(p) for p in paths], dtype=torch.int32, device=_DEV))
    if own:
        st["ctx"] = _context(c, big)
    st["answer"] = [big[:, :, b, :, p: p + A] for b, p in enumerate(lens)]
    return st


def _parents(c, seed):
    """src[b] of every sequence: a beam that survives keeps its slot, the others fork from a
    survivor of their own prompt."""
    import random
    r = random.Random(seed * 65537 + 4)
    src = []
    for p in range(0, c["batch"], c["beams"]):
        group = list(range(p, min(p + c["beams"], c["batch"])))
        alive = r.sample(group, r.randint(1, max(1, len(group) // 2)))
        src += [b if b in alive else r.choice(alive) for b in group]
    return src


def _prepare_reorder(c, seed):
    big = _layers_cache(c, seed)
    src, lens = _parents(c, seed), _lens(c, seed, 0)
    lens = [lens[b // c["beams"] * c["beams"]] for b in range(c["batch"])]   # beams of a prompt grow together
    st = dict(c=c, big=big, src=torch.tensor(src, dtype=torch.int32, device=_DEV),
              lens=torch.tensor(lens, dtype=torch.int32, device=_DEV), longest=max(lens))
    if own:
        st["ctx"] = _context(c, big)
    return st


def prepare(case, seed):
    return {"tree": _prepare_tree, "compact": _prepare_compact, "reorder": _prepare_reorder}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(x, D):
    """A cache in 32 bits."""
    if x.dtype != torch.uint8:
        return x.float()
    code = torch.stack((x[..., : D // 2] & 15, x[..., : D // 2] >> 4), -1).reshape(*x.shape[:-1], D // _GROUP, _GROUP)
    prm = x[..., D // 2: D // 2 + D // 4].contiguous().view(torch.bfloat16).float()
    prm = prm.reshape(*x.shape[:-1], D // _GROUP, 2)
    return (prm[..., 1:] + code.float() * prm[..., :1]).reshape(*x.shape[:-1], D)


def _visible(st, rows):
    """[B, T, rows]: which of the call's cache rows each node sees.  Row r of a ring holds the last
    position of its residue that has been written."""
    c, T = st["c"], st["c"]["nodes"]
    lens, tree = st["lens"].long(), st["tree"][..., 0]
    at = torch.arange(rows, device=_DEV)[None, :].expand(c["batch"], rows)
    if c["ring"]:
        last = (lens + T - 1)[:, None]
        at = last - (last - at) % c["ring"]
    node = at - lens[:, None]                                     # >= 0: a drafted row
    bits = (tree[:, :, None] >> torch.arange(T, device=_DEV)) & 1    # [B, T, T]
    depth = bits.sum(-1).clamp(min=1) - 1
    drafted = (node >= 0) & (node < T)
    pick = node.clamp(0, T - 1)
    seen = torch.gather(bits, 2, pick[:, None, :].expand(-1, T, -1)) > 0
    see = torch.where(drafted[:, None], seen, (node < 0)[:, None] & (at >= 0)[:, None])
    if c["window"]:
        pos = lens[:, None] + depth
        key = torch.where(drafted, lens[:, None] + torch.gather(depth, 1, pick), at)
        see = see & (key[:, None, :] > pos[:, :, None] - c["window"])
    return see


def _plain_tree(st):
    c = st["c"]
    B, H, D, T = c["batch"], c["kv_heads"], c["head_dim"], c["nodes"]
    rows = c["ring"] or st["longest"]
    k, v = ([_values(x[:, :, :rows], D) for x in st[n]] for n in ("k", "v"))
    a0, a1, b0, b1 = (x[None, :, None, :] for x in st["w"])
    if c["mode"] == "fused":
        k, v = a0 * k[0] + a1 * k[1], b0 * v[0] + b1 * v[1]
    elif c["mode"] == "scaled":
        k, v = a0 * k[0], b0 * v[0]
    else:
        k, v = k[0], v[0]
    q = st["q"].float().reshape(B, H, -1, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    see = _visible(st, rows)[:, None, None]
    s = s.reshape(B, H, -1, T, rows).masked_fill_(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H, -1, rows), v).reshape(B, H, -1, T, D) / torch.where(total > 0, total, 1.0)
    return o.reshape(st["q"].shape).to(st["q"].dtype)


def _plain_compact(st):
    c, big, A = st["c"], st["big"], st["A"]
    j = torch.arange(A, device=_DEV)[None, :]
    move = j < st["counts"][:, None]
    frm = st["pos"][:, None].long() + torch.where(move, st["idx"], j)     # rows read, [B, A]
    to = st["pos"][:, None].long() + j
    b = torch.arange(c["batch"], device=_DEV)[:, None].expand_as(frm)
    big[:, :, b, :, to] = big[:, :, b, :, frm]
    return st["answer"]


def _plain_reorder(st):
    big = st["big"][:, :, :, :, : st["longest"]]
    row = torch.arange(st["longest"], device=_DEV)
    write = (row[None, :] < st["lens"][:, None])[None, None, :, None, :, None]
    big.copy_(torch.where(write, big.index_select(2, st["src"]), big))
    return st["big"]


def run(state):
    op = state["c"]["op"]
    if op == "tree":
        if own:
            return state["ctx"].fkv_tree_attn(state["q"], state["layer"], state["c"]["mode"], state["lens"],
                                              state["tree"], state["out"], state["workspace"])
        return _plain_tree(state)
    if op == "compact":
        if own:
            state["ctx"].fkv_compact_rows(state["pos"], state["idx"], state["counts"])
            return state["answer"]
        return _plain_compact(state)
    if own:
        state["ctx"].fkv_reorder_seqs(state["src"], state["lens"])
        return state["big"]
    return _plain_reorder(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    D, H, B = c["head_dim"], c["kv_heads"], c["batch"]
    elem = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "tree":
        T, room = c["nodes"], c["seq"] - c["nodes"]
        # prefix rows: uniform in [room/2, room] where ragged; at most a window's
        rows = room * (0.75 if c["ragged"] else 1.0)
        rows = (min(rows, c["window"] - 1) if c["window"] else rows) + T
        row = (D // 2 + D // 4 + 15) // 16 * 16 if c["dtype"] == "q4" else D * elem
        tensors = 2 * _sources(c)
        return {"bytes": tensors * row * H * B * rows + 2 * B * c["q_heads"] * T * D * elem + 8 * B * T,
                "flops": 4.0 * B * c["q_heads"] * T * D * rows}
    planes = c["layers"] * H * D * elem          # K and V of half the layers: bytes of one position
    if c["op"] == "compact":
        moved = (1 + min(c["accept"], c["nodes"])) / 2
        return {"bytes": 2.0 * planes * B * moved + 4 * B * c["accept"], "flops": 0.0}
    # about three of four beams end; each survivor is read once
    return {"bytes": planes * (B * 0.7 + B * 0.25) * c["seq"] * 0.75, "flops": 0.0}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _wide(x, D):
    """A cache in 64 bits."""
    if x.dtype != torch.uint8:
        return x.double()
    low, high = (x[..., : D // 2] % 16).double(), (x[..., : D // 2] // 16).double()
    code = torch.empty(*x.shape[:-1], D, dtype=torch.float64, device=x.device)
    code[..., 0::2], code[..., 1::2] = low, high
    prm = x[..., D // 2: D // 2 + D // 4].contiguous().view(torch.bfloat16).double()
    return code * prm[..., 0::2].repeat_interleave(_GROUP, -1) + prm[..., 1::2].repeat_interleave(_GROUP, -1)


def exact(case, seed):
    global own
    c = case
    was, own = own, False
    st = prepare(case, seed)
    own = was
    if c["op"] == "compact":
        old = st["big"].clone()
        for b, path in enumerate(_paths(c, seed)):
            for j, node in enumerate(path):
                st["big"][:, :, b, :, st["where"][b] + j] = old[:, :, b, :, st["where"][b] + node]
        return st["answer"]
    if c["op"] == "reorder":
        old = st["big"].clone()
        for b, s in enumerate(_parents(c, seed)):
            n = int(st["lens"][b])
            st["big"][:, :, b, :, :n] = old[:, :, s, :, :n]
        return st["big"]
    D, T, G = c["head_dim"], c["nodes"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=_DEV)
    lens, trees = st["lens"].tolist(), _random_trees(c, seed)
    fused, scaled = c["mode"] == "fused", c["mode"] == "scaled"
    wt = [x.double() for x in st["w"]]
    for b in range(c["batch"]):
        P, m = lens[b], trees[b]
        first = max(0, P - c["window"] + 1) if c["window"] else 0
        pos = torch.arange(first, P + T, device=_DEV)
        at = pos % c["ring"] if c["ring"] else pos
        anc = torch.tensor([[m[i] >> j & 1 for j in range(T)] for i in range(T)], dtype=torch.bool, device=_DEV)
        see = torch.ones(T, P + T - first, dtype=torch.bool, device=_DEV)
        see[:, P - first:] = anc
        if c["window"]:
            depth = anc.sum(1) - 1
            key = torch.cat((pos[: P - first], P + depth))
            see &= (P + depth)[:, None] - key[None, :] < c["window"]
        for h in range(c["kv_heads"]):
            ks = [_wide(x[b, h][at], D) for x in st["k"]]
            vs = [_wide(x[b, h][at], D) for x in st["v"]]
            k = wt[0][h] * ks[0] + wt[1][h] * ks[1] if fused else wt[0][h] * ks[0] if scaled else ks[0]
            v = wt[2][h] * vs[0] + wt[3][h] * vs[1] if fused else wt[2][h] * vs[0] if scaled else vs[0]
            s = st["q"][b, h * G: (h + 1) * G].double() @ k.T / math.sqrt(D)
            s = s.masked_fill(~see, -math.inf)
            out[b, h * G: (h + 1) * G] = torch.softmax(s, -1) @ v
    return out
