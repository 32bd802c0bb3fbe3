"""Cases of the speculative-decoding operators over the paged KV cache, with their plain forms.

Three operators make one step of drafted-token verification:

* ``append``: RMS norm of each query and key head, rotary position, and the K and V rows written
  into their cache slots, in one pass (``qk_norm_rope_append``);
* ``tree``: attention of every drafted node over the request's cached tokens and the nodes its
  mask row names (``tree_decode_attention``);
* ``commit``: the accepted nodes' rows moved together behind the committed tokens
  (``tree_commit``).

A pool is [pages][kv heads][16][dim]; a request's position p lives in page table[p // 16], row
p % 16. ``context_lens`` counts the drafted nodes, which are a request's last ``tree_lens`` rows.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn,
         "int8": torch.int8}


def listed():
    return [
        # one request decoding without a draft: one token's rows, a latency-bound call
        {"name": "append_one_token", "op": "append", "tokens": 1, "h_q": 32, "h_kv": 8, "dim": 128,
         "rot": 128, "io": "bf16", "cache": "bf16", "interleaved": False, "norm": True},
        # a verification step's nodes (64 requests, 24 nodes each) into an 8-bit cache
        {"name": "append_drafts_fp8", "op": "append", "tokens": 1536, "h_q": 64, "h_kv": 8,
         "dim": 128, "rot": 128, "io": "bf16", "cache": "fp8", "interleaved": False, "norm": True},
        # a long prompt of odd length
        {"name": "append_prompt", "op": "append", "tokens": 12345, "h_q": 32, "h_kv": 8,
         "dim": 128, "rot": 128, "io": "bf16", "cache": "bf16", "interleaved": False, "norm": True},
        # a model kept in 32 bits, half of each head rotated in neighbouring pairs, no norm
        {"name": "append_f32_partial", "op": "append", "tokens": 777, "h_q": 12, "h_kv": 4,
         "dim": 64, "rot": 32, "io": "f32", "cache": "f32", "interleaved": True, "norm": False},
        # one interactive request with a small draft
        {"name": "tree_one_request", "op": "tree", "batch": 1, "nodes": 8, "h_q": 32, "h_kv": 8,
         "dim": 128, "io": "bf16", "cache": "bf16", "lo": 777, "hi": 777, "ragged": False},
        # a serving batch, every request with a full draft
        {"name": "tree_batch64", "op": "tree", "batch": 64, "nodes": 16, "h_q": 32, "h_kv": 8,
         "dim": 128, "io": "bf16", "cache": "bf16", "lo": 512, "hi": 4096, "ragged": False},
        # large drafts of unequal size (some requests without any)
        {"name": "tree_batch64_wide", "op": "tree", "batch": 64, "nodes": 64, "h_q": 32, "h_kv": 8,
         "dim": 128, "io": "bf16", "cache": "bf16", "lo": 512, "hi": 4096, "ragged": True},
        # an 8-bit cache under continuous batching, eight query heads to a KV head
        {"name": "tree_fp8_batch128", "op": "tree", "batch": 128, "nodes": 24, "h_q": 64,
         "h_kv": 8, "dim": 128, "io": "bf16", "cache": "fp8", "lo": 128, "hi": 8192,
         "ragged": True},
        # few requests with long contexts, INT8 codes
        {"name": "tree_int8_long", "op": "tree", "batch": 4, "nodes": 12, "h_q": 64, "h_kv": 8,
         "dim": 128, "io": "bf16", "cache": "int8", "lo": 8191, "hi": 65536, "ragged": True},
        # 32-bit cache, three query heads to a KV head of 64 dimensions
        {"name": "tree_f32_dim64", "op": "tree", "batch": 8, "nodes": 5, "h_q": 12, "h_kv": 4,
         "dim": 64, "io": "f32", "cache": "f32", "lo": 100, "hi": 2000, "ragged": True},
        # the accepted paths of a serving batch
        {"name": "commit_batch64", "op": "commit", "batch": 64, "nodes": 16, "h_kv": 8, "dim": 128,
         "cache": "bf16", "lo": 33, "hi": 512, "accept": 5},
        # a large batch with an 8-bit cache and deep drafts
        {"name": "commit_fp8_batch256", "op": "commit", "batch": 256, "nodes": 48, "h_kv": 8,
         "dim": 128, "cache": "fp8", "lo": 64, "hi": 700, "accept": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case between the smallest and the largest of its operator."""
    most = {op: [work(c) for c in listed() if c["op"] == op] for op in ("append", "tree", "commit")}
    while True:
        op = rng.choice(["append", "append", "tree", "tree", "tree", "commit"])
        h_kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128, 128])
        if op == "append":
            io = rng.choice(["bf16", "bf16", "f32"])
            c = {"op": op, "tokens": _log(rng, 1, 12345), "h_q": h_kv * rng.choice([1, 2, 3, 4, 8]),
                 "h_kv": h_kv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, 16]), "io": io,
                 "cache": rng.choice([io, "fp8"]), "interleaved": rng.random() < 0.3,
                 "norm": rng.random() < 0.8}
        elif op == "tree":
            io = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
            cache = io if io == "f32" else rng.choice(["bf16", "bf16", "fp8", "int8"])
            lo = _log(rng, 65, 4096)
            c = {"op": op, "batch": _log(rng, 1, 128), "nodes": _log(rng, 1, 64),
                 "h_q": h_kv * rng.choice([1, 2, 3, 4, 8]), "h_kv": h_kv, "dim": dim, "io": io,
                 "cache": cache, "lo": lo, "hi": _log(rng, lo, 65536), "ragged": rng.random() < 0.6}
        else:
            nodes = _log(rng, 1, 64)
            lo = _log(rng, nodes, 256)
            c = {"op": op, "batch": _log(rng, 1, 256), "nodes": nodes, "h_kv": h_kv, "dim": dim,
                 "cache": rng.choice(["bf16", "fp8", "int8", "f32"]), "lo": lo,
                 "hi": _log(rng, lo, 700), "accept": rng.randint(1, 16)}
        w = work(c)
        padded = c.get("batch", 1) * c.get("nodes", 1) * c.get("h_q", 1) * c.get("hi", 1)
        if (w["bytes"] <= max(m["bytes"] for m in most[op]) and padded <= 1 << 31 and
                w["flops"] <= max(m["flops"] for m in most[op])):
            return c


# ---- what a user's program has in hand -----------------------------------------------------------


def _lens(case, seed):
    """Context lengths (nodes included) and draft sizes of the requests, on the host."""
    r = np.random.RandomState(seed % (1 << 31))
    b, t = case["batch"], case["nodes"]
    ctx = r.randint(max(case["lo"], t), max(case["lo"], case["hi"], t) + 1, b)
    tree = np.full(b, t)
    if case.get("ragged"):
        tree = r.randint(0 if b > 1 else 1, t + 1, b)
    return ctx.astype(np.int32), tree.astype(np.int32)


def _parents(case, seed):
    """A draft tree for each request in level order: node 0 is the last committed token's, a level
    has one to eight nodes, a node's parent is any node of the level above."""
    r = np.random.RandomState((seed + 7) % (1 << 31))
    b, t = case["batch"], case["nodes"]
    parents = np.full((b, t), -1, np.int64)
    for i in range(b):
        lo, hi = 0, 1  # the level above
        while hi < t:
            n = min(t - hi, int(r.randint(1, 9)))
            parents[i, hi:hi + n] = r.randint(lo, hi, n)
            lo, hi = hi, hi + n
    return parents


def _ancestors(parents):
    """seen[b, i, j]: node j is node i or above it."""
    b, t = parents.shape
    seen = np.zeros((b, t, t + 1), bool)  # (the last column takes the roots' parent -1)
    rows = np.arange(b)
    for i in range(t):
        p = parents[:, i]
        seen[:, i, :t] = seen[rows, np.maximum(p, 0), :t] & (p >= 0)[:, None]
        seen[:, i, i] = True
    return seen[:, :, :t]


def _words(seen):
    """The mask as a program holds it: bit j % 64 of word j // 64 of a node's row."""
    b, t, n = seen.shape
    bits = np.zeros((b, t, -(-n // 64) * 64), np.uint8)
    bits[:, :, :n] = seen
    return np.packbits(bits, axis=-1, bitorder="little").view(np.int64)


def _table(case, ctx, seed):
    """Page tables with the pages handed out in random order, and the pool's size: the pages of
    these requests, or for ``commit`` (which returns the pool) of the longest ones."""
    pages = -(-ctx.astype(np.int64) // PAGE)
    used = n = int(pages.sum())
    if case["op"] == "commit":
        n = case["batch"] * -(-max(case["lo"], case["hi"], case["nodes"]) // PAGE)
    order = np.random.RandomState((seed + 3) % (1 << 31)).permutation(n).astype(np.int32)
    bt = np.zeros((len(ctx), int(pages.max())), np.int32)
    bt[np.arange(bt.shape[1])[None, :] < pages[:, None]] = order[:used]
    return bt, n


def _pool(n, case, gen):
    """A pool of cached rows. Codes use the range that per-head scales leave them."""
    shape = (n, case["h_kv"], PAGE, case["dim"])
    t = TYPES[case["cache"]]
    if case["cache"] == "int8":
        return torch.randint(-127, 128, shape, dtype=t, device="cuda", generator=gen)
    x = torch.randn(shape, device="cuda", generator=gen,
                    dtype=torch.float32 if case["cache"] == "f32" else torch.bfloat16)
    return x if x.dtype == t else (x * 64).clamp(-448, 448).to(t)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=dtype)

    def scales():  # of an 8-bit cache, one for each KV head
        if case["cache"] not in ("fp8", "int8"):
            return None
        u = torch.rand(case["h_kv"], device="cuda", generator=gen)
        return (0.012 + 0.008 * u) if case["cache"] == "fp8" else (0.03 + 0.01 * u)

    state = {"case": case, "k_scales": scales(), "v_scales": scales()}
    if case["op"] == "append":
        n, h_q, h_kv, d = case["tokens"], case["h_q"], case["h_kv"], case["dim"]
        io = TYPES[case["io"]]
        # the projection's output: queries, keys and values of a token side by side
        qkv = randn(n, (h_q + 2 * h_kv) * d, dtype=io)
        q, k, v = qkv.split([h_q * d, h_kv * d, h_kv * d], dim=-1)
        pages = -(-n // PAGE) + 1
        most = 8192
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * (
            500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) /
                         case["rot"]))
        state.update(
            q=q.view(n, h_q, d), k=k.view(n, h_kv, d), v=v.view(n, h_kv, d),
            q_weight=(1 + 0.2 * randn(d)).to(io) if case["norm"] else None,
            k_weight=(1 + 0.2 * randn(d)).to(io) if case["norm"] else None,
            table=torch.cat([angle.cos(), angle.sin()], -1).float(),
            positions=torch.randint(0, most, (n,), device="cuda", generator=gen,
                                    dtype=torch.int32),
            slots=torch.randperm(pages * PAGE, device="cuda", generator=gen)[:n],
            k_cache=_pool(pages, case, gen), v_cache=_pool(pages, case, gen))
        return state
    ctx, tree = _lens(case, seed)
    bt, n = _table(case, ctx, seed)
    parents = _parents(case, seed)
    state.update(k_cache=_pool(n, case, gen), v_cache=_pool(n, case, gen),
                 block_tables=torch.from_numpy(bt).cuda(), context_lens=torch.from_numpy(ctx).cuda(),
                 tree_lens=torch.from_numpy(tree).cuda())
    if case["op"] == "tree":
        shape = (case["batch"], case["nodes"], case["h_q"], case["dim"])
        state.update(q=randn(*shape, dtype=TYPES[case["io"]]),
                     mask=torch.from_numpy(_words(_ancestors(parents))).cuda(),
                     scale=case["dim"] ** -0.5,
                     out=torch.zeros(shape, dtype=TYPES[case["io"]], device="cuda"))
    else:
        path, count = _paths(case, seed, parents)
        state.update(path=torch.from_numpy(path).cuda(), path_lens=torch.from_numpy(count).cuda())
    return state


def _paths(case, seed, parents):
    """An accepted path from node 0 down for each request. A node that moves comes from behind the
    accepted length, as it does in a tree wider than the path is deep (so that a pass repeated on
    the same cache writes the same bytes)."""
    r = np.random.RandomState((seed + 11) % (1 << 31))
    b, t = parents.shape
    path = np.zeros((b, case["accept"]), np.int32)
    count = np.zeros(b, np.int32)
    for i in range(b):
        walk = [0]
        while len(walk) < case["accept"]:
            below = np.nonzero(parents[i] == walk[-1])[0]
            if not len(below):
                break
            walk.append(int(below[r.randint(len(below))]))
        n = int(r.randint(0, len(walk) + 1))
        while any(w != k and w < n for k, w in enumerate(walk[:n])):
            n -= 1
        path[i, :n], count[i] = walk[:n], n
    return path, count


# ---- one pass -----------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "tree": _own_tree, "commit": _own_commit}[op](s)
    return {"append": _append, "tree": _tree, "commit": _commit}[op](s)


def _own_append(s):
    import paged_kv_cache_271_gb300 as pkv
    q = pkv.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"],
                                s["v_cache"], s["table"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=EPS,
                                interleaved=s["case"]["interleaved"], k_scales=s["k_scales"],
                                v_scales=s["v_scales"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_tree(s):
    import paged_kv_cache_271_gb300 as pkv
    return pkv.tree_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                                     s["context_lens"], s["scale"], tree_mask=s["mask"],
                                     tree_lens=s["tree_lens"], out=s["out"],
                                     k_scales=s["k_scales"], v_scales=s["v_scales"])


def _own_commit(s):
    import paged_kv_cache_271_gb300 as pkv
    lens = pkv.tree_commit(s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                           s["tree_lens"], s["path"], s["path_lens"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": lens}


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _store(pool, slots, rows, scales):
    """Rows [n, kv heads, dim] in 32 bits into the pool, rounded once."""
    if pool.dtype == torch.float8_e4m3fn:
        rows = (rows / scales[:, None]).clamp(-448, 448).to(pool.dtype).view(torch.uint8)
    _bytes(pool)[slots // PAGE, :, slots % PAGE] = rows.to(_bytes(pool).dtype)


def _append(s):
    c = s["case"]
    cs = s["table"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r.chunk(2, -1)
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1)

    q = turned(s["q"], s["q_weight"]).to(s["q"].dtype)
    _store(s["k_cache"], s["slots"], turned(s["k"], s["k_weight"]), s["k_scales"])
    _store(s["v_cache"], s["slots"], s["v"].float(), s["v_scales"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _tree(s):
    q, bt = s["q"], s["block_tables"].long()
    b, t, h_q, d = q.shape
    h_kv = s["case"]["h_kv"]
    length = bt.shape[1] * PAGE

    def rows(pool, scales):  # [b, kv heads, length, dim] in 32 bits
        x = _bytes(pool)[bt].view(pool.dtype).float()
        x = x if scales is None else x * scales[:, None, None]
        return x.transpose(1, 2).reshape(b, h_kv, length, d)

    pos = torch.arange(length, device=q.device)
    base = (s["context_lens"] - s["tree_lens"])[:, None]
    bits = (s["mask"][..., None] >> torch.arange(64, device=q.device)) & 1
    bits = bits.flatten(-2).bool()
    node = (pos - base).clamp(0, bits.shape[-1] - 1)[:, None, :].expand(b, t, length)
    seen = (pos < base)[:, None, :] | (bits.gather(-1, node) & (pos >= base)[:, None, :])
    seen &= (pos < s["context_lens"][:, None])[:, None, :]
    qs = q.float().view(b, t, h_kv, h_q // h_kv, d).transpose(1, 2).reshape(b, h_kv, -1, d)
    scores = qs @ rows(s["k_cache"], s["k_scales"]).transpose(-1, -2) * s["scale"]
    scores = scores.view(b, h_kv, t, h_q // h_kv, length)
    scores.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h_kv, -1, length) @ rows(s["v_cache"], s["v_scales"])).view(*p.shape[:4], d)
    o = torch.where(total > 0, o / total, 0.0).transpose(1, 2).reshape(q.shape)
    real = torch.arange(t, device=q.device) < s["tree_lens"][:, None]
    s["out"].copy_(torch.where(real[:, :, None, None], o.to(q.dtype), s["out"]))
    return s["out"]


def _commit(s):
    bt = s["block_tables"].long()
    base = (s["context_lens"] - s["tree_lens"]).long()[:, None]
    i = torch.arange(s["path"].shape[1], device=bt.device)[None, :]
    kept = i < s["path_lens"][:, None]
    to = (base + i)
    come = base + torch.where(kept, s["path"].long(), 0)

    def page(p):
        return bt.gather(1, (p // PAGE).clamp_max(bt.shape[1] - 1))[kept]

    src, dst, r_src, r_dst = page(come), page(to), (come % PAGE)[kept], (to % PAGE)[kept]
    _bytes(s["k_cache"])[dst, :, r_dst] = _bytes(s["k_cache"])[src, :, r_src]
    _bytes(s["v_cache"])[dst, :, r_dst] = _bytes(s["v_cache"])[src, :, r_src]
    lens = (s["context_lens"] - s["tree_lens"] + s["path_lens"]).int()
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": lens}


# ---- what a pass cannot do without ----------------------------------------------------------------


def work(case):
    size = {"f32": 4, "bf16": 2, "fp8": 1, "int8": 1}
    d, h_kv, cache = case["dim"], case["h_kv"], size[case["cache"]]
    if case["op"] == "append":
        n, io = case["tokens"], size[case["io"]]
        rows_in = n * (case["h_q"] + 2 * h_kv) * d * io
        rows_out = n * case["h_q"] * d * io + 2 * n * h_kv * d * cache
        return {"bytes": rows_in + rows_out + n * (4 * case["rot"] + 12),
                "flops": n * (case["h_q"] + h_kv) * d * 8}
    seed = 0  # the lengths' distribution stands for every seed's
    ctx, tree = _lens(case, seed)
    ctx, tree = ctx.astype(np.int64), tree.astype(np.int64)
    if case["op"] == "tree":
        live = tree > 0
        base = ctx - tree
        keys = int((tree * (base + (tree + 1) // 2))[live].sum())
        rows = int(tree.sum())
        return {"bytes": int(ctx[live].sum()) * 2 * h_kv * d * cache +
                2 * rows * case["h_q"] * d * size[case["io"]],
                "flops": 4 * keys * case["h_q"] * d}
    path, count = _paths(case, seed, _parents(case, seed))
    k = np.arange(path.shape[1])[None, :]
    moved = int(((k < count[:, None]) & (path != k)).sum())
    return {"bytes": moved * 4 * h_kv * d * cache + 4 * int(count.sum()) + 16 * case["batch"],
            "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    half = c["rot"] // 2
    at = s["table"].double()[s["positions"].long()]
    turn = torch.complex(at[:, :half], at[:, half:])[:, None, :]

    def form(x, w):
        x = x.double()
        if w is not None:
            x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
        x = x.clone()
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(x[..., a], x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
        return x

    out = {"q": form(s["q"], s["q_weight"])}
    for name, rows in (("k", form(s["k"], s["k_weight"])), ("v", s["v"].double())):
        pool = s[name + "_cache"].double()
        if c["cache"] == "fp8":
            rows = (rows / s[name + "_scales"].double()[None, :, None]).clamp(-448.0, 448.0)
        flat = pool.transpose(1, 2).reshape(-1, c["h_kv"], c["dim"])
        flat[s["slots"]] = rows
        out[name + "_cache"] = flat.view(-1, PAGE, c["h_kv"], c["dim"]).transpose(1, 2)
    return out


def _exact_tree(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    seen = torch.from_numpy(_ancestors(_parents_of(s))).cuda()
    group = c["h_q"] // c["h_kv"]
    for b, (ctx, t) in enumerate(zip(s["context_lens"].tolist(), s["tree_lens"].tolist())):
        if t == 0:
            continue
        pages = s["block_tables"][b, :-(-ctx // PAGE)].long()
        for h in range(c["h_kv"]):
            k = s["k_cache"][pages, h].double().reshape(-1, c["dim"])[:ctx]
            v = s["v_cache"][pages, h].double().reshape(-1, c["dim"])[:ctx]
            if s["k_scales"] is not None:
                k, v = k * s["k_scales"][h].double(), v * s["v_scales"][h].double()
            q = s["q"][b, :t, h * group:(h + 1) * group].double()
            score = torch.einsum("tgd,kd->tgk", q, k) * c["dim"] ** -0.5
            score[:, :, ctx - t:].masked_fill_(~seen[b, :t, None, :t], -math.inf)
            out[b, :t, h * group:(h + 1) * group] = torch.softmax(score, -1) @ v
    return out


def _parents_of(s):
    """Each node's parent, read back from its mask row: the nearest node above it."""
    words = s["mask"].cpu().numpy()
    b, t, _ = words.shape
    bits = np.unpackbits(words.view(np.uint8), axis=-1, bitorder="little")[:, :, :t]
    parents = np.full((b, t), -1, np.int64)
    for i in range(1, t):
        above = bits[:, i, :i]
        parents[:, i] = np.where(above.any(-1), i - 1 - above[:, ::-1].argmax(-1), -1)
    return parents


def _exact_commit(s):
    out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    table = s["block_tables"].tolist()
    lens = []
    for b, (ctx, t, n) in enumerate(zip(s["context_lens"].tolist(), s["tree_lens"].tolist(),
                                        s["path_lens"].tolist())):
        base = ctx - t
        nodes = [base + x for x in s["path"][b, :n].tolist()]
        for pool in out.values():
            rows = [pool[table[b][p // PAGE], :, p % PAGE].clone() for p in nodes]
            for i, row in enumerate(rows):
                pool[table[b][(base + i) // PAGE], :, (base + i) % PAGE] = row
        lens.append(base + n)
    out["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return out
