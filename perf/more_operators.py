"""Cases of the prompt-chunk and eviction operators over the paged KV cache, with their plain forms.

Three operators take a prompt (or any run of new tokens) into a cache of bounded size:

* ``chunk``: attention of a chunk of new tokens of each request over its cached tokens and the
  chunk's own earlier ones (``chunk_attention``), optionally with scores capped by a tanh, a bias
  that falls with distance, or a sliding window with sinks;
* ``weigh``: the weights that the rows of a chunk give to each cached position, summed over rows and
  over the query heads of a KV head, added to earlier sums (``chunk_weights``);
* ``evict``: the positions with the largest sums chosen for each KV head (``evict_select``), their
  rows copied together onto new pages with their sums (``evict_move``).

A pool is [pages][kv heads][16][dim]; a request's position p lives in page table[p // 16], row
p % 16. ``context_lens`` counts the chunk's tokens, which are a request's last positions; the
queries of request b are rows ``query_starts[b] .. query_starts[b + 1] - 1``.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn,
         "int8": torch.int8}


def listed():
    return [
        # one request decoding with capped scores: a latency-bound call
        {"name": "chunk_one_token", "op": "chunk", "batch": 1, "new": 1, "lo": 777, "hi": 777,
         "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16", "softcap": 30.0,
         "alibi": False, "window": 0, "sinks": 0},
        # a serving batch's decode step of a model whose positions are a bias by distance
        {"name": "chunk_decode_alibi", "op": "chunk", "batch": 64, "new": 1, "lo": 512, "hi": 4096,
         "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16", "softcap": 0.0,
         "alibi": True, "window": 0, "sinks": 0},
        # a whole prompt of odd length in one chunk
        {"name": "chunk_prompt", "op": "chunk", "batch": 1, "new": 8191, "lo": 0, "hi": 0,
         "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16", "softcap": 0.0,
         "alibi": False, "window": 0, "sinks": 0},
        # the next chunk of a long prompt over an FP8 cache, eight query heads to a KV head
        {"name": "chunk_continued_fp8", "op": "chunk", "batch": 1, "new": 2048, "lo": 32768,
         "hi": 32768, "h_q": 64, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "fp8",
         "softcap": 0.0, "alibi": False, "window": 0, "sinks": 0},
        # continuous batching: chunks of every size beside one another, INT8 codes, capped scores
        {"name": "chunk_mixed_int8", "op": "chunk", "batch": 48, "new": 512, "lo": 0, "hi": 4096,
         "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "int8", "softcap": 50.0,
         "alibi": False, "window": 0, "sinks": 0},
        # prompts of a sliding-window model
        {"name": "chunk_window", "op": "chunk", "batch": 16, "new": 1500, "lo": 0, "hi": 4096,
         "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16", "softcap": 0.0,
         "alibi": False, "window": 1024, "sinks": 4},
        # a model kept in 32 bits, three query heads to a KV head of 64 dimensions
        {"name": "chunk_f32_dim64", "op": "chunk", "batch": 8, "new": 100, "lo": 0, "hi": 1000,
         "h_q": 12, "h_kv": 4, "dim": 64, "io": "f32", "cache": "f32", "softcap": 0.0,
         "alibi": False, "window": 0, "sinks": 0},
        # what the last 32 rows of each prompt look at, before its cache is cut
        {"name": "weigh_last_rows", "op": "weigh", "batch": 8, "new": 512, "last": 32, "lo": 0,
         "hi": 8192, "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16",
         "softcap": 0.0, "alibi": False, "window": 0, "sinks": 0},
        # sums kept up to date by a decode step over an FP8 cache
        {"name": "weigh_decode_fp8", "op": "weigh", "batch": 64, "new": 1, "last": 0, "lo": 512,
         "hi": 4096, "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "fp8",
         "softcap": 0.0, "alibi": False, "window": 0, "sinks": 0},
        # every row of a prompt
        {"name": "weigh_prompt", "op": "weigh", "batch": 1, "new": 4095, "last": 0, "lo": 0,
         "hi": 0, "h_q": 32, "h_kv": 8, "dim": 128, "io": "bf16", "cache": "bf16", "softcap": 0.0,
         "alibi": False, "window": 0, "sinks": 0},
        # the caches of a serving batch cut to 1024 tokens
        {"name": "evict_batch64", "op": "evict", "batch": 64, "lo": 512, "hi": 4096,
         "budget": 1024, "recent": 64, "sinks": 4, "h_kv": 8, "dim": 128, "cache": "bf16"},
        # one long context cut to an eighth
        {"name": "evict_long_fp8", "op": "evict", "batch": 1, "lo": 65536, "hi": 65536,
         "budget": 8192, "recent": 512, "sinks": 0, "h_kv": 8, "dim": 128, "cache": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case between the smallest and the largest of its operator."""
    most = {op: [work(c) for c in listed() if c["op"] == op] for op in ("chunk", "weigh", "evict")}
    while True:
        op = rng.choice(["chunk", "chunk", "chunk", "weigh", "weigh", "evict"])
        h_kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128, 128])
        if op == "evict":
            lo = _log(rng, 16, 4096)
            c = {"op": op, "batch": _log(rng, 1, 64), "lo": lo, "hi": _log(rng, lo, 65536),
                 "budget": _log(rng, 8, 8192), "recent": 0, "sinks": rng.choice([0, 0, 4]),
                 "h_kv": h_kv, "dim": dim, "cache": rng.choice(["bf16", "fp8", "int8", "f32"])}
            c["recent"] = rng.randint(0, c["budget"] - c["sinks"])
        else:
            io = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
            lo = rng.choice([0, _log(rng, 1, 4096)])
            c = {"op": op, "batch": _log(rng, 1, 64), "new": _log(rng, 1, 8191), "lo": lo,
                 "hi": _log(rng, max(lo, 1), 65536), "h_q": h_kv * rng.choice([1, 2, 3, 4, 8]),
                 "h_kv": h_kv, "dim": dim, "io": io,
                 "cache": io if io == "f32" else rng.choice(["bf16", "bf16", "fp8", "int8"]),
                 "softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "alibi": rng.random() < 0.25,
                 "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "sinks": 0}
            if c["window"]:
                c["sinks"] = rng.choice([0, 4, 30])
            if op == "weigh":
                c["last"] = rng.choice([0, _log(rng, 1, 128)])
        w = work(c)
        if (w["bytes"] <= max(m["bytes"] for m in most[op]) and
                w["flops"] <= max(m["flops"] for m in most[op]) and
                c["batch"] * (c["hi"] + c.get("new", 0)) <= 1 << 19):
            return c


# ---- what a user's program has in hand -----------------------------------------------------------


def _lens(case, seed):
    """Context lengths (the chunks included) and chunk sizes of the requests, on the host. A case has
    the same ones whatever the seed, in another order: sizes of tensors stay as they are."""
    r = np.random.RandomState(1)
    b = case["batch"]
    past = r.randint(case["lo"], max(case["lo"], case["hi"]) + 1, b)
    new = np.zeros(b, np.int64)
    if case["op"] != "evict":
        new += case["new"]
        if b > 1 and case["new"] > 1:  # chunks of unequal size, the largest among them, some empty
            new = r.randint(0, case["new"] + 1, b)
            new[0], new[1] = case["new"], 0
    order = np.random.RandomState(seed % (1 << 31)).permutation(b)
    return (past + new)[order], new[order]


def _table(lens, first, n, seed):
    """Page tables for requests of these lengths, pages first .. first + n - 1 handed out at random."""
    pages = -(-lens // PAGE)
    order = first + np.random.RandomState((seed + 3) % (1 << 31)).permutation(n).astype(np.int32)
    bt = np.zeros((len(lens), max(int(pages.max()), 1)), np.int32)
    bt[np.arange(bt.shape[1])[None, :] < pages[:, None]] = order[:int(pages.sum())]
    return bt


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
    ctx, new = _lens(case, seed)
    state = {"case": case, "ctx": ctx.tolist(), "new": new.tolist(),
             "context_lens": torch.from_numpy(ctx.astype(np.int32)).cuda()}
    n = max(int((-(-ctx // PAGE)).sum()), 1)
    state["block_tables"] = torch.from_numpy(_table(ctx, 0, n, seed)).cuda()
    if case["op"] == "evict":
        # budget pages for every request: a program reserves them before the choice is known
        kept = np.minimum(ctx, case["budget"])
        room = np.full(case["batch"], case["budget"])
        m = int((-(-room // PAGE)).sum())
        state["k_cache"], state["v_cache"] = _pool(n + m, case, gen), _pool(n + m, case, gen)
        # sums of softmax weights: a few large, most small, some equal, some not looked at
        x = torch.randn(case["batch"], case["h_kv"], int(ctx.max()), device="cuda", generator=gen)
        x = (2 * x).exp()
        x = torch.where(x < 0.1, 0.0, torch.where(x < 1, (x * 64).round() / 64, x))
        state.update(weights=x, new_tables=torch.from_numpy(_table(room, n, m, seed + 1)).cuda(),
                     new_weights=torch.zeros(case["batch"], case["h_kv"], case["budget"],
                                             device="cuda"), kept=kept.tolist())
        return state
    state["k_cache"], state["v_cache"] = _pool(n, case, gen), _pool(n, case, gen)
    state["k_scales"] = state["v_scales"] = None
    if case["cache"] in ("fp8", "int8"):  # one for each KV head
        for name in ("k_scales", "v_scales"):
            u = torch.rand(case["h_kv"], device="cuda", generator=gen)
            state[name] = (0.012 + 0.008 * u) if case["cache"] == "fp8" else (0.03 + 0.01 * u)
    rows = int(new.sum())
    padded = rows if case["batch"] == 1 else -(-rows // 8) * 8  # a batch's rows in steps of eight
    h_q = case["h_q"]
    starts = np.concatenate([[0], np.cumsum(new)])
    slopes = 2.0 ** (-8.0 * torch.arange(1, h_q + 1, device="cuda") / h_q)
    state.update(
        starts=starts.tolist(), query_starts=torch.from_numpy(starts.astype(np.int32)).cuda(),
        q=torch.randn(padded, h_q, case["dim"], device="cuda", generator=gen,
                      dtype=TYPES[case["io"]]),
        slopes=slopes.float() if case["alibi"] else None, scale=case["dim"] ** -0.5)
    state["lse"] = torch.zeros(padded, h_q, device="cuda")
    if case["op"] == "chunk":
        state["out"] = torch.zeros_like(state["q"])
    else:  # the rows' (maximum, sum) as attention left them, and sums of earlier chunks
        for b in range(case["batch"]):
            for r0, r1, s in _scores(state, b, state["new"][b]):
                at = state["starts"][b]
                state["lse"][at + r0:at + r1] = torch.logsumexp(s, -1).permute(1, 0, 2).reshape(
                    r1 - r0, h_q)
        width = max(max(state["ctx"]), 1)
        state["weights"] = torch.rand(case["batch"], case["h_kv"], width, device="cuda",
                                      generator=gen)
        state["out"] = torch.zeros_like(state["weights"])
    return state


# ---- one pass -----------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"chunk": _own_chunk, "weigh": _own_weigh, "evict": _own_evict}[op](s)
    return {"chunk": _chunk, "weigh": _weigh, "evict": _evict}[op](s)


def _own_chunk(s):
    import paged_kv_cache_271_gb300 as pkv
    c = s["case"]
    out = pkv.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                              s["context_lens"], s["query_starts"], s["scale"],
                              softcap=c["softcap"], alibi_slopes=s["slopes"], window=c["window"],
                              sink_tokens=c["sinks"], out=s["out"], lse=s["lse"],
                              k_scales=s["k_scales"], v_scales=s["v_scales"])
    return {"out": out, "lse": s["lse"]}


def _own_weigh(s):
    import paged_kv_cache_271_gb300 as pkv
    c = s["case"]
    return pkv.chunk_weights(s["q"], s["k_cache"], s["block_tables"], s["context_lens"],
                             s["query_starts"], s["lse"], s["scale"], softcap=c["softcap"],
                             alibi_slopes=s["slopes"], window=c["window"], sink_tokens=c["sinks"],
                             last_rows=c["last"], add_to=s["weights"], out=s["out"],
                             k_scales=s["k_scales"])


def _own_evict(s):
    import paged_kv_cache_271_gb300 as pkv
    c = s["case"]
    kept, lens = pkv.evict_select(s["weights"], s["context_lens"], c["budget"],
                                  recent=c["recent"], sink_tokens=c["sinks"])
    pkv.evict_move(s["k_cache"], s["v_cache"], s["block_tables"], kept, lens, s["new_tables"],
                   weights=s["weights"], new_weights=s["new_weights"])
    return {"kept": kept, "lens": lens, "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "new_weights": s["new_weights"]}


def _bytes(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def _rows(s, name, b):
    """Cached rows [kv heads, context, dim] of request b in 32 bits."""
    pool, scales = s[name + "_cache"], s[name + "_scales"]
    pages = s["block_tables"][b, :-(-s["ctx"][b] // PAGE)].long()
    x = _bytes(pool)[pages].view(pool.dtype).float()
    x = x if scales is None else x * scales[:, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :s["ctx"][b]]


def _scores(s, b, last):
    """Scores [kv heads, rows, group, positions] of the last ``last`` rows of request b's chunk, some
    rows at a time: yields (first row, behind the last row, scores over the positions up to there)."""
    c = s["case"]
    ctx, new, at = s["ctx"][b], s["new"][b], s["starts"][b]
    if new == 0:
        return
    k = _rows(s, "k", b)
    h_kv, group = c["h_kv"], c["h_q"] // c["h_kv"]
    step = max(1, min(1024, (1 << 27) // (c["h_q"] * ctx)))
    for r0 in range(max(new - last, 0), new, step):
        r1 = min(new, r0 + step)
        end = ctx - new + r1
        q = s["q"][at + r0:at + r1].float().view(r1 - r0, h_kv, group, -1).transpose(0, 1)
        x = q.reshape(h_kv, -1, c["dim"]) @ k[:, :end].transpose(1, 2) * s["scale"]
        x = x.view(h_kv, r1 - r0, group, end)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        pos = torch.arange(end, device=x.device)
        row = torch.arange(ctx - new + r0, end, device=x.device)[:, None]
        if s["slopes"] is not None:
            x = x + s["slopes"].view(h_kv, 1, group, 1) * (pos - row).float()[:, None, :]
        seen = pos <= row
        if c["window"]:
            seen &= (pos > row - c["window"]) | (pos < c["sinks"])
        yield r0, r1, x.masked_fill(~seen[:, None, :], float("-inf"))


def _chunk(s):
    c = s["case"]
    for b in range(c["batch"]):
        v = _rows(s, "v", b) if s["new"][b] else None
        for r0, r1, x in _scores(s, b, s["new"][b]):
            top = x.amax(-1, keepdim=True)
            p = (x - top).exp_()
            total = p.sum(-1, keepdim=True)
            o = p.flatten(1, 2) @ v[:, :x.shape[-1]] / total.flatten(1, 2)
            at = slice(s["starts"][b] + r0, s["starts"][b] + r1)
            o = o.view(c["h_kv"], r1 - r0, -1, c["dim"]).transpose(0, 1)
            s["out"][at] = o.reshape(r1 - r0, c["h_q"], c["dim"]).to(s["out"].dtype)
            s["lse"][at] = (top + total.log()).squeeze(-1).transpose(0, 1).reshape(r1 - r0, c["h_q"])
    return {"out": s["out"], "lse": s["lse"]}


def _weigh(s):
    c = s["case"]
    for b in range(c["batch"]):
        total = s["weights"][b, :, :s["ctx"][b]].double()  # (sums over up to 65,000 rows)
        for r0, r1, x in _scores(s, b, c["last"] or s["new"][b]):
            lse = s["lse"][s["starts"][b] + r0:s["starts"][b] + r1]
            lse = lse.view(r1 - r0, c["h_kv"], -1, 1).transpose(0, 1)
            total[:, :x.shape[-1]] += (x - lse).exp_().flatten(1, 2).sum(1)
        s["out"][b, :, :s["ctx"][b]] = total.float()
    return s["out"]


def _evict(s):
    c = s["case"]
    kept = torch.zeros(c["batch"], c["h_kv"], c["budget"], dtype=torch.int32, device="cuda")
    lens = s["context_lens"].clamp_max(c["budget"])
    k, v = _bytes(s["k_cache"]), _bytes(s["v_cache"])
    heads = torch.arange(c["h_kv"], device="cuda")[:, None]
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["kept"])):
        w = s["weights"][b, :, :ctx]
        order = w.clone()
        order[:, max(ctx - c["recent"], 0):] = float("inf")
        order[:, :c["sinks"]] = float("inf")
        # (stable: equal sums in the order of their positions)
        at = order.sort(dim=-1, descending=True, stable=True).indices[:, :n].sort(dim=-1).values
        kept[b, :, :n] = at.int()
        to = torch.arange(n, device="cuda")[None, :].expand(c["h_kv"], n)
        src, dst = s["block_tables"][b].long()[at // PAGE], s["new_tables"][b].long()[to // PAGE]
        k[dst, heads, to % PAGE] = k[src, heads, at % PAGE]
        v[dst, heads, to % PAGE] = v[src, heads, at % PAGE]
        s["new_weights"][b, :, :n] = w.gather(1, at)
        s["new_weights"][b, :, n:] = 0
    return {"kept": kept, "lens": lens, "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "new_weights": s["new_weights"]}


# ---- what a pass cannot do without ----------------------------------------------------------------


def _seen(case, ctx, new, last):
    """Pairs of (row, position seen) and positions seen by any row, for the last rows of a chunk."""
    rows = min(last, new) if last else new
    if rows == 0:
        return 0, 0
    t = np.arange(ctx - rows, ctx, dtype=np.int64)
    if not case["window"]:
        return int((t + 1).sum()), int(ctx)
    first = np.maximum(t + 1 - case["window"], 0)
    sinks = np.minimum(case["sinks"], first)
    return int((t + 1 - first + sinks).sum()), int(ctx - first[0] + sinks[0])


def work(case):
    size = {"f32": 4, "bf16": 2, "fp8": 1, "int8": 1}
    d, h_kv, cache = case["dim"], case["h_kv"], size[case["cache"]]
    ctx, new = _lens(case, 0)  # the lengths' distribution stands for every seed's
    if case["op"] == "evict":
        n, m = int(ctx.sum()), int(np.minimum(ctx, case["budget"]).sum())
        # every sum read; kept rows of K and V read and written, their positions and sums written
        return {"bytes": 4 * h_kv * n + h_kv * m * (4 * d * cache + 8) + 8 * case["batch"],
                "flops": 0}
    last = case.get("last", 0)
    pairs, cached = (int(x) for x in np.sum([_seen(case, int(c), int(n), last)
                                             for c, n in zip(ctx, new)], axis=0))
    if case["op"] == "chunk":
        rows = int(new.sum()) * case["h_q"]
        return {"bytes": cached * 2 * h_kv * d * cache + rows * (2 * d * size[case["io"]] + 4),
                "flops": 4 * pairs * case["h_q"] * d}
    rows = int((np.minimum(new, last) if last else new).sum()) * case["h_q"]
    return {"bytes": cached * h_kv * d * cache + rows * (d * size[case["io"]] + 4) +
            8 * h_kv * int(ctx.sum()), "flops": 2 * pairs * case["h_q"] * d}


# ---- the definition in 64 bits -----------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _exact_head(s, b, j, first):
    """For KV head j of request b, from row ``first`` of the chunk on: yields (rows, the cached keys'
    scores [rows, group, context], -inf where a row does not see them), in 64 bits."""
    c = s["case"]
    ctx, new, at = s["ctx"][b], s["new"][b], s["starts"][b]
    group = c["h_q"] // c["h_kv"]
    pages = s["block_tables"][b, :-(-ctx // PAGE)].long()
    k = s["k_cache"][pages, j].double().reshape(-1, c["dim"])[:ctx]
    if s["k_scales"] is not None:
        k = k * s["k_scales"][j].double()
    position = torch.arange(ctx, device="cuda")
    for row in range(first, new, 512):
        rows = torch.arange(row, min(new, row + 512), device="cuda")
        q = s["q"][at + rows, j * group:(j + 1) * group].double()
        score = torch.einsum("tgd,kd->tgk", q, k) * (c["dim"] ** -0.5)
        if c["softcap"]:
            score = torch.tanh(score / c["softcap"]) * c["softcap"]
        behind = (ctx - new + rows)[:, None] - position  # how far a position lies behind a row
        if c["alibi"]:
            slope = s["slopes"][j * group:(j + 1) * group].double()
            score = score - slope[None, :, None] * behind[:, None, :]
        hidden = behind < 0
        if c["window"]:
            hidden |= (behind >= c["window"]) & (position >= c["sinks"])
        yield rows, score.masked_fill(hidden[:, None, :], -math.inf)


def _exact_chunk(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    group = c["h_q"] // c["h_kv"]
    for b in range(c["batch"]):
        pages = s["block_tables"][b, :-(-s["ctx"][b] // PAGE)].long()
        for j in range(c["h_kv"]):
            v = s["v_cache"][pages, j].double().reshape(-1, c["dim"])[:s["ctx"][b]]
            if s["v_scales"] is not None:
                v = v * s["v_scales"][j].double()
            for rows, score in _exact_head(s, b, j, 0):
                at = s["starts"][b] + rows
                out[at, j * group:(j + 1) * group] = torch.softmax(score, -1) @ v
                lse[at, j * group:(j + 1) * group] = torch.logsumexp(score, -1)
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    c = s["case"]
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    group = c["h_q"] // c["h_kv"]
    for b in range(c["batch"]):
        ctx, new = s["ctx"][b], s["new"][b]
        out[b, :, :ctx] = s["weights"][b, :, :ctx].double()
        for j in range(c["h_kv"]):
            for rows, score in _exact_head(s, b, j, max(0, new - c["last"]) if c["last"] else 0):
                lse = s["lse"][s["starts"][b] + rows, j * group:(j + 1) * group].double()
                out[b, j, :ctx] += (score - lse[:, :, None]).exp().sum((0, 1))
    return out


def _exact_evict(s):
    c = s["case"]
    pools = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    kept = np.zeros((c["batch"], c["h_kv"], c["budget"]), np.int32)
    sums = torch.zeros(s["new_weights"].shape, dtype=torch.float64, device="cuda")
    lens = []
    for b, ctx in enumerate(s["ctx"]):
        n = min(ctx, c["budget"])
        lens.append(n)
        w = s["weights"][b, :, :ctx].cpu().numpy()
        old, new = s["block_tables"][b], s["new_tables"][b]
        for j in range(c["h_kv"]):
            always = np.zeros(ctx, bool)
            always[:c["sinks"]] = True
            always[max(0, ctx - c["recent"]):] = True
            # the last key counts most: positions always kept, then larger sums, then lower positions
            order = np.lexsort((np.arange(ctx), -w[j].astype(np.float64), ~always))
            at = np.sort(order[:n])
            kept[b, j, :n] = at
            at = torch.from_numpy(at).cuda()
            sums[b, j, :n] = s["weights"][b, j, at].double()
            to = torch.arange(n, device="cuda")
            for pool in pools.values():
                pool[new[to // PAGE].long(), j, to % PAGE] = pool[old[at // PAGE].long(), j,
                                                                 at % PAGE]
    return dict(pools, kept=torch.from_numpy(kept).cuda(), new_weights=sums,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
