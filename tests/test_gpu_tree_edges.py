"""The speculative-decoding operators in their less usual forms, on the GPU: calls on a stream of the
caller's, drafts of a single tile each, scales and scores of any size, and the whole step against
a 64-bit implementation.

A rounding to type t is off by at most eps(t) / 2 relative to the value; tolerances are derived where
they are computed.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_271_gb300 as pkv
from paged_kv_cache_271_gb300.cache import PagedKVCache
from tests import test_gpu_tree
from tests.test_gpu_tree import DT, H, KINDS, U32, Tree, gen, randn, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available()
    pkv.device_error()
    yield
    pkv.device_error()


# ---- host slots on a stream of the caller's ------------------------------------------------------


def slots_on_a_busy_stream(call, n=600, h_kv=2, d=128):
    """Runs call(cache, slots, k, v, stream) on a busy stream, then fills tensors of the slots' size
    on the current one with the slots of the pool's other half. Every row has to be where its slot
    says, and the other half as it was."""
    g = gen(50)
    k, v = (randn(g, n, h_kv, d, dtype=torch.bfloat16) for _ in range(2))
    slots = np.random.default_rng(50).permutation(1024)[:n].astype(np.int64)
    call(PagedKVCache(128, h_kv, d, torch.bfloat16), slots, k, v, None)  # (kernels are loaded here)
    for raw_handle in (False, True):
        cache = PagedKVCache(128, h_kv, d, torch.bfloat16)
        cache.k.zero_()
        cache.v.zero_()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        kept = call(cache, slots, k, v, side.cuda_stream if raw_handle else side)
        assert not side.query()  # (else nothing is tested)
        others = [torch.empty(n, dtype=torch.int64, device="cuda") for _ in range(8)]
        for x in others:
            x.copy_(torch.arange(1024, 1024 + n, device="cuda"))
        torch.cuda.synchronize()
        at = torch.from_numpy(slots).cuda()
        for pool, rows in ((cache.k, k), (cache.v, v)):
            assert torch.equal(pool[at // 16, :, at % 16], rows)
            assert not raw(pool[64:]).any()
        del kept, others
    assert pkv.device_error() == 0


def test_write_qkv_with_host_slots_on_a_busy_stream():
    slots_on_a_busy_stream(lambda c, slots, k, v, stream: c.write_qkv(
        slots, torch.cat([k, k], 1), k, v, None, None, stream=stream))


def test_write_with_host_slots_on_a_busy_stream():
    slots_on_a_busy_stream(lambda c, slots, k, v, stream: c.write(slots, k, v, stream=stream))


# ---- units of one tile -----------------------------------------------------------------------------


@pytest.mark.parametrize("nodes", [3, 70])  # up to 6 rows a KV head; 140, mostly few
@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("int8", 64)])
def test_long_runs_of_single_tile_units(cache, d, nodes):
    """Contexts of up to 64 tokens, sixteen units a block one behind the other: the second of a
    unit's two groups of threads has no step of its own and runs ahead to the unit's end."""
    r = np.random.default_rng(51)
    ctx = r.integers(1, 65, 600)
    tree = np.minimum(r.integers(1, 4, 600), ctx)
    if nodes > 3:
        tree[::97] = 63
        ctx[::97] = 64
    t = Tree(ctx.tolist(), tree.tolist(), nodes, 8, 4, d, "bf16", cache, seed=51)
    first = t.check().clone()
    for _ in range(20):
        assert torch.equal(t.run(), first)


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
@pytest.mark.parametrize("nodes", [1, 3])
def test_the_largest_batch(io, cache, nodes):
    """65,535 requests of one page; a request's value rows are all alike, so every node that sees any
    gives that row."""
    B, h_kv, d = 65535, 1, 64
    g = gen(56)
    k = randn(g, B, h_kv, 16, d).to(DT[cache])
    x = randn(g, B, h_kv, 1, d).to(DT[cache])
    v = raw(x).view(B, h_kv, 1, -1).expand(-1, -1, 16, -1).contiguous().view(DT[cache])
    q = randn(g, B, nodes, 2, d, dtype=DT[io])
    bt = torch.randperm(B, generator=g, device="cuda").to(torch.int32)[:, None]
    cl = torch.randint(0, 17, (B,), generator=g, device="cuda", dtype=torch.int32)
    tl = torch.minimum(torch.randint(0, nodes + 1, (B,), generator=g, device="cuda",
                                     dtype=torch.int32), cl)
    ks = vs = torch.full((h_kv,), 0.5, device="cuda") if cache == "fp8" else None
    out = pkv.tree_decode_attention(q, k, v, bt, cl, d ** -0.5, tree_lens=tl, k_scales=ks,
                                    v_scales=vs)
    assert pkv.device_error() == 0
    want = x.double()[bt[:, 0].long()][:, :, 0, None] * (0.5 if cache == "fp8" else 1.0)
    want = torch.where(torch.arange(nodes, device="cuda")[None, :, None, None] < tl[:, None, None, None],
                       want, 0.0)
    # the weights' rounding to the matrix type against their unrounded sum (16 terms), the division,
    # the scales, the output's rounding; weights below f16's normals
    h = {"f32": 0, "bf16": 2.0 ** -8, "fp8": 2.0 ** -11}[cache]
    tol = (h + 40 * U32) * want.abs() + (2.0 ** -20 * want.abs().max() if cache == "fp8" else 0)
    assert ((out.double() - want).abs() <= tol + H[io] * (want.abs() + tol)).all()


# ---- outputs that the call makes --------------------------------------------------------------------


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
@pytest.mark.parametrize("lens", [True, False])
def test_a_new_output_is_zero_where_there_is_no_draft(io, cache, lens):
    """With tree_lens and without: requests without a context, and ones that are left out because
    their context is shorter than the draft."""
    t = Tree([40, 0, 70, 4], [6, 0, 6, 4], 6, 4, 2, 128, io, cache, seed=52)
    t.tl = torch.tensor([6, 0, 6, 5], dtype=torch.int32, device="cuda")  # (5 of 4: left out)
    want = t.run().clone()
    assert (want[1] == 3.25).all() and (want[3] == 3.25).all()
    assert pkv.device_error() == pkv.DEVERR_BAD_TREE
    want[1] = want[3] = 0
    for _ in range(3):
        poison = torch.full_like(want, float("nan"))
        at = poison.data_ptr()
        del poison  # (the next output of this size)
        got = t.run(out=None, tree_lens=t.tl if lens else None)
        assert got.data_ptr() == at and torch.equal(got, want)
        assert pkv.device_error() == pkv.DEVERR_BAD_TREE
        del got


# ---- scales and scores of any size -------------------------------------------------------------------


@pytest.mark.parametrize("io,cache,d", [("bf16", "fp8", 128), ("bf16", "int8", 64), ("f32", "fp8", 64),
                                        ("f32", "int8", 128)])
@pytest.mark.parametrize("nodes", [7, 70])  # up to 28 rows a KV head; 280
def test_negative_zero_and_nan_scales_are_kept(io, cache, d, nodes):
    t = Tree([nodes + 9, nodes + 300], [nodes, 5], nodes, 12, 3, d, io, cache, seed=53)
    t.ks[0] *= -1
    t.ks[1] = 0  # every seen position weighs the same
    t.vs[2] *= -1
    t.check()
    want = t.out.clone()
    t.ks[1] = float("nan")
    got = t.run()
    assert torch.equal(got[:, :, :4], want[:, :, :4]) and torch.equal(got[:, :, 8:], want[:, :, 8:])
    for b, n in enumerate(t.tree):
        assert torch.isnan(got[b, :n, 4:8]).all() and (got[b, n:] == 3.25).all()


@pytest.mark.parametrize("io,cache,d", KINDS)
@pytest.mark.parametrize("power", [12, 22, 26, 28, 30, 32, 33, 60, 110])
def test_scores_of_huge_size_pick_the_largest(io, cache, d, power):
    """Queries 2^power times their usual size: where the largest score of a row leads the others by
    30 more than fp32 can tell apart, the row's output is that position's value."""
    checked = rows = 0
    for nodes, ctx in ((7, 330), (60, 130)):  # up to 21 rows a KV head; 180
        t = Tree([ctx], [nodes], nodes, 6, 2, d, io, cache, seed=54)
        t.q *= 2.0 ** power
        got = t.run()[0].double()
        assert pkv.device_error() == 0
        k, v = (x.double() for x in t.rows[0])
        if t.ks is not None:
            k, v = k * t.ks.double()[:, None], v * t.vs.double()[:, None]
        k, v = (x.repeat_interleave(3, 1) for x in (k, v))
        q = t.q[0].double()
        see = torch.ones(nodes, ctx, dtype=torch.bool, device="cuda")
        see[:, ctx - nodes:] = t.seen(0)
        s = torch.einsum("thd,chd->thc", q, k) * t.scale
        s = torch.where(see[:, None], s, torch.tensor(float("-inf"), dtype=s.dtype, device="cuda"))
        sabs = torch.einsum("thd,chd->thc", q.abs(), k.abs()) * t.scale
        # d products and sums, the scales and log2(e), and the score's own rounding, of both scores
        fuzz = 2 * (d + 8) * U32 * torch.where(see[:, None], sabs, 0).amax(-1)
        top = s.topk(2, -1)
        clear = top.values[..., 0] - top.values[..., 1] > 30 + fuzz
        want = torch.stack([v[top.indices[:, h, 0], h] for h in range(6)], 1)
        # the others weigh less than ctx e^-30 < 2^-34 of the largest value; the weight's own
        # rounding to the matrix type, the division, the scales and the output's
        h = {"f32": 0, "bf16": 2.0 ** -8, "fp8": 2.0 ** -11, "int8": 2.0 ** -11}[cache]
        tol = (h + 8 * U32) * want.abs() + 2.0 ** -33 * v.abs().max()
        tol = tol + H[io] * (want.abs() + tol)
        bad = ~((got - want).abs() <= tol) & clear[..., None]
        assert not bad.any(), (nodes, bad.any(-1).sum().item(), clear.sum().item())
        checked += int(clear.sum())
        rows += clear.numel()
    assert 2 * checked > rows


@pytest.mark.parametrize("io,cache,d", KINDS)
def test_rows_of_huge_and_usual_scores_side_by_side(io, cache, d):
    """Usual rows keep their bounds beside rows whose scores fp32 hardly tells apart (which only have
    to be finite: their bound is as wide as the values)."""
    for nodes, ctx in ((9, [40, 300, 64]), (60, [130, 700])):
        t = Tree(ctx, [nodes] * len(ctx), nodes, 6, 2, d, io, cache, seed=57)
        r = np.random.default_rng(57)
        power = np.where(r.random((len(ctx), nodes, 6, 1)) < 0.3, r.integers(20, 60, (len(ctx), nodes, 6, 1)), 0)
        t.q *= torch.from_numpy(2.0 ** power).to("cuda", t.q.dtype)
        t.check()


# ---- append: blocks with several row groups over many tokens -----------------------------------------

# Rows (query, key and value heads) of a token, in groups of 16 (32 for 64 bf16 dims, 8 for 128 fp32
# dims); calls of more than 456 groups in all give a block up to three groups of a token and several
# tokens, an odd or an even number of them.
LOOPS = [  # tokens, h_q, h_kv, d, io, cache, rot, interleaved, norm
    (1401, 16, 8, 128, "bf16", "bf16", 128, False, True),   # two groups
    (1000, 32, 8, 128, "bf16", "bf16", 128, False, True),   # three
    (2300, 32, 8, 128, "bf16", "fp8", 128, False, True),    # three, six tokens at most
    (777, 64, 8, 128, "bf16", "fp8", 128, False, True),     # three and two, in two parts
    (643, 61, 9, 128, "bf16", "int8", 96, True, True),      # the same, the last one not full
    (1500, 20, 5, 128, "bf16", "bf16", 48, True, False),    # heads of three kinds in one warp
    (919, 70, 3, 64, "bf16", "int8", 64, False, True),
    (1300, 12, 4, 128, "f32", "f32", 128, False, True),     # three groups
    (1203, 9, 4, 128, "f32", "int8", 128, True, True),
    (1100, 40, 4, 64, "f32", "fp8", 32, False, True),
    (12345, 7, 1, 64, "f32", "f32", 64, True, True),        # one group, 28 tokens
]


@pytest.mark.parametrize("case", LOOPS, ids=lambda c: "-".join(map(str, c[:6])))
def test_append_of_many_tokens_matches_the_formula(case):
    test_gpu_tree.test_append_matches_the_formula(*case)


@pytest.mark.parametrize("case", LOOPS[:10], ids=lambda c: "-".join(map(str, c[:6])))
def test_append_of_many_tokens_is_that_of_each_alone(case):
    """Bit for bit, in place as well, with padding, bad slots and bad positions among them."""
    n, h_q, h_kv, d, io, cache, rot, inter, norm = case
    q, k, v, w, pages, slots, table, pos, scales, kc, vc = test_gpu_tree.append_inputs(
        n, h_q, h_kv, d, io, cache, rot, norm, seed=55)
    slots, pos = slots.clone(), pos.clone()
    slots[7::50], slots[9::50], pos[3::50], pos[4::50] = -1, pages * 16, -1, 500
    ks, vs = scales or (None, None)

    def one(i, j, kc, vc, out):
        pkv.qk_norm_rope_append(q[i:j], k[i:j], v[i:j], pos[i:j], slots[i:j], kc, vc, table, w[0],
                                w[1], 1e-5, inter, q_out=out[i:j], k_scales=ks, v_scales=vs)

    pools = [(raw(kc).clone().view(kc.dtype), raw(vc).clone().view(vc.dtype)) for _ in range(3)]
    want = q.clone()  # (rows of tokens left out stay)
    for i in range(n):
        one(i, i + 1, *pools[0], want)
    assert pkv.device_error() == pkv.DEVERR_BAD_SLOT | pkv.DEVERR_BAD_POSITION
    apart = q.clone()
    one(0, n, *pools[1], apart)
    k0, v0 = k.clone(), v.clone()
    one(0, n, *pools[2], q)
    assert pkv.device_error() == pkv.DEVERR_BAD_SLOT | pkv.DEVERR_BAD_POSITION
    assert torch.equal(apart, want) and torch.equal(q, want)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    for p in pools[1:]:
        assert torch.equal(raw(p[0]), raw(pools[0][0])) and torch.equal(raw(p[1]), raw(pools[0][1]))


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("scale", [0.02, 2.0 ** -100, 2.0 ** 100, 1e-38, -0.5, 0.0, float("nan")])
def test_append_of_every_bf16_value_is_the_plain_appends(cache, scale):
    """Value rows byte for byte, whatever they hold (infinities, NaN, subnormal numbers), and without
    norm and rotation key rows too, but for which NaN a NaN becomes."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    x = x[torch.randperm(65536, generator=gen(58), device="cuda")].view(256, 2, 128)
    ks = vs = None if cache == "bf16" else torch.full((2,), scale, device="cuda")
    slots = torch.randperm(320, generator=gen(59), device="cuda")[:256]
    pools = [[test_gpu_tree.junk_pool(20, 2, 128, cache, 58) for _ in range(2)] for _ in range(3)]
    q = torch.zeros(256, 4, 128, dtype=torch.bfloat16, device="cuda")
    pkv.kv_append(x, x, slots, *pools[0], ks, vs)
    pkv.qk_norm_rope_append(q, x, x, None, slots, *pools[1], None, k_scales=ks, v_scales=vs)
    table = pkv.rope_table(4, 128)
    pos = torch.zeros(256, dtype=torch.int32, device="cuda")  # (another path: the keys are rotated)
    pkv.qk_norm_rope_append(q, x, x, pos, slots, *pools[2], table, k_scales=ks, v_scales=vs)
    assert torch.equal(raw(pools[1][1]), raw(pools[0][1]))
    assert torch.equal(raw(pools[2][1]), raw(pools[0][1]))
    k0, k1 = pools[0][0], pools[1][0]
    if cache == "int8":
        assert torch.equal(k0, k1)
    else:
        nan = torch.isnan(k0.float())
        assert torch.equal(torch.isnan(k1.float()), nan)
        assert torch.equal(k0.view(raw(k0).dtype if cache == "fp8" else torch.int16)[~nan],
                           k1.view(raw(k1).dtype if cache == "fp8" else torch.int16)[~nan])


# ---- the step as it is used, node by node -------------------------------------------------------------


def attention(q, k, v, see, scale, cache):
    """(out, tolerance) [n, h_q, d] in fp64 on the CPU: queries [n, h_q, d] over rows k, v [c, h_kv, d],
    of which node t sees those of see[t]."""
    n, h_q, d = q.shape
    c, h_kv, _ = k.shape
    k, v = (x.repeat_interleave(h_q // h_kv, 1) for x in (k, v))
    see = see[:, None, :]
    s = (torch.einsum("thd,chd->thc", q, k) * scale).masked_fill(~see, -math.inf)
    size = (torch.einsum("thd,chd->thc", q.abs(), k.abs()) * scale * see).amax(-1, keepdim=True)
    p = torch.softmax(s, -1)
    out, mag = (torch.einsum("thc,chd->thd", p, x) for x in (v, v.abs()))
    # fp32 scores: d products and sums, the scales, twice (the score and the row's largest); the
    # weights' exponents and the sums of c terms; the weights' rounding for the product with V
    h = 2.0 ** -8 if cache == "bf16" else 2.0 ** -11
    top = s.masked_fill(~see, 0).abs().amax(-1, keepdim=True)
    tol = (h + (2 * (d + 4) * size + 4 * top + c + 80) * U32) * mag
    if cache == "fp8":  # weights below f16's normals
        tol = tol + 2.0 ** -24 * c * v.abs().amax(0)[None]
    return out, tol + H["bf16"] * (out.abs() + tol)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_every_node_of_every_step_attends_what_it_should(cache):
    """Verification steps against a list of accepted rows kept on the CPU. The bounds tell a node that
    sees one row too few: taking a node's own row out of the implementation breaks them."""
    h_q, h_kv, d, B, T = 8, 2, 128, 3, 12
    r, g = np.random.default_rng(60), gen(60)
    ks = vs = None
    if cache == "fp8":
        ks, vs = (torch.tensor([0.02, 0.03], device="cuda") for _ in range(2))
    c = PagedKVCache(64, h_kv, d, DT[cache], k_scales=ks, v_scales=vs)
    table = pkv.rope_table(512, d)
    norm = dict(q_weight=randn(g, d).add(1).bfloat16(), k_weight=randn(g, d).add(1).bfloat16())

    def qkv(n):
        x = randn(g, n, (h_q + 2 * h_kv) * d, dtype=torch.bfloat16)
        return [y.view(n, -1, d) for y in x.split([h_q * d, h_kv * d, h_kv * d], dim=-1)]

    def rows(slots):  # K and V rows of these slots on the CPU, in fp64
        at = torch.from_numpy(np.asarray(slots)).cuda()
        got = []
        for pool, scale in ((c.k, ks), (c.v, vs)):
            x = raw(pool)[at // 16, :, at % 16].view(DT[cache]).double()
            got.append((x if scale is None else x * scale.double()[:, None]).cpu())
        return got

    lens = [45, 16, 3]
    for b in range(B):
        c.add_request(b)
    slots = c.reserve(range(B), lens)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    c.write_qkv(slots, *qkv(sum(lens)), pos, table, **norm)
    at = np.cumsum([0] + lens)
    kept = [rows(slots[at[b]:at[b + 1]]) for b in range(B)]
    for step in range(5):
        parents = np.stack([[-1] + [int(r.integers(0, i)) for i in range(1, T)] for _ in range(B)])
        masks, depths = pkv.tree_masks(parents)
        n = [int(x) for x in r.integers(1, T + 1, B)]
        n[step % B] = [T, 0, 1, T, 5][step]
        pos = np.concatenate([lens[b] + depths[b, :n[b]] for b in range(B)]).astype(np.int32)
        slots = c.reserve(range(B), n)
        rot = c.write_qkv(slots, *qkv(sum(n)), torch.from_numpy(pos).cuda(), table, **norm)
        at = np.cumsum([0] + n)
        q = torch.zeros(B, T, h_q, d, dtype=torch.bfloat16, device="cuda")
        for b in range(B):
            q[b, :n[b]] = rot[at[b]:at[b + 1]]
        bt = torch.from_numpy(c.block_table_array(range(B))).cuda()
        cl = torch.from_numpy(c.context_lens_array(range(B))).cuda()
        tl = torch.tensor(n, dtype=torch.int32, device="cuda")
        out = c.attend_tree(q, bt, cl, d ** -0.5, torch.from_numpy(masks).cuda(), tl).double().cpu()
        path = np.zeros((B, T), np.int32)
        plen = np.zeros(B, np.int32)
        for b in range(B):
            assert not out[b, n[b]:].any()
            if n[b] == 0:
                continue
            new = rows(slots[at[b]:at[b + 1]])
            k, v = (torch.cat([x, y]) for x, y in zip(kept[b], new))
            see = torch.zeros(n[b], lens[b] + n[b], dtype=torch.bool)
            see[:, :lens[b]] = True
            for i in range(n[b]):
                j = i
                while j >= 0:
                    see[i, lens[b] + j] = True
                    j = int(parents[b, j])
            qb = q[b, :n[b]].double().cpu()
            ref, tol = attention(qb, k, v, see, d ** -0.5, cache)
            assert ((out[b, :n[b]] - ref).abs() <= tol).all(), (step, b)
            for i in range(n[b]):
                see[i, lens[b] + i] = False
            ref, tol = attention(qb, k, v, see, d ** -0.5, cache)
            assert ((out[b, :n[b]] - ref).abs() > tol).flatten(1).any(1).all(), (step, b)
            walk = [0]
            while True:
                below = [i for i in range(n[b]) if parents[b, i] == walk[-1]]
                if not below or r.random() < 0.2:
                    break
                walk.append(int(r.choice(below)))
            path[b, :len(walk)], plen[b] = walk, len(walk)
            kept[b] = [torch.cat([x, y[walk]]) for x, y in zip(kept[b], new)]
        got = c.commit_tree(range(B), bt, cl, tl, torch.from_numpy(path).cuda(),
                            torch.from_numpy(plen).cuda())
        lens = [lens[b] + int(plen[b]) for b in range(B)]
        assert got == lens == [len(kept[b][0]) for b in range(B)]
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("below", [10.0, 24.6, 30.0])
@pytest.mark.parametrize("batch,nodes,h_q", [(40, 64, 16), (200, 4, 8), (2, 4, 8)])
def test_many_small_weights_beside_a_large_one(cache, below, batch, nodes, h_q):
    """One position with 2^below times the weight of each of 131,072 others, whose values alone are not 0:
    together the small ones count, though each is near the end of the matrix type's range. (All requests
    share one context.)"""
    d, past = 64, 1 << 17
    pages = -(-(past + nodes) // 16)
    one = {"bf16": 1.0, "fp8": 0x38, "int8": 1}[cache]  # (0x38: the code of 1)
    dtype = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8}[cache]
    k, v = (torch.zeros(pages, 1, 16, d, dtype=dtype, device="cuda") for _ in range(2))
    k[0, 0, 0, 0] = one
    v.fill_(one)
    v[0, 0, 0] = 0
    scales = {} if cache == "bf16" else dict(k_scales=torch.ones(1, device="cuda"),
                                             v_scales=torch.ones(1, device="cuda"))
    q = torch.zeros(batch, nodes, h_q, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 16.0
    scale = torch.tensor(below * math.log(2.0) / 16.0).item()  # (as the call takes it: fp32)
    out = pkv.tree_decode_attention(
        q, k, v, torch.arange(pages, dtype=torch.int32, device="cuda")[None].repeat(batch, 1),
        torch.full((batch,), past + nodes, dtype=torch.int32, device="cuda"), scale, **scales)
    n = torch.arange(past, past + nodes, dtype=torch.float64, device="cuda")[None, :, None, None]
    ref = n / (n + math.exp(scale * 16.0))
    # the large weight's score (4 U32 of it) and exponential (2^-21); a small weight's; sums over tiles of 64,
    # one rounding or truncation (2 U32) each, and 64 within them and over shares; a small weight's rounding
    # to the matrix type: in f16 half a step, 2^-25, of a value kept 2^7 times as large or more; the output's
    e = 4 * U32 * below + 2.0 ** -20 + 2 * (past // 64 + 64) * U32
    p = H["bf16"] if cache == "bf16" else 2.0 ** -11 + 2.0 ** (below - 32)
    tol = (2 * e + p) * ref + H["bf16"] * ref * (1 + p)
    assert ((out.double() - ref).abs() <= tol).all(), ((out.double() - ref).abs() / tol).max()
    assert pkv.device_error() == 0
