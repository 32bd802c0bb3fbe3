"""The speculative-decoding operators against plain 64-bit implementations, element by element.

Tolerances are bounds, derived where they are computed: a rounding to type t is off by at most
H[t] = eps(t) / 2 relative to the value.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_271_gb300 as pkv
from paged_kv_cache_271_gb300.cache import PagedKVCache
from tests.gpu_harness import fill_junk

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn,
      "int8": torch.int8}
U32 = 2.0 ** -24
H = {"f32": U32, "bf16": 2.0 ** -8, "fp8": 2.0 ** -4}


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available()
    pkv.device_error()
    yield
    pkv.device_error()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def junk_pool(pages, h_kv, d, cache, seed):
    x = torch.empty(pages, h_kv, 16, d, dtype=DT[cache], device="cuda")
    fill_junk(x, seed)
    return x


def raw(x):
    return x.contiguous().view(torch.uint8)


def pick(x, *index):
    """x[index] for every type (8-bit floats are not indexed everywhere)."""
    return raw(x)[index].view(x.dtype)


# ---- norm + rotation + append ------------------------------------------------------------------


def rotated(x, w, table, pos, rot, interleaved, eps):
    """(rows in fp64, magnitude of the sums they are rounded from)."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, mag = x.clone(), x.abs()
    if rot:
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = table.double()[pos.long(), :rot // 2][:, None]
        s = table.double()[pos.long(), rot // 2:][:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


# fp32 work on a row, in units of U32 relative to |a| + |b|: the sum of squares (4 in a lane, 5
# shuffles: under 12 roundings, halved by the root), the mean and eps (1, halved), rsqrt (2 ulp =
# 4 U32), two products (2), the rotation (2): under 16.
NORM_U = 16


def check_rows(got, ref, mag, t, scale=None):
    err = NORM_U * U32 * mag
    if t in ("f32", "bf16"):
        assert ((got.double() - ref).abs() <= H[t] * (ref.abs() + err) + err).all()
        return
    q = ref / scale.double()[:, None]  # the quotient a code stands for, plus its division
    err = err / scale.double()[:, None] + U32 * q.abs()
    if t == "fp8":  # half a step: 2^-4 of the value, 2^-10 below the normal codes; saturating
        q = q.clamp(-448, 448)
        assert ((got.double() - q).abs() <= (H["fp8"] * (q.abs() + err)).clamp_min(2.0 ** -10) +
                err).all()
    else:
        assert ((got.double() - q.clamp(-127, 127)).abs() <= 0.5 + err).all()


APPENDS = [  # tokens, h_q, h_kv, d, io, cache, rot, interleaved, norm
    (1, 32, 8, 128, "bf16", "bf16", 128, False, True),
    (5, 4, 4, 128, "bf16", "bf16", 128, True, True),
    (37, 6, 2, 64, "bf16", "bf16", 64, False, True),
    (19, 8, 1, 64, "bf16", "fp8", 16, False, True),
    (64, 64, 8, 128, "bf16", "fp8", 128, False, True),
    (33, 8, 2, 128, "bf16", "int8", 96, False, True),
    (9, 3, 3, 64, "bf16", "int8", 48, True, False),
    (7, 2, 1, 128, "f32", "f32", 128, False, True),
    (50, 12, 4, 64, "f32", "f32", 32, True, False),
    (11, 5, 1, 64, "f32", "fp8", 64, False, True),
    (13, 4, 2, 128, "f32", "int8", 0, False, True),
    (1300, 7, 1, 128, "bf16", "bf16", 32, False, False),
]


def append_inputs(n, h_q, h_kv, d, io, cache, rot, norm, seed=3):
    g = gen(seed)
    qkv = randn(g, n, (h_q + 2 * h_kv) * d, dtype=DT[io]) * 2
    q, k, v = (x.view(n, -1, d) for x in qkv.split([h_q * d, h_kv * d, h_kv * d], dim=-1))
    w = [randn(g, d).add(1.5).to(DT[io]) if norm else None for _ in range(2)]
    pages = -(-n // 16) + 2
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:n]
    table = pkv.rope_table(500, rot, 10000.0) if rot else None
    pos = torch.randint(0, 500, (n,), generator=g, device="cuda", dtype=torch.int32)
    scales = None
    if cache in ("fp8", "int8"):
        unit = 0.02 if cache == "fp8" else 0.06
        scales = [unit * (0.5 + torch.rand(h_kv, generator=g, device="cuda")) for _ in range(2)]
    kc, vc = (junk_pool(pages, h_kv, d, cache, seed + i) for i in (1, 2))
    return q, k, v, w, pages, slots, table, pos, scales, kc, vc


@pytest.mark.parametrize("n,h_q,h_kv,d,io,cache,rot,inter,norm", APPENDS)
def test_append_matches_the_formula(n, h_q, h_kv, d, io, cache, rot, inter, norm):
    q, k, v, w, pages, slots, table, pos, scales, kc, vc = append_inputs(
        n, h_q, h_kv, d, io, cache, rot, norm)
    before = [raw(kc).clone(), raw(vc).clone()]
    ks, vs = scales or (None, None)
    out = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, table, w[0], w[1], 1e-5, inter,
                                  k_scales=ks, v_scales=vs)
    check_rows(out, *rotated(q, w[0], table, pos, rot, inter, 1e-5), io)
    page, row = slots // 16, slots % 16
    # (8-bit rows: the stored codes, as the values they stand for before the scale)
    check_rows(pick(kc, page, slice(None), row).float(), *rotated(k, w[1], table, pos, rot, inter, 1e-5), cache, ks)
    # the value rows are the append's, byte for byte; nothing else is touched
    kc2, vc2 = before[0].clone().view(kc.dtype), before[1].clone().view(vc.dtype)
    pkv.kv_append(k.contiguous(), v.contiguous(), slots, kc2, vc2, ks, vs)
    assert torch.equal(raw(vc), raw(vc2))
    if not norm and not rot:
        assert torch.equal(raw(kc), raw(kc2))
    other = torch.ones(pages, 16, dtype=torch.bool, device="cuda")
    other[page, row] = False
    at = other.nonzero()
    assert torch.equal(raw(kc)[at[:, 0], :, at[:, 1]],
                       before[0].view(raw(kc).shape)[at[:, 0], :, at[:, 1]])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "int8")])
def test_append_without_norm_or_rotation_is_the_plain_append(io, cache):
    q, k, v, _, _, slots, _, _, scales, kc, vc = append_inputs(40, 8, 2, 128, io, cache, 0, False)
    kc2, vc2 = raw(kc).clone().view(kc.dtype), raw(vc).clone().view(vc.dtype)
    ks, vs = scales or (None, None)
    out = pkv.qk_norm_rope_append(q, k, v, None, slots, kc, vc, None, k_scales=ks, v_scales=vs)
    pkv.kv_append(k.contiguous(), v.contiguous(), slots, kc2, vc2, ks, vs)
    assert torch.equal(out, q) and torch.equal(raw(kc), raw(kc2)) and torch.equal(raw(vc), raw(vc2))


def test_append_in_place_on_a_strided_projection():
    q, k, v, w, _, slots, table, pos, _, kc, vc = append_inputs(21, 8, 2, 128, "bf16", "bf16", 128,
                                                                True)
    kc2, vc2 = raw(kc).clone().view(kc.dtype), raw(vc).clone().view(vc.dtype)
    k0, v0 = k.clone(), v.clone()
    ref = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc2, vc2, table, *w)
    out = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, table, *w, q_out=q)
    assert out.data_ptr() == q.data_ptr() and torch.equal(q, ref)
    assert torch.equal(raw(kc), raw(kc2)) and torch.equal(k, k0) and torch.equal(v, v0)


def test_append_padding_bad_slots_and_positions():
    q, k, v, w, pages, slots, table, pos, _, kc, vc = append_inputs(6, 4, 2, 64, "bf16", "bf16", 64,
                                                                    True)
    kc2, vc2 = raw(kc).clone().view(kc.dtype), raw(vc).clone().view(vc.dtype)
    ref = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc2, vc2, table, *w)
    before = raw(kc).clone()
    slots2, pos2 = slots.clone(), pos.clone()
    slots2[1] = -1          # padding: its query is still rotated
    slots2[2] = pages * 16  # past the pool
    pos2[3], pos2[4] = -1, 500  # outside the table: left out whole
    out = torch.full_like(ref, 7.0)
    pkv.qk_norm_rope_append(q, k, v, pos2, slots2, kc, vc, table, *w, q_out=out)
    assert pkv.device_error() == pkv.DEVERR_BAD_SLOT | pkv.DEVERR_BAD_POSITION
    for i in (0, 1, 2, 5):
        assert torch.equal(out[i], ref[i])
    assert (out[3:5] == 7).all()
    want = before.view(torch.bfloat16).view(kc.shape)
    for i in (0, 5):
        p, r = int(slots[i]) // 16, int(slots[i]) % 16
        want[p, :, r] = kc2[p, :, r]
    assert torch.equal(raw(kc), raw(want))


def test_append_keeps_infinities_in_their_row_and_zero_rows_zero():
    q, k, v, w, _, slots, table, pos, _, kc, vc = append_inputs(4, 2, 1, 64, "f32", "f32", 32, True)
    q = q.clone()
    q[1, 0, 40] = math.inf
    q[2] = 0
    out = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, table, *w, eps=0.0)
    ref = pkv.qk_norm_rope_append(q[:1], k[:1], v[:1], pos[:1], slots[:1], kc, vc, table, *w, eps=0.0)
    assert torch.equal(out[:1], ref) and torch.isfinite(out[1, 1]).all() and torch.isnan(out[2]).all()
    # without a norm an infinity stays in its own dim past the rotated ones
    out = pkv.qk_norm_rope_append(q, k, v, pos, slots, kc, vc, table)
    assert out[1, 0, 40] == math.inf and torch.isfinite(out[1, 0, :40]).all()
    assert (out[2] == 0).all()


# ---- tree attention --------------------------------------------------------------------------------


class Tree:
    """A batch of requests with drafts: pools with junk outside the cached rows, pages in random
    order, random trees."""

    def __init__(self, ctx, tree, nodes, h_q, h_kv, d, io, cache, seed=0, spare=3, mask=None,
                 level=None):
        g, r = gen(seed), np.random.default_rng(seed)
        self.ctx, self.tree, self.nodes = list(ctx), list(tree), nodes
        self.h_q, self.h_kv, self.d, self.io, self.cache = h_q, h_kv, d, io, cache
        B = len(self.ctx)
        pages = [-(-c // 16) for c in self.ctx]
        n = sum(pages) + spare
        order = r.permutation(n)
        self.table = np.full((B, max(pages + [1]) + 1), -12345, np.int32)
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = order[at:at + p]
            at += p
        self.k, self.v = (junk_pool(n, h_kv, d, cache, seed + i) for i in (1, 2))
        self.ks = self.vs = None
        if cache in ("fp8", "int8"):
            unit = 0.02 if cache == "fp8" else 0.02
            self.ks, self.vs = (unit * (0.5 + torch.rand(h_kv, generator=g, device="cuda"))
                                for _ in range(2))
        self.rows = []
        for b, c in enumerate(self.ctx):
            pos = torch.arange(c, device="cuda")
            page = torch.from_numpy(self.table[b])[: max(pages[b], 1)].cuda().long()
            kv = []
            for pool in (self.k, self.v):
                x = randn(g, c, h_kv, d)
                if cache == "fp8":
                    x = (x * 60).clamp(-448, 448)
                elif cache == "int8":
                    x = (x * 40).round().clamp(-127, 127)
                if level is not None and pool is self.k:
                    x[:, :, 0] = level(b, pos)[:, None]
                x = x.to(DT[cache])
                if c:
                    raw_pool = pool.view(torch.uint8) if cache == "fp8" else pool
                    raw_pool[page[pos // 16], :, pos % 16] = (x.view(torch.uint8) if cache == "fp8"
                                                             else x)
                kv.append(x)
            self.rows.append(kv)
        self.q = randn(g, B, nodes, h_q, d, dtype=DT[io])
        if mask is None:
            parents = np.stack([[-1] + [int(r.integers(max(0, i - 5), i)) for i in range(1, nodes)]
                                for _ in range(max(B, 1))])
            mask = pkv.tree_masks(parents)[0]
        self.mask = None if isinstance(mask, str) else torch.from_numpy(np.asarray(mask)).cuda()
        self.out = torch.full(self.q.shape, 3.25, dtype=DT[io], device="cuda")
        self.bt = torch.from_numpy(self.table).cuda()
        self.cl = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.tl = torch.tensor(self.tree, dtype=torch.int32, device="cuda")
        self.scale = d ** -0.5

    def run(self, **kw):
        args = dict(tree_mask=self.mask, tree_lens=self.tl, out=self.out, k_scales=self.ks,
                    v_scales=self.vs)
        args.update(kw)
        return pkv.tree_decode_attention(self.q, self.k, self.v, self.bt, self.cl, self.scale,
                                         **args)

    def seen(self, b):
        """[n, n] node mask of request b."""
        n = self.tree[b]
        if self.mask is None:
            return torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        words = self.mask[b if self.mask.shape[0] > 1 else 0].cpu().numpy()
        bits = np.unpackbits(np.ascontiguousarray(words).view(np.uint8), axis=-1, bitorder="little")
        return torch.from_numpy(bits[:n, :n].astype(bool)).cuda()

    def expect(self, b):
        """(out, tolerance) of request b's rows [n, h_q, d] in fp64."""
        c, n, G = self.ctx[b], self.tree[b], self.h_q // self.h_kv
        q = self.q[b, :n].double()
        k, v = (x.double() for x in self.rows[b])
        if self.ks is not None:
            k, v = k * self.ks.double()[:, None], v * self.vs.double()[:, None]
        k, v = (x.repeat_interleave(G, 1) for x in (k, v))
        see = torch.cat([torch.ones(n, c - n, dtype=torch.bool, device="cuda"), self.seen(b)], 1)
        see = see[:, None, :]
        s = torch.einsum("thd,chd->thc", q, k) * self.scale
        sabs = (torch.einsum("thd,chd->thc", q.abs(), k.abs()) * self.scale)
        s = torch.where(see, s, torch.tensor(-math.inf, device="cuda", dtype=torch.float64))
        p = torch.nan_to_num(torch.softmax(s, -1)) * see
        vv = torch.nan_to_num(v, 0.0, 0.0, 0.0)
        out = torch.einsum("thc,chd->thd", p, vv)
        A = torch.einsum("thc,chd->thd", p, vv.abs())  # weighted magnitude
        # fp32 scores: d products and sums, the scales (4 roundings); their error shifts weights
        ds = ((self.d + 4) * U32 * torch.where(see, torch.nan_to_num(sabs, 0., 0., 0.), 0)).amax(-1)
        # weights: 2^x to 4 U32 and its argument's rounding (|s| log2(e) U32), rounded to the
        # matrix type (bf16 cache: H[bf16]; 8-bit caches: f16, and 2^-25 of the row's largest
        # weight where that is below the f16 normals); sums of c terms
        h = {"f32": 0, "bf16": 2.0 ** -8, "fp8": 2.0 ** -11, "int8": 2.0 ** -11}[self.cache]
        arg = torch.where(see, s.abs(), 0).amax(-1) * 2 * U32
        rel = (h + 2 * ds + 2 * arg + (c + 80) * U32)[..., None]
        tiny = 0 if self.cache in ("f32", "bf16") else 2.0 ** -24 * c * vv.abs().amax(0)[None]
        tol = rel * A + tiny
        return out, tol + H[self.io] * (out.abs() + tol) + 1e-30

    def check(self, got=None):
        got = self.run() if got is None else got
        assert pkv.device_error() == 0
        for b in range(len(self.ctx)):
            n = self.tree[b]
            if n:
                ref, tol = self.expect(b)
                bad = ~((got[b, :n].double() - ref).abs() <= tol)
                assert not bad.any(), (b, bad.nonzero()[:4].tolist(),
                                       (got[b, :n].double() - ref).abs().max().item())
            assert (got[b, n:] == 3.25).all()
        return got


KINDS = [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("bf16", "fp8", 128), ("bf16", "fp8", 64),
         ("bf16", "int8", 128), ("bf16", "int8", 64), ("f32", "f32", 128), ("f32", "f32", 64),
         ("f32", "fp8", 128), ("f32", "int8", 64)]


@pytest.mark.parametrize("io,cache,d", KINDS)
@pytest.mark.parametrize("ctx,tree,nodes,h_q,h_kv", [
    ([1], [1], 1, 1, 1),                                   # one token, one head
    ([1, 16, 17, 64, 65], [1, 1, 1, 1, 1], 1, 8, 2),       # single-token decode
    ([9, 33, 64, 80, 100, 0, 31], [9, 8, 7, 0, 1, 0, 9], 9, 4, 4),  # drafts only, none, ragged
    ([300, 1000, 63, 128], [33, 5, 33, 17], 33, 6, 2),     # three heads to a KV head
    ([2000, 77], [64, 65], 65, 8, 2),                      # over one mask word
    ([1500], [40], 40, 16, 1),                             # many rows, one KV head
])
def test_tree_attention_matches_the_formula(io, cache, d, ctx, tree, nodes, h_q, h_kv):
    Tree(ctx, tree, nodes, h_q, h_kv, d, io, cache, seed=nodes).check()


@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "fp8", 128),
                                        ("f32", "f32", 64)])
def test_tree_attention_of_the_widest_draft(io, cache, d):
    Tree([700, 256], [256, 250], 256, 4, 2, d, io, cache, seed=5).check()


@pytest.mark.parametrize("io,cache,d", KINDS)
def test_tree_attention_of_a_chain_and_of_one_shared_tree(io, cache, d):
    Tree([90, 130, 64], [20, 70, 64], 70, 4, 2, d, io, cache, seed=6, mask="chain").check()
    one = pkv.tree_masks([[-1, 0, 0, 1, 1, 2, 5, 5, 3]])[0]
    Tree([90, 130, 64], [9, 4, 9], 9, 4, 2, d, io, cache, seed=7, mask=one).check()


@pytest.mark.parametrize("io,cache,d", KINDS)
def test_tree_attention_rows_that_see_nothing_are_zero(io, cache, d):
    mask = np.zeros((1, 6, 1), np.int64)
    mask[0, :, 0] = [0, 1, 0b100, 0, -1, 0b100000]  # (bits past the draft are ignored)
    t = Tree([6, 4], [6, 4], 6, 4, 2, d, io, cache, seed=8, mask=mask)
    got = t.check()
    assert (got[0, 0] == 0).all() and (got[0, 3] == 0).all() and (got[1, 3] == 0).all()


@pytest.mark.parametrize("io,cache,d", [k for k in KINDS if k[1] not in ("fp8", "int8")] +
                         [("bf16", "fp8", 128), ("f32", "fp8", 64)])
@pytest.mark.parametrize("base", [0, 5, 60, 130])
def test_tree_attention_unseen_nodes_may_hold_anything(io, cache, d, base):
    """NaN and infinite rows of nodes that a row does not see leave it alone; rows that see them
    get what the formula gives."""
    n = 12
    parents = [[-1] + [i // 2 for i in range(n - 1)]]
    t = Tree([base + n], [n], n, 4, 2, d, io, cache, seed=9, mask=pkv.tree_masks(parents)[0])
    nan = torch.tensor(math.nan, device="cuda")
    for node, value in ((11, math.nan), (10, math.inf if cache != "fp8" else math.nan)):
        p = base + node
        page, row = int(t.table[0, p // 16]), p % 16
        for pool in (t.k, t.v):
            bits = torch.full((t.h_kv, d), value, device="cuda").to(DT[cache])
            (pool.view(torch.uint8) if cache == "fp8" else pool)[page, :, row] = (
                bits.view(torch.uint8) if cache == "fp8" else bits)
        for x in t.rows[0]:
            (x.view(torch.uint8) if cache == "fp8" else x)[p] = 0
    # a value row alone that is not finite, in one dim
    p = base + 9
    page, row = int(t.table[0, p // 16]), p % 16
    hot = torch.zeros(t.h_kv, d, device="cuda")
    hot[:, 5] = math.inf if cache != "fp8" else math.nan
    hot = hot.to(DT[cache])
    (t.v.view(torch.uint8) if cache == "fp8" else t.v)[page, :, row] = (
        hot.view(torch.uint8) if cache == "fp8" else hot)
    t.rows[0][1][p] = hot if cache != "fp8" else torch.zeros_like(hot, dtype=torch.float32).to(
        DT[cache])
    got = t.run()
    ref, tol = t.expect(0)
    sees = t.seen(0)
    for i in range(n):
        if sees[i, 10] or sees[i, 11]:
            assert torch.isnan(got[0, i]).all()
            continue
        bad = ~((got[0, i].double() - ref[i]).abs() <= tol[i])
        if sees[i, 9]:
            assert not torch.isfinite(got[0, i, :, 5]).any()
            bad[:, 5] = False
        assert not bad.any(), i
    assert sees[9, 9] and not sees[0, 9]


@pytest.mark.parametrize("io,cache,d", KINDS)
def test_tree_attention_over_many_requests(io, cache, d):
    r = np.random.default_rng(4)
    ctx = r.integers(5, 90, 300)
    tree = np.minimum(r.integers(0, 6, 300), ctx)
    Tree(ctx.tolist(), tree.tolist(), 5, 4, 2, d, io, cache, seed=10).check()


@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "fp8", 128),
                                        ("bf16", "int8", 64), ("bf16", "bf16", 64),
                                        ("f32", "f32", 64)])
def test_tree_attention_of_long_contexts_is_split_and_joined(io, cache, d):
    Tree([20011, 3, 9000], [7, 3, 0], 7, 8, 2, d, io, cache, seed=11).check()


@pytest.mark.parametrize("io,cache,d", KINDS)
@pytest.mark.parametrize("nodes", [9, 40])  # rows of a KV head: up to 36, up to 160
def test_tree_attention_maxima_that_move_at_every_tile(io, cache, d, nodes):
    """Scores that jump by about 10 (2^14) from one 64 tokens to the next, up, down or in any order,
    over one to seven of them; drafts of few and of many rows side by side."""
    unit, q0 = {"f32": (1, 120), "bf16": (1, 120), "fp8": (40, 150), "int8": (18, 330)}[cache]
    r = np.random.default_rng(21)
    orders = [np.arange(1, 8), np.arange(7, 0, -1), *(r.permutation(7) + 1 for _ in range(6))]
    ctx = r.integers(nodes, 449, 48).tolist()
    tree = [int(n) for n in r.integers(1, nodes + 1, 48)]
    steps = [torch.from_numpy(unit * orders[b % 8]).float().cuda() for b in range(48)]
    t = Tree(ctx, tree, nodes, 8, 2, d, io, cache, seed=21,
             level=lambda b, pos: steps[b][pos // 64])
    t.q[..., 0] = q0 * (d / 128) ** 0.5
    t.check()


def test_tree_attention_matches_single_token_decode():
    t = Tree([100, 1000, 17], [1, 1, 1], 1, 8, 2, 128, "bf16", "bf16", seed=12)
    got = t.check()
    ref = pkv.paged_decode_attention(t.q[:, 0], t.k, t.v, t.bt, t.cl, t.scale)
    for b in range(3):  # two roundings of one value, each within its bound
        _, tol = t.expect(b)
        assert ((got[b, 0].double() - ref[b].double()).abs() <= 2 * tol[0]).all()


def test_tree_attention_scores_of_any_size():
    """Queries far outside f16's range against 8-bit caches: scores are fp32."""
    for cache in ("fp8", "int8", "bf16"):
        for power in (-30, 0, 8, 30):
            t = Tree([130], [6], 6, 4, 2, 128, "bf16", cache, seed=13)
            t.q *= 2.0 ** power
            t.scale = t.d ** -0.5 * 2.0 ** -power
            t.check()
        t = Tree([130], [6], 6, 4, 2, 128, "bf16", cache, seed=14)
        t.q[:, 2] = 0  # a zero query weighs all it sees alike
        t.q[:, 3, :, 1:] *= 2.0 ** -20  # one large component
        t.check()


@pytest.mark.parametrize("io,cache,d", KINDS)
def test_tree_attention_reports_bad_pages_and_skips_them(io, cache, d):
    t = Tree([100, 40], [5, 5], 5, 4, 2, d, io, cache, seed=15)
    good = t.run().clone()
    t.bt[0, 2] = t.k.shape[0]
    t.bt[1, 1] = -1
    got = t.run(out=torch.zeros_like(t.out))
    assert pkv.device_error() == pkv.DEVERR_BAD_PAGE
    # the same as with the positions of those pages unseen
    for b, lp in ((0, 2), (1, 1)):
        keep = [p for p in range(t.ctx[b] - 5) if p // 16 != lp]
        n0 = t.ctx[b] - 5
        nodes = [p for p in range(n0, t.ctx[b])]
        see = t.seen(b)
        for i, p in enumerate(nodes):
            if p // 16 == lp:
                see[:, i] = False
        idx = torch.tensor(keep + nodes, device="cuda")
        sub = Tree([len(idx)], [5], 5, 4, 2, d, io, cache, seed=15)
        sub.rows[0] = [pick(x, idx) for x in t.rows[b]]
        sub.q, sub.ks, sub.vs = t.q[b:b + 1], t.ks, t.vs
        sub.seen = lambda _, see=see: see
        ref, tol = sub.expect(0)
        assert ((got[b].double() - ref).abs() <= tol).all()
    assert torch.isfinite(good).all()


def test_tree_attention_leaves_out_requests_with_bad_drafts():
    t = Tree([50, 60, 3, 20], [5, 5, 3, 5], 5, 4, 2, 128, "bf16", "bf16", seed=16)
    t.tl = torch.tensor([5, 6, 4, -1], dtype=torch.int32, device="cuda")
    got = t.run()
    assert pkv.device_error() == pkv.DEVERR_BAD_TREE
    ref, tol = t.expect(0)
    assert ((got[0].double() - ref).abs() <= tol).all() and (got[1:] == 3.25).all()
    t.tl = torch.tensor([5, 5, 3, 5], dtype=torch.int32, device="cuda")
    t.check()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_tree_attention_cuts_a_context_longer_than_its_table(cache):
    t = Tree([100], [5], 5, 4, 2, 128, "bf16", cache, seed=17)
    t.bt = t.bt[:, :4].contiguous()  # 64 positions: the drafted nodes are past the table
    got = t.run()
    assert pkv.device_error() == pkv.DEVERR_BAD_PAGE
    sub = Tree([69], [5], 5, 4, 2, 128, "bf16", cache, seed=17)
    sub.rows[0] = [x[:69] for x in t.rows[0]]
    sub.q, sub.ks, sub.vs = t.q, t.ks, t.vs
    sub.seen = lambda _: torch.zeros(5, 5, dtype=torch.bool, device="cuda")
    ref, tol = sub.expect(0)
    assert ((got[0].double() - ref).abs() <= tol).all()


def test_tree_attention_without_tree_lens_takes_full_drafts():
    t = Tree([40, 0, 70], [6, 0, 6], 6, 4, 2, 128, "bf16", "bf16", seed=18)
    t.check(t.run(tree_lens=None))


@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "int8", 128),
                                        ("bf16", "fp8", 64)])
def test_tree_attention_past_32_bit_offsets(io, cache, d):
    h_kv = 8
    t = Tree([200, 90], [9, 4], 9, 16, h_kv, d, io, cache, seed=19)
    page_bytes = h_kv * 16 * d * t.k.element_size()
    far = (1 << 32) // page_bytes + 7  # pages whose bytes lie past 2^32
    n = t.k.shape[0]
    for name in ("k", "v"):
        big = torch.empty(far + n, h_kv, 16, d, dtype=DT[cache], device="cuda")
        big.view(torch.uint8)[far:] = getattr(t, name).view(torch.uint8)
        setattr(t, name, big)
    t.bt = t.bt + far
    t.check()


@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "fp8", 128),
                                        ("f32", "f32", 64)])
def test_tree_attention_in_a_graph_follows_its_inputs(io, cache, d):
    """Captured once; lengths, trees and queries change between replays. Replays give the eager
    call's bits."""
    a = Tree([700, 130, 64], [7, 3, 0], 7, 8, 2, d, io, cache, seed=20)
    need = pkv.tree_decode_workspace_size(DT[io], DT[cache], 3, 7, 8, 2, d, a.bt.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    eager = a.check(a.run(workspace=ws)).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(workspace=ws)
    a.out.fill_(3.25)
    ws.random_(0, 255)  # its contents do not matter
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, eager)
    a.ctx, a.tree = [690, 130, 20], [2, 7, 5]
    a.rows = [[x[:c] for x in kv] for kv, c in zip(a.rows, a.ctx)]
    a.cl.copy_(torch.tensor(a.ctx))
    a.tl.copy_(torch.tensor(a.tree))
    a.q.mul_(-1)
    a.out.fill_(3.25)
    g.replay()
    a.check(a.out)


def test_tree_attention_two_streams_two_workspaces():
    trees = [Tree([5000, 800], [16, 9], 16, 8, 2, 128, "bf16", c, seed=21) for c in ("bf16", "fp8")]
    want = [t.check().clone() for t in trees]
    streams = [torch.cuda.Stream() for _ in trees]
    ws = [torch.empty(pkv.tree_decode_workspace_size(torch.bfloat16, DT[t.cache], 2, 16, 8, 2, 128,
                                                     t.bt.shape[1]), dtype=torch.uint8,
                      device="cuda") for t in trees]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, s, w in zip(trees, streams, ws):
            t.run(stream=s, workspace=w)
    torch.cuda.synchronize()
    for t, w in zip(trees, want):
        assert torch.equal(t.out, w)


def test_calls_on_another_stream_make_their_tensors_there(monkeypatch):
    """What a call allocates belongs to the stream it is given, and a new output's zeros come before
    the attention: the current stream is kept busy so that a fill on it would come after."""
    t = Tree([100, 30], [6, 3], 6, 4, 2, 128, "bf16", "bf16", seed=23)
    want = t.check().clone()
    x = t.q[0].contiguous()
    nowhere = torch.full((6,), -1, device="cuda")
    path = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    none = path[:, 0].contiguous()
    side, seen = torch.cuda.Stream(), []
    for name in ("empty", "zeros"):
        def spy(*a, _make=getattr(torch, name), **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return _make(*a, **k)
        monkeypatch.setattr(torch, name, spy)
    for stream in (side, side.cuda_stream):
        del seen[:]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        out = t.run(out=None, stream=stream)
        qo = pkv.qk_norm_rope_append(x, x[:, :2], x[:, 2:], None, nowhere, t.k, t.v, None,
                                     stream=stream)
        lens = pkv.tree_commit(t.k, t.v, t.bt, t.cl, t.tl, path, none, stream=stream)
        torch.cuda.synchronize()
        assert seen == [side.cuda_stream] * 4  # zeros of out, workspace, q_out, new lengths
        assert torch.equal(out[0], want[0]) and torch.equal(out[1, :3], want[1, :3])
        assert (out[1, 3:] == 0).all() and torch.equal(qo, x) and lens.tolist() == [94, 27]
    assert pkv.device_error() == 0


def test_tree_attention_refuses_what_it_cannot_take():
    t = Tree([40], [4], 4, 4, 2, 128, "bf16", "bf16", seed=22)
    for change in (dict(tree_mask=t.mask.int()), dict(tree_mask=t.mask[:, :3].contiguous()),
                   dict(tree_lens=t.tl.long()), dict(out=t.out.float()),
                   dict(tree_mask=t.mask.cpu()), dict(workspace=torch.empty(16, device="cuda"))):
        with pytest.raises(pkv.PkvError):
            t.run(**change)
    with pytest.raises(pkv.PkvError):
        pkv.tree_decode_attention(t.q.transpose(1, 2), t.k, t.v, t.bt, t.cl, 1.0)
    f = Tree([40], [4], 4, 4, 2, 128, "bf16", "fp8", seed=22)
    for change in (dict(k_scales=None), dict(v_scales=f.vs[:1]), dict(k_scales=f.ks.double())):
        with pytest.raises(pkv.PkvError):
            f.run(**change)


# ---- commit ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("fp8", 64), ("int8", 128), ("f32", 64),
                                     ("f32", 128)])
def test_commit_moves_the_path(cache, d):
    nodes = 40
    ctx, tree = [100, 47, 40, 16, 5, 200], [40, 33, 40, 1, 0, 17]
    paths = [[0, 1, 2, 3], [1, 3, 4, 7, 12, 13, 20, 31, 32], list(range(40)), [0], [],
             [2, 3, 4, 5, 6, 7, 8, 9, 10, 16]]
    t = Tree(ctx, tree, nodes, 4, 3, d, "f32" if cache == "f32" else "bf16", cache, seed=30,
             mask="chain")  # (h_q is not used)
    width = 40
    path = torch.full((6, width), -7, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    plen = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    want = [raw(t.k).clone(), raw(t.v).clone()]
    for pool, src in zip(want, (raw(t.k), raw(t.v))):
        for b, p in enumerate(paths):
            for i, node in enumerate(p):
                a, z = (ctx[b] - tree[b] + x for x in (node, i))
                pool[t.table[b, z // 16], :, z % 16] = src[t.table[b, a // 16], :, a % 16]
    lens = pkv.tree_commit(t.k, t.v, t.bt, t.cl, t.tl, path.cuda(), plen.cuda())
    assert pkv.device_error() == 0
    assert lens.tolist() == [c - n + len(p) for c, n, p in zip(ctx, tree, paths)]
    assert torch.equal(raw(t.k), want[0]) and torch.equal(raw(t.v), want[1])


def test_commit_leaves_out_bad_paths():
    t = Tree([50] * 7, [6] * 7, 6, 4, 2, 128, "bf16", "bf16", seed=31, mask="chain")
    path = torch.tensor([[0, 0, 3], [2, 1, 3], [-1, 2, 3], [1, 2, 6], [1, 3, 5], [1, 3, 5],
                         [1, 3, 5]], dtype=torch.int32, device="cuda")
    plen = torch.tensor([3, 3, 3, 3, 4, -1, 3], dtype=torch.int32, device="cuda")
    before = raw(t.k).clone()
    lens = pkv.tree_commit(t.k, t.v, t.bt, t.cl, t.tl, path, plen)
    assert pkv.device_error() == pkv.DEVERR_BAD_TREE
    assert lens.tolist() == [50] * 6 + [47]
    for p, i in ((1, 0), (3, 1), (5, 2)):
        a, z = 44 + p, 44 + i
        before[t.table[6, z // 16], :, z % 16] = before[t.table[6, a // 16], :, a % 16]
    assert torch.equal(raw(t.k), before)
    t.bt[6, 2] = t.k.shape[0]
    pkv.tree_commit(t.k, t.v, t.bt, t.cl, t.tl, path[6:].expand(7, 3).contiguous(),
                    torch.tensor([0] * 6 + [3], dtype=torch.int32, device="cuda"))
    assert pkv.device_error() == pkv.DEVERR_BAD_PAGE
    with pytest.raises(pkv.PkvError):
        pkv.tree_commit(t.k, t.v, t.bt, t.cl, t.tl, path, plen, new_lens=t.cl)


# ---- the step as it is used --------------------------------------------------------------------


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_verification_steps_leave_the_cache_of_plain_decoding(cache):
    """Prompts, then verification steps: the nodes appended, attended, the accepted path kept. A
    second cache that gets only the accepted tokens, one plain append at a time, ends with the same
    rows and page counts, and the accepted nodes' attention is the one it gives."""
    h_q, h_kv, d, B, T = 8, 2, 128, 3, 10
    r, g = np.random.default_rng(40), gen(40)
    ks = vs = None
    if cache == "fp8":
        ks, vs = (torch.full((h_kv,), 0.02, device="cuda") for _ in range(2))
    tree, plain = (PagedKVCache(64, h_kv, d, DT[cache], k_scales=ks, v_scales=vs)
                   for _ in range(2))
    table = pkv.rope_table(512, d)
    norm = dict(q_weight=randn(g, d).add(1).bfloat16(), k_weight=randn(g, d).add(1).bfloat16())
    lens = [37, 16, 3]

    def qkv(n):
        x = randn(g, n, (h_q + 2 * h_kv) * d, dtype=torch.bfloat16)
        return [y.view(n, -1, d) for y in x.split([h_q * d, h_kv * d, h_kv * d], dim=-1)]

    prompt = qkv(sum(lens))
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    for c in (tree, plain):
        for b in range(B):
            c.add_request(b)
        c.write_qkv(c.reserve(range(B), lens), *prompt, pos, table, **norm)
    for step in range(4):
        parents = np.stack([[-1] + [int(r.integers(0, i)) for i in range(1, T)] for _ in range(B)])
        masks, depths = pkv.tree_masks(parents)
        n = [int(x) for x in r.integers(1, T + 1, B)]
        if step == 2:
            n[1] = 0  # a request without a draft in this step
        new = qkv(sum(n))
        pos = np.concatenate([lens[b] + depths[b, :n[b]] for b in range(B)]).astype(np.int32)
        slots = tree.reserve(range(B), n)
        rot = tree.write_qkv(slots, *new, torch.from_numpy(pos).cuda(), table, **norm)
        q = torch.zeros(B, T, h_q, d, dtype=torch.bfloat16, device="cuda")
        at = np.cumsum([0] + n)
        for b in range(B):
            q[b, :n[b]] = rot[at[b]:at[b + 1]]
        bt = torch.from_numpy(tree.block_table_array(range(B))).cuda()
        cl = torch.from_numpy(tree.context_lens_array(range(B))).cuda()
        tl = torch.tensor(n, dtype=torch.int32, device="cuda")
        out = tree.attend_tree(q, bt, cl, d ** -0.5, torch.from_numpy(masks).cuda(), tl)
        path = np.zeros((B, T), np.int32)
        plen = np.zeros(B, np.int32)
        for b in range(B):
            walk = [0] if n[b] else []
            while walk:
                below = [i for i in range(n[b]) if parents[b, i] == walk[-1]]
                if not below or r.random() < 0.2:
                    break
                walk.append(int(r.choice(below)))
            path[b, :len(walk)], plen[b] = walk, len(walk)
        got = tree.commit_tree(range(B), bt, cl, tl, torch.from_numpy(path).cuda(),
                               torch.from_numpy(plen).cuda())
        # the same tokens, plainly
        for i in range(int(plen.max())):
            who = [b for b in range(B) if i < plen[b]]
            rows = torch.tensor([at[b] + path[b, i] for b in who], device="cuda")
            slots = plain.reserve(who, [1] * len(who))
            p = torch.tensor([lens[b] + i for b in who], dtype=torch.int32, device="cuda")
            pq = plain.write_qkv(slots, *(x[rows] for x in new), p, table, **norm)
            ref = pkv.paged_decode_attention(
                pq, plain.k, plain.v, torch.from_numpy(plain.block_table_array(who)).cuda(),
                torch.from_numpy(plain.context_lens_array(who)).cuda(), d ** -0.5, k_scales=ks,
                v_scales=vs)
            for k, b in enumerate(who):
                # both within 2^-8 (weights) + 2^-8 (output) of the value plus the values' size
                # (|V| < 8): 4 * 2^-8 * 8 bounds their difference
                assert ((out[b, path[b, i]].float() - ref[k].float()).abs() <= 4 * 2.0 ** -8 * 8).all()
        lens = [lens[b] + int(plen[b]) for b in range(B)]
        assert got == lens == [tree.lens[b] for b in range(B)] == [plain.lens[b] for b in range(B)]
        assert [len(tree.pages[b]) for b in range(B)] == [len(plain.pages[b]) for b in range(B)]
        assert tree.allocator.num_free() == plain.allocator.num_free()
        for b in range(B):
            p = np.arange(lens[b])
            for x, y in ((tree.k, plain.k), (tree.v, plain.v)):
                a, z = (raw(c)[np.array(t.pages[b])[p // 16], :, p % 16]
                        for c, t in ((x, tree), (y, plain)))
                assert torch.equal(a, z)
    assert pkv.device_error() == 0
