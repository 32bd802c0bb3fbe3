"""Attention of chunks of new tokens, the sums of its weights and the eviction by them, against plain
64-bit implementations, element by element.

Tolerances are bounds, derived where they are computed: a rounding to type t is off by at most
H[t] = eps(t) / 2 relative to the value.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_271_gb300 as pkv
from paged_kv_cache_271_gb300.cache import PagedKVCache
from tests.test_gpu_tree import DT, U32, gen, junk_pool, randn, raw

pytestmark = pytest.mark.gpu

H = {"f32": U32, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(autouse=True)
def _clean_error_word():
    assert torch.cuda.is_available()
    pkv.device_error()
    yield
    pkv.device_error()


class Chunk:
    """Requests with `past` cached tokens and `new` further ones on random pages of a pool of junk."""

    def __init__(self, past, new, h_q=8, h_kv=2, d=128, io="bf16", cache="bf16", seed=1, softcap=0.0,
                 alibi=False, window=0, sinks=0, spread=1.0, pad=3, spare=2):
        g, r = gen(seed), np.random.default_rng(seed)
        self.new = list(new)
        self.ctx = [p + n for p, n in zip(past, new)]
        self.h_q, self.h_kv, self.d, self.io, self.cache = h_q, h_kv, d, io, cache
        self.group = h_q // h_kv
        self.softcap, self.window, self.sinks = softcap, window, sinks
        B = len(self.new)
        pages = [-(-c // 16) for c in self.ctx]
        n = sum(pages) + spare
        order = r.permutation(n)
        table = np.full((B, max(max(pages), 1) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.table, self.spare_pages = table, order[at:]
        self.k_cache, self.v_cache = (junk_pool(n, h_kv, d, cache, seed + i) for i in (1, 2))
        self.k_scales = self.v_scales = None
        if cache in ("fp8", "int8"):
            unit = 0.03 if cache == "fp8" else 0.02
            self.k_scales, self.v_scales = (unit * (0.5 + torch.rand(h_kv, generator=g, device="cuda"))
                                            for _ in range(2))
        for b in range(B):  # the rows of the contexts; what lies behind them stays junk
            for pool in (self.k_cache, self.v_cache):
                x = randn(g, self.ctx[b], h_kv, d) * (1 if cache in ("f32", "bf16") else 40)
                x = (x.round().clamp(-127, 127).to(torch.int8) if cache == "int8" else
                     x.to(DT[cache]))
                pos = torch.arange(self.ctx[b])
                page = torch.from_numpy(table[b].astype(np.int64))[pos // 16].cuda()
                raw8 = pool.view(torch.uint8) if pool.element_size() == 1 else pool
                raw8[page, :, (pos % 16).cuda()] = (x.view(torch.uint8) if pool.element_size() == 1
                                                    else x)
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.starts[-1])
        self.q = randn(g, self.rows + pad, h_q, d).mul(spread).to(DT[io])
        self.scale = d ** -0.5
        self.slopes = (torch.rand(h_q, generator=g, device="cuda") * 0.3) if alibi else None
        self.dev()

    def dev(self):
        self.bt = torch.from_numpy(self.table).cuda()
        self.cl = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.qs = torch.from_numpy(self.starts).cuda()

    def form(self):
        return dict(softcap=self.softcap, alibi_slopes=self.slopes, window=self.window,
                    sink_tokens=self.sinks)

    def attend(self, **kw):
        kw = {**self.form(), "k_scales": self.k_scales, "v_scales": self.v_scales, **kw}
        return pkv.chunk_attention(self.q, self.k_cache, self.v_cache, self.bt, self.cl, self.qs,
                                   self.scale, **kw)

    def weigh(self, lse, **kw):
        kw = {**self.form(), "k_scales": self.k_scales, **kw}
        return pkv.chunk_weights(self.q, self.k_cache, self.bt, self.cl, self.qs, lse, self.scale,
                                 **kw)

    def cached(self, pool, scales, b, j):
        """Rows of KV head j of request b in 64 bits; a page that is not there: None rows."""
        ids = self.table[b, :-(-self.ctx[b] // 16)].astype(np.int64)
        good = (ids >= 0) & (ids < pool.shape[0])
        x = pool[torch.from_numpy(np.where(good, ids, 0)).cuda()][:, j].double().reshape(-1, self.d)
        there = torch.from_numpy(np.repeat(good, 16)).cuda()[:self.ctx[b]]
        x = x[:self.ctx[b]]
        return (x if scales is None else x * scales[j].double()), there

    def score_error(self, q, k):
        """Bound of the fp32 scores' errors (natural units): d products, summed in any order and
        truncated (2 U32 each), the scale's and the K scale's roundings; the cap's tanh is off by at
        most 2^-21 besides."""
        e = self.scale * (2 * self.d + 8) * U32 * (q.abs() @ k.abs().T).amax(-1)
        return e + self.softcap * 2.0 ** -21

    def reference(self, b, j):
        """(scores [new, group, ctx] with -inf where unseen, bound of their error [new, group])."""
        k, there = self.cached(self.k_cache, self.k_scales, b, j)
        k = torch.where(there[:, None], k, 0.0).nan_to_num(0.0, 0.0, 0.0) if not there.all() else k
        at = int(self.starts[b])
        q = self.q[at:at + self.new[b], j * self.group:(j + 1) * self.group].double()
        s = q @ k.T * self.scale
        err = self.score_error(q, k.nan_to_num(0.0, 0.0, 0.0))
        if self.softcap:
            s = self.softcap * torch.tanh(s / self.softcap)
        pos = torch.arange(self.ctx[b], device="cuda")
        behind = torch.arange(self.ctx[b] - self.new[b], self.ctx[b], device="cuda")[:, None] - pos
        if self.slopes is not None:
            slope = self.slopes[j * self.group:(j + 1) * self.group].double()
            s = s - slope[None, :, None] * behind[:, None, :]
            err = err + 3 * U32 * slope * 60  # (a bias beyond 60 takes the weight below 2^-80)
        seen = (behind >= 0) & there
        if self.window:
            seen &= (behind < self.window) | (pos < self.sinks)
        return s.masked_fill(~seen[:, None, :], -math.inf), err

    def check(self, out, lse=None):
        # P is rounded to the cache's matrix type; for fp32 queries it is not
        p_type = None if self.io == "f32" else "bf16" if self.cache == "bf16" else "f16"
        for b in range(len(self.new)):
            if self.new[b] == 0:
                continue
            for j in range(self.h_kv):
                s, err = self.reference(b, j)
                v, there = self.cached(self.v_cache, self.v_scales, b, j)
                v = torch.where(there[:, None], v, 0.0)
                at = slice(int(self.starts[b]), int(self.starts[b]) + self.new[b])
                heads = slice(j * self.group, (j + 1) * self.group)
                ref_lse = torch.logsumexp(s, -1)
                p = torch.exp(s - ref_lse.clamp_min(-1e300)[..., None])
                ref, size = p @ v, p @ v.abs()
                # a weight: the score's error, 2^-21 of the exponential and the running maximum's
                # FMA (|s| U32 shared by a row's weights), its rounding; the sums over tiles, groups and
                # shares in fp32: up to 40 roundings; f16 weights below 2^-14 step by 2^-25
                sums = 40 * U32 + 2.0 ** -21
                e = 2 * err[..., None] + sums + (H[p_type] if p_type else 0)
                tiny = v.abs().amax() * (2.0 ** -24 * self.ctx[b] if p_type == "f16" else 0.0)
                got = out[at, heads].double()
                tol = e * size + H[self.io] * (ref.abs() + e * size) + tiny * 2 ** -8 + 1e-30
                bad = (got - ref).abs() > tol
                assert not bad.any(), (b, j, bad.sum().item(), ((got - ref).abs() / tol).max())
                if lse is not None:
                    x = lse[at, heads].double()
                    empty = torch.isinf(ref_lse)
                    assert torch.equal(torch.isinf(x), empty)
                    tol = err + sums + 4 * U32 * (ref_lse.abs() + s.nan_to_num(0., 0., 0.).abs().amax(-1))
                    assert ((x - ref_lse).abs() <= tol)[~empty].all(), (b, j)

    def sums(self, lse, last=0, add_to=None):
        """(reference sums, bounds) of the weights that the rows give, with this lse."""
        B, width = len(self.new), self.bt.shape[1] * 16
        ref = torch.zeros(B, self.h_kv, width, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(ref)
        for b in range(B):
            n, c = self.new[b], self.ctx[b]
            first = max(0, n - last) if last else 0
            at = int(self.starts[b])
            for j in range(self.h_kv):
                if n:
                    s, err = self.reference(b, j)
                    x = lse[at:at + n, j * self.group:(j + 1) * self.group].double()
                    # (a row that saw nothing gives nothing)
                    w = torch.where(torch.isinf(x)[..., None], 0.0, torch.exp(s - x[..., None]))[first:]
                    # a weight: the score's error, roundings of its product and of the lse in the
                    # log2 domain, 2^-21 of the exponential; a step's sum 16 + 4 roundings, the
                    # compensated sum, four places, the partials
                    e = 2 * err + 4 * U32 * (x.nan_to_num(0., 0., 0.).abs() + 30) + 2.0 ** -21 + 40 * U32
                    ref[b, j, :c] = w.sum((0, 1))
                    tol[b, j, :c] = (w * e[first:, :, None]).sum((0, 1)) + 1e-30
                if add_to is not None:
                    ref[b, j] += add_to[b, j].double()
        tol += 2 * U32 * ref.abs()
        return ref, tol


KINDS = [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("bf16", "fp8", 128), ("bf16", "int8", 64),
         ("bf16", "int8", 128), ("bf16", "fp8", 64), ("f32", "f32", 128), ("f32", "f32", 64),
         ("f32", "fp8", 64), ("f32", "int8", 128)]
SIZES = [  # past, new, h_q, h_kv
    ([0], [1], 4, 2), ([0], [129], 4, 1), ([777], [1], 32, 8), ([130], [63], 8, 2),
    ([5, 0, 300, 1000, 40], [60, 1, 0, 200, 16], 6, 2), ([0, 63], [257, 300], 3, 3),
    ([100, 17, 2000], [1, 1, 1], 16, 2), ([50], [70], 128, 1), ([31], [20], 40, 1),
]


@pytest.mark.parametrize("past,new,h_q,h_kv", SIZES)
@pytest.mark.parametrize("io,cache,d", KINDS)
def test_attention_and_sums_match_the_formula(io, cache, d, past, new, h_q, h_kv):
    c = Chunk(past, new, h_q, h_kv, d, io, cache)
    lse = torch.full((c.q.shape[0], h_q), 7.0, device="cuda")
    out = torch.full_like(c.q, 3.0)
    assert c.attend(out=out, lse=lse) is out
    assert pkv.device_error() == 0
    c.check(out, lse)
    assert (out[c.rows:] == 3).all() and (lse[c.rows:] == 7).all()  # rows of no request
    w = c.weigh(lse)
    ref, tol = c.sums(lse)
    assert ((w.double() - ref).abs() <= tol).all()
    for b in range(len(new)):
        assert (w[b, :, c.ctx[b]:] == 0).all()
    assert pkv.device_error() == 0


FORMS = [dict(softcap=5.0), dict(softcap=30.0, alibi=True), dict(alibi=True),
         dict(window=1), dict(window=100, sinks=4), dict(window=300, sinks=150),
         dict(window=64, sinks=1, softcap=20.0), dict(window=2000), dict(spread=300.0),
         dict(spread=60.0, softcap=50.0)]


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("io,cache,d", [KINDS[i] for i in (0, 1, 2, 3, 6, 8)])
def test_forms_match_the_formula(io, cache, d, form):
    c = Chunk([0, 517, 1300], [400, 130, 33], 8, 2, d, io, cache, seed=2, **form)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.check(c.attend(lse=lse), lse)
    for last in (0, 1, 50):
        w = c.weigh(lse, last_rows=last)
        ref, tol = c.sums(lse, last)
        assert ((w.double() - ref).abs() <= tol).all()
    assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "int8"), ("f32", "f32")])
@pytest.mark.parametrize("softcap", [1e-42, 1e-35, 1e-6, 1e6, 1e29, 1e36, 3e38])
def test_caps_far_from_the_scores(io, cache, softcap):
    """A cap far below the scores leaves every position seen the same weight, one far above them the scores;
    a query of zeros has scores of 0 under any."""
    c = Chunk([100, 0], [70, 200], 8, 2, 64, io, cache, seed=17, softcap=softcap)
    c.q[7] = 0
    lse = torch.empty(c.q.shape[:2], device="cuda")
    out = c.attend(lse=lse)
    # (the cap's own error is relative to it, or to the score: 2^-21 of the smaller)
    c.softcap = 0.0 if softcap >= 1e6 else softcap
    if softcap < 1:
        c.check(out, lse)
    else:
        c.score_error = lambda q, k, e=c.score_error: e(q, k) + 2.0 ** -19 * c.scale * (
            q.abs() @ k.abs().T).amax(-1)
        c.check(out, lse)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
def test_one_long_context_and_many_requests(io, cache):
    c = Chunk([9000], [3], 16, 2, 128, io, cache)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.check(c.attend(lse=lse), lse)
    ref, tol = c.sums(lse)
    assert ((c.weigh(lse).double() - ref).abs() <= tol).all()
    r = np.random.default_rng(5)
    new = r.integers(0, 4, 700)
    c = Chunk(r.integers(0, 90, 700), new, 2, 1, 64, io, cache)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.check(c.attend(lse=lse), lse)
    ref, tol = c.sums(lse)
    assert ((c.weigh(lse).double() - ref).abs() <= tol).all()
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("new,group", [(32, 4), (9, 4), (13, 3)])
def test_sums_of_many_short_runs(cache, d, new, group):
    """A CTA's share is tens of items of one step each, some of one half and some of two, whose rings
    begin before the first copies land; every call gives the same bits."""
    r = np.random.default_rng(8)
    c = Chunk(r.integers(0, 1700, 96), [new] * 96, 6 * group, 6, d, "bf16", cache, seed=8)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.check(c.attend(lse=lse), lse)
    ref, tol = c.sums(lse)
    first = c.weigh(lse)
    assert ((first.double() - ref).abs() <= tol).all()
    spoil = torch.empty(1 << 26, device="cuda")
    for i in range(30):
        if i % 3 == 0:
            spoil.fill_(i)  # (K comes from memory again, in another order)
        assert torch.equal(c.weigh(lse), first)
    assert pkv.device_error() == 0


FEW = [  # new tokens of each request, h_q, h_kv: on the mean few rows to a KV head
    ([4] * 20, 8, 2), ([3] * 20, 8, 2), ([6, 7, 8, 5], 8, 2), ([8] * 9, 4, 1),
    ([1] * 64 + [300], 3, 1), ([1] * 64 + [40], 2, 2), ([1] * 30 + [300] + [1] * 34, 3, 3),
    ([0, 1, 2] * 20 + [77, 0], 4, 2),
]


@pytest.mark.parametrize("new,h_q,h_kv", FEW, ids=lambda x: str(x)[:30])
@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64), ("int8", 128),
                                     ("int8", 64)])
@pytest.mark.parametrize("form", [dict(), dict(window=37, sinks=5), dict(alibi=True, softcap=20.0)], ids=str)
def test_sums_of_few_rows_in_several_passes(cache, d, new, h_q, h_kv, form):
    """Calls of few rows on the mean, whose requests have one to many times the rows that are taken at
    once; with earlier sums, in place too, and the same bits every time."""
    past = np.random.default_rng(3).integers(0, 700, len(new))
    c = Chunk(past, new, h_q, h_kv, d, "bf16", cache, seed=13, pad=0, **form)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.attend(lse=lse)
    for last in (0, 40):
        add = torch.rand(len(new), h_kv, c.bt.shape[1] * 16, generator=gen(14), device="cuda") * 3
        ref, tol = c.sums(lse, last, add)
        w = c.weigh(lse, last_rows=last, add_to=add)
        assert ((w.double() - ref).abs() <= tol).all()
        assert torch.equal(c.weigh(lse, last_rows=last, add_to=add), w)
        assert c.weigh(lse, last_rows=last, add_to=add, out=add) is add
        assert torch.equal(add, w)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_small_sums_join_large_earlier_ones_once(cache):
    """900 rows of one request beside 200 decode steps add some 0.001 each to sums of 1000 before: every
    addition by itself would be half a step or less."""
    c = Chunk([700] + [20] * 200, [300] + [1] * 200, 3, 1, 64, "bf16", cache, seed=15, pad=0)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.attend(lse=lse)
    add = torch.full((201, 1, c.bt.shape[1] * 16), 1000.0, device="cuda")
    ref, tol = c.sums(lse, 0, add)
    assert ((c.weigh(lse, add_to=add).double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("io,cache", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")])
@pytest.mark.parametrize("new", [[300] + [1] * 64, [200, 100, 3]], ids=["few", "many"])
def test_infinite_earlier_sums_stay_that(io, cache, new):
    """Positions that a program pins, or gives up, by sums of either infinity."""
    c = Chunk([100] * len(new), new, 3, 1, 64, io, cache, seed=16, pad=0)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.attend(lse=lse)
    add = torch.zeros(len(new), 1, c.bt.shape[1] * 16, device="cuda")
    plain = c.weigh(lse, add_to=add)
    add[:, :, 3::7] = math.inf
    add[:, :, 5::11] = -math.inf
    w = c.weigh(lse, add_to=add)
    pinned = torch.isinf(add)
    assert torch.equal(w[pinned], add[pinned]) and torch.equal(w[~pinned], plain[~pinned])


@pytest.mark.parametrize("cache,d,new", [("bf16", 64, 20), ("fp8", 64, 20), ("fp8", 64, 2)])
def test_sums_of_long_contexts_behind_a_window(cache, d, new):
    """Most items have no rows: more of them in a share than the kernel keeps at a time."""
    c = Chunk([20000] * 6, [new] * 6, 16, 8, d, "bf16", cache, seed=9, window=40, sinks=3)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.check(c.attend(lse=lse), lse)
    ref, tol = c.sums(lse)
    for _ in range(5):
        out = torch.full((6, 8, c.bt.shape[1] * 16), 5.0, device="cuda")
        c.weigh(lse, out=out, add_to=None)
        for b in range(6):
            n = c.ctx[b]
            assert ((out[b, :, :n].double() - ref[b, :, :n]).abs() <= tol[b, :, :n]).all()
            assert (out[b, :, n:] == 5).all()
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("below", [10.0, 15.0, 24.6, 30.0])
@pytest.mark.parametrize("new,h_q", [(400, 128), (3, 8)])
def test_many_small_weights_beside_a_large_one(cache, below, new, h_q):
    """One position with 2^below times the weight of each of 131,072 others, whose values alone are not 0:
    together the small ones count, though each is near the end of the matrix type's range."""
    d, past = 64, 1 << 17
    ctx = past + new
    pages = -(-ctx // 16)
    one = {"bf16": 1.0, "fp8": 0x38, "int8": 1}[cache]  # (0x38: the code of 1)
    dtype = {"bf16": torch.bfloat16, "fp8": torch.uint8, "int8": torch.int8}[cache]
    k, v = (torch.zeros(pages, 1, 16, d, dtype=dtype, device="cuda") for _ in range(2))
    k[0, 0, 0, 0] = one
    v.fill_(one)
    v[0, 0, 0] = 0
    scales = dict(k_scales=torch.ones(1, device="cuda"), v_scales=torch.ones(1, device="cuda"))
    q = torch.zeros(new, h_q, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 16.0
    q[:, :, 1] = torch.arange(new, device="cuda")[:, None]  # (meets zeros)
    scale = below * math.log(2.0) / 16.0
    lse = torch.empty(new, h_q, device="cuda")
    out = pkv.chunk_attention(q, k, v, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                              torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, new], dtype=torch.int32, device="cuda"), scale, lse=lse,
                              **(scales if cache != "bf16" else {}))
    scale = torch.tensor(scale).item()  # (as the call took it: fp32)
    top = math.exp(torch.tensor(scale, dtype=torch.float32).double().item() * 16.0)
    n = torch.arange(past, past + new, dtype=torch.float64, device="cuda")[:, None, None]  # small ones
    ref = n / (n + top)
    # the large weight's score: its product with the scale and log2(e) and the exponential (4 U32 of the
    # score, 2^-21); a small weight: 2^-21; sums over tiles, one rounding or truncation (2 U32) each, and
    # 64 within them and over shares; a small weight's rounding to the matrix type: in f16 half a step,
    # 2^-25, of a value kept 2^7 times as large or more; the output's
    e = 4 * U32 * below + 2.0 ** -20 + 2 * (past // 128 + 64) * U32
    p = H["bf16"] if cache == "bf16" else H["f16"] + 2.0 ** (below - 32)
    tol = (2 * e + p) * ref + H["bf16"] * ref * (1 + p) + 1e-30
    assert ((out.double() - ref).abs() <= tol).all(), ((out.double() - ref).abs() / tol).max()
    want = torch.log(n + top).expand(new, h_q, 1)[..., 0]
    assert ((lse.double() - want).abs() <= 2 * e + 4 * U32 * want).all()
    assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache,d", [KINDS[i] for i in (0, 1, 2, 5, 6, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_values_and_keys_that_are_not_finite_reach_only_rows_that_see_them(io, cache, d, window, sinks):
    past, new = [40, 300], [200, 90]
    c = Chunk(past, new, 4, 1, d, io, cache, window=window, sinks=sinks)
    clean = c.attend()
    # a late value NaN, an earlier one infinite (8-bit floats have NaN alone), a key NaN
    spots = {0: (110, 230), 1: (310, 350)}
    for b, (k_pos, v_pos) in spots.items():
        for pool, pos, value in ((c.k_cache, k_pos, math.nan),
                                 (c.v_cache, v_pos, math.nan if cache == "fp8" else math.inf)):
            page = int(c.table[b, pos // 16])
            if cache == "fp8":
                pool.view(torch.uint8)[page, 0, pos % 16, 3] = 0x7f
            else:
                pool[page, 0, pos % 16, 3] = value
    out = c.attend()
    for b, (k_pos, v_pos) in spots.items():
        pq = torch.arange(past[b], past[b] + new[b], device="cuda")

        def sees(p):
            x = pq >= p
            return x & ((pq - p < window) | (p < sinks)) if window else x

        rows = slice(int(c.starts[b]), int(c.starts[b]) + new[b])
        got, was = out[rows], clean[rows]
        nan_rows = sees(k_pos)
        assert torch.isnan(got[nan_rows]).all()
        inf_rows = sees(v_pos) & ~nan_rows
        assert not torch.isfinite(got[inf_rows][:, :, 3]).any()
        others = [i for i in range(d) if i != 3]
        assert torch.equal(got[inf_rows][:, :, others], was[inf_rows][:, :, others])
        free = ~nan_rows & ~sees(v_pos)
        assert free.any() and torch.equal(got[free], was[free])
    assert pkv.device_error() == 0


def test_bad_pages_are_skipped_and_flagged():
    for io, cache in (("bf16", "bf16"), ("bf16", "int8"), ("f32", "f32")):
        c = Chunk([300, 20, 0], [40, 10, 12], 4, 2, 64, io, cache)
        c.table[0, 3], c.table[0, 18], c.table[2, 0] = -1, c.k_cache.shape[0], -7
        c.dev()
        lse = torch.empty(c.q.shape[:2], device="cuda")
        out = c.attend(lse=lse)
        assert pkv.device_error() == pkv.DEVERR_BAD_PAGE
        c.check(out, lse)
        assert not out[50:62].any() and torch.isinf(lse[50:62]).all()  # a request without a page
        w = c.weigh(lse)
        assert pkv.device_error() == pkv.DEVERR_BAD_PAGE
        ref, tol = c.sums(lse)
        assert ((w.double() - ref).abs() <= tol).all()


def test_bad_requests_are_left_out_and_flagged():
    for io in ("bf16", "f32"):
        c = Chunk([30, 20, 70, 10], [10, 12, 9, 30], 4, 2, 64, io, io)
        good = c.attend()
        lse = torch.empty(c.q.shape[:2], device="cuda")
        c.attend(lse=lse)
        sums = c.weigh(lse)
        width = c.bt.shape[1] * 16
        for what, bit in (("start", pkv.DEVERR_BAD_CHUNK), ("short", pkv.DEVERR_BAD_CHUNK),
                          ("long", pkv.DEVERR_BAD_PAGE)):
            qs, cl = c.qs.clone(), c.cl.clone()
            if what == "start":
                qs[2] = -5  # request 1 ends, request 2 begins outside
            elif what == "short":
                cl[1] = 11
            else:
                cl[1] = width + 1
            out = torch.full_like(c.q, 2.0)
            pkv.chunk_attention(c.q, c.k_cache, c.v_cache, c.bt, cl, qs, c.scale, out=out)
            assert pkv.device_error() == bit
            w = torch.full_like(sums, 2.0)
            pkv.chunk_weights(c.q, c.k_cache, c.bt, cl, qs, lse, c.scale, out=w)
            assert pkv.device_error() in (bit, pkv.DEVERR_BAD_CHUNK)
            left = (1, 2) if what == "start" else (1,)
            for b in range(4):
                rows = slice(int(c.starts[b]), int(c.starts[b + 1]))
                if b in left:
                    assert (out[rows] == 2).all() and (w[b] == 2).all()
                else:
                    assert torch.allclose(out[rows].float(), good[rows].float(), atol=0.02, rtol=0.02)
                    assert torch.allclose(w[b, :, :c.ctx[b]], sums[b, :, :c.ctx[b]], rtol=1e-4)
                    assert (w[b, :, c.ctx[b]:] == 2).all()


@pytest.mark.parametrize("io,cache,new", [("bf16", "bf16", 20), ("bf16", "fp8", 20), ("bf16", "fp8", 2),
                                          ("f32", "f32", 20)])
def test_rows_given_to_several_requests_leave_every_request_out(io, cache, new):
    """Starts that rise and fall: the work that the plan counts is bounded for rows that belong to one request
    each. A fall that gives no row twice leaves out its own request alone."""
    n = 40
    c = Chunk([900] * n, [new] * n, 4, 2, 64, io, cache)  # (a request could hold all rows)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.attend(lse=lse)
    sums = c.weigh(lse)
    for last, every in ((c.rows, True), (new, False)):
        c.qs = torch.tensor([0, last] * (n // 2) + [0], dtype=torch.int32, device="cuda")
        assert (last * (n // 2) > c.q.shape[0]) == every
        out, w = torch.full_like(c.q, 2.0), torch.full_like(sums, 2.0)
        c.attend(out=out)
        assert pkv.device_error() == pkv.DEVERR_BAD_CHUNK
        c.weigh(lse, out=w)
        assert pkv.device_error() == pkv.DEVERR_BAD_CHUNK
        assert (out[new:] == 2).all() and (w[1::2] == 2).all()
        assert (out[:new] == 2).all() == every and (w[::2, :, :900] == 2).all() == every


def test_released_pages_outside_the_window_are_not_read():
    for io, cache in (("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32")):
        c = Chunk([700], [50], 4, 2, 128, io, cache, window=100, sinks=20)
        lse = torch.empty(c.q.shape[:2], device="cuda")
        before = c.attend(lse=lse)
        w = c.weigh(lse)
        c.table[0, 2:37] = -1  # positions 32 .. 591; the first row's window begins at 601
        c.dev()
        assert torch.equal(c.attend(), before) and torch.equal(c.weigh(lse), w)
        assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache,d", [KINDS[i] for i in (0, 2, 6)])
def test_chunks_of_a_prompt_equal_the_whole(io, cache, d):
    """A prompt cut into chunks gives each row the same answer as at once, to rounding; its sums add
    up, in place too."""
    whole = Chunk([0], [700], 8, 2, d, io, cache, pad=0)
    lse = torch.empty(700, 8, device="cuda")
    out = whole.attend(lse=lse)
    sums = whole.weigh(lse)
    parts, acc = torch.empty_like(out), torch.zeros_like(sums)
    part_lse = torch.empty_like(lse)
    at = 0
    for n in (1, 130, 256, 313):
        cl = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        args = (whole.bt, cl, qs)
        q, o, l = (x[at:at + n].contiguous() for x in (whole.q, parts, part_lse))
        kw = dict(k_scales=whole.k_scales)
        pkv.chunk_attention(q, whole.k_cache, whole.v_cache, *args, whole.scale, out=o, lse=l,
                            v_scales=whole.v_scales, **kw)
        assert pkv.chunk_weights(q, whole.k_cache, *args, l, whole.scale, add_to=acc, out=acc,
                                 **kw) is acc
        parts[at:at + n], part_lse[at:at + n] = o, l
        at += n
    whole.check(parts, part_lse)
    ref, tol = whole.sums(lse)
    assert ((acc.double() - ref).abs() <= 2 * tol).all()


def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph():
    c = Chunk([3000, 10, 0], [70, 300, 1], 8, 2, 128, "bf16", "bf16")
    lse = torch.empty(c.q.shape[:2], device="cuda")
    out = c.attend(lse=lse)
    w = c.weigh(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l2 = torch.empty_like(lse)
    a = c.attend(lse=l2, stream=side)
    b = c.weigh(l2, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(b, w) and torch.equal(lse[:c.rows], l2[:c.rows])
    static, sums = torch.zeros_like(out), torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(out=static, lse=l2)
        c.weigh(l2, out=sums)
    for _ in range(2):
        l2.zero_(), static.zero_(), sums.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(static, out) and torch.equal(sums, w)


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("int8", 128)])
@pytest.mark.parametrize("form", [dict(window=1, sinks=4), dict(window=300, sinks=20), dict()])
def test_capped_scores_do_not_depend_on_what_is_not_seen(cache, d, form):
    """Pages that no row sees are not read: what memory held before has no say in the cap's rounding."""
    c = Chunk([4220, 1100, 2700], [130, 170, 5], 16, 1, d, "bf16", cache, seed=6, softcap=20.0, **form)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    out = c.attend(lse=lse)
    c.check(out, lse)
    w = c.weigh(lse)
    other = Chunk([3000, 900, 2000], [130, 170, 40], 16, 1, d, "bf16", cache, seed=7)
    for i in range(12):
        other.q.mul_(3.0 if i % 2 else 1 / 3.0)
        other.attend()  # (leaves other rows in shared memory)
        lse2 = torch.empty_like(lse)
        out2 = c.attend(lse=lse2)
        assert torch.equal(out2[:c.rows], out[:c.rows]) and torch.equal(lse2[:c.rows], lse[:c.rows])
        assert torch.equal(c.weigh(lse2), w)
    assert pkv.device_error() == 0


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_query_rows_of_others_take_no_part(cache, d, value):
    """Rows behind the last request, and a request's own, that are not finite: the others' results do not
    change by a bit (steps of sums read whole boxes of rows)."""
    c = Chunk([40, 300, 0, 1000], [20, 5, 33, 70], 8, 2, d, "bf16", cache, seed=4)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    out = c.attend(lse=lse)
    w = c.weigh(lse)
    c.q[c.rows:] = value
    c.q[20:25] = value  # request 1
    lse2 = torch.empty_like(lse)
    out2 = c.attend(lse=lse2)
    keep = [i for i in range(c.rows) if not 20 <= i < 25]
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[keep], lse[keep])
    w2 = c.weigh(lse2)
    assert torch.equal(w2[[0, 2, 3]], w[[0, 2, 3]])
    assert pkv.device_error() == 0


@pytest.mark.parametrize("io,cache,d", [("bf16", "bf16", 128), ("bf16", "bf16", 64), ("bf16", "fp8", 128),
                                        ("bf16", "int8", 64), ("f32", "f32", 64), ("f32", "int8", 128)])
@pytest.mark.parametrize("new", [[200, 90, 3], [1, 2, 2]], ids=["many", "few"])
@pytest.mark.parametrize("form", [dict(), dict(softcap=10.0), dict(window=33, sinks=4, alibi=True)], ids=str)
def test_sums_take_nothing_from_rows_that_saw_nothing_nor_for_what_is_not_seen(io, cache, d, new, form):
    """A row whose lse is -infinity gives nothing, whatever its queries hold; one whose lse is NaN gives NaN
    to the positions that it sees, and to no other."""
    c = Chunk([40, 300, 700], new, 8, 2, d, io, cache, seed=12, **form)
    lse = torch.empty(c.q.shape[:2], device="cuda")
    c.attend(lse=lse)
    none, nan = int(c.starts[1]) - 1, int(c.starts[2]) - 2  # the last row of request 0, one of request 1
    dropped = lse.clone()
    dropped[none], dropped[nan, 5] = -math.inf, -math.inf
    ref, tol = c.sums(dropped)
    assert ((c.weigh(dropped).double() - ref).abs() <= tol).all()
    clean = c.q.clone()
    for value in (math.nan, math.inf, -math.inf):
        c.q.copy_(clean)
        c.q[none] = value
        assert ((c.weigh(dropped).double() - ref).abs() <= tol).all(), value
    c.q[nan, 5] = math.nan
    poison = dropped.clone()
    poison[nan, 5] = math.nan
    w = c.weigh(poison)
    pos = torch.arange(w.shape[2], device="cuda")
    at = c.ctx[1] - 2
    seen = (pos <= at) & (pos < c.ctx[1])
    if c.window:
        seen &= (pos > at - c.window) | (pos < c.sinks)
    assert torch.isnan(w[1, 1, seen]).all()
    keep = torch.ones_like(w, dtype=torch.bool)
    keep[1, 1, seen] = False
    assert ((w.double() - ref).abs() <= tol)[keep].all()
    assert pkv.device_error() == 0


def test_two_calls_at_once_on_two_streams():
    calls = []
    for seed, cache, d in ((1, "bf16", 128), (2, "fp8", 64)):
        c = Chunk([100, 900, 0, 33], [300, 1, 200, 40], 8, 2, d, "bf16", cache, seed=seed)
        B, P = len(c.new), c.bt.shape[1]
        ws = [torch.empty(1 << 26, dtype=torch.uint8, device="cuda") for _ in range(2)]
        lse = torch.empty(c.q.shape[:2], device="cuda")
        out = torch.zeros_like(c.q)
        w = torch.zeros(B, 2, P * 16, device="cuda")

        def call(c=c, ws=ws, lse=lse, out=out, w=w):
            c.attend(out=out, lse=lse, workspace=ws[0])
            c.weigh(lse, out=w, workspace=ws[1])
        call()
        calls.append((call, out, lse, w, out.clone(), lse.clone(), w.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for call, out, lse, w, *_ in calls:
        for x in (out, lse, w):
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (call, *_) in zip(streams, calls):
            with torch.cuda.stream(st):
                call()
    torch.cuda.synchronize()
    for _, out, lse, w, *want in calls:
        n = sum((300, 1, 200, 40))
        assert torch.equal(out[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])
        assert torch.equal(w, want[2])
    assert pkv.device_error() == 0


def test_empty_calls():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.chunk_attention(q, pool, pool, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                              zero[:0], zero, 0.1)
    assert out.shape == q.shape
    # no new token: the sums are carried over
    bt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cl = torch.tensor([5], dtype=torch.int32, device="cuda")
    qs = torch.zeros(2, dtype=torch.int32, device="cuda")
    add = torch.rand(1, 2, 16, device="cuda")
    got = pkv.chunk_weights(q, pool, bt, cl, qs, torch.empty(0, 4, device="cuda"), 0.1, add_to=add,
                            out=torch.zeros_like(add))
    assert torch.equal(got[:, :, :5], add[:, :, :5]) and (got[:, :, 5:] == 0).all()
    new = pkv.chunk_weights(q, pool, bt, cl, qs, torch.empty(0, 4, device="cuda"), 0.1, add_to=add)
    assert torch.equal(new, add) and new.data_ptr() != add.data_ptr()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cache", ["fp8", "int8"])
def test_sums_without_rows_are_carried_over_without_scales(io, cache):
    """num_rows = 0: neither queries nor lse nor scales are needed, in the C call (the contexts are there)."""
    d, h_kv, width = 64, 2, 300
    pool = torch.zeros(3, h_kv, 16, d, dtype=torch.uint8, device="cuda")
    desc = pkv._Desc(3, 16, h_kv, d, pkv.FP8_E4M3 if cache == "fp8" else pkv.INT8)
    cl = torch.tensor([300, 0, 70], dtype=torch.int32, device="cuda")
    qs = torch.zeros(4, dtype=torch.int32, device="cuda")
    add = torch.rand(3, h_kv, width, device="cuda")
    out = torch.full_like(add, 7.0)
    code = pkv.F32 if io == "f32" else pkv.BF16
    need = pkv.chunk_weights_workspace_size(code, 0, 3, 4, h_kv, d, width)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    form = pkv._ScoreForm(0.1, 0.0, None, 0, 0)
    st = pkv.lib().pkv_chunk_weights(
        None, code, 0, 3, 4, pool.data_ptr(), desc, None, 1, cl.data_ptr(), qs.data_ptr(), form, None,
        None, 0, add.data_ptr(), out.data_ptr(), width, ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0 and pkv.device_error() == 0
    for b, n in enumerate((300, 0, 70)):
        assert torch.equal(out[b, :, :n], add[b, :, :n]) and (out[b, :, n:] == 7).all()


# ---- eviction ----------------------------------------------------------------------------------


def kept_positions(w, ctx, budget, recent, sinks):
    """The definition: positions always kept, then larger sums, then lower positions."""
    n = min(ctx, budget)
    always = np.zeros(ctx, bool)
    always[:sinks] = True
    always[max(0, ctx - recent):] = True
    return np.sort(np.lexsort((np.arange(ctx), -w.astype(np.float64), ~always))[:n])


SELECTS = [  # contexts, width, budget, recent, sinks
    ([1], 1, 1, 0, 0), ([0, 5, 16, 17], 20, 16, 0, 0), ([100, 33], 128, 32, 32, 0),
    ([1000, 999, 31, 2], 1024, 30, 10, 4), ([4096], 4096, 1, 0, 1), ([5000, 70000], 70001, 4097, 64, 4),
    ([300], 300, 299, 100, 50), ([513, 1025, 2049], 3000, 512, 0, 0), ([140000], 140000, 100, 7, 3),
]


@pytest.mark.parametrize("ctx,width,budget,recent,sinks", SELECTS)
@pytest.mark.parametrize("kind", ["spread", "ties", "same", "odd"])
def test_select_matches_a_sort(ctx, width, budget, recent, sinks, kind):
    g, h_kv = gen(9), 3
    w = torch.rand(len(ctx), h_kv, width, generator=g, device="cuda")
    if kind == "spread":
        w = torch.exp(20 * w - 15)
    elif kind == "ties":
        w = (w * 8).floor() / 8
    elif kind == "same":
        w = torch.zeros_like(w)
        w[:, 1] = -0.0
        w[:, 2, ::2] = -0.0
    else:  # negative, huge, infinite, tiny
        w = torch.where(w < 0.3, -w * 1e30, torch.where(w < 0.5, w * 1e-42, w))
        w[:, :, ::97] = math.inf
        w[:, 0, ::89] = -math.inf
    cl = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    kept, lens = pkv.evict_select(w, cl, budget, recent, sinks)
    assert lens.tolist() == [min(c, budget) for c in ctx]
    for b, c in enumerate(ctx):
        n = min(c, budget)
        for j in range(h_kv):
            want = kept_positions(w[b, j, :c].cpu().numpy(), c, budget, recent, sinks)
            assert np.array_equal(kept[b, j, :n].cpu().numpy(), want)
            assert not kept[b, j, n:].any()
    assert pkv.device_error() == 0


def test_select_puts_nan_above_everything_and_flags_a_long_request():
    w = torch.arange(64, dtype=torch.float32, device="cuda").repeat(2, 1, 1)
    w[0, 0, 5], w[0, 0, 9], w[0, 0, 20] = math.nan, math.inf, -math.nan
    cl = torch.tensor([64, 65], dtype=torch.int32, device="cuda")
    kept, lens = pkv.evict_select(w, cl, 4)
    assert kept[0, 0].tolist() == [5, 9, 20, 63] and lens.tolist() == [4, 0]
    assert not kept[1].any() and pkv.device_error() == pkv.DEVERR_BAD_CHUNK


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("f32", 64), ("fp8", 64), ("int8", 128)])
def test_move_copies_bits_and_leaves_the_rest(cache, d):
    c = Chunk([200, 37, 16, 5], [1, 1, 1, 0], 2, 2, d, "f32" if cache == "f32" else "bf16", cache, spare=9)
    budget = 24
    w = torch.rand(4, 2, 220, device="cuda")
    kept, lens = pkv.evict_select(w, c.cl, budget, 3, 2)
    nt = torch.from_numpy(c.spare_pages[:8].reshape(4, 2).astype(np.int32)).cuda()
    before = [raw(x).view(x.shape[0], 2, 16, -1).clone() for x in (c.k_cache, c.v_cache)]
    sums = torch.full((4, 2, 30), 5.0, device="cuda")
    pkv.evict_move(c.k_cache, c.v_cache, c.bt, kept, lens, nt, w, sums)
    assert pkv.device_error() == 0
    for x, old in zip((c.k_cache, c.v_cache), before):
        want = old.clone()
        for b in range(4):
            for j in range(2):
                for i in range(int(lens[b])):
                    p = int(kept[b, j, i])
                    want[int(nt[b, i // 16]), j, i % 16] = old[int(c.table[b, p // 16]), j, p % 16]
        assert torch.equal(raw(x).view_as(want), want)
    for b in range(4):
        n = int(lens[b])
        assert torch.equal(sums[b, :, :n], w[b].gather(1, kept[b, :, :n].long()))
        assert not sums[b, :, n:].any()


def test_move_skips_and_flags_what_is_not_there():
    c = Chunk([100, 50], [1, 1], 2, 1, 64, "bf16", "bf16", spare=9)
    kept = torch.arange(32, dtype=torch.int32, device="cuda").repeat(2, 1, 1)
    nt = torch.from_numpy(c.spare_pages[:4].reshape(2, 2).astype(np.int32)).cuda()
    lens = torch.tensor([32, 20], dtype=torch.int32, device="cuda")
    for what, bit in (("position", pkv.DEVERR_BAD_PAGE), ("source", pkv.DEVERR_BAD_PAGE),
                      ("target", pkv.DEVERR_BAD_PAGE), ("count", pkv.DEVERR_BAD_CHUNK),
                      ("negative", pkv.DEVERR_BAD_CHUNK)):
        k, t, new, n = kept.clone(), c.bt.clone(), nt.clone(), lens.clone()
        if what == "position":
            k[0, 0, 3] = t.shape[1] * 16
        elif what == "source":
            t[0, 0] = -1
        elif what == "target":
            new[0, 0] = c.k_cache.shape[0]
        else:
            n[0] = 33 if what == "count" else -1
        c.k_cache[nt.long()] = 0
        before = raw(c.k_cache).clone()
        pkv.evict_move(c.k_cache, c.v_cache, t, k, n, new)
        assert pkv.device_error() == bit
        rows = c.k_cache[nt[1].long()].reshape(32, 64)[:20]
        assert torch.equal(rows, c.k_cache[c.bt[1, :2].long()].reshape(32, 64)[:20])
        if what in ("count", "negative"):
            assert not raw(c.k_cache[nt[0].long()]).any()
        other = torch.ones(c.k_cache.shape[0], dtype=torch.bool, device="cuda")
        other[nt.flatten().long()] = False
        assert torch.equal(raw(c.k_cache).view(len(other), -1)[other], before.view(len(other), -1)[other])


def test_eviction_and_decode_sums_in_a_graph_and_on_two_streams():
    """Sums of a decode step, the choice and the move, captured once and replayed over other sums and over
    other lengths; and two such calls at the same time."""
    calls = []
    for seed, cache in ((21, "bf16"), (22, "fp8")):
        c = Chunk([300, 1000, 40], [1, 1, 1], 4, 2, 64, "bf16", cache, seed=seed, spare=12)
        lse = torch.empty(c.q.shape[:2], device="cuda")
        c.attend(lse=lse)
        w = torch.rand(3, 2, c.bt.shape[1] * 16, device="cuda")
        nt = torch.from_numpy(c.spare_pages[:12].reshape(3, 4).astype(np.int32)).cuda()
        kept = torch.zeros(3, 2, 64, dtype=torch.int32, device="cuda")
        lens = torch.zeros(3, dtype=torch.int32, device="cuda")
        sums, moved = torch.zeros_like(w), torch.zeros(3, 2, 70, device="cuda")

        def call(c=c, lse=lse, w=w, nt=nt, kept=kept, lens=lens, sums=sums, moved=moved):
            c.weigh(lse, add_to=w, out=sums)
            pkv.evict_select(sums, c.cl, 64, 8, 2, kept=kept, kept_lens=lens)
            pkv.evict_move(c.k_cache, c.v_cache, c.bt, kept, lens, nt, sums, moved)

        def wrong(c=c, nt=nt, kept=kept, lens=lens, sums=sums, moved=moved):
            for b, n in enumerate(c.cl.tolist()):
                m = min(n, 64)
                assert int(lens[b]) == m
                for j in range(2):
                    at = kept_positions(sums[b, j, :n].cpu().numpy(), n, 64, 8, 2)
                    if not np.array_equal(kept[b, j, :m].cpu().numpy(), at):
                        return "kept"
                    at = torch.from_numpy(at).cuda()
                    if not torch.equal(moved[b, j, :m], sums[b, j, at]) or moved[b, j, m:].any():
                        return "sums"
                    for pool in (c.k_cache, c.v_cache):
                        x = pool.view(torch.uint8) if pool.element_size() == 1 else pool
                        new = x[nt[b].long(), j].reshape(-1, 64)[:m]
                        if not torch.equal(raw(new), raw(x[c.bt[b].long()[at // 16], j, at % 16])):
                            return "rows"
            return None
        calls.append((c, w, call, wrong, kept, lens, moved))
    for c, w, call, wrong, kept, lens, moved in calls:
        call()
        assert wrong() is None
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for i in range(3):
            w.copy_(torch.rand_like(w))
            if i == 2:
                c.cl.copy_(torch.tensor([200, 3, 30], dtype=torch.int32))
            for x in (kept, lens, moved):
                x.fill_(-1)
            graph.replay()
            torch.cuda.synchronize()
            assert wrong() is None
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (_, _, call, *_) in zip(streams, calls):
            with torch.cuda.stream(st):
                call()
    torch.cuda.synchronize()
    assert [wrong() for _, _, _, wrong, *_ in calls] == [None, None]
    assert pkv.device_error() == 0


# ---- as they are used together -------------------------------------------------------------------


@pytest.mark.parametrize("cache_type", ["bf16", "fp8"])
def test_prompts_in_chunks_then_eviction_then_decoding(cache_type):
    """Two prompts (one forked) go into the cache in chunks, their last rows' weights decide what stays,
    and decoding over the cut cache equals 64-bit attention over the kept rows."""
    g = gen(11)
    h_q, h_kv, d, budget, recent = 8, 2, 128, 100, 20
    scales = {}
    if cache_type == "fp8":
        scales = dict(k_scales=torch.full((h_kv,), 0.02, device="cuda"),
                      v_scales=torch.full((h_kv,), 0.015, device="cuda"))
    cache = PagedKVCache(100, h_kv, d, DT[cache_type], **scales)
    table = pkv.rope_table(2000, d)
    rids, lens = [0, 1], [333, 210]
    for rid in rids:
        cache.add_request(rid)
    done = [0, 0]
    q = lse = qs = None
    while any(done[i] < lens[i] for i in range(2)):
        n = [min(128, lens[i] - done[i]) for i in range(2)]
        slots = cache.reserve(rids, n)
        rows = sum(n)
        qkv = randn(g, rows, (h_q + 2 * h_kv) * d, dtype=torch.bfloat16)
        a, b, c = (x.view(rows, -1, d) for x in qkv.split([h_q * d, h_kv * d, h_kv * d], -1))
        pos = torch.cat([torch.arange(done[i], done[i] + n[i]) for i in range(2)]).int().cuda()
        q = cache.write_qkv(slots, a, b, c, pos, table)
        bt = torch.from_numpy(cache.block_table_array(rids)).cuda()
        cl = torch.from_numpy(cache.context_lens_array(rids)).cuda()
        qs = torch.tensor([0, n[0], rows], dtype=torch.int32, device="cuda")
        lse = torch.empty(rows, h_q, device="cuda")
        out = cache.attend_chunk(q, bt, cl, qs, d ** -0.5, lse=lse)
        assert torch.isfinite(out).all()
        done = [x + y for x, y in zip(done, n)]
    # (the second prompt ended in an earlier chunk: its last call had no row of it)
    w = cache.chunk_weights(q, bt, cl, qs, lse, d ** -0.5, last_rows=16, width=400)
    w[1] = torch.rand(h_kv, 400, generator=g, device="cuda")
    cache.fork(0, 7)
    held = {rid: cache.pages[rid] for rid in (0, 7)}
    free = cache.allocator.num_free()

    def rows_of(rid, j):
        pages = torch.tensor(cache.pages[rid], device="cuda")
        out = []
        for pool, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            x = pool if s is None else pool.view(torch.float8_e4m3fn)
            x = x.view(torch.uint8)[pages].view(x.dtype) if s is not None else x[pages]
            x = x[:, j].double().reshape(-1, d)[:cache.lens[rid]]
            out.append(x if s is None else x * s[j].double())
        return out

    before = {(rid, j): rows_of(rid, j) for rid in (0, 1) for j in range(h_kv)}
    new_w = cache.evict(rids, w, budget, recent=recent, sink_tokens=4)
    torch.cuda.synchronize()
    assert [cache.lens[r] for r in (0, 1, 7)] == [budget, budget, 333]
    assert cache.pages[7] == held[7]  # the fork keeps its rows
    # seven new pages each; the forked request's old ones stay with the fork
    assert cache.allocator.num_free() == free - 2 * 7 + (-(-210 // 16))
    for i, rid in enumerate(rids):
        for j in range(h_kv):
            at = torch.from_numpy(kept_positions(w[i, j, :lens[i]].cpu().numpy(), lens[i], budget,
                                                 recent, 4)).cuda()
            for new, old in zip(rows_of(rid, j), before[rid, j]):
                assert torch.equal(new, old[at])
            assert torch.equal(new_w[i, j, :budget], w[i, j, at]) and not new_w[i, j, budget:].any()
    for j in range(h_kv):
        assert all(torch.equal(x, y) for x, y in zip(rows_of(7, j), before[0, j]))
    # decoding goes on over the cut caches: one token each, in both of the framework's ways
    for step in range(3):
        slots = cache.reserve(rids, [1, 1])
        k1, v1 = (randn(g, 2, h_kv, d, dtype=torch.bfloat16) for _ in range(2))
        cache.write(slots, k1, v1)
        bt = torch.from_numpy(cache.block_table_array(rids)).cuda()
        cl = torch.from_numpy(cache.context_lens_array(rids)).cuda()
        q1 = randn(g, 2, h_q, d, dtype=torch.bfloat16)
        qs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        lse = torch.empty(2, h_q, device="cuda")
        got = cache.attend_chunk(q1, bt, cl, qs, d ** -0.5, lse=lse)
        same = pkv.paged_decode_attention(q1, cache.k, cache.v, bt, cl, d ** -0.5,
                                          k_scales=cache.k_scales, v_scales=cache.v_scales)
        cache.chunk_weights(q1, bt, cl, qs, lse, d ** -0.5, add_to=new_w, out=new_w)
        for i, rid in enumerate(rids):
            for j in range(h_kv):
                k, v = rows_of(rid, j)
                s = q1[i, 4 * j:4 * j + 4].double() @ k.T * d ** -0.5
                p = torch.softmax(s, -1)
                ref, size = p @ v, p @ v.abs()
                tol = (2 * H["bf16"] + 1e-5) * size + H["bf16"] * ref.abs()
                for x in (got, same):
                    assert ((x[i, 4 * j:4 * j + 4].double() - ref).abs() <= tol).all()
                assert abs(new_w[i, j, budget + step].item() - p[:, -1].sum().item()) < 1e-5
    assert pkv.device_error() == 0


def test_evict_leaves_short_requests_and_changes_nothing_when_pages_run_out():
    cache = PagedKVCache(20, 1, 64, torch.bfloat16)
    for rid, n in ((3, 100), (4, 20), (5, 90)):
        cache.add_request(rid)
        slots = cache.reserve([rid], [n])
        cache.write(slots, *(torch.randn(n, 1, 64, device="cuda").bfloat16() for _ in range(2)))
    w = torch.rand(3, 1, 128, device="cuda")
    state = {r: (cache.pages[r], cache.lens[r]) for r in (3, 4, 5)}
    with pytest.raises(pkv.PkvError):  # 15 of 20 pages are in use; ten are asked for
        cache.evict([3, 4, 5], w, 70)
    assert {r: (cache.pages[r], cache.lens[r]) for r in (3, 4, 5)} == state
    assert cache.allocator.num_free() == 5
    out = cache.evict([3, 4, 5], w, 32)
    assert [cache.lens[r] for r in (3, 4, 5)] == [32, 20, 32] and cache.pages[4] == state[4][0]
    assert torch.equal(out[1], w[1]) and cache.allocator.num_free() == 20 - 2 - 2 - 2
    assert torch.equal(cache.evict([4], w[1:2], 32), w[1:2])
    for bad in (dict(budget=0), dict(budget=10, recent=8, sink_tokens=3), dict(budget=10, recent=-1)):
        with pytest.raises(pkv.PkvError):
            cache.evict([3], w[:1], **bad)
    for rids, x in (([3, 3], w[:2]), ([3], w), ([3], w[:1, :, :16]), ([3], w[:1].double())):
        with pytest.raises(pkv.PkvError):
            cache.evict(rids, x, 8)
    with pytest.raises(pkv.PkvError):
        cache.evict([99], w[:1], 8)
