"""Host side of the operators on chunks of new tokens and of the eviction: refusals, found before
anything is launched, and workspace sizes. No GPU."""
import ctypes

import pytest

import paged_kv_cache_271_gb300 as pkv
from tests.test_tree_ops_host import ODD, P, call, desc

EINVAL, ESHAPE, EDTYPE, EALIGN = -1, -2, -3, -4
F32, BF16, FP8, INT8 = pkv.F32, pkv.BF16, pkv.FP8_E4M3, pkv.INT8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_271_gb300 import build
    build.build()


def form(scale=0.1, softcap=0.0, slopes=None, window=0, sinks=0):
    return ctypes.byref(pkv._ScoreForm(scale, softcap, slopes, window, sinks))


NAN, INF = float("nan"), float("inf")
CHUNK = dict(q=P, dtype=BF16, rows=40, batch=2, h_q=8, k_cache=P, v_cache=P, desc=desc(), tables=P,
             max_pages=4, ctx=P, starts=P, form=form(), k_scales=None, v_scales=None, out=P,
             lse=None, ws=P, ws_bytes=1 << 40, stream=None)
SHARED = [  # what both chunk calls refuse
    (dict(rows=-1), EINVAL), (dict(batch=-1), EINVAL), (dict(h_q=0), EINVAL),
    (dict(max_pages=0), EINVAL), (dict(h_q=7), ESHAPE), (dict(h_q=2 * 129), ESHAPE),
    (dict(batch=65536), ESHAPE), (dict(max_pages=(1 << 27) - 15), ESHAPE),
    (dict(rows=1 << 28), ESHAPE), (dict(dtype=FP8), EDTYPE), (dict(dtype=F32), EDTYPE),
    (dict(desc=desc(F32)), EDTYPE), (dict(desc=desc(d=96)), ESHAPE),
    (dict(desc=desc(page_size=8)), EINVAL), (dict(desc=desc(FP8)), EINVAL),
    (dict(desc=desc(pages=(1 << 26))), ESHAPE), (dict(form=None), EINVAL),
    (dict(form=form(scale=0.0)), EINVAL), (dict(form=form(scale=INF)), EINVAL),
    (dict(form=form(scale=NAN)), EINVAL), (dict(form=form(softcap=-1.0)), EINVAL),
    (dict(form=form(softcap=NAN)), EINVAL), (dict(form=form(softcap=INF)), EINVAL),
    (dict(form=form(scale=1e38)), EINVAL), (dict(form=form(scale=1e37, softcap=1.0)), EINVAL),
    (dict(form=form(window=-1)), EINVAL), (dict(form=form(window=5, sinks=-1)), EINVAL),
    (dict(form=form(sinks=1)), EINVAL), (dict(q=None), EINVAL), (dict(k_cache=None), EINVAL),
    (dict(tables=None), EINVAL), (dict(ctx=None), EINVAL), (dict(starts=None), EINVAL),
    (dict(q=ODD), EALIGN), (dict(k_cache=ODD), EALIGN), (dict(ws=None), EINVAL),
    (dict(ws_bytes=64), EINVAL), (dict(ws=ODD), EALIGN)]


@pytest.mark.parametrize("changed,code", SHARED + [
    (dict(v_cache=None), EINVAL), (dict(out=None), EINVAL), (dict(out=ODD), EALIGN),
    (dict(v_cache=ODD), EALIGN), (dict(desc=desc(FP8), k_scales=P), EINVAL),
    (dict(rows=1 << 25, max_pages=(1 << 27) - 16), ESHAPE)], ids=str)
def test_chunk_attention_refusals(changed, code):
    st, msg = call("pkv_chunk_attention", CHUNK, **changed)
    assert st == code and msg


WEIGHTS = dict(q=P, dtype=BF16, rows=40, batch=2, h_q=8, k_cache=P, desc=desc(), tables=P,
               max_pages=4, ctx=P, starts=P, form=form(), k_scales=None, lse=P, last_rows=0,
               add_to=None, out=P, width=64, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("changed,code", SHARED + [
    (dict(lse=None), EINVAL), (dict(out=None), EINVAL), (dict(width=-1), EINVAL),
    (dict(last_rows=-1), EINVAL), (dict(width=1 << 31), ESHAPE),
    (dict(rows=1 << 25, width=1 << 30), ESHAPE)], ids=str)
def test_chunk_weights_refusals(changed, code):
    st, msg = call("pkv_chunk_weights", WEIGHTS, **changed)
    assert st == code and msg


SELECT = dict(weights=P, width=64, ctx=P, batch=2, h_kv=2, budget=16, recent=4, sinks=2, kept=P,
              kept_lens=ctypes.c_void_p(8192), stream=None)


@pytest.mark.parametrize("changed,code", [
    (dict(batch=-1), EINVAL), (dict(h_kv=0), EINVAL), (dict(width=-1), EINVAL),
    (dict(budget=0), EINVAL), (dict(recent=-1), EINVAL), (dict(sinks=-1), EINVAL),
    (dict(recent=15), EINVAL), (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), EINVAL),
    (dict(batch=65536), ESHAPE), (dict(h_kv=65536), ESHAPE), (dict(width=1 << 31), ESHAPE),
    (dict(weights=None), EINVAL), (dict(ctx=None), EINVAL), (dict(kept=None), EINVAL),
    (dict(kept_lens=None), EINVAL), (dict(kept_lens=P), EINVAL)], ids=str)
def test_evict_select_refusals(changed, code):
    st, msg = call("pkv_evict_select", SELECT, **changed)
    assert st == code and msg


MOVE = dict(k_cache=P, v_cache=P, desc=desc(), tables=P, max_pages=4, kept=P, kept_lens=P, batch=2,
            budget=16, new_tables=P, new_pages=1, weights=P, width=64,
            new_weights=ctypes.c_void_p(8192), new_width=64, stream=None)


@pytest.mark.parametrize("changed,code", [
    (dict(batch=-1), EINVAL), (dict(budget=0), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(new_pages=0), EINVAL), (dict(width=-1), EINVAL), (dict(new_width=-1), EINVAL),
    (dict(batch=65536), ESHAPE), (dict(k_cache=None), EINVAL), (dict(v_cache=None), EINVAL),
    (dict(tables=None), EINVAL), (dict(kept=None), EINVAL), (dict(kept_lens=None), EINVAL),
    (dict(new_tables=None), EINVAL), (dict(new_weights=None), EINVAL), (dict(new_weights=P), EINVAL),
    (dict(k_cache=ODD), EALIGN), (dict(v_cache=ODD), EALIGN),
    (dict(desc=desc(page_size=32)), EINVAL)], ids=str)
def test_evict_move_refusals(changed, code):
    st, msg = call("pkv_evict_move", MOVE, **changed)
    assert st == code and msg


def test_empty_calls_launch_nothing():
    none = dict(q=None, k_cache=None, tables=None, ctx=None, starts=None, out=None, ws=None, ws_bytes=0)
    assert call("pkv_chunk_attention", CHUNK, batch=0, v_cache=None, **none)[0] == 0
    assert call("pkv_chunk_attention", CHUNK, rows=0, **{**none, "ctx": P, "starts": P})[0] == 0
    assert call("pkv_chunk_weights", WEIGHTS, batch=0, lse=None, **none)[0] == 0
    assert call("pkv_evict_select", SELECT, batch=0, weights=None, ctx=None, kept=None,
                kept_lens=None)[0] == 0
    assert call("pkv_evict_move", MOVE, batch=0, k_cache=None, v_cache=None, tables=None)[0] == 0


def test_workspace_sizes():
    size = pkv.chunk_workspace_size
    assert size(BF16, BF16, 0, 1, 8, 2, 128, 10) == 0 and size(BF16, BF16, 5, 0, 8, 2, 128, 10) == 0
    small, large = (size(BF16, BF16, n, 4, 32, 8, 128, 512) for n in (4, 4096))
    assert 0 < small <= large
    # no more than two partials of 256 rows for each of 152 CTAs, their (max, sum) and records
    assert large <= 152 * (2 * 256 * (128 + 2) * 4 + 16) + 1024
    assert size(F32, F32, 4096, 4, 32, 8, 64, 512) > 0
    w = pkv.chunk_weights_workspace_size
    assert w(BF16, 5, 0, 8, 2, 128, 100) == 0
    assert 0 < w(BF16, 0, 1, 8, 2, 128, 100) <= w(BF16, 4096, 4, 8, 2, 128, 8192)


def test_shared_arrays_read_in_wider_words_say_their_alignment():
    """A shared array of scalars is aligned to its element; where a kernel reads it in words of 16 bytes, its
    declaration has to ask for them (the order of a block's variables is the compiler's)."""
    import glob
    import os
    import re
    wide = r"reinterpret_cast<(?:const )?(?:u?int4|float4|ulonglong2)\s*\*>\(([^;]*?)\)"
    looked = 0
    for path in glob.glob(os.path.join(os.path.dirname(pkv.__file__), "csrc", "*.cu*")):
        text = open(path).read()
        for line in re.findall(r"^\s*(?:static )?__shared__ [^;]*;", text, re.M):
            kind = re.match(r"\s*__shared__\s+(__align__\(16\)|alignas\(16\))?\s*(\w+)\s+(\w+)\[", line)
            if not kind or kind[2] not in ("int", "float", "uint32_t", "uint8_t", "int32_t"):
                continue
            reads = [r for r in re.findall(wide, text) if re.search(r"\b%s\b" % kind[3], r)]
            looked += len(reads)
            assert kind[1] or not reads, (os.path.basename(path), line.strip(), reads)
    assert looked >= 1


def test_numbers_beyond_32_bits_are_refused():
    """ctypes would cut them to others without a word: a window of 2^32 + 5 to one of 5."""
    import torch
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32)
    args = (ints(0)[None], ints(5), ints(0, 2))
    big = 2 ** 32 + 5
    for kw in (dict(window=big), dict(window=8, sink_tokens=big), dict(window=-big)):
        with pytest.raises(pkv.PkvError, match="32 bits"):
            pkv.chunk_attention(q, pool, pool, *args, 0.1, **kw)
        with pytest.raises(pkv.PkvError, match="32 bits"):
            pkv.chunk_weights(q, pool, *args, torch.zeros(2, 2), 0.1, **kw)
    with pytest.raises(pkv.PkvError, match="32 bits"):
        pkv.chunk_weights(q, pool, *args, torch.zeros(2, 2), 0.1, last_rows=big)
    w = torch.zeros(1, 1, 16)
    for kw in (dict(budget=big), dict(budget=8, recent=big), dict(budget=8, sink_tokens=big)):
        with pytest.raises(pkv.PkvError, match="32 bits"):
            pkv.evict_select(w, ints(5), **kw)
