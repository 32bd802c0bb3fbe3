"""Host side of the speculative-decoding operators: refusals (found before anything is launched),
draft-tree masks, and truncating requests. No GPU."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_271_gb300 as pkv

EINVAL, ESHAPE, EDTYPE, EALIGN = -1, -2, -3, -4
F32, BF16, FP8, INT8 = pkv.F32, pkv.BF16, pkv.FP8_E4M3, pkv.INT8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_271_gb300 import build
    build.build()


P = ctypes.c_void_p(4096)    # an aligned address nothing may touch
ODD = ctypes.c_void_p(4100)


def desc(cache=BF16, h_kv=2, d=128, pages=8, page_size=16):
    return ctypes.byref(pkv._Desc(pages, page_size, h_kv, d, cache))


def call(fn, args, **changed):
    assert set(changed) <= set(args)
    args = {**args, **changed}
    st = getattr(pkv.lib(), fn)(*args.values())
    return st, pkv.lib().pkv_last_error().decode()


APPEND = dict(q=P, q_stride=1024, k=P, k_stride=256, v=P, v_stride=256, dtype=BF16, n=4, h_q=8,
              q_weight=P, k_weight=P, eps=1e-6, cos_sin=P, max_positions=64, rot_dim=128,
              interleaved=0, positions=P, slots=P, q_out=P, q_out_stride=1024, k_cache=P,
              v_cache=P, desc=desc(), k_scales=None, v_scales=None, stream=None)


@pytest.mark.parametrize("changed,code", [
    (dict(n=-1), EINVAL), (dict(h_q=0), EINVAL), (dict(q=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(q_out=None), EINVAL), (dict(v_cache=None), EINVAL), (dict(dtype=FP8), EDTYPE),
    (dict(dtype=F32), EDTYPE), (dict(desc=desc(FP8)), EINVAL), (dict(desc=desc(d=96)), ESHAPE),
    (dict(desc=desc(page_size=8)), EINVAL), (dict(rot_dim=120), ESHAPE),
    (dict(rot_dim=144), ESHAPE), (dict(rot_dim=-16), ESHAPE), (dict(cos_sin=None), EINVAL),
    (dict(positions=None), EINVAL), (dict(max_positions=0), EINVAL), (dict(interleaved=2), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(q_stride=1023), ESHAPE), (dict(k_stride=128), ESHAPE), (dict(q_out_stride=8), ESHAPE),
    (dict(q_stride=1028), EALIGN), (dict(v=ODD), EALIGN), (dict(q_weight=ODD), EALIGN),
    (dict(cos_sin=ODD), EALIGN)])
def test_append_refusals(changed, code):
    st, msg = call("pkv_qk_norm_rope_append", APPEND, **changed)
    assert st == code and msg


TREE = dict(q=P, dtype=BF16, batch=2, nodes=5, h_q=8, k_cache=P, v_cache=P, desc=desc(), tables=P,
            max_pages=4, ctx=P, tree_lens=P, mask=P, mask_stride=5, scale=0.1, k_scales=None,
            v_scales=None, out=P, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("changed,code", [
    (dict(batch=-1), EINVAL), (dict(nodes=-1), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(max_pages=1 << 27), ESHAPE), (dict(h_q=7), ESHAPE), (dict(nodes=257), ESHAPE),
    (dict(h_q=258), ESHAPE), (dict(batch=65536), ESHAPE), (dict(dtype=F32), EDTYPE),
    (dict(dtype=INT8), EDTYPE), (dict(desc=desc(F32)), EDTYPE), (dict(desc=desc(FP8)), EINVAL),
    (dict(q=None), EINVAL), (dict(ctx=None), EINVAL), (dict(out=None), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(mask_stride=4), ESHAPE), (dict(mask=ODD), EALIGN),
    (dict(out=ODD), EALIGN), (dict(ws=None), EINVAL), (dict(ws_bytes=16), EINVAL),
    (dict(ws=ODD), EALIGN), (dict(desc=desc(h_kv=1, pages=1 << 27)), ESHAPE),  # 2^31 rows
    (dict(batch=60000, max_pages=1 << 20), ESHAPE)])  # 2^30 half tiles
def test_tree_attention_refusals(changed, code):
    st, msg = call("pkv_tree_decode_attention", TREE, **changed)
    assert st == code and msg


COMMIT = dict(k_cache=P, v_cache=P, desc=desc(), tables=P, max_pages=4, ctx=ctypes.c_void_p(64),
              tree_lens=ctypes.c_void_p(128), path=ctypes.c_void_p(192),
              path_lens=ctypes.c_void_p(256), batch=2, max_path=3, new_lens=P, stream=None)


@pytest.mark.parametrize("changed,code", [
    (dict(batch=-1), EINVAL), (dict(max_path=-1), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(k_cache=None), EINVAL), (dict(tree_lens=None), EINVAL), (dict(path=None), EINVAL),
    (dict(path_lens=None), EINVAL), (dict(new_lens=ctypes.c_void_p(64)), EINVAL),
    (dict(new_lens=ctypes.c_void_p(192)), EINVAL), (dict(v_cache=ODD), EALIGN),
    (dict(desc=desc(d=32)), ESHAPE)])
def test_commit_refusals(changed, code):
    st, msg = call("pkv_tree_commit", COMMIT, **changed)
    assert st == code and msg


def test_empty_calls_take_null_pointers():
    assert call("pkv_qk_norm_rope_append", APPEND, n=0, q=None, k=None, v=None, slots=None)[0] == 0
    assert call("pkv_tree_decode_attention", TREE, batch=0, q=None, out=None, ws=None)[0] == 0
    assert call("pkv_tree_decode_attention", TREE, nodes=0, q=None, out=None, ws=None)[0] == 0
    assert call("pkv_tree_commit", COMMIT, batch=0, ctx=None, path=None, new_lens=None)[0] == 0


@pytest.mark.parametrize("q,cache,d", [(BF16, BF16, 128), (BF16, FP8, 128), (F32, F32, 64),
                                       (BF16, INT8, 64)])
def test_workspace_size_is_bounded_by_the_grid_and_zero_for_empty_calls(q, cache, d):
    size = lambda b, t, pages: pkv.tree_decode_workspace_size(q, cache, b, t, 32, 8, d, pages)
    assert size(0, 8, 4) == size(4, 0, 4) == 0
    assert 0 < size(1, 1, 1) <= size(64, 64, 256) == size(64, 256, 4096) < 1 << 28


def test_masks_and_depths_of_a_tree():
    masks, depths = pkv.tree_masks([-1, 0, 0, 1, 3, -1])
    assert masks.shape == (1, 6, 1) and masks.dtype == np.int64
    assert masks[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b11011, 0b100000]
    assert depths[0].tolist() == [0, 1, 1, 2, 3, 0]


def test_masks_cross_words():
    t = 200
    masks, depths = pkv.tree_masks(np.arange(-1, t - 1))  # a chain
    bits = np.unpackbits(masks[0].view(np.uint8), axis=-1, bitorder="little")
    assert masks.shape == (1, t, 4)
    assert (bits == np.pad(np.tril(np.ones((t, t), int)), ((0, 0), (0, 56)))).all()
    assert depths[0].tolist() == list(range(t))


@pytest.mark.parametrize("parents", [[0], [-1, 1], [-1, 2, 0], [-2], [-1, 0, 3]])
def test_masks_refuse_a_parent_that_is_no_earlier_node(parents):
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks(parents)


def test_masks_refuse_wide_trees():
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks(np.full((1, 257), -1))
    assert pkv.tree_masks(np.zeros((0, 4)))[0].shape == (0, 4, 1)


# ---- truncate --------------------------------------------------------------------------------


def table(pages=16):
    a = pkv.PageAllocator(pages)
    return a, pkv.SeqTable(a)


@pytest.mark.parametrize("new,kept", [(40, 3), (33, 3), (32, 2), (31, 2), (17, 2), (16, 1), (1, 1),
                                      (0, 0)])
def test_truncate_returns_whole_pages(new, kept):
    a, t = table()
    t.add(5)
    t.reserve([5], [40])
    row = t.pages(5)
    t.truncate([5], [new])
    assert t.length(5) == new and t.pages(5) == row[:kept] and a.num_free() == 16 - kept
    slots, _ = t.reserve([5], [41 - new])  # grows again from there
    assert t.length(5) == 41 and len(t.pages(5)) == 3
    assert slots[0] == t.pages(5)[new // 16] * 16 + new % 16


def test_truncate_keeps_a_fork_s_pages():
    a, t = table()
    t.add(1)
    t.reserve([1], [48])
    row = t.pages(1)
    t.fork([1], [2])
    t.truncate([1], [20])
    assert t.pages(2) == row and t.length(2) == 48 and a.num_free() == 13
    assert [a.refcount(p) for p in row] == [2, 2, 1]
    _, copies = t.reserve([1], [1])  # its partly filled page is shared: copied first
    assert copies and copies[0][0] == row[1] and t.pages(1)[1] != row[1]


def test_truncate_skips_released_pages():
    a, t = table()
    t.add(1)
    t.reserve([1], [64])
    assert t.release_outside_window(1, 10) == 3
    t.truncate([1], [16])
    assert t.pages(1) == [-1] and a.num_free() == 16


def test_truncate_refuses_and_changes_nothing():
    a, t = table()
    t.add(1)
    t.add(2)
    t.reserve([1, 2], [20, 20])
    for rids, lens in (([1, 3], [4, 4]), ([1, 1], [4, 4]), ([1, 2], [4, 21]), ([2, 1], [4, -1])):
        with pytest.raises(pkv.PkvError):
            t.truncate(rids, lens)
    with pytest.raises(pkv.PkvError):
        t.truncate([1], [1, 2])
    assert t.length(1) == t.length(2) == 20 and a.num_free() == 12


def test_truncate_and_the_incremental_export():
    _, t = table(32)
    t.add(1)
    t.add(2)
    t.reserve([1, 2], [60, 30])
    bt, cl = np.full((2, 6), 77, np.int32), np.zeros(2, np.int32)
    t.step([], [], [], [1, 2], 6, bt, cl, incremental=True)
    t.truncate([1], [10])
    t.step([], [], [], [1, 2], 6, bt, cl, incremental=True)
    assert cl.tolist() == [11, 32]
    for i, rid in enumerate((1, 2)):
        row = t.pages(rid)
        assert bt[i].tolist() == row + [0] * (6 - len(row))
