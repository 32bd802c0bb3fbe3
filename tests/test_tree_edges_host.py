"""Host side of the speculative-decoding calls in their less usual forms. No GPU."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_271_gb300 as pkv
from paged_kv_cache_271_gb300 import cache as cache_module
from paged_kv_cache_271_gb300.cache import PagedKVCache
from tests.test_tree_ops_host import APPEND, BF16, ESHAPE, F32, INT8, TREE, call, desc


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_271_gb300 import build
    build.build()


# ---- host slots on a stream of the caller's ------------------------------------------------------


class FakeStream:
    """Stands for torch.cuda.Stream where there is no GPU."""

    def __init__(self, handle=77, device=None):
        self.cuda_stream = handle


@pytest.fixture
def recorded(monkeypatch):
    """[(address, stream handle)] of the tensors whose use on a stream was recorded, and the slots
    that reached the operator, kept alive: (records, slots)."""
    records, slots = [], []
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: records.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(cache_module, "qk_norm_rope_append",
                        lambda q, k, v, positions, slot_mapping, *a, **kw: slots.append(slot_mapping))
    monkeypatch.setattr(cache_module, "kv_append",
                        lambda k, v, slot_mapping, *a, **kw: slots.append(slot_mapping))
    return records, slots


@pytest.mark.parametrize("stream", [FakeStream(), 77])
def test_write_qkv_keeps_host_slots_until_the_stream_is_done(recorded, stream):
    """The device copy of host slots is the call's own: it must outlive the work on the stream it
    was given."""
    records, slots = recorded
    c = PagedKVCache(2, 1, 64, torch.float32, device="cpu")
    c.write_qkv(np.array([3, 4]), None, None, None, None, None, stream=stream)
    assert slots[0].tolist() == [3, 4] and slots[0].dtype == torch.int64
    assert records == [(slots[0].data_ptr(), 77)]


def test_write_qkv_leaves_the_callers_slots_alone(recorded):
    records, slots = recorded
    c = PagedKVCache(2, 1, 64, torch.float32, device="cpu")
    mine = torch.tensor([3, 4])
    c.write_qkv(mine, None, None, None, None, None, stream=77)
    c.write_qkv([3, 4], None, None, None, None, None)  # the current stream: freed in its order
    assert slots[0] is mine and slots[1].tolist() == [3, 4] and not records


@pytest.mark.parametrize("stream", [FakeStream(), 77])
def test_write_keeps_host_slots_until_the_stream_is_done(recorded, stream):
    records, slots = recorded
    c = PagedKVCache(2, 1, 64, torch.float32, device="cpu")
    c.write([5], None, None, stream=stream)
    assert slots[0].tolist() == [5] and records == [(slots[0].data_ptr(), 77)]
    c.write([5], None, None)
    assert len(records) == 1


# ---- sizes past what the kernels count with ----------------------------------------------------------


@pytest.mark.parametrize("d", [64, 128])
def test_append_refuses_rows_and_pages_of_2_31_elements(d):
    """Offsets within a token's row, and within a page, are 32 bits in the kernel."""
    most_q, most_kv = (2 ** 31 - 1) // d, (2 ** 31 - 1) // (16 * d)
    wide = dict(q_stride=1 << 40, k_stride=1 << 40, v_stride=1 << 40, q_out_stride=1 << 40)
    big = dict(desc=desc(h_kv=2, d=d, pages=1), rot_dim=d, n=2, h_q=most_q, **wide)
    st, msg = call("pkv_qk_norm_rope_append", APPEND, **dict(big, h_q=most_q + 1))
    assert st == ESHAPE and "2^31" in msg
    st, msg = call("pkv_qk_norm_rope_append", APPEND,
                   **dict(big, h_q=8, desc=desc(h_kv=most_kv + 1, d=d, pages=1)))
    assert st == ESHAPE and "2^31" in msg
    # (one less is not refused for its size: the call gets to its next check)
    st, msg = call("pkv_qk_norm_rope_append", APPEND, **dict(big, q=ctypes.c_void_p(4100)))
    assert st == -4
    st, msg = call("pkv_qk_norm_rope_append", APPEND, **dict(
        big, h_q=8, desc=desc(h_kv=most_kv, d=d, pages=1), q=ctypes.c_void_p(4100)))
    assert st == -4


@pytest.mark.parametrize("batch,h_kv,group,pages", [(65535, 65535, 128, (1 << 27) - 16),
                                                    (32768, 32768, 128, (1 << 27) - 16),
                                                    (65535, 32768, 64, 1 << 25)])
def test_tree_attention_refuses_tables_whose_work_passes_64_bits(batch, h_kv, group, pages):
    """The work that these tables could hold, counted in half tiles, is negative modulo 2^64."""
    st, msg = call("pkv_tree_decode_attention", TREE, dtype=F32, batch=batch, nodes=256,
                   h_q=h_kv * group, max_pages=pages, desc=desc(F32, h_kv=h_kv, d=64, pages=1),
                   mask=None)
    assert st == ESHAPE and "2^30" in msg


def test_workspace_size_of_absurd_sizes_is_a_whole_wave():
    whole = pkv.tree_decode_workspace_size(F32, F32, 64, 256, 8, 8, 64, 4096)
    for sizes in ((65535, 256, 65535 * 128, 65535, 64, (1 << 27) - 16),
                  (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1, 64, 2 ** 31 - 1)):
        assert pkv.tree_decode_workspace_size(F32, F32, *sizes) == whole


# ---- commit ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("rids", [[1], [1, 2, 2], [1, 2, 3], [1, 2, 4, 5], iter([1, 2])])
def test_commit_tree_refuses_requests_before_it_moves_rows(monkeypatch, rids):
    """One listed request for each row of the batch, all known, none twice: found before the rows in
    the pools are moved, so that a refused call leaves cache and table as they were."""
    moved = []
    monkeypatch.setattr(cache_module, "tree_commit",
                        lambda *a, **kw: moved.append(1) or torch.full((3,), 20))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream())
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    c = PagedKVCache(8, 1, 64, torch.float32, device="cpu")
    for rid in (1, 2, 4):
        c.add_request(rid)
    c.reserve([1, 2, 4], [20, 20, 20])
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(pkv.PkvError):
        c.commit_tree(rids, ints[:, None], ints, ints, ints[:, None], ints)
    assert not moved
    assert c.commit_tree(iter([4, 1, 2]), ints[:, None], ints, ints, ints[:, None], ints) == [20] * 3
    assert len(moved) == 1 and [c.lens[r] for r in (1, 2, 4)] == [20, 20, 20]
