"""One layer's paged KV cache: the two pools plus the host bookkeeping around them.

"KV cache and PagedAttention", section 4: a physical pool of fixed-size pages and, per
request, a page table listing its pages; the allocator is O(1); requests with a common
prefix point at the same pages (reference-counted here). Section 5 (continuous batching):
requests join and leave the running batch every step, so pages are freed and reused.

Page accounting, the allocator and the per-request page tables (fork, free, reserve with
copy-on-write, window release, table export) run in the C library (``pkv_alloc``/``pkv_incref``/
``pkv_decref``, ``pkv_seq_*``); this class holds the pools and hands tensors to the kernels.
"""
from __future__ import annotations

from collections.abc import Mapping

import numpy as np
import torch

from . import (PageAllocator, PkvError, SeqTable, _ids, chunk_attention, chunk_weights, copy_pages,
               evict_move, evict_select, kv_append, qk_norm_rope_append, tree_commit,
               tree_decode_attention)


class _RowView(Mapping):
    """Read-only view of the request table: rid -> page row (list) or token count (int)."""

    def __init__(self, table: SeqTable, what: str):
        self._t, self._what = table, what

    def __getitem__(self, rid):
        return self._t.pages(rid) if self._what == "pages" else self._t.length(rid)

    def __iter__(self):
        return iter(self._t.ids())

    def __len__(self):
        return len(self._t.ids())

    def __contains__(self, rid):
        try:
            self._t.length(rid)
        except KeyError:
            return False
        return True


class PagedKVCache:
    def __init__(self, num_pages: int, num_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 device="cuda", page_size: int = 16, initial_free_order=None,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
        if dtype == torch.float8_e4m3fn:
            dtype = torch.uint8  # FP8 E4M3 codes; torch.int8 pools hold INT8 codes
        self.k = torch.empty(num_pages, num_kv_heads, page_size, head_dim, dtype=dtype,
                             device=device)
        self.v = torch.empty_like(self.k)
        self.page_size = page_size
        self.num_pages = num_pages
        self.allocator = PageAllocator(num_pages, initial_free_order)
        self.table = SeqTable(self.allocator, page_size)
        self.k_scales = k_scales
        self.v_scales = v_scales
        self.pages = _RowView(self.table, "pages")  # rid -> list of page ids (-1: released)
        self.lens = _RowView(self.table, "lens")    # rid -> tokens held

    @property
    def is_fp8(self) -> bool:
        return self.k.dtype == torch.uint8

    @property
    def is_int8(self) -> bool:
        return self.k.dtype == torch.int8

    # ---- requests ---------------------------------------------------------------------------

    def add_request(self, rid: int, shared_pages=None, shared_len: int = 0, adopt: bool = False):
        """New request; optionally starting on ``shared_pages`` that already hold its first
        ``shared_len`` tokens (a prefix, whole pages only). ``adopt``: the request takes over
        references the caller holds on those pages instead of taking new ones."""
        self.table.add(rid, shared_pages, shared_len, adopt)

    def add_request_from_prefix_cache(self, rid: int, prefix_cache, tenant: int, tokens) -> int:
        """New request whose prompt is ``tokens``: it starts on the longest prefix of whole
        pages that ``prefix_cache`` holds for this tenant (the lookup's references become the
        request's). Returns the number of prompt tokens already in the cache; the caller
        reserves and writes the rest."""
        return prefix_cache.add_request(self.table, rid, tenant, tokens)

    def register_prompt(self, rid: int, prefix_cache, tenant: int, tokens):
        """Puts the full pages of request ``rid``'s prompt (``tokens``, already written) into
        ``prefix_cache`` for later requests of the same tenant."""
        prefix_cache.insert_request(tenant, tokens, self.table, rid)

    def fork(self, src_rid: int, new_rid: int):
        """A new request sharing every page of ``src_rid`` (parallel sampling, beam search);
        writes into a shared, partly filled page first copy it (``reserve`` does that)."""
        self.table.fork([src_rid], [new_rid])

    def fork_many(self, src_rids, new_rids):
        """``fork`` for several requests in one call (a parent may be forked earlier in it)."""
        self.table.fork(src_rids, new_rids)

    def free_request(self, rid: int):
        self.table.free([rid])

    def free_many(self, rids):
        self.table.free(rids)

    def release_outside_window(self, rid: int, window: int, sink_tokens: int = 0) -> int:
        """Sliding window ("KV cache and PagedAttention", section 8): return to the allocator
        every page of the request whose positions all lie outside the first ``sink_tokens``
        and the last ``window`` positions (the window only moves forward, so they are never
        read again). Their table entries become -1. Returns the number of pages released."""
        return self.table.release_outside_window(rid, window, sink_tokens)

    def truncate(self, rids, new_lens):
        """Cut requests back to ``new_lens`` tokens (rejected drafts, a restarted answer): pages
        that hold none of the kept tokens go back to the allocator."""
        self.table.truncate(rids, new_lens)

    def reserve(self, rids, counts, copies_out=None) -> np.ndarray:
        """Grow each request by counts[i] tokens (allocating pages on page boundaries) and
        return the int64 slots of the new positions, request by request. Shared, partly filled
        pages about to be written are copied first (copy-on-write): on the device here, or,
        when ``copies_out`` is a list, appended to it as (source, destination) page pairs for
        the caller to copy (``copy_pages``) before the writes."""
        slots, copies = self.table.reserve(rids, counts)
        if copies_out is not None:
            copies_out.extend(copies)
        elif copies:
            src = torch.tensor([c[0] for c in copies], dtype=torch.int32, device=self.k.device)
            dst = torch.tensor([c[1] for c in copies], dtype=torch.int32, device=self.k.device)
            copy_pages(self.k, self.v, src, dst)
        return slots

    def step(self, finished, joining, prompt_lens, live, width: int | None = None,
             tables_out=None, lens_out=None, copies_out=None, incremental: bool = False):
        """One continuous-batching step of bookkeeping in one library call: the ``finished``
        requests are freed, the ``joining`` ones added and grown by their ``prompt_lens``, every
        ``live`` request (joining ones included) gets room for one new token, and the live
        requests' page-table rows and lengths are exported (into ``tables_out``/``lens_out``
        when given). Returns (prompt slots, tables, lengths). Shared pages about to be written
        are copied as in ``reserve``. If the pages run out, the frees stand and the joining
        requests are not added (PkvError). ``incremental``: rows of ``tables_out`` that still
        hold the same request as after the previous incremental step are only patched."""
        slots, bt, cl, copies = self.table.step(finished, joining, prompt_lens, live, width,
                                                tables_out, lens_out, incremental=incremental)
        if copies_out is not None:
            copies_out.extend(copies)
        elif copies:
            src = torch.tensor([c[0] for c in copies], dtype=torch.int32, device=self.k.device)
            dst = torch.tensor([c[1] for c in copies], dtype=torch.int32, device=self.k.device)
            copy_pages(self.k, self.v, src, dst)
        return slots, bt, cl

    def _device_slots(self, slots, stream) -> torch.Tensor:
        """``slots`` on the device, for a call on ``stream``. Host slots are copied here, on the
        current stream; the copy is complete on return, and its memory is not handed out again
        before the work then queued on ``stream`` is done."""
        if isinstance(slots, torch.Tensor):
            return slots
        slots = torch.from_numpy(np.asarray(slots, dtype=np.int64)).to(self.k.device)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):  # a raw cudaStream_t handle
                stream = torch.cuda.ExternalStream(int(stream), device=self.k.device)
            slots.record_stream(stream)
        return slots

    def write(self, slots, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        """Append rows k_new/v_new [N, h_kv, d] at the given slots (host array or CUDA int64)."""
        kv_append(k_new, v_new, self._device_slots(slots, stream), self.k, self.v, self.k_scales,
                  self.v_scales, stream)

    def write_qkv(self, slots, q, k_new, v_new, positions, cos_sin, q_out=None, stream=None,
                  **norm):
        """Norm, rotate and append in one pass (qk_norm_rope_append; ``norm``: q_weight, k_weight,
        eps, interleaved); returns the rotated queries."""
        slots = self._device_slots(slots, stream)
        return qk_norm_rope_append(q, k_new, v_new, positions, slots, self.k, self.v, cos_sin,
                                   q_out=q_out, k_scales=self.k_scales, v_scales=self.v_scales,
                                   stream=stream, **norm)

    # ---- drafted tokens ----------------------------------------------------------------------

    def attend_tree(self, q, block_tables, context_lens, scale, tree_mask=None, tree_lens=None,
                    out=None, workspace=None, stream=None):
        """Attention of drafted nodes q [B, T, h_q, d] (tree_decode_attention over these pools)."""
        return tree_decode_attention(q, self.k, self.v, block_tables, context_lens, scale,
                                     tree_mask, tree_lens, out, self.k_scales, self.v_scales,
                                     workspace, stream)

    def commit_tree(self, rids, block_tables, context_lens, tree_lens, path, path_lens,
                    stream=None) -> list:
        """Keep the accepted path of each request's draft: move its rows together (tree_commit),
        read the new lengths back (this waits for the stream) and truncate the requests to them.
        Returns the new lengths. The drafted rows' pages must be the request's own, as ``reserve``
        leaves them: fork a request before its draft or after this, not in between."""
        rids = _ids(rids)
        self.table.lengths(rids)  # (refuses an unknown request)
        if rids.size != context_lens.numel() or np.unique(rids).size != rids.size:
            raise PkvError(-1, "rids must name each request of the batch once")
        if stream is None:
            stream = torch.cuda.current_stream(self.k.device)
        elif not isinstance(stream, torch.cuda.Stream):  # a raw cudaStream_t handle
            stream = torch.cuda.ExternalStream(int(stream), device=self.k.device)
        with torch.cuda.stream(stream):
            new = tree_commit(self.k, self.v, block_tables, context_lens, tree_lens, path,
                              path_lens, stream=stream).tolist()
        self.table.truncate(rids, new)
        return new

    # ---- chunks of new tokens, and a bounded cache -------------------------------------------

    def attend_chunk(self, q, block_tables, context_lens, query_starts, scale, stream=None, **form):
        """Attention of chunks of new tokens q [N, h_q, d], whose rows are in the cache already
        (chunk_attention over these pools; ``form``: softcap, alibi_slopes, window, sink_tokens, out,
        lse, workspace)."""
        return chunk_attention(q, self.k, self.v, block_tables, context_lens, query_starts, scale,
                               k_scales=self.k_scales, v_scales=self.v_scales, stream=stream, **form)

    def chunk_weights(self, q, block_tables, context_lens, query_starts, lse, scale, stream=None,
                      **form):
        """Sums of the weights that the chunks' rows give to each cached position (chunk_weights;
        ``form``: the attention's, last_rows, add_to, out, width, workspace)."""
        return chunk_weights(q, self.k, block_tables, context_lens, query_starts, lse, scale,
                             k_scales=self.k_scales, stream=stream, **form)

    def evict(self, rids, weights, budget: int, recent: int = 0, sink_tokens: int = 0,
              stream=None) -> torch.Tensor:
        """Cut each request longer than ``budget`` tokens to its first ``sink_tokens``, its last
        ``recent`` and the positions with the largest ``weights`` (fp32 [len(rids), h_kv, width], as
        ``chunk_weights`` makes them) between them, ``budget`` in all, chosen for each KV head on its
        own. The kept rows move together onto new pages, so that shared pages (a fork's, a cached
        prefix's) stay as they are for their other holders, and the request gives its old pages back:
        what is written into them later must be ordered after this call's work on ``stream``. Returns
        the sums in the new order, zeros behind them. If the new pages are not there, PkvError is
        raised and nothing changes."""
        rids = _ids(rids)
        lens = self.table.lengths(rids)  # (refuses an unknown request)
        if np.unique(rids).size != rids.size:
            raise PkvError(-1, "rids must name each request once")
        if (weights.dtype != torch.float32 or weights.dim() != 3 or
                tuple(weights.shape[:2]) != (rids.size, self.k.shape[1])):
            raise PkvError(-2, "weights must be float32 [len(rids), num_kv_heads, width]")
        budget = int(budget)
        if budget <= 0 or recent < 0 or sink_tokens < 0 or recent + sink_tokens > budget:
            raise PkvError(-1, "budget must be positive and hold recent and sink_tokens")
        if rids.size and int(lens.max()) > weights.shape[2]:
            raise PkvError(-2, "a request is longer than its row of weights")
        cut = np.nonzero(lens > budget)[0]
        if stream is None:
            stream = torch.cuda.current_stream(self.k.device)
        elif not isinstance(stream, torch.cuda.Stream):  # a raw cudaStream_t handle
            stream = torch.cuda.ExternalStream(int(stream), device=self.k.device)
        with torch.cuda.stream(stream):
            if cut.size == 0:
                return weights.clone()
            old = self.table.tables(rids[cut])
            if any((old[i, :-(-int(lens[c]) // self.page_size)] < 0).any()
                   for i, c in enumerate(cut)):
                raise PkvError(-1, "a request that gave pages back (release_outside_window) cannot "
                                   "be cut")
            per = -(-budget // self.page_size)
            pages = np.asarray(self.allocator.alloc(per * cut.size), dtype=np.int32)
            try:
                dev = self.k.device
                new = pages.reshape(cut.size, per)
                rows = None if cut.size == rids.size else torch.from_numpy(cut).to(dev)
                w = weights if rows is None else weights[rows]
                bt, nt, cl = (torch.from_numpy(np.ascontiguousarray(x)).to(dev)
                              for x in (old, new, lens[cut]))
                kept, kept_lens = evict_select(w.contiguous(), cl, budget, recent, sink_tokens,
                                               stream=stream)
                moved = torch.empty_like(w, memory_format=torch.contiguous_format)
                evict_move(self.k, self.v, bt, kept, kept_lens, nt, w.contiguous(), moved,
                           stream=stream)
                if rows is not None:
                    moved = weights.clone().index_copy_(0, rows, moved)
            except BaseException:
                self.allocator.decref(pages)
                raise
            for i, rid in enumerate(rids[cut].tolist()):
                self.table.free([rid])
                self.table.add(rid, new[i].tolist(), per * self.page_size, adopt=True)
            self.table.truncate(rids[cut], np.full(cut.size, budget))
        return moved

    # ---- views for the decode ---------------------------------------------------------------

    def block_table_array(self, rids, width: int | None = None, out=None) -> np.ndarray:
        """Page-table rows of the requests (unused columns 0, released pages -1); ``out`` (a
        contiguous int32 array or CPU tensor of [len(rids)][width]) is filled in place."""
        return self.table.tables(rids, width, out=out)

    def context_lens_array(self, rids, out=None) -> np.ndarray:
        return self.table.lengths(rids, out=out)
