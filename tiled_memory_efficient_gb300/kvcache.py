"""A paged KV cache in 8 bits for decoding with the tiled kernels.

``PagedKVCache`` owns the device memory that include/kvcache.h describes -- e4m3
pages with one power-of-two scale per (page, KV head), a page table, lengths and
holder counts -- and offers the calls of a decoding loop over it::

    cache = PagedKVCache(n_layers=24, n_seqs=8, n_kv_heads=2, head_dim=64, n_pages=4096)
    cache.reserve(n_new)                     # room for this step's tokens, every layer
    for layer in range(24):
        cache.append(layer, k, v, n_new)     # this layer's new keys and values
        out, lse = cache.attend(layer, q, n_new=n_new)   # the same tokens over the cache
    cache.reassign(parents)                  # fork, reorder or free sequences
    cache.compact()                          # held pages to the front of the pools

Nothing here reads device memory on the host: lengths and tables stay on the
device, so a step captures into a CUDA graph.  ``sync_status()`` reports what a
call could not do (a full pool: ATTN_ERR_POOL), ``info`` holds the last
bookkeeping call's counts.  After a ``reserve`` that found no room ``granted`` is 0
and every ``append`` leaves the cache as it is, until a ``reserve`` succeeds.

A step may give each sequence its own number of tokens: ``n_new`` goes to all three
calls, and both the keys and the queries of sequence b are the first n_new[b] rows.

With a ``rope.Rope`` the append also turns the keys, and the step's queries, to the
positions that ``reserve`` gave them::

    q = cache.append(layer, k, v, n_new, rope=rope, q=q)

``share=True`` is for sequences that begin alike (samples or beams of one prompt, many
questions about one text).  One sequence takes the prompt, ``reassign`` forks it, and
``attend`` then reads the common pages once for all of them.
"""
from __future__ import annotations

import torch

from . import _lib

__all__ = ["PagedKVCache"]

# Attention over a shared prefix keeps all query rows in fp32 twice, and takes 2^20 rows a KV head.  A call whose
# rows would take more is kv8_attn's.  (16 sequences of 2048 queries, 32:8 heads, D = 128, 1.1 GB: 17.0 ms where
# 16384 positions are shared and 45.5 with every sequence for itself; 10.4 and 10.9 where it is 256.)
_SHARED_BYTES = 4 << 30
_SHARED_ROWS = 1 << 20
# What prefixes have to save in keys and values before attention with a plan that leaves the choice follows it.  (8 beams
# under 4096 positions, 14:2 heads, D = 64: 13.3 us with a plan that is not followed, 12 by kv8_attn.)
_WORTH_BYTES = 128 << 20


class PagedKVCache:
    """Keys and values of n_seqs sequences in n_layers layers.

    page_size is 16, 32, 64 or 128 tokens; max_pages (default: all n_pages) the
    most pages one sequence can hold.  With window > 0 queries see the last
    `window` positions and the first `sinks`, and ``reserve`` gives back pages
    the window has left behind.

    share (without a window): ``reassign`` looks which sequences begin with the same
    pages, and ``attend`` reads those once for all of them where that saves enough (128 MB of
    keys and values, in groups of enough sequences (include/kvcache.h); or min_saved
    positions, for each group).  A NaN or infinity among a prefix's values then reaches every
    query of the sequences that share it, those before its position too.  Whoever writes `table`
    by hand calls ``find_shared`` afterwards.  Such an ``attend`` asks for 8 bytes of workspace per
    value of q, and for parts of up to 40 MB beside; with over 4 GB of them, or more than 2^20
    queries a KV head (its query heads'), it reads every sequence for itself.  So does a
    cache that can never save 128 MB: n_seqs - 1 tables of max_pages pages hold less (give
    max_pages, where sequences cannot take the whole pool), and min_saved is -1.
    """

    def __init__(self, n_layers: int, n_seqs: int, n_kv_heads: int, head_dim: int, n_pages: int,
                 page_size: int = 64, max_pages: int | None = None, window: int = 0, sinks: int = 0,
                 device="cuda", share: bool = False, min_saved: int = -1):
        if head_dim not in (64, 128):
            raise NotImplementedError(f"head dim {head_dim} is not one of (64, 128)")
        if page_size not in (16, 32, 64, 128):
            raise NotImplementedError(f"page size {page_size} is not one of (16, 32, 64, 128)")
        if min(n_layers, n_seqs, n_kv_heads, n_pages) < 1 or window < 0 or sinks < 0:
            raise ValueError("sizes must be positive, window and sinks not negative")
        if share and window:
            raise ValueError("a cache with a window does not share the reading of prefixes")
        max_pages = n_pages if max_pages is None else max_pages
        if max_pages < 1:
            raise ValueError("max_pages must be positive")
        self.page_size, self.window, self.sinks = page_size, window, sinks
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        self.k_pages = torch.zeros(shape, device=device, dtype=torch.float8_e4m3fn)
        self.v_pages = torch.zeros(shape, device=device, dtype=torch.float8_e4m3fn)
        self.k_scale = torch.ones(shape[:3], device=device)
        self.v_scale = torch.ones(shape[:3], device=device)
        i32 = dict(device=device, dtype=torch.int32)
        self.table = torch.full((n_seqs, max_pages), -1, **i32)
        self.lens = torch.zeros(n_seqs, **i32)
        self.refs = torch.zeros(n_pages, **i32)
        self.info = torch.zeros(4, **i32)
        self.granted = torch.ones(1, **i32)   # did the last reserve make room?
        self._count = self.info[1:2]
        # pairs of pages to copy: at most one a sequence, or half the pool
        pairs = max(n_seqs, n_pages // 2)
        self._src, self._dst = torch.zeros(pairs, **i32), torch.zeros(pairs, **i32)
        self._ws = torch.empty(_lib.kvp_workspace_size(n_seqs, max_pages, n_pages), device=device,
                               dtype=torch.uint8)
        self._all = torch.empty(n_seqs, **i32)
        self.plan = None   # which sequences share a prefix
        if share:
            self.min_saved = min_saved
            # whether a plan of this cache can ever be followed
            self._worth = min_saved >= 0 or \
                (n_seqs - 1) * max_pages * page_size * 2 * n_kv_heads * head_dim >= _WORTH_BYTES
            self.plan = _lib.kvp_find_shared(self.table, self.lens, page_size, min_saved)

    def _counts(self, n):
        if isinstance(n, int):
            return self._all.fill_(n)
        return n

    def reserve(self, n_new):
        """Makes room for n_new tokens of every sequence (an int, or an int32 tensor
        [n_seqs]; 0: the sequence rests) and adds them to the lengths; with too few
        free pages it changes nothing but ``granted``."""
        _lib.kvp_reserve(self.table, self.lens, self.refs, self._counts(n_new), self.page_size,
                         self.info, window=self.window, sinks=self.sinks, workspace=self._ws,
                         granted=self.granted)

    def append(self, layer: int, k, v, n_new=None, rope=None, q=None):
        """Stores the keys and values [n_seqs, n_kv_heads, T, head_dim] of the tokens
        that ``reserve`` made room for (n_new of the T each; None: all T); none when it
        found no room.  With rope (a ``rope.Rope``) the keys are turned to their positions
        on the way, and the step's queries q [n_seqs, Hq, T, head_dim], if given, as
        well: they are returned, rows from n_new on as 0.  (Without a gradient: a q that
        autograd follows is refused.)"""
        return _lib.kv8_append(k, v, self.k_pages[layer], self.v_pages[layer], self.k_scale[layer],
                               self.v_scale[layer], self.table, self.lens,
                               n_new=None if n_new is None else self._counts(n_new), granted=self.granted,
                               rope=rope, q=q)

    def attend(self, layer: int, q, scale: float | None = None, n_new=None):
        """(out, lse) of the newest positions q [n_seqs, Hq, Nq, head_dim].  n_new as in
        ``append``: the first n_new rows of each sequence, the others (and all rows
        of a step that found no room) get 0 and -inf.  None: all Nq rows are the
        newest positions; with a window no more than the sequence's last ``reserve``
        made room for, since older queries want pages that it gave back."""
        if self.plan is not None and self._worth and not self._too_many(q):
            return _lib.kv8_attn_shared(q, self.k_pages[layer], self.v_pages[layer], self.k_scale[layer],
                                        self.v_scale[layer], self.table, self.lens, self.plan, scale=scale,
                                        n_new=None if n_new is None else self._counts(n_new),
                                        granted=None if n_new is None else self.granted)
        return _lib.kv8_attn(q, self.k_pages[layer], self.v_pages[layer], self.k_scale[layer],
                             self.v_scale[layer], self.table, self.lens, scale=scale,
                             window=self.window, sinks=self.sinks,
                             n_new=None if n_new is None else self._counts(n_new),
                             granted=None if n_new is None else self.granted)

    def _too_many(self, q):
        return q.dim() == 4 and (8 * q.numel() > _SHARED_BYTES or
                                 q.shape[1] * q.shape[2] > _SHARED_ROWS * self.k_scale.shape[2])

    def reassign(self, parents):
        """Sequence c becomes a copy-on-write child of parents[c] (int32 tensor
        [n_seqs]; c: kept, -1: freed), all at once, in every layer.  With too few free
        pages every sequence keeps its own content (``info[0]`` is 0 then)."""
        _lib.kvp_reassign(self.table, self.lens, self.refs, parents, self.page_size, self._src,
                          self._dst, self.info, workspace=self._ws)
        self._copy(self.table.shape[0])
        if self.plan is not None and self._worth:
            self.find_shared()

    def find_shared(self):
        """With share: looks anew which sequences begin with the same pages."""
        if self.plan is None:
            raise ValueError("the cache was made without share")
        _lib.kvp_find_shared(self.table, self.lens, self.page_size, self.min_saved, plan=self.plan)

    def compact(self):
        """Moves the held pages of every layer to the front of the pools."""
        _lib.kvp_compact(self.table, self.refs, self._src, self._dst, self.info, workspace=self._ws)
        self._copy(self.refs.numel() // 2)

    def _copy(self, most: int):
        _lib.kv8_copy_pages(self.k_pages, self.v_pages, self.k_scale, self.v_scale, self._src,
                            self._dst, self._count, max_count=most)
