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
"""
from __future__ import annotations

import torch

from . import _lib

__all__ = ["PagedKVCache"]


class PagedKVCache:
    """Keys and values of n_seqs sequences in n_layers layers.

    page_size is 16, 32, 64 or 128 tokens; max_pages (default: all n_pages) the
    most pages one sequence can hold.  With window > 0 queries see the last
    `window` positions and the first `sinks`, and ``reserve`` gives back pages
    the window has left behind.
    """

    def __init__(self, n_layers: int, n_seqs: int, n_kv_heads: int, head_dim: int, n_pages: int,
                 page_size: int = 64, max_pages: int | None = None, window: int = 0, sinks: int = 0,
                 device="cuda"):
        if head_dim not in (64, 128):
            raise NotImplementedError(f"head dim {head_dim} is not one of (64, 128)")
        if page_size not in (16, 32, 64, 128):
            raise NotImplementedError(f"page size {page_size} is not one of (16, 32, 64, 128)")
        if min(n_layers, n_seqs, n_kv_heads, n_pages) < 1 or window < 0 or sinks < 0:
            raise ValueError("sizes must be positive, window and sinks not negative")
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

    def append(self, layer: int, k, v, n_new=None):
        """Stores the keys and values [n_seqs, n_kv_heads, T, head_dim] of the tokens
        that ``reserve`` made room for (n_new of the T each; None: all T); none when it
        found no room."""
        _lib.kv8_append(k, v, self.k_pages[layer], self.v_pages[layer], self.k_scale[layer],
                        self.v_scale[layer], self.table, self.lens,
                        n_new=None if n_new is None else self._counts(n_new), granted=self.granted)

    def attend(self, layer: int, q, scale: float | None = None, n_new=None):
        """(out, lse) of the newest positions q [n_seqs, Hq, Nq, head_dim].  n_new as in
        ``append``: the first n_new rows of each sequence, the others (and all rows
        of a step that found no room) get 0 and -inf.  None: all Nq rows are the
        newest positions; with a window no more than the sequence's last ``reserve``
        made room for, since older queries want pages that it gave back."""
        return _lib.kv8_attn(q, self.k_pages[layer], self.v_pages[layer], self.k_scale[layer],
                             self.v_scale[layer], self.table, self.lens, scale=scale,
                             window=self.window, sinks=self.sinks,
                             n_new=None if n_new is None else self._counts(n_new),
                             granted=None if n_new is None else self.granted)

    def reassign(self, parents):
        """Sequence c becomes a copy-on-write child of parents[c] (int32 tensor
        [n_seqs]; c: kept, -1: freed), all at once, in every layer.  With too few free
        pages every sequence keeps its own content (``info[0]`` is 0 then)."""
        _lib.kvp_reassign(self.table, self.lens, self.refs, parents, self.page_size, self._src,
                          self._dst, self.info, workspace=self._ws)
        self._copy(self.table.shape[0])

    def compact(self):
        """Moves the held pages of every layer to the front of the pools."""
        _lib.kvp_compact(self.table, self.refs, self._src, self._dst, self.info, workspace=self._ws)
        self._copy(self.refs.numel() // 2)

    def _copy(self, most: int):
        _lib.kv8_copy_pages(self.k_pages, self.v_pages, self.k_scale, self.v_scale, self._src,
                            self._dst, self._count, max_count=most)
