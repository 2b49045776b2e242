"""A serving step over a paged KV cache, through the C ABI.

Requests of unlike lengths share one pool of pages per layer. A step runs

  plan      paged_build_tables      pages, slots and positions of the step's new tokens, from the lengths
  append    paged_norm_rope_append  per layer: norms and rotation of q and k, k and v into the pages
  attend    gqa_paged_attn          per layer: every new token over its request's pages
  commit                            the lengths after the step
  release   paged_release_pages     pages of requests that ended, or of a rejected tail of drafted tokens

with one plan for all layers: every layer's pools use the same page indices. Over 8-bit pages append and attend
are paged_norm_rope_append_e4m3 and gqa_paged_attn_e4m3. A planned step is
committed or released before the next is planned (its pages are otherwise lost to the pool). Everything
a step reads or writes on the device lies in buffers that this object keeps, so the five can be captured
in a CUDA graph (after one eager step) and replayed with new contents of new_len and keep_len.

This module only sequences library calls and owns the buffers they share.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import (PAGE_SIZE, alloc_paged_workspace, gqa_paged_attn, gqa_paged_attn_e4m3, make_paged_dims, new_pages,
               new_pages_e4m3, num_pages, paged_build_tables, paged_norm_rope_append, paged_norm_rope_append_e4m3,
               paged_release_pages)


class PagedCache:
    """Pools, block table and free list of up to ``batch`` requests of at most ``max_len`` tokens each.

    ``max_tokens`` is the most new tokens of a step. A step's q, k and v have the rows that its plan was
    given (max_tokens, or fewer); rows behind the step's tokens are padding.

    ``dtype`` is the type of q, k and v, and of the pages unless ``kv_dtype`` says torch.float8_e4m3fn: then
    k_pages and v_pages hold E4M3 codes, k_exp and v_exp the exponents of each layer's pages. A released tail of large
    rows (a rejected draft) leaves the exponent of the page it began in where it put it: rows that join the page later are
    rounded to it, until the page is begun again. Infinite keys and values become their page's largest number."""

    def __init__(self, num_layers: int, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, pool_pages: int,
                 max_len: int, max_tokens: int, device, page_size: int = PAGE_SIZE, dtype=torch.float16, kv_dtype=None):
        if kv_dtype not in (None, dtype, torch.float8_e4m3fn):
            raise ValueError(f"pages hold {dtype} or torch.float8_e4m3fn, not {kv_dtype}")
        self.device, self.page_size, self.max_len, self.max_tokens = torch.device(device), page_size, max_len, max_tokens
        self.scale = 1.0 / math.sqrt(head_dim)
        width = num_pages(max_len, page_size)
        dims = make_paged_dims(batch, num_q_heads, num_kv_heads, head_dim, page_size, pool_pages, width, max_tokens, dtype)
        self.workspace = alloc_paged_workspace(dims, self.device)
        self.k_exp = self.v_exp = None
        if kv_dtype == torch.float8_e4m3fn:
            pools = [new_pages_e4m3(pool_pages, num_kv_heads, page_size, head_dim, self.device) for _ in range(2 * num_layers)]
            self.k_exp, self.v_exp = ([e for _, e in pools[i::2]] for i in range(2))
            self.k_pages, self.v_pages = ([c for c, _ in pools[i::2]] for i in range(2))
        else:
            pool = lambda: new_pages(pool_pages, num_kv_heads, page_size, head_dim, self.device, dtype)  # noqa: E731
            self.k_pages = [pool() for _ in range(num_layers)]
            self.v_pages = [pool() for _ in range(num_layers)]
        i32 = dict(dtype=torch.int32, device=self.device)
        self.block_table = torch.full((batch, width), -1, **i32)
        self.free_pages = torch.arange(pool_pages - 1, -1, -1, **i32)  # page 0 is taken first
        self.free_count = torch.full((1,), pool_pages, **i32)
        self.cache_len = torch.zeros(batch, **i32)   # tokens of each request in the cache
        self.kv_len = torch.zeros(batch, **i32)      # with the step's new ones (0: refused)
        self.cu_q = torch.zeros(batch + 1, **i32)
        self.positions = torch.zeros(max_tokens, **i32)
        self.slots = torch.full((max_tokens,), -1, **i32)
        self._rows = (self.positions, self.slots)    # of the planned step

    def plan(self, new_len: torch.Tensor, rows: Optional[int] = None):
        """Place the step's new_len [batch] tokens in as many rows (None: max_tokens). A request that does not
        fit them is refused (GQAQ_DEV_BAD_POS). A request the pool has no pages for is refused
        (kv_len 0, GQAQ_DEV_NO_PAGES), and so is one that would pass max_len (GQAQ_DEV_BAD_LEN): its rows
        of the step have no effect and out is 0 there."""
        n = self.max_tokens if rows is None else int(rows)
        if not 1 <= n <= self.max_tokens:
            raise ValueError(f"rows must lie in 1 .. max_tokens = {self.max_tokens}, got {n}")
        positions, slots = self.positions[:n], self.slots[:n]
        paged_build_tables(self.cache_len, new_len, self.free_pages, self.free_count, self.block_table, n, self.page_size,
                           kv_len=self.kv_len, cu_q=self.cu_q, positions=positions, slots=slots,
                           free_count_out=self.free_count, max_len=self.max_len)
        self._rows = (positions, slots)

    def append(self, layer: int, q, k, v, q_weight=None, k_weight=None, eps: float = 1e-6, cos_sin=None,
               interleaved: bool = False, q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The layer's projected q [rows,Hq,D] and k, v [rows,Hkv,D]: returns q for attend."""
        positions, slots = self._rows
        more = dict(q_weight=q_weight, k_weight=k_weight, eps=eps, cos_sin=cos_sin, interleaved=interleaved, q_out=q_out)
        if self.k_exp is not None:
            return paged_norm_rope_append_e4m3(q, k, v, positions, slots, self.k_pages[layer], self.v_pages[layer],
                                               self.k_exp[layer], self.v_exp[layer], **more)
        return paged_norm_rope_append(q, k, v, positions, slots, self.k_pages[layer], self.v_pages[layer], **more)

    def attend(self, layer: int, q, max_q_len: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of the step's tokens, q [rows,Hq,D]; max_q_len bounds the new tokens of a request."""
        if q.shape[0] != self._rows[0].shape[0]:
            raise ValueError(f"q must have the {self._rows[0].shape[0]} rows of the step's plan, got {q.shape[0]}")
        tables = (self.block_table, self.cu_q, self.kv_len, self.scale, max_q_len)
        if self.k_exp is not None:
            return gqa_paged_attn_e4m3(q, self.k_pages[layer], self.v_pages[layer], self.k_exp[layer], self.v_exp[layer], *tables,
                                       out=out, workspace=self.workspace)
        return gqa_paged_attn(q, self.k_pages[layer], self.v_pages[layer], *tables, out=out, workspace=self.workspace)

    def commit(self):
        """The step's tokens are part of the cache (refused requests keep their length)."""
        torch.maximum(self.cache_len, self.kv_len, out=self.cache_len)

    def release(self, keep_len: torch.Tensor):
        """Requests keep their first keep_len [batch] tokens; the pages past them are free again. Before commit the
        planned step counts, so keep_len can give it up, or keep part of it. A request whose keep_len is negative or
        above its length keeps its lengths and all its pages (GQAQ_DEV_BAD_LEN)."""
        held = torch.maximum(self.cache_len, self.kv_len)  # with a planned step that commit has not seen
        paged_release_pages(held, keep_len, self.block_table, self.free_pages, self.free_count, self.page_size,
                            free_count_out=self.free_count)
        # both lengths follow the library's rule, so that neither they nor a later commit pass the tokens that the pages hold
        kept = (keep_len >= 0) & (keep_len <= held)
        torch.where(kept, keep_len, self.cache_len, out=self.cache_len)
        torch.where(kept, keep_len, self.kv_len, out=self.kv_len)
