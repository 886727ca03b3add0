"""Serving with the learned-relative attention: a paged key-value cache and its step.

:class:`PagedKVCache` holds one attention layer's pages, the block table and the lengths of
``max_requests`` request rows, and a stack of free pages, all on the GPU. A step is

* ``plan = cache.reserve(new_lens, max_tokens)``: sets the rows' lengths (a growing row gets
  pages, one that shrinks gives pages back, 0 ends it) and returns the new tokens' slots;
* ``cache.append(k, v, plan["slots"])``: their keys and values, clipped on the way if asked;
* ``out, lse = cache.decode(q, profiles, sink)``: attention of each row's newest token.

Prompts use ``binding.forward`` for their attention and ``append`` to fill the cache; rows
without a request have length 0 and get ``out = 0``. No call waits for the GPU or reads a
length on the host, and all state is updated in place, so a step can be captured in a CUDA
graph (with ``new_lens`` in a tensor that the caller rewrites) and replayed. The calls are
the C ABI of ``include/inkling_paged_attn.h`` through :mod:`learned_relative_gqa_b200.binding`.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding


class PagedKVCache:
    """Pages, block table [max_requests, ceil(max_len / page_size)] and lengths of one layer.

    ``dtype`` is ``torch.bfloat16`` or ``torch.float8_e4m3fn`` (then with ``k_scale`` and
    ``v_scale``, fp32 [heads_kv]). Pools are [num_pages, page_size, heads_kv, head_dim],
    laid out with each page's tokens of a head next to each other.
    """

    def __init__(self, *, max_requests: int, max_len: int, num_pages: int, page_size: int, heads_kv: int,
                 head_dim: int, dtype=torch.bfloat16, k_scale=None, v_scale=None, device="cuda"):
        if min(max_requests, max_len, num_pages, page_size, heads_kv) < 1:
            raise ValueError("PagedKVCache: sizes must be positive")
        if dtype not in binding.KV_DTYPES:
            raise ValueError(f"PagedKVCache: a cache is bfloat16 or float8_e4m3fn, got {dtype}")
        device = torch.zeros((), device=device).device  # with its index
        self.page_size, self.num_pages = int(page_size), int(num_pages)
        width = -(-max_len // page_size)
        pool = (num_pages, heads_kv, page_size, head_dim)
        self.k_cache = torch.zeros(pool, dtype=dtype, device=device).transpose(1, 2)
        self.v_cache = torch.zeros(pool, dtype=dtype, device=device).transpose(1, 2)
        self.k_scale, self.v_scale = k_scale, v_scale
        for name, scale in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (scale is not None) != (dtype == torch.float8_e4m3fn):
                raise ValueError(f"PagedKVCache: {name}: an e4m3 cache needs its scales, a bfloat16 cache takes none")
        i32 = dict(dtype=torch.int32, device=device)
        self.block_table = torch.full((max_requests, width), -1, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)  # page 0 on top
        # lengths and the four plan results, and the same of the step that is being planned:
        # the plan may not write what it reads, so one small copy follows it
        at = (max_requests + 3) // 4 * 4
        self._state = torch.zeros(at + 4, **i32)
        self._state[at] = num_pages
        self._next = torch.zeros_like(self._state)
        self.lens = self._state[:max_requests]
        self.info, self._free_count = self._state[at:], self._state[at:at + 1]
        self._next_lens, self._next_info = self._next[:max_requests], self._next[at:]

    def reserve(self, new_lens: torch.Tensor, max_tokens: int, stream=None):
        """Brings the rows to ``new_lens`` [max_requests] int32 tokens; dict of ``slots`` [max_tokens] int64,
        ``positions`` [max_tokens] and ``query_start`` [max_requests + 1] of the new tokens.

        ``cache.lens`` holds the lengths that the free pages allowed and ``cache.info`` the
        pages left, the new tokens, the pages that were missing and the pages taken. With
        more new tokens than ``max_tokens`` the last ones get no slot, though ``cache.lens``
        counts them: what ``decode`` reads for those is whatever their pages held before.
        """
        plan = binding.kv_plan(self.lens, new_lens, self.block_table, self.free_pages, self._free_count,
                               page_size=self.page_size, num_pages=self.num_pages, max_tokens=max_tokens,
                               lens=self._next_lens, info=self._next_info, stream=stream)
        if stream is None:
            self._state.copy_(self._next)
        else:
            with torch.cuda.stream(stream):
                self._state.copy_(self._next)
        return {name: plan[name] for name in ("slots", "positions", "query_start")}

    def append(self, k, v, slots, *, threshold: Optional[float] = None, clip_scale=None, tau=None, stream=None) -> None:
        """Stores ``k``, ``v`` [T, heads_kv, head_dim] BF16 in their slots (see ``binding.kv_append``)."""
        binding.kv_append(k, v, slots, self.k_cache, self.v_cache, k_scale=self.k_scale, v_scale=self.v_scale,
                          threshold=threshold, clip_scale=clip_scale, tau=tau, stream=stream)

    def decode(self, q, profiles=None, sink=None, *, window: int = 0, scale: Optional[float] = None, workspace=None,
               stream=None):
        """out [max_requests, heads_q, head_dim], lse [max_requests, heads_q] of each row's newest token."""
        return binding.paged_decode(q, self.k_cache, self.v_cache, self.block_table, self.lens, profiles, sink,
                                    window=window, scale=scale, k_scale=self.k_scale, v_scale=self.v_scale,
                                    workspace=workspace, stream=stream)
