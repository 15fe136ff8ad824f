"""Exact attention of many requests of different lengths over one pool of cache pages.

    cache = PagedAttentionCache(n_pages=4096, page=64, H=8, E=128, D=128, dtype=torch.bfloat16,
                                max_requests=64, max_length=32768, bounds=True)
    step = cache.plan(new_lengths, max_tokens)      # pages, slots and positions of the step's tokens
    cache.append(k, v, step.slots)                  # (N, H, E), (N, H, D): their keys and values
    out = cache.attend(q)                           # (R, Hq, E): one query token per request
    out = cache.attend_sparse(q, top=64)            # the same over the 64 best pages of each request
    cache.release(keep)                             # 0 for requests that have ended

Everything stays on the device: no call waits for the GPU or reads a value back, and all of them can
be captured into a CUDA graph.  The functions under the class take the caller's own tensors.  A page
holds ``page`` tokens of every key head, k_pages (n_pages, H, page, E) and v_pages (n_pages, H, page,
D), in any strides with a contiguous last axis; query head j reads key head j // (Hq // H).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

_binding = None


def _calls():
    """The compiled binding (_paged.so, built beside the library), with the library's entry points handed to it."""
    global _binding
    if _binding is None:
        from . import lib
        L = lib()
        try:
            from . import _paged
        except ImportError as e:
            raise ImportError(f"{e}: build it with `python -m thinned_softmax_attention_b200.build`") from e
        _paged.bind(*(ctypes.cast(getattr(L, f"thin_attn_paged_{f}"), ctypes.c_void_p).value
                      for f in ("plan", "release", "append", "attention_workspace", "attention")))
        _binding = _paged
    return _binding


def _raise(status: int):
    from . import _check
    _check(status)


class PagedPlan(NamedTuple):
    """A step's places.  ``lengths`` (R) and ``n_free`` (1) after the step; ``cu`` (R + 1) the prefix
    sums of the new lengths; per token of the step ``slots`` int64, ``rows`` (its request) and
    ``context`` (the keys it sees, itself among them), -1, -1 and 0 where there is none; ``status``
    (R): 0 placed, 1 out of pages, 2 table row too narrow or a negative length, 3 behind max_tokens (a
    request without new tokens too, where those before it fill the step)."""
    lengths: torch.Tensor
    n_free: torch.Tensor
    cu: torch.Tensor
    slots: torch.Tensor
    rows: torch.Tensor
    context: torch.Tensor
    status: torch.Tensor


def paged_plan(lengths: torch.Tensor, new: torch.Tensor, table: torch.Tensor, free: torch.Tensor, n_free: torch.Tensor,
               page: int, max_tokens: int, inplace: bool = False) -> PagedPlan:
    """Block tables and slots of a step that gives request r ``new[r]`` more tokens, on the device.

    lengths, new (R) int32; table (R, W) int32, whose fresh entries are written; free int32, its
    first ``n_free[0]`` entries the free pages (the last one is taken first).  Requests are served
    in order; one that finds no room keeps its length and gets nothing (``status``).  The step's
    tokens are laid out request by request, ``max_tokens`` places in all.  ``lengths`` and
    ``n_free`` themselves change only with ``inplace=True``."""
    got = _calls().plan(lengths, new, table, free, n_free, page, max_tokens, inplace)
    if type(got) is int:
        _raise(got)
    return PagedPlan._make(got)


def paged_release(keep: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor, free: torch.Tensor,
                  n_free: torch.Tensor, page: int) -> None:
    """Shorten request r to ``keep[r]`` tokens (0: it has ended; negative: as it is) and give the pages
    behind them back; lengths, table, free and n_free change in place."""
    status = _calls().release(keep, lengths, table, free, n_free, page)
    if status:
        _raise(status)


def paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, *,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 bounds: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> None:
    """Write k (N, H, E) and v (N, H, D) into their slots; a slot outside the pool (-1) is skipped.

    float8_e4m3fn pages hold x / scale[h], rounded to the nearest value, at most 448 in magnitude.  k and
    v may not be rows that the call writes.
    ``bounds`` = (int8 (n_pages, H, 2, E), int8 (n_pages, H)): the pages' key bounds for
    ``paged_sparse_attention``, widened by the new keys, or started anew where a page's first slot
    is written; the tokens of one page must then be neighbours, as ``paged_plan`` lays them, with no skipped
    one between them (to take tokens back, shorten the request: ``paged_release``)."""
    lohi, exps = (None, None) if bounds is None else bounds
    status = _calls().append(k, v, slots, k_pages, v_pages, k_scale, v_scale, lohi, exps)
    if status:
        _raise(status)


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                    lengths: torch.Tensor, *, rows: Optional[torch.Tensor] = None, window: int = 0,
                    scale: Optional[float] = None, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, return_lse: bool = False):
    """Attention of query tokens q (N, Hq, E) over the paged cache: out (N, Hq, D), or (out, lse) with
    ``return_lse=True`` (lse (N, Hq) fp32, implied by a given ``lse``).

    Token n belongs to request ``rows[n]`` (without ``rows``: request n) and sees its first
    ``lengths[n]`` keys, with ``window`` the last ``window`` of those.  Several tokens of a request
    are several rows of q with lengths that grow by one (``paged_plan``'s ``rows`` and ``context``).  One that sees
    nothing gets zeros and -inf; one whose row is negative is padding and leaves its rows of
    ``out`` and ``lse`` as they were (zeros in buffers made here).
    ``scale`` (without it 1 / sqrt(E)) is positive and at most 2.3e38.
    The keys are read once per query token: made for decode and short drafts, not for long prompts."""
    got = _calls().attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, window, None, None, 0, 0, 0, out, lse,
                             return_lse, False)
    if type(got) is int:
        _raise(got)
    return got[0] if got[1] is None else got[:2]


def paged_sparse_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                           lengths: torch.Tensor, bounds: Tuple[torch.Tensor, torch.Tensor], top: int, *, first: int = 1,
                           last: int = 1, rows: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           return_lse: bool = False, return_pages: bool = False):
    """``paged_attention`` over at most ``top`` pages per token and key head: the request's first
    ``first`` and last ``last`` ones, and those whose ``bounds`` (``paged_append``) promise the largest
    q . k to any of the head's queries.  Returns out, then lse and pages as asked; pages (N, H, top)
    int32 holds the chosen pages' places in the request in ascending order, then -1."""
    if top < 1:
        raise ValueError(f"top={top}: expected at least one page")
    got = _calls().attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, 0, *bounds, top, first, last, out, lse,
                             return_lse, return_pages)
    if type(got) is int:
        _raise(got)
    out, lse, pages = got
    got = (out,) + ((lse,) if lse is not None else ()) + ((pages,) if return_pages else ())
    return got if len(got) > 1 else out


class PagedAttentionCache:
    """A pool of cache pages and the block tables of up to ``max_requests`` requests.

    ``plan``, ``append``, ``attend``, ``attend_sparse`` and ``release`` are the module's functions over the cache's
    own tensors: ``k_pages``, ``v_pages``, ``table``, ``lengths``, ``free``, ``n_free`` and, with ``bounds=True``,
    ``bounds``.  They are updated in place, so a captured step replays on the cache as it then
    stands.  ``cache_dtype=torch.float8_e4m3fn`` halves the pool; ``k_scale`` and ``v_scale`` (H) fp32 are
    then required.  One cache's calls share these tensors: issue them on one stream, or order the
    streams."""

    def __init__(self, n_pages: int, page: int, H: int, E: int, D: int, dtype: torch.dtype, max_requests: int,
                 max_length: int, *, cache_dtype: Optional[torch.dtype] = None, bounds: bool = False,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, device: int = 0):
        dev = torch.device("cuda", device)
        ct = cache_dtype or dtype
        if min(n_pages, page, H, E, D, max_requests, max_length) < 1:
            raise ValueError(f"n_pages={n_pages} page={page} H={H} E={E} D={D} max_requests={max_requests} max_length={max_length}: "
                             "all must be >= 1")
        if (ct == torch.float8_e4m3fn) != (k_scale is not None and v_scale is not None):
            raise ValueError("k_scale and v_scale go with float8_e4m3fn pages, and those need them")
        self.dtype, self.device, self.page, self.scale = dtype, dev, page, scale
        self.k_scale, self.v_scale = k_scale, v_scale
        self.k_pages = torch.zeros((n_pages, H, page, E), dtype=ct, device=dev)
        self.v_pages = torch.zeros((n_pages, H, page, D), dtype=ct, device=dev)
        self.bounds = None
        if bounds:
            self.bounds = (torch.zeros((n_pages, H, 2, E), dtype=torch.int8, device=dev),
                           torch.zeros((n_pages, H), dtype=torch.int8, device=dev))
        self.table = torch.full((max_requests, -(-max_length // page)), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(max_requests, dtype=torch.int32, device=dev)
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=dev)
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=dev)

    def plan(self, new: torch.Tensor, max_tokens: int) -> PagedPlan:
        return paged_plan(self.lengths, new, self.table, self.free, self.n_free, self.page, max_tokens, inplace=True)

    def release(self, keep: torch.Tensor) -> None:
        paged_release(keep, self.lengths, self.table, self.free, self.n_free, self.page)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
        paged_append(k, v, slots, self.k_pages, self.v_pages, k_scale=self.k_scale, v_scale=self.v_scale, bounds=self.bounds)

    def attend(self, q: torch.Tensor, *, rows: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
               window: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               return_lse: bool = False):
        """q (max_requests, Hq, E), one token per request that sees all of its keys; or with ``rows``
        and ``lengths`` (``plan``'s ``rows`` and ``context``) any tokens."""
        return paged_attention(q, self.k_pages, self.v_pages, self.table, self._seen(rows, lengths), rows=rows, window=window,
                               scale=self.scale, k_scale=self.k_scale, v_scale=self.v_scale, out=out, lse=lse,
                               return_lse=return_lse)

    def attend_sparse(self, q: torch.Tensor, top: int, *, first: int = 1, last: int = 1,
                      rows: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                      return_pages: bool = False):
        if self.bounds is None:
            raise ValueError("attend_sparse needs a cache made with bounds=True")
        return paged_sparse_attention(q, self.k_pages, self.v_pages, self.table, self._seen(rows, lengths), self.bounds, top,
                                      first=first, last=last, rows=rows, scale=self.scale, k_scale=self.k_scale,
                                      v_scale=self.v_scale, out=out, lse=lse, return_lse=return_lse,
                                      return_pages=return_pages)

    def _seen(self, rows, lengths):
        if rows is not None and lengths is None:
            raise ValueError("rows need lengths: the keys that each token sees")
        return self.lengths if lengths is None else lengths
