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
import struct
from functools import lru_cache
from typing import NamedTuple, Optional, Tuple

import torch

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3}
# the argument structs of include/thin_attn.h, field by field
_PLAN = struct.Struct("@I7iPPPqPPPPPPPPP")
_RELEASE = struct.Struct("@I5iPPPqPP")
_APPEND = struct.Struct("@I9iPqqPqqPPqqqPqqqPPPP")
_ATTENTION = struct.Struct("@I16ifPqqPqqqPqqqPqPPPPPPPPqqPPN")

_fns = None
_empty = torch.empty_strided   # half the time of torch.empty for more than one dimension
_stream = torch._C._cuda_getCurrentRawStream   # of a device ordinal; what current_stream(...).cuda_stream reads


def _functions():
    global _fns
    if _fns is None:
        from . import lib
        L = lib()
        L.thin_attn_paged_attention_workspace.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)]
        for f in ("plan", "release", "append", "attention"):
            getattr(L, f"thin_attn_paged_{f}").argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        _fns = L
    return _fns


def _raise(status: int):
    from . import _check
    _check(status)


# The checks below cost a decode step as much as its kernels: they read each tensor's properties once, and
# put messages together only when one of them fails.
def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _place(t: torch.Tensor) -> str:
    return f"{t.dtype} {tuple(t.shape)} on {t.device}"


def _index(t: torch.Tensor, name: str) -> int:
    """Ordinal of the CUDA device that holds t."""
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return dev


def _vector(t: torch.Tensor, name: str, n: int, dtype: torch.dtype, dev: int) -> int:
    """Address of a contiguous vector of n entries."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} ({n},) on cuda:{dev}, got {_place(t)}")
    return t.data_ptr()


def _table(t: torch.Tensor, dev: int) -> Tuple[int, int, int]:
    """(R, W, ids from row to row) of a block table."""
    shape, strides = t.shape, t.stride()
    if t.dtype is not torch.int32 or t.get_device() != dev or len(shape) != 2 or (shape[1] > 1 and strides[1] != 1):
        raise ValueError(f"table: expected int32 (R, W) with contiguous rows on cuda:{dev}, got {_place(t)}")
    return shape[0], shape[1], strides[0]


def _pool(k_pages: torch.Tensor, v_pages: torch.Tensor, dev: int):
    """(n_pages, H, page, E, D) of the pool and its strides of pages, heads and rows."""
    ks, vs, kt, vt = k_pages.shape, v_pages.shape, k_pages.stride(), v_pages.stride()
    if (len(ks) != 4 or ks[:3] != vs[:3] or len(vs) != 4 or k_pages.dtype is not v_pages.dtype or k_pages.get_device() != dev
            or v_pages.get_device() != dev or kt[3] != 1 or vt[3] != 1):
        raise ValueError(f"k_pages (n_pages, H, page, E) and v_pages (n_pages, H, page, D): expected one type on cuda:{dev} and a "
                         f"contiguous last axis, got {_place(k_pages)} and {_place(v_pages)}")
    return ks, vs[3], kt, vt


def _types(dtype: torch.dtype, cache: torch.dtype) -> Tuple[int, int]:
    dt, ct = _DTYPES.get(dtype, 3), _DTYPES.get(cache, -1)
    if dt == 3:
        raise ValueError(f"dtype {dtype}: expected float32, bfloat16 or float16")
    if ct != dt and (ct != 3 or dt == 0):
        raise ValueError(f"pages of {cache} with {dtype}: expected {dtype}, or float8_e4m3fn with bfloat16 or float16")
    return dt, ct


def _scales(k_scale, v_scale, ct: int, H: int, dev: int) -> Tuple[int, int]:
    if ct != 3:
        _need(k_scale is None and v_scale is None, "k_scale and v_scale belong to float8_e4m3fn pages")
        return 0, 0
    _need(k_scale is not None and v_scale is not None, "float8_e4m3fn pages need k_scale and v_scale")
    return _vector(k_scale, "k_scale", H, torch.float32, dev), _vector(v_scale, "v_scale", H, torch.float32, dev)


def _bounds(bounds, n_pages: int, H: int, E: int, dev: int) -> Tuple[int, int]:
    lohi, exps = bounds
    if lohi.dtype is not torch.int8 or lohi.get_device() != dev or lohi.shape != (n_pages, H, 2, E) or not lohi.is_contiguous():
        raise ValueError(f"bounds[0]: expected contiguous int8 {(n_pages, H, 2, E)} on cuda:{dev}, got {_place(lohi)}")
    if exps.dtype is not torch.int8 or exps.get_device() != dev or exps.shape != (n_pages, H) or not exps.is_contiguous():
        raise ValueError(f"bounds[1]: expected contiguous int8 {(n_pages, H)} on cuda:{dev}, got {_place(exps)}")
    return lohi.data_ptr(), exps.data_ptr()


class PagedPlan(NamedTuple):
    """A step's places.  ``lengths`` (R) and ``n_free`` (1) after the step; ``cu`` (R + 1) the prefix
    sums of the new lengths; per token of the step ``slots`` int64, ``rows`` (its request) and
    ``context`` (the keys it sees, itself among them), -1, -1 and 0 where there is none; ``status``
    (R): 0 placed, 1 out of pages, 2 table row too narrow or a negative length, 3 behind max_tokens."""
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
    dev = _index(lengths, "lengths")
    R, T = lengths.numel(), max_tokens
    i32 = torch.int32
    at = _vector(lengths, "lengths", R, i32, dev), _vector(new, "new", R, i32, dev)
    rows_, W, row = _table(table, dev)
    n_pages = free.numel()
    pool = _vector(free, "free", n_pages, i32, dev), _vector(n_free, "n_free", 1, i32, dev)
    if rows_ != R or T < 0 or page < 1:
        raise ValueError(f"table of {rows_} rows, {R} requests, page={page}, max_tokens={T}: expected a row per request, page >= 1, "
                         "max_tokens >= 0")
    device = lengths.device
    slots = _empty((T,), (1,), dtype=torch.int64, device=device)
    sizes = (T, T, R + 1, R) if inplace else (T, T, R + 1, R, R, 1)
    parts = torch.unsafe_split_with_sizes(_empty((sum(sizes),), (1,), dtype=i32, device=device), sizes)   # one allocation
    rows, context, cu, status = parts[:4]
    lengths_out, n_free_out = (lengths, n_free) if inplace else parts[4:]
    p = _PLAN.pack(_PLAN.size, dev, R, W, page, n_pages, T, 0, *at, table.data_ptr(), row, *pool, lengths_out.data_ptr(),
                   n_free_out.data_ptr(), cu.data_ptr(), slots.data_ptr(), rows.data_ptr(), context.data_ptr(),
                   status.data_ptr())
    s = _functions().thin_attn_paged_plan(p, _stream(dev))
    if s:
        _raise(s)
    return PagedPlan(lengths_out, n_free_out, cu, slots, rows, context, status)


def paged_release(keep: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor, free: torch.Tensor,
                  n_free: torch.Tensor, page: int) -> None:
    """Shorten request r to ``keep[r]`` tokens (0: it has ended; negative: as it is) and give the pages
    behind them back; lengths, table, free and n_free change in place."""
    dev = _index(lengths, "lengths")
    R, i32 = lengths.numel(), torch.int32
    at = _vector(keep, "keep", R, i32, dev), _vector(lengths, "lengths", R, i32, dev)
    rows, W, row = _table(table, dev)
    _need(rows == R and page >= 1, f"table of {rows} rows, {R} requests, page={page}: expected a row per request, page >= 1")
    pool = _vector(free, "free", free.numel(), i32, dev), _vector(n_free, "n_free", 1, i32, dev)
    p = _RELEASE.pack(_RELEASE.size, dev, R, W, page, free.numel(), *at, table.data_ptr(), row, *pool)
    s = _functions().thin_attn_paged_release(p, _stream(dev))
    if s:
        _raise(s)


def paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, *,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 bounds: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> None:
    """Write k (N, H, E) and v (N, H, D) into their slots; a slot outside the pool (-1) is skipped.

    float8_e4m3fn pages hold x / scale[h], rounded to the nearest value, at most 448 in magnitude.
    ``bounds`` = (int8 (n_pages, H, 2, E), int8 (n_pages, H)): the pages' key bounds for
    ``paged_sparse_attention``, widened by the new keys, or started anew where a page's first slot
    is written; the tokens of one page must then be neighbours, as ``paged_plan`` lays them."""
    dev = _index(k, "k")
    (P, H, page, E), D, kt, vt = _pool(k_pages, v_pages, dev)
    N, kst, vst = k.shape[0], k.stride(), v.stride()
    if (k.shape != (N, H, E) or v.shape != (N, H, D) or k.dtype is not v.dtype or v.get_device() != dev or kst[2] != 1
            or vst[2] != 1):
        raise ValueError(f"k and v: expected {(N, H, E)} and {(N, H, D)} of one type on cuda:{dev} with a contiguous last axis, got "
                         f"{_place(k)} and {_place(v)}")
    at = _vector(slots, "slots", N, torch.int64, dev)
    dt, ct = _types(k.dtype, k_pages.dtype)
    ks, vs = _scales(k_scale, v_scale, ct, H, dev)
    b, x = (0, 0) if bounds is None else _bounds(bounds, P, H, E, dev)
    p = _APPEND.pack(_APPEND.size, dev, dt, ct, N, H, E, D, page, P, k.data_ptr(), kst[0], kst[1], v.data_ptr(), vst[0], vst[1], at,
                     k_pages.data_ptr(), kt[0], kt[1], kt[2], v_pages.data_ptr(), vt[0], vt[1], vt[2], ks, vs, b, x)
    s = _functions().thin_attn_paged_append(p, _stream(dev))
    if s:
        _raise(s)


@lru_cache(maxsize=1024)
def _workspace_bytes(dt, ct, N, R, W, Hq, H, E, D, page, P, window, top, first, last, has_rows) -> int:
    p = _ATTENTION.pack(_ATTENTION.size, 0, dt, ct, N, R, W, Hq, H, E, D, page, P, window, top, first, last, 0.0,
                        *[0] * 14, int(has_rows), *[0] * 11)   # of the pointers only whether there are rows counts
    n = ctypes.c_size_t()
    _raise(_functions().thin_attn_paged_attention_workspace(p, ctypes.byref(n)))
    return n.value


def _attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, window, bounds, top, first, last, out,
               lse, return_lse, return_pages):
    """(out, lse, pages): the last two None unless asked for."""
    dev = _index(q, "q")
    (P, H, page, E), D, kt, vt = _pool(k_pages, v_pages, dev)
    shape, qst = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != E or qst[2] != 1 or shape[1] % H or not shape[1]:
        raise ValueError(f"q: expected (N, Hq, {E}) with a contiguous last axis, Hq a multiple of {H}, got {_place(q)}")
    N, Hq, _ = shape
    R, W, row = _table(table, dev)
    seen = _vector(lengths, "lengths", N, torch.int32, dev)
    of = 0 if rows is None else _vector(rows, "rows", N, torch.int32, dev)
    dt, ct = _types(q.dtype, k_pages.dtype)
    ks, vs = _scales(k_scale, v_scale, ct, H, dev)
    device = q.device
    # rows of padding tokens are not written: zeros there where the buffer is made here
    if out is None:
        out = _empty((N, Hq, D), (Hq * D, D, 1), dtype=q.dtype, device=device)
        if rows is not None:
            out.zero_()
    ost = out.stride()
    if out.shape != (N, Hq, D) or out.dtype is not q.dtype or out.get_device() != dev or ost[2] != 1:
        raise ValueError(f"out: expected {q.dtype} {(N, Hq, D)} with a contiguous last axis on cuda:{dev}, got {_place(out)}")
    if lse is None:
        if return_lse:
            lse = _empty((N, Hq), (Hq, 1), dtype=torch.float32, device=device)
            if rows is not None:
                lse.zero_()
    elif lse.shape != (N, Hq) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError(f"lse: expected contiguous float32 {(N, Hq)} on cuda:{dev}, got {_place(lse)}")
    b, x = (0, 0) if bounds is None else _bounds(bounds, P, H, E, dev)
    pages = None
    if return_pages:
        pages = _empty((N, H, top), (H * top, top, 1), dtype=torch.int32, device=device)
        if rows is not None:
            pages.fill_(-1)
    n = _workspace_bytes(dt, ct, N, R, W, Hq, H, E, D, page, P, window, top, first, last, rows is not None)
    # scratch of this call alone: the caching allocator hands it on in stream order, and a capture
    # gets its own from the graph's pool
    ws = _empty((n,), (1,), dtype=torch.uint8, device=device)
    p = _ATTENTION.pack(_ATTENTION.size, dev, dt, ct, N, R, W, Hq, H, E, D, page, P, window, top, first, last,
                        0.0 if scale is None else scale, q.data_ptr(), qst[0], qst[1], k_pages.data_ptr(), kt[0], kt[1], kt[2],
                        v_pages.data_ptr(), vt[0], vt[1], vt[2], table.data_ptr(), row, seen, of, ks, vs, b, x,
                        0 if pages is None else pages.data_ptr(), out.data_ptr(), ost[0], ost[1],
                        0 if lse is None else lse.data_ptr(), ws.data_ptr(), n)
    s = _functions().thin_attn_paged_attention(p, _stream(dev))
    if s:
        _raise(s)
    return out, lse, pages


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
    The keys are read once per query token: made for decode and short drafts, not for long prompts."""
    out, lse, _ = _attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, window, None, 0, 0, 0, out, lse,
                             return_lse, False)
    return out if lse is None else (out, lse)


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
    _need(top >= 1, f"top={top}: expected at least one page")
    out, lse, pages = _attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, 0, bounds, top, first, last,
                                 out, lse, return_lse, return_pages)
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
        _need(min(n_pages, page, H, E, D, max_requests, max_length) >= 1,
              f"n_pages={n_pages} page={page} H={H} E={E} D={D} max_requests={max_requests} max_length={max_length}: all >= 1")
        _scales(k_scale, v_scale, _types(dtype, ct)[1], H, device)
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
        _need(self.bounds is not None, "attend_sparse needs a cache made with bounds=True")
        return paged_sparse_attention(q, self.k_pages, self.v_pages, self.table, self._seen(rows, lengths), self.bounds, top,
                                      first=first, last=last, rows=rows, scale=self.scale, k_scale=self.k_scale,
                                      v_scale=self.v_scale, out=out, lse=lse, return_lse=return_lse,
                                      return_pages=return_pages)

    def _seen(self, rows, lengths):
        _need(rows is None or lengths is not None, "rows need lengths: the keys that each token sees")
        return self.lengths if lengths is None else lengths
