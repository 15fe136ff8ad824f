"""Measured cases of the paged-cache operators, with each operator's plain form and its value in 64 bits.

The operators serve many requests of different lengths from one pool of cache pages:

  plan       block tables, slot maps and the free-page stack of a step, from request lengths
  append     new keys and values into their slots (kept as they are, or in e4m3 with a scale per
             head), with the bounds of every page's keys that block selection scores
  attention  one query token against its request's cached keys, through the block table
  sparse     the same over the pages that a cheap score selects for the query

Layouts: q (N, Hq, E); k_pages (P, H, page, E), v_pages (P, H, page, D); table (R, W) int32 page
ids; lengths (N) int32 keys that query token n sees; slot = page id * page + offset.  Query head
h * (Hq / H) + g reads key head h.

Page bounds.  For the keys k of a page and head, as the cache holds them: m = max |k|, x the least
integer in [-40, 48] with 127 * 2^x >= m (48 if there is none), lo = floor(min k / 2^x) and
hi = ceil(max k / 2^x) as int8 (clamped to +-127; a NaN counts as 0).  The query is rounded alike:
q8 = round(q / 2^y), half to even, y from max |q| of its head.  A page's score for key head h is
max over the group's heads g of 2^(x + y) * sum_e max(q8 * hi, q8 * lo), a whole number times a
power of two, so that it has one value however it is summed.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
_X_MIN, _X_MAX = -40, 48


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _plan_case(requests, page, lo, hi, new, room, tight=False, lens=1):
    return {"op": "plan", "requests": requests, "page": page, "lo": lo, "hi": hi, "new": new, "room": room,
            "tight": tight, "lens": lens}


def _append_case(requests, tokens, heads, E, D, page, dtype, cache, bounds, pad=0, lens=1):
    return {"op": "append", "requests": requests, "tokens": tokens, "heads": heads, "E": E, "D": D, "page": page,
            "dtype": dtype, "cache": cache, "bounds": bounds, "pad": pad, "lens": lens}


def _attention_case(requests, lo, hi, q_heads, heads, E, D, page, dtype, cache, draft=1, window=0, lens=1):
    return {"op": "attention", "requests": requests, "lo": lo, "hi": hi, "q_heads": q_heads, "heads": heads, "E": E,
            "D": D, "page": page, "dtype": dtype, "cache": cache, "draft": draft, "window": window, "lens": lens}


def _sparse_case(requests, lo, hi, q_heads, heads, E, D, page, dtype, cache, top, draft=1, first=1, last=1, lens=1):
    return {"op": "sparse", "requests": requests, "lo": lo, "hi": hi, "q_heads": q_heads, "heads": heads, "E": E,
            "D": D, "page": page, "dtype": dtype, "cache": cache, "top": top, "draft": draft, "first": first,
            "last": last, "lens": lens}


def listed():
    return [
        # a decode step of a busy server: every request grows by one token, a few need a fresh page
        {"name": "plan_step", **_plan_case(64, 16, 1, 32768, 1, 64)},
        # admission of prompts in chunks: hundreds of requests, up to 1024 new tokens each, the pool
        # too small for the last of them
        {"name": "plan_prompts", **_plan_case(512, 16, 0, 8192, 1024, 65536, tight=True, lens=2)},
        # the keys and values of one decode step
        {"name": "append_step", **_append_case(64, 64, 8, 128, 128, 16, "bf16", "bf16", True)},
        # prompts of a few thousand tokens each into fresh and half-full pages
        {"name": "append_prompts", **_append_case(12, 16384, 8, 128, 128, 64, "bf16", "bf16", True, lens=3)},
        # a ragged chunk with padding rows into an 8-bit cache
        {"name": "append_8bit", **_append_case(5, 1999, 8, 128, 128, 32, "fp16", "e4m3", True, pad=49, lens=4)},
        # one conversation early on, a key head per query head (the Express workloads' 32 heads)
        {"name": "attention_one", **_attention_case(1, 500, 500, 32, 32, 128, 128, 16, "bf16", "bf16")},
        # a mixed batch: lengths from one token to 8192, four query heads to a key head
        {"name": "attention_mixed", **_attention_case(48, 1, 8192, 32, 8, 128, 128, 16, "bf16", "bf16", lens=5)},
        # long documents up to the Express 128K workload's length
        {"name": "attention_long", **_attention_case(16, 65536, 131072, 32, 8, 128, 128, 64, "bf16", "bf16", lens=6)},
        # an 8-bit cache read by bf16 queries, eight query heads to a key head
        {"name": "attention_8bit", **_attention_case(40, 100, 32768, 32, 4, 128, 128, 32, "bf16", "e4m3", lens=7)},
        # fp32 with the BigGAN layer's widths, an odd page size and a sliding window
        {"name": "attention_odd", **_attention_case(7, 0, 5000, 12, 3, 64, 256, 20, "fp32", "fp32", window=1000, lens=8)},
        # one long conversation, 64 of 1024 pages
        {"name": "sparse_one", **_sparse_case(1, 32768, 32768, 32, 8, 128, 128, 32, "bf16", "bf16", 64)},
        # a batch of long documents, 32 pages of up to 2048 each
        {"name": "sparse_batch", **_sparse_case(32, 4096, 131072, 32, 8, 128, 128, 64, "bf16", "bf16", 32, lens=9)},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "sparse"])
    lens = rng.randrange(1, 1 << 30)
    if op == "plan":
        new = _log(rng, 1, 1024)
        requests = _log(rng, 1, min(2048, 131072 // new))
        room = _log(rng, max(1, requests * new // 8), min(65536, max(2, requests * new)))
        return _plan_case(requests, rng.choice([1, 8, 16, 20, 64, 128]), rng.choice([0, 1, 100]), _log(rng, 100, 32768),
                          new, room, tight=rng.random() < 0.4, lens=lens)
    heads, group = rng.choice([(32, 1), (8, 4), (4, 8), (1, 16), (3, 4), (8, 1), (8, 5), (2, 16), (1, 32)])
    E, D = rng.choice([(128, 128), (128, 128), (64, 64), (64, 256), (128, 64), (192, 128), (96, 96), (256, 256)])
    page = rng.choice([8, 16, 16, 20, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    cache = "e4m3" if dtype != "fp32" and rng.random() < 0.3 else dtype
    if op == "append":
        most = 16384 * 8 * 256 * 2 // (heads * (E + D) * _SIZE[dtype])
        tokens = _log(rng, 1, min(16384, most))
        return _append_case(_log(rng, 1, tokens), tokens, heads, E, D, page, dtype, cache, rng.random() < 0.7,
                            pad=rng.choice([0, 0, 1, 37]), lens=lens)
    # keys of all query tokens together: no more bytes than the longest listed batch's
    most = 16 * 98304 * 8 * 256 * 2 // (heads * (E + D) * _SIZE[cache])
    hi = _log(rng, 1, 131072)
    draft = rng.choice([1, 1, 1, 2, 4])
    requests = _log(rng, 1, max(1, min(256, most // (4 * hi * draft * max(1, group // 8)))))
    lo = rng.choice([0, 1, max(1, hi // 4), hi])
    if op == "attention":
        return _attention_case(requests, lo, hi, heads * group, heads, E, D, page, dtype, cache, draft,
                               rng.choice([0, 0, 1, 100, 4000]), lens)
    first, last = rng.choice([(1, 1), (0, 1), (2, 3)])
    return _sparse_case(requests, lo, hi, heads * group, heads, E, D, page, dtype, cache, _log(rng, 5, 128), draft,
                        first, last, lens)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _spread(lens, n, lo, hi):
    """n whole numbers between lo and hi, spread over their logarithm, both ends among them: the case's alone."""
    r = random.Random(lens)
    v = [int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _plan_sizes(case):
    lengths = _spread(case["lens"], case["requests"], case["lo"], case["hi"])
    new = _spread(case["lens"] + 1, case["requests"], min(1, case["new"]), case["new"])
    if case["new"] > 1 and len(new) > 2:
        new[len(new) // 2] = 0   # a request that waits this step out
    return lengths, new


def _ceil(a, b):
    return -(-a // b)


def _shuffled(v, seed):
    v = list(v)
    random.Random(seed * 7919 + 13).shuffle(v)
    return v


def _tables(lengths, page, pages, gen, dev, width):
    """Block tables over a shuffled pool, and the pages that stay free."""
    L = torch.tensor(lengths, device=dev)
    used = (L + page - 1) // page
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device=dev)
    mask = torch.arange(width, device=dev)[None, :] < used[:, None]
    n = int(used.sum())
    table[mask] = order[:n]
    return table, order[n:].clone()


def _pow2(x):
    """2^x for whole x in [-126, 127], exactly."""
    return ((x.int() + 127) << 23).view(torch.float32)


def _bounds(keys, dim):
    """Bounds over dimension `dim` of keys (..., E), as whole numbers in floats, and their exponent."""
    k = torch.nan_to_num(keys, nan=0.0)
    lo, hi = k.amin(dim).float(), k.amax(dim).float()
    x = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    lo8 = torch.floor(lo * _pow2(-x)[..., None]).clamp(-127, 127)
    hi8 = torch.ceil(hi * _pow2(-x)[..., None]).clamp(-127, 127)
    return lo8, hi8, x


def _exponent(m):
    """The least integer x in [-40, 48] with 127 * 2^x >= m, as a float."""
    f, x = torch.frexp(m.float())
    x = torch.where(f <= 127 / 128, x - 7, x - 6)
    x = torch.where(m > 0, x, torch.full_like(x, _X_MIN))
    return torch.where(torch.isinf(m), torch.full_like(x, _X_MAX), x).clamp(_X_MIN, _X_MAX).float()


def _prepare_plan(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    page = case["page"]
    lengths, new = _plan_sizes(case)
    pairs = _shuffled(zip(lengths, new), seed)
    lengths, new = [a for a, _ in pairs], [b for _, b in pairs]
    used = sum(_ceil(a, page) for a in lengths)
    need = sum(_ceil(a + b, page) - _ceil(a, page) for a, b in pairs)
    pages = used + (need * 3 // 4 if case["tight"] else need + need // 8 + 8)
    width = _ceil(max(a + b for a, b in pairs), page) + 1
    table, free = _tables(lengths, page, max(1, pages), gen, dev, width)
    stack = torch.zeros(max(1, pages), dtype=torch.int32, device=dev)
    stack[:free.numel()] = free
    return {"case": case, "lengths": torch.tensor(lengths, dtype=torch.int32, device=dev),
            "new": torch.tensor(new, dtype=torch.int32, device=dev), "table": table, "free": stack,
            "n_free": torch.tensor([free.numel()], dtype=torch.int32, device=dev)}


def _prepare_append(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    R, page, H, E, D = case["requests"], case["page"], case["heads"], case["E"], case["D"]
    r = random.Random(case["lens"])
    cut = sorted(r.randrange(case["tokens"] + 1) for _ in range(R - 1)) if R < case["tokens"] else list(range(1, R))
    new = [b - a for a, b in zip([0] + cut, cut + [case["tokens"]])]
    pairs = _shuffled([(r.randrange(4 * page), b) for b in new], seed)
    before, new = [a for a, _ in pairs], [b for _, b in pairs]
    total = [a + b for a, b in zip(before, new)]
    pages = sum(_ceil(t, page) for t in total) + 8
    table, _ = _tables(total, page, pages, gen, dev, max(1, _ceil(max(total), page)))
    row = torch.repeat_interleave(torch.arange(R), torch.tensor(new)).to(dev)
    at = torch.cat([torch.arange(a, a + b) for a, b in zip(before, new)]).to(dev)
    slots = table[row, at // page].long() * page + at % page
    if case["pad"]:
        slots = torch.cat([slots, torch.full((case["pad"],), -1, device=dev)])
    n = slots.numel()
    dt, ct = _TYPES[case["dtype"]], _TYPES[case["cache"]]

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    k, v = rnd(n, H, E).to(dt), rnd(n, H, D).to(dt)
    s = {"case": case, "k": k, "v": v, "slots": slots, "k_scale": None, "v_scale": None, "bounds": None}
    if case["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = rnd(H).abs() * 0.02 + 0.01, rnd(H).abs() * 0.02 + 0.01
    kp, vp = rnd(pages, H, page, E), rnd(pages, H, page, D)
    if s["k_scale"] is not None:
        kp, vp = kp / s["k_scale"][:, None, None], vp / s["v_scale"][:, None, None]
        kp, vp = kp.clamp(-448, 448), vp.clamp(-448, 448)
    s["k_pages"], s["v_pages"] = kp.to(ct), vp.to(ct)
    if case["bounds"]:
        lo, hi, x = _bounds(s["k_pages"].float(), 2)
        s["bounds"] = (torch.stack([lo, hi], 2).to(torch.int8), x.to(torch.int8))
    return s


def _prepare_attention(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    R, page, H, E, D, draft = (case[c] for c in ("requests", "page", "heads", "E", "D", "draft"))
    Hq, dt, ct = case["q_heads"], _TYPES[case["dtype"]], _TYPES[case["cache"]]
    lengths = _shuffled(_spread(case["lens"], R, case["lo"], case["hi"]), seed)
    width = max(1, _ceil(max(lengths), page))
    pages = sum(_ceil(a, page) for a in lengths) + 8
    table, _ = _tables(lengths, page, pages, gen, dev, width)
    wide = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16

    def rnd(*shape, t=wide):
        return torch.randn(*shape, generator=gen, device=dev, dtype=t)

    # the keys of a page lie about a direction of their own, and a query looks towards one page's
    near = rnd(pages, H, 1, E)
    kp, vp = rnd(pages, H, page, E).add_(near), rnd(pages, H, page, D)
    s = {"case": case, "k_scale": None, "v_scale": None, "table": table, "rows": None}
    if case["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = rnd(H, t=torch.float32).abs() * 0.02 + 0.02, rnd(H, t=torch.float32).abs() * 0.02 + 0.02
        kp = kp.div_(s["k_scale"][:, None, None]).clamp_(-448, 448)
        vp = vp.div_(s["v_scale"][:, None, None]).clamp_(-448, 448)
    s["k_pages"], s["v_pages"] = kp.to(ct), vp.to(ct)
    del kp, vp
    row = torch.arange(R, device=dev).repeat_interleave(draft)
    L = torch.tensor(lengths, device=dev)
    s["lengths"] = (L[row] - draft + 1 + torch.arange(draft, device=dev).repeat(R)).clamp(min=0).to(torch.int32)
    if draft > 1:
        s["rows"] = row.to(torch.int32)
    seen = (s["lengths"].long() + page - 1) // page
    goal = (torch.rand(R * draft, generator=gen, device=dev) * seen).long()
    goal = table[row, goal.clamp(max=width - 1)].long().clamp(min=0)
    q = rnd(R * draft, H, Hq // H, E) + 0.35 * near[goal]
    s["q"] = q.reshape(R * draft, Hq, E).to(dt)
    if case["op"] == "sparse":
        b = [_bounds(c.to(wide), 2) for c in s["k_pages"].split(4096)]
        s["bounds"] = (torch.cat([torch.stack([lo, hi], 2).to(torch.int8) for lo, hi, _ in b]),
                       torch.cat([x.to(torch.int8) for _, _, x in b]))
    return s


def prepare(case, seed):
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    if case["op"] == "append":
        return _prepare_append(case, seed)
    return _prepare_attention(case, seed)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention,
            "sparse": _plain_sparse}[state["case"]["op"]](state)


def _own(s):
    import thinned_softmax_attention_b200 as T
    c = s["case"]
    if c["op"] == "plan":
        p = T.paged_plan(s["lengths"], s["new"], s["table"], s["free"], s["n_free"], c["page"], c["room"])
        return {"lengths": p.lengths, "n_free": p.n_free, "cu": p.cu, "slots": p.slots, "rows": p.rows,
                "context": p.context, "status": p.status, "table": s["table"]}
    if c["op"] == "append":
        T.paged_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], k_scale=s["k_scale"],
                       v_scale=s["v_scale"], bounds=s["bounds"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "bounds": s["bounds"]}
    if c["op"] == "attention":
        out, lse = T.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], rows=s["rows"],
                                     window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
        return {"out": out, "lse": lse}
    out, lse, pages = T.paged_sparse_attention(
        s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["bounds"], c["top"], first=c["first"],
        last=c["last"], rows=s["rows"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True, return_pages=True)
    return {"out": out, "lse": lse, "pages": pages}


def _plain_plan(s):
    """Requests are served in order: one whose pages, table row or token room run out gets nothing (status 1, 2, 3),
    and once the pool is short no later request gets a page.  Pages come off the top of the free stack."""
    page, room = s["case"]["page"], s["case"]["room"]
    L, n, table = s["lengths"].long(), s["new"].long(), s["table"]
    R, W = table.shape
    have, want = (L + page - 1) // page, (L + n.clamp(min=0) + page - 1) // page
    cu = torch.cat([n.new_zeros(1), n.clamp(min=0).cumsum(0)])
    narrow = (want > W) | (n < 0) | (L < 0)
    late = ~narrow & (cu[1:] > room)
    need = torch.where(narrow | late, torch.zeros_like(want), want - have)
    top = need.cumsum(0)
    short = (need > 0) & (top > s["n_free"].long())
    status = torch.where(narrow, 2, torch.where(late, 3, torch.where(short, 1, 0)))
    placed = status == 0
    at = torch.arange(W, device=L.device)[None, :]
    fresh = placed[:, None] & (at >= have[:, None]) & (at < want[:, None])
    pick = s["n_free"].long() - 1 - ((top - need)[:, None] + at - have[:, None])
    table[:] = torch.where(fresh, s["free"][pick.clamp(0, s["free"].numel() - 1)], table)
    t = torch.arange(room, device=L.device)
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    live = (t < cu[-1]) & placed[row]
    pos = L[row] + t - cu[row]
    slot = table[row, (pos // page).clamp(0, W - 1)].long() * page + pos % page
    none = torch.full_like(t, -1)
    return {"lengths": torch.where(placed, L + n, L).int(),
            "n_free": s["n_free"] - torch.where(placed, need, 0).sum().int(), "cu": cu.int(),
            "slots": torch.where(live, slot, none), "rows": torch.where(live, row, none).int(),
            "context": torch.where(live, pos + 1, torch.zeros_like(pos)).int(), "status": status.int(), "table": table}


def _held(x, scale, like):
    """x as the cache holds it."""
    if scale is None:
        return x.to(like.dtype)
    return (x.float() / scale[:, None]).clamp(-448, 448).to(like.dtype)


def _plain_append(s):
    kp, vp, page = s["k_pages"], s["v_pages"], s["case"]["page"]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    pg, off = slots // page, slots % page
    k = _held(s["k"][live], s["k_scale"], kp)
    kp[pg, :, off] = k
    vp[pg, :, off] = _held(s["v"][live], s["v_scale"], vp)
    if s["bounds"] is not None:
        # a page whose first slot is written starts anew; another keeps its bounds and widens them
        lohi, exps = s["bounds"]
        touched, which = torch.unique(pg, return_inverse=True)
        anew = torch.zeros(touched.numel(), dtype=torch.bool, device=pg.device)
        anew[which[off == 0]] = True
        step = _pow2(exps[touched].float())[..., None]
        lo = torch.where(anew[:, None, None], math.inf, lohi[touched, :, 0].float() * step)
        hi = torch.where(anew[:, None, None], -math.inf, lohi[touched, :, 1].float() * step)
        kf = torch.nan_to_num(k.float(), nan=0.0)
        idx = which[:, None, None].expand_as(kf)
        lo_k = torch.full_like(lo, math.inf).scatter_reduce(0, idx, kf, "amin")
        hi_k = torch.full_like(hi, -math.inf).scatter_reduce(0, idx, kf, "amax")
        x = _exponent(torch.maximum(lo_k.abs(), hi_k.abs()).amax(-1))
        x = torch.where(anew[:, None], x, torch.maximum(x, exps[touched].float()))
        down = _pow2(-x)[..., None]
        lo = torch.floor(torch.minimum(lo, lo_k) * down).clamp(-127, 127)
        hi = torch.ceil(torch.maximum(hi, hi_k) * down).clamp(-127, 127)
        lohi[touched] = torch.stack([lo, hi], 2).to(torch.int8)
        exps[touched] = x.to(torch.int8)
    return {"k_pages": kp, "v_pages": vp, "bounds": s["bounds"]}


def _softmax_pv(q, K, V, seen, dtype):
    """q (N, H, G, E), K (N, H, S, E), V (N, H, S, D), seen (N, H or 1, S): out (N, H G, D), lse (N, H G)."""
    N, H, G, E = q.shape
    z = (q @ K.transpose(-1, -2)) * (1.0 / math.sqrt(E))
    z = z.masked_fill(~seen[:, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = (p @ torch.where(seen[..., None], V, 0.0)) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    return o.reshape(N, H * G, -1).to(dtype), lse.reshape(N, H * G)


def _cached(pages, ids, scale):
    """Pages ids (N, W) of the pool in 32 bits, (N, H, W * page, width)."""
    x = pages[ids.clamp(min=0)].float()
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
    c, q = s["case"], s["q"]
    H, G = c["heads"], c["q_heads"] // c["heads"]
    ids = (s["table"] if s["rows"] is None else s["table"][s["rows"].long()]).long()
    at = torch.arange(ids.shape[1] * c["page"], device=q.device)[None, :]
    L = s["lengths"].long()[:, None]
    seen = at < L
    if c["window"]:
        seen = seen & (at >= L - c["window"])
    out, lse = _softmax_pv(q.float().reshape(-1, H, G, c["E"]), _cached(s["k_pages"], ids, s["k_scale"]),
                           _cached(s["v_pages"], ids, s["v_scale"]), seen[:, None], q.dtype)
    return {"out": out, "lse": lse}


def _plain_sparse(s):
    c, q = s["case"], s["q"]
    H, G, E, page, top = c["heads"], c["q_heads"] // c["heads"], c["E"], c["page"], c["top"]
    ids = (s["table"] if s["rows"] is None else s["table"][s["rows"].long()]).long()
    N, W = ids.shape
    L = s["lengths"].long()
    n_pages = (L + page - 1) // page
    qf = torch.nan_to_num(q.float().reshape(N, H, G, E), nan=0.0)
    y = _exponent(qf.abs().amax(-1))
    q8 = torch.round(qf * _pow2(-y)[..., None]).clamp(-127, 127)
    lohi, exps = s["bounds"]
    held = ids.clamp(min=0)
    b = lohi[held].float().permute(0, 2, 3, 4, 1)                       # (N, H, 2, E, W), whole numbers
    dot = q8.clamp(min=0) @ b[:, :, 1] + q8.clamp(max=0) @ b[:, :, 0]   # below 2^24: exact in any order
    score = dot * _pow2(exps[held].float().permute(0, 2, 1))[:, :, None] * _pow2(y)[..., None]
    score = score.amax(2)                                               # (N, H, W)
    j = torch.arange(W, device=q.device)
    forced = (j < c["first"]) | (j >= (n_pages - c["last"])[:, None])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((j < n_pages[:, None])[:, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    take = torch.arange(order.shape[-1], device=q.device) < n_pages[:, None, None]
    order = torch.sort(torch.where(take, order, W), dim=-1).values
    got = order < W
    held = torch.gather(ids[:, None].expand(N, H, W), 2, order.clamp(max=W - 1)).clamp(min=0)
    h = torch.arange(H, device=q.device)[None, :, None]
    K, V = s["k_pages"][held, h].float().flatten(2, 3), s["v_pages"][held, h].float().flatten(2, 3)
    if s["k_scale"] is not None:
        K, V = K * s["k_scale"][:, None, None], V * s["v_scale"][:, None, None]
    at = order[..., None] * page + torch.arange(page, device=q.device)
    seen = (got[..., None] & (at < L[:, None, None, None])).flatten(2, 3)
    out, lse = _softmax_pv(q.float().reshape(N, H, G, E), K, V, seen, q.dtype)
    pages = torch.full((N, H, top), -1, dtype=torch.int32, device=q.device)
    pages[..., :order.shape[-1]] = torch.where(got, order, -1).int()
    return {"out": out, "lse": lse, "pages": pages}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "plan":
        lengths, new = _plan_sizes(case)
        R, page = case["requests"], case["page"]
        fresh = sum(_ceil(a + b, page) - _ceil(a, page) for a, b in zip(lengths, new))
        # lengths, new, statuses and sums; free ids in, table entries out; a slot, row and context per token of room
        return {"bytes": R * 20 + fresh * 8 + case["room"] * 16, "flops": R * 8 + case["room"] * 8}
    H, E, D = case["heads"], case["E"], case["D"]
    qb = _SIZE[case["dtype"]]
    if case["op"] == "append":
        rows = case["tokens"] * H
        touched = (case["tokens"] // case["page"] + case["requests"]) * H if case["bounds"] else 0
        return {"bytes": rows * (E + D) * (qb + _SIZE[case["cache"]]) + touched * 2 * (2 * E + 1) + case["tokens"] * 8,
                "flops": rows * (E + D) * (2 if case["cache"] == "e4m3" else 0) + (rows * E * 3 if case["bounds"] else 0)}
    Hq, draft, page = case["q_heads"], case["draft"], case["page"]
    lengths = _spread(case["lens"], case["requests"], case["lo"], case["hi"])
    N = case["requests"] * draft
    io = N * Hq * ((E + D) * qb + 4) + N * 4
    kv = H * (E + D) * _SIZE[case["cache"]]
    if case["op"] == "attention":
        seen = [[max(0, a - draft + 1 + i) for i in range(draft)] for a in lengths]
        if case["window"]:
            keys = sum(min(a, case["window"] + draft - 1) for a in lengths)
            pairs = sum(min(b, case["window"]) for a in seen for b in a)
        else:
            keys, pairs = sum(lengths), sum(b for a in seen for b in a)
        return {"bytes": keys * kv + io + _ceil(keys, page) * 4, "flops": pairs * Hq * 2 * (E + D)}
    pages = [_ceil(a, page) for a in lengths]
    # the drafts of a request may choose the same pages: counted once
    keys = sum(min(a, case["top"] * page) for a in lengths)
    return {"bytes": sum(pages) * (H * (2 * E + 1) + 4) + keys * kv + io + N * H * case["top"] * 4,
            "flops": draft * (sum(pages) * Hq * 4 * E + keys * Hq * 2 * (E + D))}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attention": _exact_attention,
            "sparse": _exact_attention}[case["op"]](s)


def _exact_plan(s):
    page, room = s["case"]["page"], s["case"]["room"]
    lengths, new, table = s["lengths"].tolist(), s["new"].tolist(), s["table"].tolist()
    free = s["free"].tolist()[:int(s["n_free"])]
    width, cu, status = len(table[0]), [0], []
    slots, rows, context = [-1] * room, [-1] * room, [0] * room
    dry = False
    for i, (L, n) in enumerate(zip(list(lengths), new)):
        first = cu[-1]
        cu.append(first + max(0, n))
        have, want = _ceil(L, page), _ceil(L + max(0, n), page)
        if want > width or n < 0 or L < 0:
            status.append(2)
            continue
        if cu[-1] > room:
            status.append(3)
            continue
        if want > have and (dry or want - have > len(free)):
            dry = True
            status.append(1)
            continue
        status.append(0)
        for j in range(have, want):
            table[i][j] = free.pop()
        lengths[i] = L + n
        for t in range(n):
            p = L + t
            slots[first + t], rows[first + t], context[first + t] = table[i][p // page] * page + p % page, i, p + 1

    def whole(v, t=torch.int32):
        return torch.tensor(v, dtype=t, device=s["table"].device)

    return {"lengths": whole(lengths), "n_free": whole([len(free)]), "cu": whole(cu), "slots": whole(slots, torch.int64),
            "rows": whole(rows), "context": whole(context), "status": whole(status), "table": whole(table)}


def _exact_exponent(m):
    """The exponents of a float64 tensor of magnitudes, one by one."""
    x = [next((e for e in range(_X_MIN, _X_MAX) if 127 * 2.0 ** e >= v), _X_MAX) for v in m.flatten().tolist()]
    return torch.tensor(x, dtype=torch.int64, device=m.device).reshape(m.shape)


def _exact_pow2(x):
    return ((x.long() + 1023) << 52).view(torch.float64)


def _exact_append(s):
    page = s["case"]["page"]
    out = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(), "bounds": None}
    rows = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][rows]
    for name, x, scale in (("k_pages", s["k"], s["k_scale"]), ("v_pages", s["v"], s["v_scale"])):
        y = x[rows].double()
        if scale is not None:
            y = (y / scale.double()[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
        out[name][slots // page, :, slots % page] = y
    if s["bounds"] is None:
        return out
    lohi, exps = s["bounds"][0].clone(), s["bounds"][1].clone()
    at = (slots // page).tolist()
    off = (slots % page).tolist()
    runs = [i for i in range(len(at)) if i == 0 or at[i] != at[i - 1]] + [len(at)]
    kept = s["k_pages"].clone()
    kept[slots // page, :, slots % page] = _held(s["k"][rows], s["k_scale"], kept)
    for a, b in zip(runs, runs[1:]):
        keys = torch.nan_to_num(kept[at[a], :, off[a]:off[b - 1] + 1].double(), nan=0.0)   # a run's slots ascend
        x = _exact_exponent(keys.abs().amax((1, 2)))
        lo, hi = keys.amin(1), keys.amax(1)
        if off[a] != 0:
            x0 = exps[at[a]].long()
            lo = torch.minimum(lo, lohi[at[a], :, 0].double() * _exact_pow2(x0)[:, None])
            hi = torch.maximum(hi, lohi[at[a], :, 1].double() * _exact_pow2(x0)[:, None])
            x = torch.maximum(x, x0)
        lohi[at[a], :, 0] = torch.floor(lo / _exact_pow2(x)[:, None]).clamp(-127, 127).to(torch.int8)
        lohi[at[a], :, 1] = torch.ceil(hi / _exact_pow2(x)[:, None]).clamp(-127, 127).to(torch.int8)
        exps[at[a]] = x.to(torch.int8)
    return {**out, "bounds": (lohi, exps)}


def _exact_attention(s):
    c = s["case"]
    H, G, E, page = c["heads"], c["q_heads"] // c["heads"], c["E"], c["page"]
    N = s["q"].shape[0]
    if sum(s["lengths"].tolist()) * H * (E + c["D"]) > 6 << 30:
        return None
    dev = s["q"].device
    outs, lses, chosen = [], [], []
    for n, L in enumerate(s["lengths"].tolist()):
        ids = s["table"][n if s["rows"] is None else int(s["rows"][n])][:_ceil(L, page)].long()
        q = s["q"][n].double().reshape(H, G, E)
        K = s["k_pages"][ids].double().transpose(0, 1).reshape(H, -1, E)[:, :L]
        V = s["v_pages"][ids].double().transpose(0, 1).reshape(H, -1, c["D"])[:, :L]
        if s["k_scale"] is not None:
            K, V = K * s["k_scale"].double()[:, None, None], V * s["v_scale"].double()[:, None, None]
        at = torch.arange(L, device=dev)
        seen = (at >= (L - c["window"] if c.get("window") else 0)).expand(H, L)
        if c["op"] == "sparse":
            pick = torch.full((H, c["top"]), -1, dtype=torch.int32, device=dev)
            if L:
                pick = _exact_pages(s, q, ids, pick)
            chosen.append(pick)
            seen = (pick[:, :, None] == (at // page)[None, None, :]).any(1) if L else seen
        z = torch.einsum("hge,hse->hgs", q, K) / math.sqrt(E)
        z = torch.where(seen[:, None], z, -math.inf)
        if L == 0:
            outs.append(torch.zeros(H * G, c["D"], dtype=torch.float64, device=dev))
            lses.append(torch.full((H * G,), -math.inf, dtype=torch.float64, device=dev))
            continue
        lse = torch.logsumexp(z, -1)
        outs.append(torch.einsum("hgs,hsd->hgd", torch.exp(z - lse[..., None]), V).reshape(H * G, c["D"]))
        lses.append(lse.reshape(H * G))
    got = {"out": torch.stack(outs), "lse": torch.stack(lses)}
    return got if c["op"] == "attention" else {**got, "pages": torch.stack(chosen)}


def _exact_pages(s, q, ids, pick):
    """The pages of one query token (H, top), its scores summed as whole numbers."""
    c = s["case"]
    q = torch.nan_to_num(q, nan=0.0)
    y = _exact_exponent(q.abs().amax(-1))
    q8 = torch.round(q / _exact_pow2(y)[..., None]).clamp(-127, 127)
    n = ids.numel()
    best = torch.full((q.shape[0], n), -math.inf, dtype=torch.float64, device=q.device)
    lo, hi = s["bounds"][0][ids, :, 0].double(), s["bounds"][0][ids, :, 1].double()   # (n, H, E)
    x = s["bounds"][1][ids].long()
    for g in range(q.shape[1]):
        part = torch.maximum(q8[:, g] * hi, q8[:, g] * lo).sum(-1) * _exact_pow2(x + y[:, g])
        best = torch.maximum(best, part.T)
    best[:, :c["first"]] = math.inf
    best[:, max(0, n - c["last"]):] = math.inf
    for h, row in enumerate(best.tolist()):
        got = sorted(sorted(range(n), key=lambda j: (-row[j], j))[:c["top"]])
        pick[h, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return pick
