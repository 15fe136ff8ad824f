"""Paged cache on the GPU: plans, appends, attention and page selection against plain 64-bit forms."""
import math
import random

import pytest
import torch

import thinned_softmax_attention_b200 as T
from tests import plain_paged as P

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def pool(gen, n_pages, H, page, E, D, cache, layout="heads"):
    """k_pages, v_pages and e4m3 scales; every slot holds poison until something is written there."""
    ct = TYPES[cache]
    poison = float("nan")
    if layout == "heads":          # (n_pages, H, page, width)
        kp, vp = (torch.full((n_pages, H, page, w), poison, device=DEV).to(ct) for w in (E, D))
    elif layout == "rows":         # (n_pages, page, H, width)
        kp, vp = (torch.full((n_pages, page, H, w), poison, device=DEV).to(ct).transpose(1, 2) for w in (E, D))
    else:                          # one buffer, a page's keys and values side by side
        kv = torch.full((n_pages, H, page, E + D + 16), poison, device=DEV).to(ct)
        kp, vp = kv[..., :E], kv[..., E:E + D]
    scales = (None, None)
    if cache == "e4m3":
        scales = (rnd(gen, H).abs() * 0.02 + 0.01, rnd(gen, H).abs() * 0.02 + 0.01)
    return kp, vp, scales


def filled(lengths, H, E, D, page, dtype, cache, seed=0, layout="heads", spare=3):
    """A pool with shuffled pages that holds random keys and values of the lengths, NaN elsewhere, its
    table, and per request the keys and values that it stands for (float64, (H, L, width))."""
    gen = torch.Generator(DEV).manual_seed(seed)
    used = [-(-L // page) for L in lengths]
    n_pages = sum(used) + spare
    kp, vp, scales = pool(gen, n_pages, H, page, E, D, cache, layout)
    order = torch.randperm(n_pages, generator=gen, device=DEV).tolist()
    table = torch.full((len(lengths), max(used + [1]) + 1), -1, dtype=torch.int32, device=DEV)
    held = []
    for r, L in enumerate(lengths):
        ids = [order.pop() for _ in range(used[r])]
        table[r, :used[r]] = i32(ids)
        k, v = rnd(gen, H, L, E).to(TYPES[dtype]), rnd(gen, H, L, D).to(TYPES[dtype])
        if cache == "e4m3":
            k = (k.float() / scales[0][:, None, None]).clamp(-448, 448).to(TYPES[cache])
            v = (v.float() / scales[1][:, None, None]).clamp(-448, 448).to(TYPES[cache])
        at = torch.arange(L, device=DEV)
        if L:
            ids = i32(ids).long()
            kp[ids[at // page], :, at % page] = k.transpose(0, 1)
            vp[ids[at // page], :, at % page] = v.transpose(0, 1)
        k, v = k.double(), v.double()
        if cache == "e4m3":
            k, v = k * scales[0].double()[:, None, None], v * scales[1].double()[:, None, None]
        held.append((k, v))
    return kp, vp, scales, table, held


def check(out, lse, q, keys, dtype, cache, scale=None):
    """out (Hq, D), lse (Hq) of one token against its visible keys: per key head a pair (K, V)."""
    H, G = len(keys), q.shape[0] // len(keys)
    for h, (K, V) in enumerate(keys):
        ref, l, spread, dz = P.attention(q[h * G:(h + 1) * G], K, V, scale)
        to, tl = P.tolerance(ref, l, spread, dz, K.shape[0], TYPES[dtype], cache)
        got, gl = out[h * G:(h + 1) * G].double(), lse[h * G:(h + 1) * G].double()
        if K.shape[0] == 0:
            assert (got == 0).all() and (gl == -math.inf).all()
            continue
        assert torch.isfinite(got).all() and torch.isfinite(gl).all()
        assert ((got - ref).abs() <= to).all(), float(((got - ref).abs() / to).max())
        assert ((gl - l).abs() <= tl).all(), float(((gl - l).abs() / tl).max())


# lengths, H, G, E, D, page, dtype, cache, layout
SHAPES = [
    ([0, 1, 2, 15, 16, 17, 33], 2, 4, 128, 128, 16, "bf16", "bf16", "heads"),
    ([1], 1, 1, 64, 64, 16, "bf16", "bf16", "heads"),
    ([700], 8, 4, 128, 128, 64, "bf16", "bf16", "rows"),
    ([5000, 3, 0, 1200], 2, 8, 128, 128, 64, "fp16", "fp16", "mixed"),
    ([2500, 100, 65], 3, 1, 64, 256, 20, "fp32", "fp32", "heads"),
    ([31, 257, 1023], 2, 5, 96, 96, 7, "bf16", "bf16", "rows"),
    ([40, 41, 42], 1, 16, 192, 128, 1, "bf16", "bf16", "heads"),
    ([513, 64], 2, 32, 128, 64, 32, "fp16", "fp16", "heads"),
    ([300, 17], 1, 40, 256, 256, 128, "bf16", "bf16", "heads"),
    ([900, 0, 77, 1], 4, 8, 128, 128, 32, "bf16", "e4m3", "heads"),
    ([333, 2049], 2, 3, 64, 96, 48, "fp16", "e4m3", "mixed"),
    ([129, 130], 2, 2, 256, 240, 16, "bf16", "e4m3", "rows"),
    ([77, 200], 2, 2, 8, 8, 16, "fp32", "fp32", "heads"),
    ([77, 200], 2, 2, 72, 40, 16, "bf16", "bf16", "rows"),
    ([100, 999], 2, 20, 128, 128, 256, "fp32", "fp32", "rows"),
    ([20000], 1, 8, 128, 128, 64, "bf16", "bf16", "heads"),
    ([i % 50 for i in range(300)], 1, 4, 64, 64, 16, "bf16", "bf16", "heads"),
    ([4096 + 13 * i for i in range(9)], 4, 4, 128, 128, 64, "bf16", "bf16", "heads"),
]


@pytest.mark.parametrize("case", SHAPES, ids=[f"{i}-{c[6]}-{c[7]}" for i, c in enumerate(SHAPES)])
def test_attention_matches_the_definition(case):
    lengths, H, G, E, D, page, dtype, cache, layout = case
    kp, vp, (ks, vs), table, held = filled(lengths, H, E, D, page, dtype, cache, 1, layout)
    q = rnd(torch.Generator(DEV).manual_seed(2), len(lengths), H * G, E).to(TYPES[dtype])
    out, lse = T.paged_attention(q, kp, vp, table, i32(lengths), k_scale=ks, v_scale=vs, return_lse=True)
    assert out.shape == (len(lengths), H * G, D) and out.dtype == q.dtype
    for r in range(len(lengths)):
        k, v = held[r]
        check(out[r], lse[r], q[r], [(k[h], v[h]) for h in range(H)], dtype, cache)
    again = T.paged_attention(q, kp, vp, table, i32(lengths), k_scale=ks, v_scale=vs)
    assert torch.equal(again, out)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
def test_window_and_scale(window, dtype, cache):
    lengths, H, G, E, D = [0, 1, 4, 5, 6, 99, 100, 101, 1500], 2, 4, 64, 64
    kp, vp, (ks, vs), table, held = filled(lengths, H, E, D, 16, dtype, cache, 3)
    q = rnd(torch.Generator(DEV).manual_seed(4), len(lengths), H * G, E).to(TYPES[dtype])
    # what the window hides must not matter: not even infinities and NaN
    for r, L in enumerate(lengths):
        for j in range(0, max(0, L - window)):
            kp[int(table[r, j // 16]), :, j % 16] = float("nan") if cache == "e4m3" else float("inf")
            vp[int(table[r, j // 16]), :, j % 16] = float("nan")
    out, lse = T.paged_attention(q, kp, vp, table, i32(lengths), window=window, scale=0.3, k_scale=ks, v_scale=vs, return_lse=True)
    for r, L in enumerate(lengths):
        k, v = held[r]
        lo = max(0, L - window)
        check(out[r], lse[r], q[r], [(k[h, lo:], v[h, lo:]) for h in range(H)], dtype, cache, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tokens_of_one_request_and_padding(dtype):
    """Draft tokens share a request; padding rows keep what the buffers held, in strided buffers too."""
    lengths, H, G, E, D = [40, 700, 9], 2, 4, 128, 64
    kp, vp, _, table, held = filled(lengths, H, E, D, 16, dtype, dtype, 5)
    rows, seen = [1, 1, 1, -1, 0, 3, 2, 2, 1], [698, 699, 700, 5, 40, 7, 0, 9, 1]
    wide = rnd(torch.Generator(DEV).manual_seed(6), len(rows), H * G + 3, E + 8).to(TYPES[dtype])
    q = wide[:, 1:1 + H * G, :E]
    buf = torch.full((len(rows) + 2, H * G, D + 16), 7.0, dtype=TYPES[dtype], device=DEV)
    lse = torch.full((len(rows), H * G), 7.0, device=DEV)
    out = buf[:len(rows), :, :D]
    got, got_lse = T.paged_attention(q, kp, vp, table, i32(seen), rows=i32(rows), out=out, lse=lse)
    assert got.data_ptr() == out.data_ptr() and got_lse is lse
    for t, (r, L) in enumerate(zip(rows, seen)):
        if r in (-1, 3):
            assert (out[t] == 7).all() and (lse[t] == 7).all()
            continue
        k, v = held[r]
        check(out[t], lse[t], q[t], [(k[h, :L], v[h, :L]) for h in range(H)], dtype, dtype)
    assert (buf[len(rows):] == 7).all() and (buf[..., D:] == 7).all()
    fresh = T.paged_attention(q, kp, vp, table, i32(seen), rows=i32(rows))
    assert (fresh[3] == 0).all() and (fresh[5] == 0).all() and torch.equal(fresh[0], out[0])


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "e4m3")])
def test_pages_outside_the_pool_are_not_seen(dtype, cache):
    lengths, H, G, E, D, page = [100, 64, 50, 333], 2, 4, 64, 64, 16
    kp, vp, (ks, vs), table, held = filled(lengths, H, E, D, page, dtype, cache, 7)
    bad = {0: [0, 3], 1: [0, 1, 2, 3], 3: [20, 7]}   # request 1 has none left, request 3 loses its tail
    ids = [-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31]
    for r, places in bad.items():
        for i, j in enumerate(places):
            table[r, j] = ids[i % 4]
    given = [100, 64, 10 ** 9, 333, ]
    given[2] = 10 ** 9          # clamped to the table, whose further entries are no pages
    q = rnd(torch.Generator(DEV).manual_seed(8), 4, H * G, E).to(TYPES[dtype])
    # the last page of request 2 ends behind its 50 keys: fill it, since the length says it is full
    for j in range(50, 64):
        kp[int(table[2, 3]), :, j % page] = torch.zeros(H, E, device=DEV).to(kp.dtype)
        vp[int(table[2, 3]), :, j % page] = torch.zeros(H, D, device=DEV).to(vp.dtype)
    out, lse = T.paged_attention(q, kp, vp, table, i32(given), k_scale=ks, v_scale=vs, return_lse=True)
    for r in range(4):
        k, v = held[r]
        if r == 2:
            k, v = torch.cat([k, k.new_zeros(H, 14, E)], 1), torch.cat([v, v.new_zeros(H, 14, D)], 1)
        keep = [j for j in range(k.shape[1]) if j // page not in bad.get(r, [])]
        check(out[r], lse[r], q[r], [(k[h, keep], v[h, keep]) for h in range(H)], dtype, cache)
    none, l = T.paged_attention(q, kp, vp, table, i32([-5, -2 ** 31, 0, 0]), k_scale=ks, v_scale=vs, return_lse=True)
    assert (none == 0).all() and (l == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_extreme_scores(dtype):
    """Scores far apart, all very low, the type's lowest finite value as a key: weights 0 and 1, no NaN."""
    H, G, E, D, page, L = 1, 2, 64, 64, 16, 200
    kp, vp, _, table, held = filled([L, L, L], H, E, D, page, dtype, dtype, 9)
    low = torch.finfo(TYPES[dtype]).min
    q = torch.zeros(3, G, E, device=DEV, dtype=TYPES[dtype])
    q[0, :, 0] = 1.0
    q[1, :, 0] = 1.0
    q[2, :, 0] = 100.0
    for r in range(3):
        for j in range(L):
            kp[int(table[r, j // page]), 0, j % page] = 0
    for j in range(L):          # request 0: one ordinary key among the lowest; request 1: all the lowest
        for r, x in ((0, 1.0 if j == 37 else low), (1, low), (2, 100.0 if j == 3 else -100.0)):
            kp[int(table[r, j // page]), 0, j % page, 0] = x
    out = T.paged_attention(q, kp, vp, table, i32([L] * 3))
    v = held[0][1][0].to(TYPES[dtype])
    # a weight of 1: the value itself; an fp32 value enters the product as hi + lo with lo cut to 11 of its 12
    # bits, so it may lose 2^-23 of its leading bit, and hi + lo' is exact in fp32
    near = lambda a, b: ((a.double() - b.double()).abs() <= (2.0 ** -23 * b.double().abs() if dtype == "fp32" else 0)).all()
    assert near(out[0], v[37].expand(G, D))
    mean = held[1][1][0].mean(0)
    tol = torch.finfo(TYPES[dtype]).eps * mean.abs() + (2.0 ** -16 + 2 * L * 2.0 ** -24) * held[1][1][0].abs().mean(0)
    assert ((out[1].double() - mean).abs() <= tol).all()
    assert near(out[2], held[2][1][0].to(TYPES[dtype])[3].expand(G, D))


def bounds_of(kp, table, lengths, page):
    """Bounds of the pages that the lengths fill, from their keys together; the others zero."""
    n, H, _, E = kp.shape
    b, x = torch.zeros(n, H, 2, E, dtype=torch.int8), torch.full((n, H), -1, dtype=torch.int8)
    for r, L in enumerate(lengths):
        for j in range(-(-L // page)):
            i = int(table[r, j])
            for h in range(H):
                b[i, h], x[i, h] = P.key_bounds(kp[i, h, :min(page, L - j * page)])
    return b.to(DEV), x.to(DEV)


SPARSE = [
    ([0, 1, 16, 17, 400, 900], 2, 4, 128, 128, 16, "bf16", "bf16", 8, 1, 1),
    ([2000, 31], 8, 4, 64, 64, 8, "bf16", "bf16", 5, 1, 1),
    ([640], 1, 1, 128, 64, 64, "fp16", "fp16", 4, 0, 1),
    ([700, 64, 65], 2, 3, 72, 40, 20, "bf16", "bf16", 6, 2, 3),
    ([1500], 2, 16, 96, 96, 16, "fp32", "fp32", 33, 1, 1),
    ([1500, 5, 0], 2, 8, 128, 128, 32, "bf16", "e4m3", 9, 1, 2),
    ([300], 1, 32, 256, 256, 4, "bf16", "bf16", 70, 1, 1),
    ([900, 77], 1, 20, 64, 256, 1, "fp32", "fp32", 100, 3, 1),
    ([5000], 2, 4, 128, 128, 2, "fp16", "e4m3", 1000, 1, 1),
    ([5000, 100], 1, 4, 64, 64, 16, "bf16", "bf16", 1, 0, 1),
]


@pytest.mark.parametrize("case", SPARSE, ids=[f"{i}-{c[6]}-{c[7]}" for i, c in enumerate(SPARSE)])
def test_sparse_attention_matches_the_definition(case):
    lengths, H, G, E, D, page, dtype, cache, top, first, last = case
    kp, vp, (ks, vs), table, held = filled(lengths, H, E, D, page, dtype, cache, 11)
    b, x = bounds_of(kp, table, lengths, page)
    q = rnd(torch.Generator(DEV).manual_seed(12), len(lengths), H * G, E).to(TYPES[dtype])
    out, lse, pages = T.paged_sparse_attention(q, kp, vp, table, i32(lengths), (b, x), top, first=first, last=last,
                                               k_scale=ks, v_scale=vs, return_lse=True, return_pages=True)
    for r, L in enumerate(lengths):
        n = -(-L // page)
        keys = []
        for h in range(H):
            ids = table[r, :n].long()
            want = P.choose(q[r, h * G:(h + 1) * G], b[ids, h], x[ids, h], top, first, last)
            assert pages[r, h].tolist() == want + [-1] * (top - len(want))
            at = [j for j in range(L) if j // page in set(want)]
            keys.append((held[r][0][h, at], held[r][1][h, at]))
        check(out[r], lse[r], q[r], keys, dtype, cache)
    # every page taken: the dense result
    everything = max(table.shape[1], first + last)
    if everything <= 4096:
        full, lse = T.paged_sparse_attention(q, kp, vp, table, i32(lengths), (b, x), everything, first=first, last=last,
                                             k_scale=ks, v_scale=vs, return_lse=True)
        for r in range(len(lengths)):
            check(full[r], lse[r], q[r], [(held[r][0][h], held[r][1][h]) for h in range(H)], dtype, cache)


def _lse(q, kv, H):
    G = q.shape[0] // H
    return torch.cat([P.attention(q[h * G:(h + 1) * G], kv[0][h], kv[1][h])[1] for h in range(H)]).float()


def test_equal_scores_go_to_the_lowest_pages_and_padding_is_left():
    lengths, H, G, E, page = [320, 320], 2, 2, 64, 16
    kp, vp, _, table, held = filled(lengths, H, E, E, page, "bf16", "bf16", 13)
    b = torch.ones(kp.shape[0], H, 2, E, dtype=torch.int8, device=DEV)
    x = torch.zeros(kp.shape[0], H, dtype=torch.int8, device=DEV)
    x[table[1, 11].item()] = 1                       # one page above the others
    q = torch.ones(3, H * G, E, dtype=torch.bfloat16, device=DEV)
    out = torch.full((3, H * G, E), 7.0, dtype=torch.bfloat16, device=DEV)
    o, pages = T.paged_sparse_attention(q, kp, vp, table, i32([320, 9, 320]), (b, x), 5, rows=i32([0, -1, 1]), out=out, return_pages=True)
    assert pages[0].tolist() == [[0, 1, 2, 3, 19]] * H and pages[2].tolist() == [[0, 1, 2, 11, 19]] * H
    assert (pages[1] == -1).all() and (out[1] == 7).all()
    # a page outside the pool scores lowest, and is not seen when it is taken all the same
    table[0, 2], table[0, 0] = -1, kp.shape[0]
    o, pages = T.paged_sparse_attention(q, kp, vp, table, i32([320, 9, 320]), (b, x), 5, rows=i32([0, -1, 1]), return_pages=True)
    assert pages[0].tolist() == [[0, 1, 3, 4, 19]] * H
    at = [j for j in range(320) if j // page in (1, 3, 4, 19)]
    check(o[0], _lse(q[0], (held[0][0][:, at], held[0][1][:, at]), H), q[0], [(held[0][0][h, at], held[0][1][h, at]) for h in range(H)], "bf16", "bf16")
    # NaN and infinities in a query: the choice is still made (a NaN counts as 0, an infinity as the largest)
    q2 = q.clone()
    q2[0, :, 3], q2[0, :, 5] = float("nan"), float("inf")
    pages = T.paged_sparse_attention(q2, kp, vp, table, i32([320, 9, 320]), (b, x), 5, rows=i32([0, -1, 1]), return_pages=True)[1]
    assert pages[0].tolist() == [P.choose(q2[0, :G], torch.where(torch.arange(20)[:, None, None] == 2, -127, 1).expand(20, 2, E),
                                          [0] * 20, 5, 1, 1)] * H


@pytest.mark.parametrize("dtype,cache,E,D,page,layout", [
    ("bf16", "bf16", 128, 128, 16, "heads"), ("fp32", "fp32", 64, 256, 20, "rows"), ("fp16", "e4m3", 96, 112, 8, "mixed"),
    ("bf16", "e4m3", 128, 128, 64, "heads"), ("fp16", "fp16", 72, 8, 1, "heads"), ("bf16", "bf16", 256, 64, 7, "rows"),
    ("bf16", "bf16", 8, 256, 300, "heads")])
def test_append_in_steps_keeps_rows_and_bounds(dtype, cache, E, D, page, layout):
    """Tokens that arrive in steps of any size: the rows as one rounding gives them, the bounds those of
    all of a page's keys together, nothing else touched."""
    r = random.Random(E + page)
    gen = torch.Generator(DEV).manual_seed(page)
    H, R = 3, 4
    kp, vp, (ks, vs) = pool(gen, 60 if page < 16 else 40, H, page, E, D, cache, layout)
    n_pages = kp.shape[0]
    b = torch.zeros(n_pages, H, 2, E, dtype=torch.int8, device=DEV)
    x = torch.full((n_pages, H), -1, dtype=torch.int8, device=DEV)
    lengths, table = i32([0] * R), torch.full((R, n_pages), -1, dtype=torch.int32, device=DEV)
    free, n_free = i32(r.sample(range(n_pages), n_pages)), i32([n_pages])
    rows = [[] for _ in range(R)]
    for step in range(6):
        new = [r.choice([0, 1, 1, 2, 5, page, 2 * page + 1]) if step else 1 for _ in range(R)]
        step_plan = T.paged_plan(lengths, i32(new), table, free, n_free, page, sum(new) + 3, inplace=True)
        N = sum(new) + 3
        wide = rnd(gen, N, H + 1, E + D + 16) * 10.0 ** r.randrange(-2, 3)
        wide = wide.to(TYPES[dtype])
        if cache != "e4m3" and step == 3:
            wide[0, :, :8] = float("inf")
        if step == 2:
            wide[0, :, :3] = float("nan")
        k, v = wide[:, :H, :E], wide[:, 1:, E:E + D]
        T.paged_append(k, v, step_plan.slots, kp, vp, k_scale=ks, v_scale=vs, bounds=(b, x))
        status, cu = step_plan.status.tolist(), step_plan.cu.tolist()
        for i in range(R):
            if status[i] == 0:
                rows[i] += [(k[t].clone(), v[t].clone()) for t in range(cu[i], cu[i + 1])]
    got = lengths.tolist()
    assert got == [len(a) for a in rows] and sum(got) > 10
    want_k, want_v = torch.full_like(kp, float("nan")), torch.full_like(vp, float("nan"))
    for i in range(R):
        for t, (k, v) in enumerate(rows[i]):
            at = int(table[i, t // page]), slice(None), t % page
            if cache == "e4m3":
                k, v = ((y.float() / s[:, None]).clamp(-448, 448).to(TYPES[cache]) for y, s in ((k, ks), (v, vs)))
            want_k[at], want_v[at] = k, v
    for got_p, want in ((kp, want_k), (vp, want_v)):
        assert torch.equal(got_p.float().nan_to_num(nan=12345.0), want.float().nan_to_num(nan=12345.0))
    bw, xw = bounds_of(kp, table, got, page)
    assert torch.equal(x, xw) and torch.equal(b, bw)


def test_append_skips_slots_outside_the_pool():
    kp, vp, _ = pool(torch.Generator(DEV).manual_seed(0), 2, 1, 16, 64, 64, "bf16")
    b = (torch.zeros(2, 1, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(2, 1, dtype=torch.int8, device=DEV))
    k = torch.ones(6, 1, 64, dtype=torch.bfloat16, device=DEV)
    T.paged_append(k, k, torch.tensor([-1, 32, 2 ** 62, -2 ** 63, 31, -16], device=DEV), kp, vp, bounds=b)
    assert torch.isnan(kp).sum() == 31 * 64 and (kp[1, 0, 15] == 1).all() and torch.isnan(vp).sum() == 31 * 64
    assert (b[0][0] == 0).all() and b[1].tolist() == [[0], [0]]
    T.paged_append(k[:0], k[:0], torch.zeros(0, dtype=torch.int64, device=DEV), kp, vp, bounds=b)


def check_plan(lengths, new, table, free, n_free, page, max_tokens):
    """paged_plan against the plain plan; returns the state after it."""
    want = P.plan(lengths, new, table, free[:n_free], page, max_tokens)
    W = len(table[0])
    dt = i32(table).reshape(len(table), W)
    got = T.paged_plan(i32(lengths), i32(new), dt, i32(free), i32([n_free]), page, max_tokens)
    assert got.status.tolist() == want[6]
    assert got.lengths.tolist() == want[0] and got.n_free.tolist() == [len(want[1])] and got.cu.tolist() == want[2]
    assert got.slots.tolist() == want[3] and got.rows.tolist() == want[4] and got.context.tolist() == want[5]
    assert dt.tolist() == want[7]
    return want


def test_plan_matches_the_plain_plan():
    r = random.Random(5)
    for trial in range(40):
        R = r.choice([1, 2, 7, 33, 64, 300])
        page = r.choice([1, 3, 16, 64])
        hi = r.choice([1, 20, 200])
        lengths = [r.choice([0, 1, page, r.randrange(hi + 1), -3 if trial % 5 == 0 else 2]) for _ in range(R)]
        new = [r.choice([0, 1, 1, page, r.randrange(hi + 1), -2 if trial % 7 == 0 else 1]) for _ in range(R)]
        W = r.choice([1, 4, -(-2 * hi // page) + 2])
        n_pages = max(1, R * W // 2)
        ids = r.sample(range(10 * n_pages), n_pages)
        table = [[ids.pop() if ids and j < -(-max(L, 0) // page) else -1 for j in range(W)] for L in lengths]
        free = ids + [99] * 3
        total = sum(max(n, 0) for n in new)
        check_plan(lengths, new, table, free, len(ids), page, r.choice([total, total + 5, total // 2, 0, 1]))


def test_plan_of_many_requests_and_long_prompts():
    r = random.Random(6)
    R, page = 16384, 16
    lengths, new = [r.randrange(40) for _ in range(R)], [r.randrange(3) for _ in range(R)]
    table = [[3 * i + j if j < -(-L // page) else -1 for j in range(3)] for i, L in enumerate(lengths)]
    check_plan(lengths, new, table, list(range(50000, 54000)), 4000, page, 16384)
    check_plan([5], [200000], [[7] + [-1] * 12600], list(range(12600)), 12600, page, 200001)
    got = T.paged_plan(i32([]), i32([]), torch.zeros(0, 4, dtype=torch.int32, device=DEV), i32([3]), i32([1]), 16, 5)
    assert got.slots.tolist() == [-1] * 5 and got.cu.tolist() == [0] and got.n_free.tolist() == [1]
    # sums beyond 32 bits end as refusals
    big = T.paged_plan(i32([0, 2 ** 31 - 5, 3]), i32([2 ** 31 - 1, 100, 2 ** 31 - 1]), torch.zeros(3, 4, dtype=torch.int32, device=DEV),
                       i32([1]), i32([1]), 2 ** 30, 8)
    assert big.status.tolist() == [3, 2, 2] and big.lengths.tolist() == [0, 2 ** 31 - 5, 3] and big.rows.tolist() == [-1] * 8


def test_a_server_s_life():
    """Requests arrive, grow, are rolled back and end, over 40 steps: tables, stack and slots as the plain
    allocator has them, and the attention of every step's tokens as of contiguous keys."""
    r = random.Random(7)
    gen = torch.Generator(DEV).manual_seed(7)
    R, H, G, E, page, n_pages, W = 6, 2, 2, 64, 8, 40, 12
    cache = T.PagedAttentionCache(n_pages, page, H, E, E, torch.bfloat16, R, W * page, bounds=True)
    lengths, free, table = [0] * R, cache.free.tolist(), cache.table.tolist()
    held = [[] for _ in range(R)]
    for step in range(40):
        new = [r.choice([0, 1, 1, 1, 3, 20 if not lengths[i] else 1]) for i in range(R)]
        room = sum(new) + r.choice([0, 4, -2])
        room = max(room, 1)
        p = cache.plan(i32(new), room)
        lengths, free, cu, slots, rows, context, status, table = P.plan(lengths, new, table, free, page, room)
        assert p.slots.tolist() == slots and p.rows.tolist() == rows and p.status.tolist() == status
        assert cache.lengths.tolist() == lengths and cache.table.tolist() == table
        assert int(cache.n_free) == len(free) and cache.free.tolist()[:len(free)] == free
        k, v = rnd(gen, room, H, E).bfloat16(), rnd(gen, room, H, E).bfloat16()
        cache.append(k, v, p.slots)
        for t, i in enumerate(rows):
            if i >= 0:
                held[i].append((k[t], v[t]))
        q = rnd(gen, room, H * G, E).bfloat16()
        out, lse = cache.attend(q, rows=p.rows, lengths=p.context, return_lse=True)
        some, lse_s, pages = cache.attend_sparse(q, 4, rows=p.rows, lengths=p.context, return_lse=True, return_pages=True)
        for t, i in enumerate(rows):
            if i < 0:
                assert (out[t] == 0).all() and (some[t] == 0).all()
                continue
            K = torch.stack([a for a, _ in held[i][:context[t]]], 1)
            V = torch.stack([b for _, b in held[i][:context[t]]], 1)
            check(out[t], lse[t], q[t], [(K[h], V[h]) for h in range(H)], "bf16", "bf16")
            for h in range(H):
                at = [j for j in range(context[t]) if j // page in pages[t, h].tolist()]
                check(some[t, h * G:(h + 1) * G], lse_s[t, h * G:(h + 1) * G], q[t, h * G:(h + 1) * G], [(K[h, at], V[h, at])], "bf16", "bf16")
        keep = [r.choice([-1, -1, -1, -1, 0, max(0, lengths[i] - 3), 10 ** 6]) for i in range(R)]
        cache.release(i32(keep))
        lengths, free, table = P.release(keep, lengths, table, free, page)
        held = [a[:n] for a, n in zip(held, lengths)]
        assert cache.lengths.tolist() == lengths and cache.table.tolist() == table
        assert int(cache.n_free) == len(free) and cache.free.tolist()[:len(free)] == free
    one = cache.attend(rnd(gen, R, H * G, E).bfloat16())
    assert torch.isfinite(one).all()


def test_captured_steps_replay_on_two_streams():
    """A whole decode step in a graph: replayed steps continue the cache, and two caches' graphs run at once."""
    H, G, E, page, R, steps = 2, 4, 64, 16, 5, 12

    def make(seed):
        gen = torch.Generator(DEV).manual_seed(seed)
        cache = T.PagedAttentionCache(60, page, H, E, E, torch.bfloat16, R, 128, bounds=True)
        q, k, v = (rnd(gen, steps + 1, R, n, E).bfloat16() for n in (H * G, H, H))
        return cache, q, k, v

    def step(cache, q, k, v, one):
        p = cache.plan(one, R)
        cache.append(k, v, p.slots)
        return cache.attend(q), cache.attend_sparse(q, 3)

    one = i32([1] * R)
    made = [make(1), make(2)]
    graphs = []
    for cache, q, k, v in made:
        sq, sk, sv = q[0].clone(), k[0].clone(), v[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(cache, sq, sk, sv, one)      # first use of every kernel outside the capture
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(cache, sq, sk, sv, one)
        graphs.append((g, sq, sk, sv, res))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    kept = [[], []]
    for s in range(1, steps + 1):
        for i, (cache, q, k, v) in enumerate(made):
            with torch.cuda.stream(streams[i]):
                g, sq, sk, sv, res = graphs[i]
                sq.copy_(q[s]); sk.copy_(k[s]); sv.copy_(v[s])
                g.replay()
                kept[i].append([t.clone() for t in res])
    torch.cuda.synchronize()
    for i, seed in enumerate((1, 2)):
        cache, q, k, v = make(seed)
        for s in range(steps + 1):
            want = step(cache, q[s], k[s], v[s], one)
            if s:
                assert all(torch.equal(a, b) for a, b in zip(want, kept[i][s - 1]))
        assert torch.equal(cache.lengths, made[i][0].lengths) and cache.lengths.tolist() == [steps + 1] * R


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements: pages at both of its ends."""
    n_pages, H, page, E = 2 ** 31 // (2 * 256 * 128) + 40, 2, 256, 128
    kp = torch.zeros((n_pages, H, page, E), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros((n_pages, H, page, E), dtype=torch.bfloat16, device=DEV)
    ids = [n_pages - 1, 0, n_pages - 2]
    gen = torch.Generator(DEV).manual_seed(3)
    table, L = i32([ids]), 600
    at = torch.arange(L, device=DEV)
    slots = i32(ids).long()[at // page] * page + at % page
    k, v = rnd(gen, L, H, E).bfloat16(), rnd(gen, L, H, E).bfloat16()
    b = (torch.zeros(n_pages, H, 2, E, dtype=torch.int8, device=DEV), torch.zeros(n_pages, H, dtype=torch.int8, device=DEV))
    T.paged_append(k, v, slots, kp, vp, bounds=b)
    assert torch.equal(kp[ids[2], :, 600 - 513], k[599]) and torch.equal(vp[ids[0], :, 255], v[255])
    q = rnd(gen, 1, 8, E).bfloat16()
    out, lse = T.paged_attention(q, kp, vp, table, i32([L]), return_lse=True)
    check(out[0], lse[0], q[0], [(k[:, h], v[:, h]) for h in range(H)], "bf16", "bf16")
    out, lse = T.paged_sparse_attention(q, kp, vp, table, i32([L]), b, 3, return_lse=True)
    check(out[0], lse[0], q[0], [(k[:, h], v[:, h]) for h in range(H)], "bf16", "bf16")


def test_no_tokens_and_no_table():
    kp, vp, _, table, _ = filled([5], 1, 64, 64, 16, "bf16", "bf16")
    q = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert T.paged_attention(q, kp, vp, table, i32([])).shape == (0, 2, 64)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = T.paged_attention(q, kp, vp, torch.zeros(2, 0, dtype=torch.int32, device=DEV), i32([4, 0]), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    b = (torch.zeros(4, 1, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 1, dtype=torch.int8, device=DEV))
    out, pages = T.paged_sparse_attention(q, kp, vp, torch.zeros(2, 0, dtype=torch.int32, device=DEV), i32([4, 0]), b, 2, return_pages=True)
    assert (out == 0).all() and (pages == -1).all()


def test_refusals_on_the_device():
    kp, vp, _, table, _ = filled([5], 2, 64, 64, 16, "bf16", "bf16")
    q, L = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV), i32([5])
    b = (torch.zeros(4, 2, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 2, dtype=torch.int8, device=DEV))
    for bad in (lambda: T.paged_attention(q[:, :3], kp, vp, table, L), lambda: T.paged_attention(q.float(), kp, vp, table, L),
                lambda: T.paged_attention(q, kp, vp[:2], table, L), lambda: T.paged_attention(q, kp, vp, table.long(), L),
                lambda: T.paged_attention(q, kp, vp, table, L.long()), lambda: T.paged_attention(q, kp, vp, table, L.cpu()),
                lambda: T.paged_attention(q, kp, vp, table, i32([5, 5])), lambda: T.paged_attention(q, kp.cpu(), vp, table, L),
                lambda: T.paged_attention(q, kp, vp, table, L, rows=i32([0, 0])),
                lambda: T.paged_attention(q, kp, vp, table, L, k_scale=torch.ones(2, device=DEV)),
                lambda: T.paged_attention(q, kp, vp, table, L, lse=torch.ones(1, 3, device=DEV)),
                lambda: T.paged_attention(q, kp, vp, table, L, out=q[:, :, :32]),
                lambda: T.paged_attention(q, kp.to(torch.float8_e4m3fn), vp.to(torch.float8_e4m3fn), table, L),
                lambda: T.paged_sparse_attention(q, kp, vp, table, L, b, 0),
                lambda: T.paged_sparse_attention(q, kp, vp, table, L, (b[0][:3], b[1]), 4),
                lambda: T.paged_append(q[:, :2], q[:, :2], i32([0]), kp, vp),
                lambda: T.paged_append(q, q, torch.zeros(1, dtype=torch.int64, device=DEV), kp, vp),
                lambda: T.paged_plan(L, i32([1, 1]), table, i32([0]), i32([1]), 16, 4),
                lambda: T.paged_plan(L, i32([1]), table, i32([0]), i32([1]), 0, 4),
                lambda: T.paged_release(i32([1, 1]), L, table, i32([0]), i32([1]), 16)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(1, 4, 72, dtype=torch.bfloat16, device=DEV)[:, :, 4:68]
    for bad in (lambda: T.paged_attention(odd, kp, vp, table, L),                                # not 16-byte aligned
                lambda: T.paged_attention(q.repeat(2, 1, 1), kp, vp, table, i32([5, 5])),         # more tokens than requests
                lambda: T.paged_attention(q, kp, vp, table, L, window=-1),
                lambda: T.paged_sparse_attention(q, kp, vp, table, L, b, 4097),
                lambda: T.paged_sparse_attention(q, kp, vp, table, L, b, 2, last=0),
                lambda: T.paged_sparse_attention(q, kp, vp, table, L, b, 2, first=2),
                lambda: T.paged_plan(i32([0] * 16385), i32([0] * 16385), i32([[0]] * 16385), i32([0]), i32([1]), 16, 4)):
        with pytest.raises(T.ThinAttnError, match="EINVAL|EUNSUPPORTED"):
            bad()


@pytest.mark.parametrize("dtype,cache,G", [("fp16", "fp16", 4), ("fp16", "fp16", 12), ("bf16", "e4m3", 4), ("bf16", "bf16", 4), ("fp32", "fp32", 4)])
def test_a_long_tail_of_small_weights(dtype, cache, G):
    """One key with weight near 1 and 60000 others at 2^-25 of it: together 0.2% of the sum, which a 16-bit weight
    rounds up or away unless it is scaled."""
    L, E, page = 60001, 64, 64
    kp, vp, (ks, vs), table, _ = filled([L], 1, E, E, page, dtype, cache, 21)
    q = torch.zeros(1, G, E, dtype=TYPES[dtype], device=DEV)
    q[..., 0] = 1.0
    ids = table[0, :-(-L // page)].long()
    K, V = torch.zeros(L, E, dtype=torch.float64), torch.ones(L, E, dtype=torch.float64)
    K[0, 0], V[0] = 16.0, 0.0
    if cache == "e4m3":
        ks.fill_(1.0)
        vs.fill_(1.0)
    k, v = torch.zeros(len(ids) * page, E), torch.zeros(len(ids) * page, E)
    k[:L], v[:L] = K.float(), V.float()
    kp[ids] = k.view(len(ids), 1, page, E).to(DEV).to(kp.dtype)
    vp[ids] = v.view(len(ids), 1, page, E).to(DEV).to(vp.dtype)
    scale = 25.4 * math.log(2) / 16.0
    out, lse = T.paged_attention(q, kp, vp, table, i32([L]), scale=scale, k_scale=ks, v_scale=vs, return_lse=True)
    check(out[0], lse[0], q[0], [(K.to(DEV), V.to(DEV))], dtype, cache, scale)


def test_output_in_place_of_the_queries():
    kp, vp, _, table, held = filled([300, 1, 4097], 2, 64, 64, 16, "bf16", "bf16", 22)
    q = rnd(torch.Generator(DEV).manual_seed(23), 3, 8, 64).bfloat16()
    want = T.paged_attention(q, kp, vp, table, i32([300, 1, 4097]))
    T.paged_attention(q, kp, vp, table, i32([300, 1, 4097]), out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("page,tokens", [(2048, 5000), (65536, 3000), (100, 777)])
def test_append_of_long_runs(page, tokens):
    """Runs that span many blocks of tokens, beginning within a page and at its start."""
    gen = torch.Generator(DEV).manual_seed(page)
    kp, vp, _ = pool(gen, 4, 3, page, 16, 16, "bf16")
    b = (torch.zeros(4, 3, 2, 16, dtype=torch.int8, device=DEV), torch.zeros(4, 3, dtype=torch.int8, device=DEV))
    table, L = [2, 0, 3, 1], 0
    for n in (37, tokens if page > 1000 else 300):
        n = min(n, 4 * page - L)
        at = torch.arange(L, L + n, device=DEV)
        slots = i32(table).long()[at // page] * page + at % page
        k, v = rnd(gen, n, 3, 16).bfloat16(), rnd(gen, n, 3, 16).bfloat16()
        T.paged_append(k, v, slots, kp, vp, bounds=b)
        assert torch.equal(kp[slots // page, :, slots % page], k) and torch.equal(vp[slots // page, :, slots % page], v)
        L += n
    bw, xw = bounds_of(kp, i32([table]), [L], page)
    used = i32(table[:-(-L // page)]).long()
    assert torch.equal(b[0][used], bw[used]) and torch.equal(b[1][used], xw[used])


def test_an_8_bit_cache_through_its_class():
    gen = torch.Generator(DEV).manual_seed(31)
    H, G, E, D, R = 2, 4, 64, 32, 3
    ks, vs = torch.full((H,), 0.02, device=DEV), torch.full((H,), 0.03, device=DEV)
    cache = T.PagedAttentionCache(20, 16, H, E, D, torch.float16, R, 100, cache_dtype=torch.float8_e4m3fn, bounds=True, k_scale=ks,
                                  v_scale=vs, scale=0.2)
    p = cache.plan(i32([30, 0, 17]), 50)
    k, v = rnd(gen, 50, H, E).half(), rnd(gen, 50, H, D).half()
    cache.append(k, v, p.slots)
    q = rnd(gen, R, H * G, E).half()
    out, lse = cache.attend(q, return_lse=True)
    both, lse2, pages = cache.attend_sparse(q, 8, return_lse=True, return_pages=True)
    held = lambda x, s: (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s.double()[:, None]
    for r, (a, b) in enumerate([(0, 30), (30, 30), (30, 47)]):
        K, V = held(k[a:b], ks), held(v[a:b], vs)
        for o, l in ((out, lse), (both, lse2)):
            check(o[r], l[r], q[r], [(K[:, h], V[:, h]) for h in range(H)], "fp16", "e4m3", 0.2)
    assert pages[0].tolist() == [[0, 1] + [-1] * 6] * H and pages[1].tolist() == [[-1] * 8] * H
    with pytest.raises(ValueError):
        T.PagedAttentionCache(20, 16, H, E, D, torch.float16, R, 100, cache_dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="bounds"):
        T.PagedAttentionCache(20, 16, H, E, D, torch.float16, R, 100).attend_sparse(q, 4)


def test_calls_from_two_threads_and_streams():
    """Concurrent calls that share only inputs: each gets the result that it gets alone."""
    import threading
    lengths = [700, 0, 64, 5000]
    kp, vp, _, table, _ = filled(lengths, 2, 64, 64, 16, "bf16", "bf16", 41)
    b = bounds_of(kp, table, lengths, 16)
    qs = [rnd(torch.Generator(DEV).manual_seed(50 + i), 4, 8, 64).bfloat16() for i in range(4)]
    n = i32(lengths)
    want = [(T.paged_attention(q, kp, vp, table, n), T.paged_sparse_attention(q, kp, vp, table, n, b, 6)) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [(T.paged_attention(qs[i], kp, vp, table, n), T.paged_sparse_attention(qs[i], kp, vp, table, n, b, 6)) for _ in range(30)]
            torch.cuda.current_stream().synchronize()
        wrong.extend(1 for g in got if not (torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_first_use_inside_a_capture():
    """A process whose first call of every operator is captured."""
    import subprocess
    import sys
    code = """
import torch, thinned_softmax_attention_b200 as T
c = T.PagedAttentionCache(20, 16, 2, 64, 64, torch.bfloat16, 3, 100, bounds=True)
new = torch.tensor([5, 20, 1], dtype=torch.int32, device="cuda")
k = torch.randn(26, 2, 64, device="cuda").bfloat16(); q = torch.randn(3, 8, 64, device="cuda").bfloat16()
keep = torch.tensor([-1, 4, 0], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    p = c.plan(new, 26); c.append(k, k, p.slots); a = c.attend(q); b = c.attend_sparse(q, 8); c.release(keep)
assert c.lengths.tolist() == [0, 0, 0]
g.replay(); torch.cuda.synchronize()
assert c.lengths.tolist() == [5, 4, 0], c.lengths
assert torch.isfinite(a).all() and (a - b).abs().max() < 1e-1 and a.abs().max() > 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert "captured" in r.stdout, r.stdout + r.stderr


def test_lengths_close_to_31_bits():
    """A table that names one page 42949 times: 2147450000 keys, whose count plus a page passes 31 bits."""
    gen = torch.Generator(DEV).manual_seed(32)
    page, W, E = 50000, 42949, 64
    kp, vp = (rnd(gen, 1, 1, page, E).bfloat16() for _ in range(2))
    b = (torch.zeros(1, 1, 2, E, dtype=torch.int8, device=DEV), torch.zeros(1, 1, dtype=torch.int8, device=DEV))
    q, table = rnd(gen, 1, 4, E).bfloat16(), torch.zeros(1, W, dtype=torch.int32, device=DEV)
    K, V = kp[0, 0].double(), vp[0, 0].double()
    for last in (page, 49000):
        length = i32([(W - 1) * page + last])
        out, lse, pages = T.paged_sparse_attention(q, kp, vp, table, length, b, 4, return_lse=True, return_pages=True)
        assert pages.tolist() == [[[0, 1, 2, W - 1]]]
        check(out[0], lse[0], q[0], [(torch.cat((K, K, K, K[:last])), torch.cat((V, V, V, V[:last])))], "bf16", "bf16")
        out, lse = T.paged_attention(q, kp, vp, table, length, window=70, return_lse=True)
        check(out[0], lse[0], q[0], [(K[last - 70:last], V[last - 70:last])], "bf16", "bf16")


def test_strides_of_axes_of_one_are_free():
    """One token, one key head, one page: what their axes' strides say is never used."""
    gen = torch.Generator(DEV).manual_seed(31)
    E, L = 64, 16
    new = [rnd(gen, L, 1, E).bfloat16().as_strided((L, 1, E), (E, 3, 1)) for _ in range(2)]
    kp, vp = (torch.zeros(L * E, dtype=torch.bfloat16, device=DEV).as_strided((1, 1, L, E), (5, 7, E, 1)) for _ in range(2))
    T.paged_append(*new, torch.arange(L, device=DEV), kp, vp)
    assert torch.equal(kp[0, 0], new[0][:, 0]) and torch.equal(vp[0, 0], new[1][:, 0])
    q = rnd(gen, 4, E).bfloat16().as_strided((1, 4, E), (9, E, 1))
    out, lse = torch.empty(4 * E, dtype=torch.bfloat16, device=DEV).as_strided((1, 4, E), (11, E, 1)), torch.empty(1, 4, device=DEV)
    T.paged_attention(q, kp, vp, i32([[0]]), i32([L]), out=out, lse=lse)
    check(out[0], lse[0], q[0], [(kp[0, 0].double(), vp[0, 0].double())], "bf16", "bf16")


def test_overlapping_tensors_and_odd_scales_are_refused():
    kp, vp, _, table, _ = filled([5, 5], 2, 64, 64, 16, "bf16", "bf16")
    buf, L = torch.zeros(2 * 4 * 64 + 64, dtype=torch.bfloat16, device=DEV), i32([5, 5])
    q, n = buf[:512].view(2, 4, 64), torch.zeros(1, dtype=torch.int32, device=DEV)
    row, one = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    for bad in (lambda: T.paged_attention(q, kp, vp, table, L, out=buf[64:].view(2, 4, 64)),
                lambda: T.paged_attention(q, kp, vp, table, L, out=row.expand(2, 4, 64)),
                lambda: T.paged_append(row[:, :2], row[:, :2], one, kp, kp),
                lambda: T.paged_append(row[:, :2], row[:, :2], one, kp[:1].expand(4, -1, -1, -1), vp[:1].expand(4, -1, -1, -1))):
        with pytest.raises(ValueError, match="overlap"):
            bad()
    for bad in (lambda: T.paged_plan(L, L, table[:1].expand(2, -1), i32([0]), n, 16, 4),
                lambda: T.paged_release(L, L, table[:1].expand(2, -1), i32([0]), n, 16),
                lambda: T.paged_attention(q, kp, vp, table, L, scale=-1.0),
                lambda: T.paged_attention(q, kp, vp, table, L, scale=float("nan"))):
        with pytest.raises(T.ThinAttnError, match="EINVAL"):
            bad()


@pytest.mark.parametrize("inplace", [False, True])
def test_a_plan_s_tensors_are_tensors_of_their_own(inplace):
    """They lie in one allocation, and stay right when one is changed, outlives the others or is used in inference mode."""
    lengths, new, table = i32([3, 0, 30]), i32([2, 5, 40]), torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    table[0, 0] = 9
    want = P.plan([3, 0, 30], [2, 5, 40], table.tolist(), [1, 2, 3], 16, 9)
    for mode in (torch.enable_grad, torch.no_grad, torch.inference_mode):
        with mode():
            args = lengths.clone(), new, table.clone(), i32([1, 2, 3]), i32([3])
            got = T.paged_plan(*args, 16, 9, inplace=inplace)
            assert [t.dtype for t in got] == [torch.int32] * 3 + [torch.int64] + [torch.int32] * 3
            assert (got.lengths is args[0]) == inplace and (got.n_free is args[4]) == inplace
            assert got.lengths.tolist() == want[0] and got.n_free.tolist() == [len(want[1])]
            assert got.cu.tolist() == want[2] and got.rows.tolist() == want[4] and got.status.tolist() == want[6]
            assert got.slots.is_contiguous() and not got.slots.requires_grad
            got.slots.fill_(-7)
            got.cu.add_(100)
            got.status.zero_()
            assert got.context.tolist() == want[5] and got.rows.tolist() == want[4]
            rows = got.rows
            del got, args
            torch.full((4096,), 5, dtype=torch.int32, device=DEV)
            assert rows.tolist() == want[4] and rows.clone().add_(1).tolist() == [r + 1 for r in want[4]]
