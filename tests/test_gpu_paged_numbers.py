"""Paged operators where numbers are hardest: long sums, infinities, ends of the types' ranges, values next to a border."""
import io
import math

import pytest
import torch

import thinned_softmax_attention_b200 as T
from tests.test_gpu_paged import DEV, TYPES, check, filled, i32, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,width,tokens,G", [("fp32", 64, 111, 1), ("fp32", 128, 74, 4), ("fp32", 256, 37, 2)])
def test_long_sums_do_not_drift(dtype, width, tokens, G):
    """65536 keys to a pair, as many pairs as CTAs: each sum runs through one CTA from end to end.  The values of a column
    are one number c, so the output is c whatever the weights.

    fp32: a value enters as two tf32 numbers (2^-23 lost); a stage's sum, two chained products of 8 terms, is cut by under
    18 steps of 2^-23 = 2^-18.8; the stages' sums, 2048 of 8 keys per warp, are added with rounding to nearest: each off by
    at most 2^-24 of a partial that grows evenly, a spread of 2^-24 / sqrt(3) sqrt(2048 / 3) = 9e-7, four of which are
    3.6e-6; the sum of the weights likewise, over four lanes each: 1.8e-6.  With the cut 7.5e-6 together."""
    H, page, L = 4, 64, 65536
    gen = torch.Generator(DEV).manual_seed(width)
    kp = rnd(gen, L // page, H, page, width).to(TYPES[dtype])
    c = (torch.rand(H, width, generator=gen, device=DEV) * 0.5 + 0.5).to(TYPES[dtype])
    vp = c[None, :, None].expand(L // page, H, page, width).contiguous()
    q = rnd(gen, tokens, H * G, width).to(TYPES[dtype])
    table = torch.arange(L // page, dtype=torch.int32, device=DEV).repeat(tokens, 1)
    out = T.paged_attention(q, kp, vp, table, i32([L] * tokens)).view(tokens, H, G, width)
    off = ((out.double() - c.double()[None, :, None]) / c.double()[None, :, None]).abs().max()
    assert float(off) <= 7.5e-6, float(off)


@pytest.mark.parametrize("dtype,cache,width,G,keys", [("fp16", "fp16", 128, 4, 1 << 18), ("fp16", "fp16", 64, 12, 1 << 18), ("fp16", "fp16", 256, 4, 1 << 18),
                                                       ("fp16", "e4m3", 128, 4, 1 << 18), ("fp16", "e4m3", 256, 16, 1 << 18), ("bf16", "bf16", 128, 4, 1 << 21)])
def test_very_long_sums_of_16_bit_types_do_not_drift(dtype, cache, width, G, keys):
    """As above, with values that the output's type holds: the output is the value itself as long as the sums are right to
    half its step, 2^-12 of it at least in fp16 and 2^-9 in bf16.  Added with rounding, 4096 and 32768 stages of 16 keys per
    warp are off by four times 2^-24 / sqrt(3) sqrt(n / 3), 5e-6 and 1.5e-5; the cut within a stage is 32 steps of 2^-23."""
    H, page, n, tokens = 4, 64, 128, 74
    gen = torch.Generator(DEV).manual_seed(width)
    kp = rnd(gen, n, H, page, width).to(TYPES[cache])
    c = (torch.rand(H, width, generator=gen, device=DEV) * 0.5 + 0.5).to(TYPES[cache])
    vp = c[None, :, None].expand(n, H, page, width).contiguous()
    q = rnd(gen, tokens, H * G, width).to(TYPES[dtype])
    table = (torch.arange(keys // page, dtype=torch.int32, device=DEV) % n).repeat(tokens, 1)
    one = torch.ones(H, device=DEV) if cache == "e4m3" else None
    out = T.paged_attention(q, kp, vp, table, i32([keys] * tokens), k_scale=one, v_scale=one).view(tokens, H, G, width)
    off = ((out.double() - c.double()[None, :, None]) / c.double()[None, :, None]).abs().max()
    assert float(off) == 0.0, float(off)


@pytest.mark.parametrize("G", [4, 8, 12, 16])
def test_weights_against_an_8_bit_cache_keep_more_than_16_bits(G):
    """Two keys of nearly equal weight and opposite values: what a weight loses is the output's error.  A weight in one
    fp16 number would be off by up to 2^-11, the tolerance takes it as good to 2^-16 (its two parts: 2^-22)."""
    E, page = 64, 16
    kp, vp = (torch.zeros(1, 1, page, E, device=DEV) for _ in range(2))
    kp[0, 0, 0, 0], kp[0, 0, 1, 0], vp[0, 0, 0], vp[0, 0, 1] = 1.0, -1.0, 1.0, -1.0
    one, q = torch.ones(1, device=DEV), torch.zeros(8, G, E, dtype=torch.float16, device=DEV)
    q[..., 0] = (torch.arange(1, 8 * G + 1, device=DEV) * 1.37e-4).view(8, G).half()
    out, lse = T.paged_attention(q, kp.to(TYPES["e4m3"]), vp.to(TYPES["e4m3"]), i32([[0]] * 8), i32([2] * 8), scale=1.0, k_scale=one,
                                 v_scale=one, return_lse=True)
    for n in range(8):   # held to the 16-bit caches' bound of a weight
        check(out[n], lse[n], q[n], [(kp[0, 0, :2], vp[0, 0, :2])], "fp16", "fp16", 1.0)


@pytest.mark.parametrize("L", [1, 40, 5000])
@pytest.mark.parametrize("dtype,G", [("fp32", 4), ("fp32", 12), ("bf16", 4), ("bf16", 12), ("fp16", 4), ("fp16", 12)])
def test_infinite_keys_have_no_weight(dtype, G, L):
    """A visible key whose score is -inf counts as none, whatever the bits of the query."""
    H, E, page = 2, 64, 16
    kp, vp, _, table, held = filled([L], H, E, E, page, dtype, dtype, 51)
    q = rnd(torch.Generator(DEV).manual_seed(52), 1, H * G, E)
    q[0, :, 5] = torch.tensor([1.0, 0.3, 1.1, 2.0], device=DEV).repeat(H * G // 4)
    q = q.to(TYPES[dtype])
    hidden = [j for j in {0, 7, 17, L - 1} if j < L]
    for j in hidden:
        kp[int(table[0, j // page]), :, j % page, 5] = -math.inf
    keep = [j for j in range(L) if j not in hidden]
    out, lse = T.paged_attention(q, kp, vp, table, i32([L]), return_lse=True)
    check(out[0], lse[0], q[0], [(held[0][0][h, keep], held[0][1][h, keep]) for h in range(H)], dtype, dtype)


@pytest.mark.parametrize("L", [40, 5000])
@pytest.mark.parametrize("dtype,G", [("fp32", 4), ("fp32", 12), ("bf16", 4), ("bf16", 12), ("fp16", 4), ("fp16", 12)])
def test_infinite_values(dtype, G, L):
    """A column with an infinite value is that infinity, with both infinities NaN; the other columns are as without.  Key 2
    of the longer request has weights from 2^-22 down to below 2^-38 of the largest, where an fp16 weight may be none."""
    H, E, page = 2, 64, 16
    kp, vp, _, table, held = filled([L], H, E, E, page, dtype, dtype, 53)
    q = rnd(torch.Generator(DEV).manual_seed(54), 1, H * G, E).to(TYPES[dtype])
    place = lambda j: (int(table[0, j // page]), slice(None), j % page)
    if L > 40:
        q[0, :, 7] = 8.0
        kp[place(2)][:, 7] = held[0][0][:, 2, 7] = -20.0
    for j, d, x in ([(2, 1, math.inf)] if L > 40 else []) + [(3, 1, math.inf), (20, 9, -math.inf), (L - 1, 63, math.inf),
                                                             (L - 2, 63, math.inf), (8, 30, math.inf), (30, 30, -math.inf)]:
        vp[place(j)][:, d] = x
        held[0][1][:, j, d] = 0.0
    out, lse = T.paged_attention(q, kp, vp, table, i32([L]), return_lse=True)
    z = torch.einsum("hge,hse->hgs", q[0].double().view(H, G, E), held[0][0]).flatten(0, 1) / math.sqrt(E)
    none = (z[:, 2] - z.amax(-1) < -38 * math.log(2)) & torch.tensor(dtype == "fp16" and L > 40, device=DEV)
    assert ((out[0, :, 1] == math.inf) | (none & torch.isnan(out[0, :, 1]))).all() and not none.all()
    assert (out[0, :, 9] == -math.inf).all() and (out[0, :, 63] == math.inf).all()
    assert torch.isnan(out[0, :, 30]).all()
    rest = [d for d in range(E) if d not in (1, 9, 30, 63)]
    check(out[0][:, rest], lse[0], q[0], [(held[0][0][h], held[0][1][h][:, rest]) for h in range(H)], dtype, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-50])
def test_a_scale_of_zero_is_refused(scale):
    """The C entry reads 0 as 1 / sqrt(E): a zero that a caller gives may not turn into that."""
    kp, vp, _, table, _ = filled([5], 1, 64, 64, 16, "bf16", "bf16")
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    b = (torch.zeros(4, 1, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 1, dtype=torch.int8, device=DEV))
    for call in (lambda: T.paged_attention(q, kp, vp, table, i32([5]), scale=scale),
                 lambda: T.paged_sparse_attention(q, kp, vp, table, i32([5]), b, 2, scale=scale)):
        with pytest.raises(ValueError, match="scale"):
            call()


@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("size", [-125, -110, -60, 0, 100, 120, 124])
def test_bf16_queries_of_any_size_against_an_8_bit_cache(size, G):
    """Queries near the ends of bf16's range, keys scaled the other way: the scores are ordinary numbers."""
    L, H, E, page = 300, 2, 64, 16
    kp, vp, (ks, vs), table, held = filled([L], H, E, E, page, "bf16", "e4m3", 55)
    q = (rnd(torch.Generator(DEV).manual_seed(56), 1, H * G, E) * 2.0 ** size).bfloat16()
    assert torch.isfinite(q).all()
    K = [held[0][0][h] / ks[h].double() * 2.0 ** (-size - 5) for h in range(H)]
    ks.fill_(2.0 ** (-size - 5))
    out, lse = T.paged_attention(q, kp, vp, table, i32([L]), k_scale=ks, v_scale=vs, return_lse=True)
    check(out[0], lse[0], q[0], [(K[h], held[0][1][h]) for h in range(H)], "bf16", "e4m3")


def test_a_plan_can_be_saved():
    plan = T.paged_plan(i32([3, 0]), i32([2, 5]), i32([[9, -1], [-1, -1]]), i32([1, 2, 3]), i32([3]), 16, 9)
    buf = io.BytesIO()
    torch.save(tuple(plan), buf)
    buf.seek(0)
    for a, b in zip(plan, torch.load(buf)):
        assert torch.equal(a, b)


def test_a_gradient_is_not_dropped_in_silence():
    kp, vp, _, table, _ = filled([5], 1, 64, 64, 16, "bf16", "bf16")
    b = (torch.zeros(4, 1, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(4, 1, dtype=torch.int8, device=DEV))
    q, k = (torch.zeros(1, n, 64, dtype=torch.bfloat16, device=DEV) for n in (2, 1))
    slot, one = torch.zeros(1, dtype=torch.int64, device=DEV), torch.ones(1, device=DEV)
    leaf = lambda x: x.clone().requires_grad_()
    for call in (lambda: T.paged_attention(leaf(q), kp, vp, table, i32([5])), lambda: T.paged_attention(q, leaf(kp), vp, table, i32([5])),
                 lambda: T.paged_attention(q, kp, leaf(vp), table, i32([5])), lambda: T.paged_attention(leaf(q) * 2, kp, vp, table, i32([5])),
                 lambda: T.paged_sparse_attention(leaf(q), kp, vp, table, i32([5]), b, 2),
                 lambda: T.paged_attention(q, kp, vp, table, i32([5]), out=leaf(q)),
                 lambda: T.paged_attention(q, kp, vp, table, i32([5]), lse=torch.zeros(1, 2, device=DEV, requires_grad=True)),
                 lambda: T.paged_attention(q, kp.to(TYPES["e4m3"]), vp.to(TYPES["e4m3"]), table, i32([5]), k_scale=leaf(one), v_scale=one),
                 lambda: T.paged_append(leaf(k), k, slot, kp, vp), lambda: T.paged_append(k, leaf(k), slot, kp, vp)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quotients_next_to_the_borders_of_e4m3(dtype):
    """x / scale on and one step either side of every border between two e4m3 values, at every mantissa of x, up to where
    it is clamped: the bytes of the rounded quotient."""
    bits = 10 if dtype == "fp16" else 7
    border = [(k + 0.5) * 2.0 ** -9 for k in range(8)] + [(1 + (k + 0.5) / 8) * 2.0 ** e for e in range(-6, 9) for k in range(8)]
    E, page = 64, 1 << bits
    x = (1 + torch.arange(1 << bits, device=DEV) / (1 << bits)).to(TYPES[dtype])
    m = torch.tensor(border, device=DEV)
    near = (x.float()[:, None] / m).view(-1)                                  # scales that lead to the border
    steps = torch.arange(-2, 3, device=DEV, dtype=torch.int32)
    scales = (near.view(torch.int32)[:, None] + steps).view(torch.float32)    # (mantissas x borders, 5)
    n = 4096                                                                  # heads of a call: a scale each
    xs = x[:, None].expand(-1, m.numel()).reshape(-1)
    for u in range(5):
        for i in range(0, xs.numel(), n):
            s, y = scales[i:i + n, u].contiguous(), xs[i:i + n]
            H = s.numel()
            k = torch.stack([y, -y], -1).repeat(1, 8)[None].contiguous()      # (1, H, 16)
            kp, vp = (torch.zeros(1, H, 1, 16, device=DEV).to(TYPES["e4m3"]) for _ in range(2))
            T.paged_append(k, k, torch.zeros(1, dtype=torch.int64, device=DEV), kp, vp, k_scale=s, v_scale=s)
            want = (k[0].float() / s[:, None]).clamp(-448, 448).to(TYPES["e4m3"])
            assert torch.equal(kp[0, :, 0].float(), want.float()) and torch.equal(vp[0, :, 0].float(), want.float())


@pytest.mark.parametrize("G", [1, 8, 20])
def test_weights_in_fp32_keep_21_bits(G):
    """Two keys of nearly equal weight and opposite values.  The larger weight is 1; the other is off by the exponential's
    2^-22 and the 2^-22 that it is cut by, half of which reaches the output, whose sum of weights is rounded by 2^-24."""
    E, page = 64, 16
    kp, vp = (torch.zeros(1, 1, page, E, device=DEV) for _ in range(2))
    kp[0, 0, 0, 0], kp[0, 0, 1, 0], vp[0, 0, 0], vp[0, 0, 1] = 1.0, -1.0, 1.0, -1.0
    q = torch.zeros(8, G, E, device=DEV)
    q[..., 0] = (torch.arange(1, 8 * G + 1, device=DEV) * 1.37e-4).view(8, G)
    out = T.paged_attention(q, kp, vp, i32([[0]] * 8), i32([2] * 8), scale=1.0)
    assert ((out.double() - torch.tanh(q[..., :1].double())).abs() <= 2.0 ** -21).all()
