"""Paged operators where numbers are hardest: long sums, infinities, ends of the types' ranges, values next to a border."""
import pytest
import torch

import thinned_softmax_attention_b200 as T
from tests.test_gpu_paged import DEV, TYPES, i32, rnd

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
