"""Plain 64-bit implementations of the paged-cache operators, written from their definitions.

Attention and page choice run in float64 (on any device), the step plan and the key bounds in Python
numbers.  ``tolerance`` derives how far a kernel's output may be from them.
"""
import math

import torch

LOG2E = 1.4426950408889634


def plan(lengths, new, table, free, page, max_tokens):
    """(lengths, free, cu, slots, rows, context, status, table) of a step; lists in, lists out."""
    lengths, free, table = list(lengths), list(free), [list(r) for r in table]
    W = len(table[0]) if table else 0
    cu, status = [0], []
    slots, rows, context = [-1] * max_tokens, [-1] * max_tokens, [0] * max_tokens
    dry = False
    for r, (L, n) in enumerate(zip(list(lengths), new)):
        t0 = cu[-1]
        cu.append(t0 + max(n, 0))
        have, want = -(-max(L, 0) // page), -(-(max(L, 0) + max(n, 0)) // page)
        if want > W or n < 0 or L < 0:
            status.append(2)
        elif cu[-1] > max_tokens:
            status.append(3)
        elif want > have and (dry or want - have > len(free)):
            dry = True
            status.append(1)
        else:
            status.append(0)
            for j in range(have, want):
                table[r][j] = free.pop()
            for i in range(n):
                p = L + i
                slots[t0 + i], rows[t0 + i], context[t0 + i] = table[r][p // page] * page + p % page, r, p + 1
            lengths[r] = L + n
    return lengths, free, cu, slots, rows, context, status, table


def release(keep, lengths, table, free, page):
    lengths, free, table = list(lengths), list(free), [list(r) for r in table]
    for r, (k, L) in enumerate(zip(keep, list(lengths))):
        k = L if k < 0 else min(k, L)
        for j in range(-(-k // page), -(-L // page)):
            free.append(table[r][j])
            table[r][j] = -1
        lengths[r] = k
    return lengths, free, table


def exponent(m):
    """The least x in [-40, 48] with 127 * 2^x >= m."""
    return next((x for x in range(-40, 48) if 127 * 2.0 ** x >= m), 48)


def key_bounds(keys):
    """(int8 (2, E), exponent) of one page and head's keys (n, E), the values the cache holds."""
    k = keys.double().cpu()
    k = torch.where(torch.isnan(k), torch.zeros_like(k), k)
    x = exponent(float(k.abs().max()))
    lo, hi = torch.floor(k.amin(0) / 2.0 ** x), torch.ceil(k.amax(0) / 2.0 ** x)
    return torch.stack([lo, hi]).clamp(-127, 127).to(torch.int8), x


def choose(q, bounds, exps, top, first, last):
    """Places of the chosen pages, ascending: q (G, E), bounds (P, 2, E), exps (P), Python's own sums."""
    P = bounds.shape[0]
    scores = []
    qs = []
    for row in q.double().cpu():
        row = torch.where(torch.isnan(row), torch.zeros_like(row), row)
        y = exponent(float(row.abs().max()))
        qs.append((y, torch.round(row / 2.0 ** y).clamp(-127, 127)))
    b = bounds.double().cpu()
    for j in range(P):
        if j < first or j >= P - last:
            scores.append(math.inf)
            continue
        scores.append(max(float(torch.maximum(r * b[j, 1], r * b[j, 0]).sum()) * 2.0 ** (int(exps[j]) + y) for y, r in qs))
    return sorted(sorted(range(P), key=lambda j: (-scores[j], j))[:top])


def attention(q, K, V, scale=None):
    """q (G, E), K (n, E), V (n, D) in any type: out (G, D), lse (G), and the tolerance's parts, float64.

    ``spread`` is sum_j p_j |v_j| and ``dz`` a bound of the error of any z_j = scale q.k_j summed in
    fp32 in any order (E products, each sum off by 2^-24 of the magnitudes' sum)."""
    q, K, V = q.double(), K.double(), V.double()
    G, E = q.shape
    s = 1 / math.sqrt(E) if scale is None else scale
    if K.shape[0] == 0:
        z = q.new_zeros(G, V.shape[1])
        return z, q.new_full((G,), -math.inf), z, q.new_zeros(G)
    z = s * (q @ K.T)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    dz = (E + 4) * 2.0 ** -24 * s * (q.abs() @ K.abs().T).amax(-1)
    return p @ V, lse, p @ V.abs(), dz


# How exactly the kernels keep p and V in their product (fp32: each as two tf32 numbers, 2^-22 both).
P_STEP = {"fp32": 2.0 ** -21, "bf16": 2.0 ** -16, "fp16": 2.0 ** -16, "e4m3": 2.0 ** -11}


def tolerance(ref, lse, spread, dz, n_keys, dtype, cache):
    """Largest |out - ref| and |lse - lse_ref| that the arithmetic allows.

    A weight is off by e^(2 dz) - 1 (its own z and the sum's), by the exponential and its argument's
    product with log2 e (8 steps of 2^-24 over |z - m|, below 2^-17 for the arguments that count), by its
    rounding before the product, and each of the fp32 sums over the keys by n 2^-24 of the
    magnitudes; the result is rounded once to its type."""
    p = torch.expm1(2 * dz)[:, None] + 2.0 ** -17 + P_STEP[cache] + 2 * (n_keys + 8) * 2.0 ** -24
    out = torch.finfo(dtype).eps / 2 * (ref.abs() + p * spread) + p * spread + torch.finfo(dtype).tiny
    dl = dz + 2.0 ** -17 + (n_keys + 8) * 2.0 ** -24 + 2.0 ** -22 * lse.abs().clamp(max=1e30)
    return out, dl
