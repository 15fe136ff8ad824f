"""Paged-cache entry points without a GPU: what they refuse, before anything is enqueued."""
import ctypes
import re
import os

import pytest
import torch

import thinned_softmax_attention_b200 as T
from thinned_softmax_attention_b200 import paged

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "thin_attn.h")
P = 0x1000   # an aligned pointer that no refused call follows


def call(name, fmt, values):
    s = getattr(paged._functions(), f"thin_attn_paged_{name}")(fmt.pack(fmt.size, *values), None)
    return s, T.lib().thin_attn_last_error().decode()


def refused(name, fmt, fields, good, **change):
    """Status of a call with the good values changed."""
    v = dict(zip(fields, good))
    assert set(change) <= set(v)
    v.update(change)
    s, msg = call(name, fmt, list(v.values()))
    assert s in (1, 5) and msg, (change, s, msg)


def fields_of(struct):
    """Field names of an argument struct in the header, without struct_size, with its C types' sizes."""
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + struct + ";", src).group(1)
    names, code = [], ""
    for decl in body.split(";"):
        decl = " ".join(decl.split())
        if not decl:
            continue
        m = re.match(r"((?:const )?[a-z0-9_]+)\s*(.*)", decl)
        for n in m.group(2).split(","):
            n = n.strip()
            t = m.group(1).replace("const ", "")
            code += "P" if "*" in n else {"int32_t": "i", "uint32_t": "I", "int64_t": "q", "float": "f", "size_t": "N"}[t]
            names.append(n.strip("* "))
    return names[1:], code


STRUCTS = {"plan": paged._PLAN, "release": paged._RELEASE, "append": paged._APPEND, "attention": paged._ATTENTION}


@pytest.mark.parametrize("name", list(STRUCTS))
def test_argument_structs_match_the_header(name):
    fields, code = fields_of(f"thin_attn_paged_{name}_args")
    import struct
    assert struct.Struct("@" + code).size == STRUCTS[name].size
    expanded = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), STRUCTS[name].format)
    assert expanded == "@" + code
    wrong = b"\7" * STRUCTS[name].size
    assert getattr(paged._functions(), f"thin_attn_paged_{name}")(wrong, None) == 1
    assert "struct_size" in T.lib().thin_attn_last_error().decode()
    assert getattr(paged._functions(), f"thin_attn_paged_{name}")(None, None) == 1


def test_plan_and_release_refusals():
    f, _ = fields_of("thin_attn_paged_plan_args")
    good = [0, 4, 8, 16, 10, 32, 0, P, P, P, 8, P, P, P, P, P, P, P, P, P]
    for change in (dict(R=-1), dict(W=-1), dict(page=0), dict(n_pages=-1), dict(max_tokens=-1), dict(R=16385), dict(lengths=0),
                   dict(n_new=0), dict(table=0), dict(free_pages=0), dict(n_free=0), dict(lengths_out=0), dict(n_free_out=0),
                   dict(cu=0), dict(slots=0), dict(rows=0), dict(context=0), dict(status=0)):
        refused("plan", paged._PLAN, f, good, **change)
    f, _ = fields_of("thin_attn_paged_release_args")
    good = [0, 4, 8, 16, 10, P, P, P, 8, P, P]
    for change in (dict(R=-1), dict(W=-1), dict(page=0), dict(n_pages=-1), dict(R=16385), dict(keep=0), dict(lengths=0),
                   dict(table=0), dict(free_pages=0), dict(n_free=0)):
        refused("release", paged._RELEASE, f, good, **change)


def test_append_refusals():
    f, _ = fields_of("thin_attn_paged_append_args")
    good = [0, 1, 1, 4, 2, 64, 64, 16, 10, P, 128, 64, P, 128, 64, P, P, 2048, 1024, 64, P, 2048, 1024, 64, 0, 0, 0, 0]
    for change in (dict(dtype=3), dict(dtype=7), dict(cache_dtype=0), dict(cache_dtype=2), dict(cache_dtype=3), dict(N=-1), dict(H=0),
                   dict(E=0), dict(E=12), dict(E=264), dict(D=4), dict(D=512), dict(page=0), dict(page=65537), dict(n_pages=0),
                   dict(N=2 ** 31 - 1), dict(k=0), dict(v=0), dict(slots=0), dict(k_pages=0), dict(v_pages=0), dict(k=P + 8),
                   dict(v_pages=P + 2), dict(k_token=132), dict(k_head=63), dict(v_head=4), dict(kp_row=65), dict(vp_page=1),
                   dict(kp_head=1020), dict(bounds=P), dict(exps=P), dict(bounds=P + 4, exps=P),
                   dict(dtype=0, cache_dtype=3, k_scale=P, v_scale=P), dict(cache_dtype=3, k_scale=P, v_scale=P, E=72)):
        refused("append", paged._APPEND, f, good, **change)
    v = dict(zip(f, good))
    v["N"] = 0
    assert call("append", paged._APPEND, list(v.values()))[0] == 0   # nothing to do


def test_attention_refusals():
    f, _ = fields_of("thin_attn_paged_attention_args")
    good = [0, 1, 1, 4, 4, 8, 8, 2, 64, 64, 16, 10, 0, 0, 0, 0, 0.0, P, 512, 64, P, 2048, 1024, 64, P, 2048, 1024, 64, P, 8, P, 0,
            0, 0, 0, 0, 0, P, 512, 64, 0, P, 1 << 30]
    for change in (dict(dtype=3), dict(cache_dtype=0), dict(cache_dtype=3), dict(N=-1), dict(R=-1), dict(W=-1), dict(N=5), dict(Hq=7),
                   dict(Hq=1), dict(H=0), dict(E=12), dict(E=264), dict(D=0), dict(page=0), dict(n_pages=0), dict(window=-1),
                   dict(top=-1), dict(top=4097, last=1), dict(top=4, last=0), dict(top=4, first=-1, last=1),
                   dict(top=4, first=4, last=1), dict(top=4, last=1), dict(top=4, last=1, bounds=P + 8, exps=P),
                   dict(top=4, last=1, window=3, bounds=P, exps=P), dict(W=2 ** 27, page=16), dict(N=2 ** 28, R=2 ** 28),
                   dict(q=0), dict(k_pages=0), dict(v_pages=0), dict(table=0), dict(lengths=0), dict(out=0), dict(q=P + 4),
                   dict(out=P + 8), dict(q_token=516), dict(q_head=60), dict(kp_page=3), dict(vp_row=68), dict(out_head=36),
                   dict(cache_dtype=3, k_scale=P), dict(workspace=0), dict(workspace=P + 16), dict(workspace_bytes=0)):
        if "workspace" in " ".join(change) and paged._workspace_bytes(1, 1, 4, 4, 8, 8, 2, 64, 64, 16, 10, 0, 0, 0, 0, False) == 0:
            continue
        refused("attention", paged._ATTENTION, f, good, **change)
    v = dict(zip(f, good))
    v["N"] = 0
    assert call("attention", paged._ATTENTION, list(v.values()))[0] == 0
    n = ctypes.c_size_t()
    assert paged._functions().thin_attn_paged_attention_workspace(None, ctypes.byref(n)) == 1


def test_workspace_grows_with_the_call():
    size = lambda N, W, top: paged._workspace_bytes(1, 1, N, N, W, 8, 2, 64, 64, 16, 100, 0, top, 1 if top else 0, 1 if top else 0, False)
    assert 0 < size(4, 8, 0) <= size(64, 8, 0) and size(4, 8, 4) < size(64, 8, 4) < size(64, 8, 400)


def test_tensors_off_the_gpu_are_refused():
    q, kp = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    for bad in (lambda: T.paged_attention(q, kp, kp, i(0)[None], i(3)), lambda: T.paged_attention(q, kp, kp, i(0)[None], i(3), return_lse=True),
                lambda: T.paged_append(q[:, :2], q[:, :2], torch.zeros(1, dtype=torch.int64), kp, kp),
                lambda: T.paged_plan(i(3), i(1), i(0)[None], i(0), i(1), 16, 4),
                lambda: T.paged_release(i(3), i(1), i(0)[None], i(0), i(1), 16)):
        with pytest.raises(ValueError, match="CUDA"):
            bad()


def test_plain_plan_and_release_are_inverse():
    """The oracle itself: releasing everything gives every page back."""
    from tests import plain_paged as PP
    lengths, free, cu, slots, rows, context, status, table = PP.plan([0, 5], [9, 4], [[-1] * 3, [7, -1, -1]], [1, 2, 3], 8, 20)
    assert status == [0, 0] and lengths == [9, 9] and free == [] and table == [[3, 2, -1], [7, 1, -1]]
    assert slots[:13] == [24 + i for i in range(8)] + [16] + [56 + 5, 56 + 6, 56 + 7, 8] and context[12] == 9
    assert sorted(PP.release([0, 0], lengths, table, free, 8)[1]) == [1, 2, 3, 7]


def test_plain_bounds_by_hand():
    from tests import plain_paged as PP
    b, x = PP.key_bounds(torch.tensor([[127.0, -0.4], [3.2, 0.0]]))
    assert x == 0 and b.tolist() == [[3, -1], [127, 0]]
    assert [PP.exponent(m) for m in (0, 127, 127.5, 1.0, float("inf"))] == [-40, 0, 1, -6, 48]
    assert PP.choose(torch.tensor([[1.0, -1.0]]), torch.tensor([[[0, 0], [1, 1]], [[-5, -5], [0, 0]], [[1, 0], [2, 0]], [[0, 0], [0, 0]]]),
                     [0, 0, 1, 0], 3, 0, 1) == [1, 2, 3]
