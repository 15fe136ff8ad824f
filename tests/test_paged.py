"""Paged-cache entry points without a GPU: what they refuse, before anything is enqueued."""
import ctypes
import os
import re
import struct

import pytest
import torch

import thinned_softmax_attention_b200 as T

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "thin_attn.h")
P = 0x1000   # an aligned pointer that no refused call follows


def entry(name):
    f = getattr(T.lib(), f"thin_attn_paged_{name}")
    f.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
    return f


def packed(name, **change):
    """The argument struct of a good call with some values changed."""
    fields, code = fields_of(f"thin_attn_paged_{name}_args")
    v = dict(zip(fields, GOOD[name]))
    assert len(fields) == len(GOOD[name]) and set(change) <= set(v)
    v.update(change)
    fmt = struct.Struct("@" + code)
    return fmt.pack(fmt.size, *v.values())


def refused(name, **change):
    s = entry(name)(packed(name, **change), None)
    msg = T.lib().thin_attn_last_error().decode()
    assert s in (1, 5) and msg, (change, s, msg)


GOOD = {
    "plan": [0, 4, 8, 16, 10, 32, 0, P, P, P, 8, P, P, P, P, P, P, P, P, P],
    "release": [0, 4, 8, 16, 10, P, P, P, 8, P, P],
    "append": [0, 1, 1, 4, 2, 64, 64, 16, 10, P, 128, 64, P, 128, 64, P, P, 2048, 1024, 64, P, 2048, 1024, 64, 0, 0, 0, 0],
    "attention": [0, 1, 1, 4, 4, 8, 8, 2, 64, 64, 16, 10, 0, 0, 0, 0, 0.0, P, 512, 64, P, 2048, 1024, 64, P, 2048, 1024, 64, P, 8, P,
                  0, 0, 0, 0, 0, 0, P, 512, 64, 0, P, 1 << 30],
}


def fields_of(name):
    """Field names of an argument struct in the header, without struct_size, with its C types' sizes."""
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", src).group(1)
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


@pytest.mark.parametrize("name", list(GOOD))
def test_struct_size_and_null_are_refused(name):
    assert entry(name)(b"\7" * 512, None) == 1
    assert "struct_size" in T.lib().thin_attn_last_error().decode()
    assert entry(name)(None, None) == 1


def test_plan_and_release_refusals():
    for change in (dict(R=-1), dict(W=-1), dict(page=0), dict(n_pages=-1), dict(max_tokens=-1), dict(R=16385), dict(lengths=0),
                   dict(n_new=0), dict(table=0), dict(free_pages=0), dict(n_free=0), dict(lengths_out=0), dict(n_free_out=0),
                   dict(cu=0), dict(slots=0), dict(rows=0), dict(context=0), dict(status=0)):
        refused("plan", **change)
    for change in (dict(R=-1), dict(W=-1), dict(page=0), dict(n_pages=-1), dict(R=16385), dict(keep=0), dict(lengths=0),
                   dict(table=0), dict(free_pages=0), dict(n_free=0)):
        refused("release", **change)


def test_append_refusals():
    for change in (dict(dtype=3), dict(dtype=7), dict(cache_dtype=0), dict(cache_dtype=2), dict(cache_dtype=3), dict(N=-1), dict(H=0),
                   dict(E=0), dict(E=12), dict(E=264), dict(D=4), dict(D=512), dict(page=0), dict(page=65537), dict(n_pages=0),
                   dict(N=2 ** 31 - 1), dict(k=0), dict(v=0), dict(slots=0), dict(k_pages=0), dict(v_pages=0), dict(k=P + 8),
                   dict(v_pages=P + 2), dict(k_token=132), dict(k_head=63), dict(v_head=4), dict(kp_row=65), dict(vp_page=1),
                   dict(kp_head=1020), dict(bounds=P), dict(exps=P), dict(bounds=P + 4, exps=P),
                   dict(dtype=0, cache_dtype=3, k_scale=P, v_scale=P), dict(cache_dtype=3, k_scale=P, v_scale=P, E=72)):
        refused("append", **change)
    assert entry("append")(packed("append", N=0), None) == 0   # nothing to do


def test_attention_refusals():
    for change in (dict(dtype=3), dict(cache_dtype=0), dict(cache_dtype=3), dict(N=-1), dict(R=-1), dict(W=-1), dict(N=5), dict(Hq=7),
                   dict(Hq=1), dict(H=0), dict(E=12), dict(E=264), dict(D=0), dict(page=0), dict(n_pages=0), dict(window=-1),
                   dict(top=-1), dict(top=4097, last=1), dict(top=4, last=0), dict(top=4, first=-1, last=1),
                   dict(top=4, first=4, last=1), dict(top=4, last=1), dict(top=4, last=1, bounds=P + 8, exps=P),
                   dict(top=4, last=1, window=3, bounds=P, exps=P), dict(W=2 ** 27, page=16), dict(N=2 ** 28, R=2 ** 28),
                   dict(N=70000, R=70000, top=4, last=1, bounds=P, exps=P), dict(Hq=1024, top=4, last=1, bounds=P, exps=P),
                   dict(q=0), dict(k_pages=0), dict(v_pages=0), dict(table=0), dict(lengths=0), dict(out=0), dict(q=P + 4),
                   dict(out=P + 8), dict(q_token=516), dict(q_head=60), dict(kp_page=3), dict(vp_row=68), dict(out_head=36),
                   dict(cache_dtype=3, k_scale=P), dict(workspace=0), dict(workspace=P + 16), dict(workspace_bytes=0)):
        refused("attention", **change)
    assert entry("attention")(packed("attention", N=0), None) == 0


def workspace(**change):
    n = ctypes.c_size_t()
    f = T.lib().thin_attn_paged_attention_workspace
    f.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)]
    assert f(packed("attention", **change), ctypes.byref(n)) == 0
    assert f(None, ctypes.byref(n)) == 1 and f(packed("attention"), None) == 1
    return f(packed("attention", **change), ctypes.byref(n)) or n.value


def test_workspace_grows_with_the_call():
    pick = dict(top=4, first=1, last=1)
    assert 0 < workspace() <= workspace(N=64, R=64) and workspace(**pick) < workspace(N=64, R=64, **pick)
    assert workspace(**pick) < workspace(W=4096, **pick)


def test_tensors_off_the_gpu_are_refused():
    q, kp = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    b = (torch.zeros(2, 2, 2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.int8))
    for bad in (lambda: T.paged_attention(q, kp, kp, i(0)[None], i(3)), lambda: T.paged_attention(q, kp, kp, i(0)[None], i(3), return_lse=True),
                lambda: T.paged_sparse_attention(q, kp, kp, i(0)[None], i(3), b, 4),
                lambda: T.paged_append(q[:, :2], q[:, :2], torch.zeros(1, dtype=torch.int64), kp, kp),
                lambda: T.paged_plan(i(3), i(1), i(0)[None], i(0), i(1), 16, 4),
                lambda: T.paged_release(i(3), i(1), i(0)[None], i(0), i(1), 16)):
        with pytest.raises(ValueError, match="CUDA"):
            bad()
    for bad in (lambda: T.paged_attention(None, kp, kp, i(0)[None], i(3)), lambda: T.paged_plan([3], i(1), i(0)[None], i(0), i(1), 16, 4)):
        with pytest.raises(ValueError, match="tensor"):
            bad()


def test_binding_without_the_library(monkeypatch):
    monkeypatch.setattr(T, "_lib", None)
    monkeypatch.setattr(T, "LIB_PATH", "/no_such_dir/libthin_attn.so")
    from thinned_softmax_attention_b200 import paged
    monkeypatch.setattr(paged, "_binding", None)
    with pytest.raises(ImportError, match="is missing"):
        T.paged_plan(None, None, None, None, None, 1, 1)


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


def test_overlapping_table_rows_and_odd_scales_are_refused():
    for name in ("plan", "release"):
        refused(name, table_row=7)
        refused(name, table_row=0)
        refused(name, table_row=-8)
    for scale in (-1.0, float("inf"), float("nan")):
        refused("attention", scale=scale)


def test_more_places_than_a_plan_counts_are_refused():
    refused("plan", max_tokens=2 ** 31 - 1)
    refused("plan", max_tokens=2 ** 30)
