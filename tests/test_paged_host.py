"""The paged operators' host side without a GPU: the binding's refusals and its build."""
import pytest
import torch

import thinned_softmax_attention_b200 as T


def test_inputs_that_require_a_gradient_are_refused():
    q, kp = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    b = (torch.zeros(2, 2, 2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.int8))
    leaf = lambda x: x.clone().requires_grad_()
    slot = torch.zeros(1, dtype=torch.int64)
    for call in (lambda: T.paged_attention(leaf(q), kp, kp, i(0)[None], i(3)), lambda: T.paged_attention(q, leaf(kp), kp, i(0)[None], i(3)),
                 lambda: T.paged_attention(q, kp, leaf(kp), i(0)[None], i(3)), lambda: T.paged_attention(leaf(q) * 2, kp, kp, i(0)[None], i(3)),
                 lambda: T.paged_sparse_attention(leaf(q), kp, kp, i(0)[None], i(3), b, 4),
                 lambda: T.paged_append(leaf(q[:, :2]), q[:, :2], slot, kp, kp), lambda: T.paged_append(q[:, :2], leaf(q[:, :2]), slot, kp, kp)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # then the next refusal
            call()


def test_the_library_is_built_first_and_without_the_binding(monkeypatch, tmp_path):
    """Neither g++, nor torch's headers are needed for libthin_attn.so, and a binding that fails to build does not keep it back."""
    from thinned_softmax_attention_b200 import build as B
    done = []

    def no_binding():
        done.append("binding")
        raise OSError("no compiler")

    monkeypatch.setattr(B, "build_library", lambda verbose=False: done.append("library"))
    monkeypatch.setattr(B, "build_binding", no_binding)
    for force, current in ((True, True), (False, False)):
        monkeypatch.setattr(B, "newer", lambda target, inputs: current)
        del done[:]
        with pytest.raises(OSError):
            B.build(force=force)
        assert done == ["library", "binding"]


def test_the_binding_is_built_anew_for_another_torch(monkeypatch, tmp_path):
    from thinned_softmax_attention_b200 import build as B
    stamp = tmp_path / "torch"
    monkeypatch.setattr(B, "BINDING_TORCH", str(stamp))
    monkeypatch.setattr(B, "newer", lambda target, inputs: True)
    assert not B.binding_up_to_date()
    stamp.write_text(B.torch_version())
    assert B.binding_up_to_date() and B.up_to_date()
    monkeypatch.setattr(B, "torch_version", lambda: "0.0")
    assert not B.binding_up_to_date()
    built = []
    monkeypatch.setattr(B, "build_binding", lambda: built.append(1))
    B.build()
    assert built == [1]


def test_scales_beyond_fp32_are_refused():
    """scale log2 e, which the kernel multiplies scores by, would be infinite, and a score of 0 NaN."""
    from tests.test_paged import refused
    for scale in (2.4e38, 3.4e38, float("inf"), float("nan"), -1e-30):
        refused("attention", scale=scale)
