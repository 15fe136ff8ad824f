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
