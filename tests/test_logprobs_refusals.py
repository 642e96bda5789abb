"""Calls of the log-probability and distillation entry points that the binding
turns down, on the CPU: nothing is computed, allocated or written by them."""
import pytest
import torch

import linear_layers_b200 as tpl

T, V, K = 6, 40, 5
X, R = torch.zeros(T, V), torch.zeros(T)
IDS, TEACHER = torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)


def test_a_loss_alone_takes_no_gradient_buffer():
    """with_grad=False writes no gradient: not into a buffer, not over the logits."""
    for d in (torch.zeros(T, V), X):
        with pytest.raises(ValueError, match="with_grad"):
            tpl.vp_distill(X, IDS, TEACHER, 4, with_grad=False, dlogits=d)
    with pytest.raises(RuntimeError, match="no CPU path"):
        tpl.vp_distill(X, IDS, TEACHER, 4, dlogits=X)
