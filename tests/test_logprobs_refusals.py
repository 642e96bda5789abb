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


def test_refused_calls_allocate_nothing(monkeypatch):
    """A refused [T, v] gradient would be the largest tensor of the step."""
    I64, BF = torch.int64, torch.bfloat16
    y, h, E = torch.zeros(T, dtype=I64), torch.zeros(T, 16, dtype=BF), torch.zeros(V, 16, dtype=BF)
    short, half, ids3 = torch.zeros(T - 1), X.half(), IDS[:3]
    f16, f64 = torch.float16, torch.float64

    def empty(*a, **k):
        raise AssertionError("allocated")

    monkeypatch.setattr(torch, "empty", empty)
    fwd, bwd, distill = tpl.vp_logprobs_fwd, tpl.vp_logprobs_bwd, tpl.vp_distill
    lfwd, lbwd = tpl.tp_linear_logprobs_fwd, tpl.tp_linear_logprobs_dlogits
    for call in (lambda: fwd(half, y, 4), lambda: fwd(X, y[:3], 4, top_k=3),
                 lambda: bwd(X, y, short, R, R, R, 4), lambda: bwd(half, y, R, R, R, R, 4),
                 lambda: bwd(X, y, R, R, R, R, 4, grad_dtype=f16),
                 lambda: bwd(X.t(), y, R, R, R, R, 4),
                 lambda: distill(half, IDS, TEACHER, 4), lambda: distill(X, ids3, TEACHER, 4),
                 lambda: distill(X, IDS, TEACHER, 4, grad_dtype=f64),
                 lambda: lfwd(h, E, y[:3], 4), lambda: lbwd(h, E, y, short, R, R, R, 4),
                 lambda: lbwd(h, E.float(), y, R, R, R, R, 4)):
        with pytest.raises((ValueError, TypeError)):
            call()
