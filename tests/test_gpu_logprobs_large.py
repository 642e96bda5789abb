"""Matrices of more than 2^32 elements: the last rows, whose offsets pass 32
bits, are bit for bit what a call on those rows alone gives (every row is
worked on by the same kernel in the same order, so nothing but an offset can
differ)."""
import pytest
import torch

import linear_layers_b200 as tpl

pytestmark = pytest.mark.gpu

T, V, LAST = 86016, 50257, 2048
assert T * V > 2**32


@pytest.fixture(scope="module")
def logits():
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    for rows in (slice(0, LAST), slice(T - LAST, T)):
        x[rows].normal_(0.0, 2.0, generator=g)
    x[LAST:T - LAST] = 0.0
    x[LAST:T - LAST, ::7] = 1.0
    return x


def _teacher(g):
    ids = torch.randint(0, V, (T, 8), generator=g, device="cuda", dtype=torch.int32)
    return ids, torch.randn(T, 8, generator=g, device="cuda")


def test_log_probabilities_and_their_gradient(logits):
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    st = tpl.new_status()
    r = tpl.vp_logprobs_fwd(logits, y, 1, top_k=3, dev_status=st)
    tail = logits[T - LAST:]
    want = tpl.vp_logprobs_fwd(tail, y[T - LAST:], 1, top_k=3)
    for k, w in want.items():
        assert torch.equal(r[k][T - LAST:], w), k
    dlp = torch.randn(T, generator=g, device="cuda")
    de = torch.randn(T, generator=g, device="cuda")
    d = tpl.vp_logprobs_bwd(logits, y, r["lse"], r["entropy"], dlp, de, 1, dev_status=st)
    last = tpl.vp_logprobs_bwd(tail, y[T - LAST:], want["lse"], want["entropy"], dlp[T - LAST:],
                               de[T - LAST:], 1)
    assert torch.equal(d[T - LAST:], last) and last.any()
    assert int(st.item()) == 0


def test_distillation(logits):
    ids, t = _teacher(torch.Generator(device="cuda").manual_seed(2))
    st = tpl.new_status()
    r = tpl.vp_distill(logits, ids, t, 1, dev_status=st)
    want = tpl.vp_distill(logits[T - LAST:], ids[T - LAST:], t[T - LAST:], 1)
    for k in ("loss", "lse", "dlogits"):
        assert torch.equal(r[k][T - LAST:], want[k]), k
    assert want["dlogits"].any()
    alone = tpl.vp_distill(logits, ids, t, 1, with_grad=False, dev_status=st)
    last = tpl.vp_distill(logits[T - LAST:], ids[T - LAST:], t[T - LAST:], 1, with_grad=False)
    assert torch.equal(alone["loss"][T - LAST:], last["loss"])
    assert int(st.item()) == 0


def test_gradient_without_the_logits():
    v, h = 50304, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    H = torch.randn(T, h, generator=g, device="cuda").bfloat16()
    E = (torch.randn(v, h, generator=g, device="cuda") * 0.2).bfloat16()
    y = torch.randint(0, v, (T,), generator=g, device="cuda")
    gr = torch.randn(T, generator=g, device="cuda")
    r = tpl.tp_linear_logprobs_fwd(H, E, y, 1)
    d = tpl.tp_linear_logprobs_dlogits(H, E, y, r["lse"], r["entropy"], gr, gr, 1)
    s = slice(T - LAST, T)
    rl = tpl.tp_linear_logprobs_fwd(H[s], E, y[s], 1)
    for k in rl:
        assert torch.equal(r[k][s], rl[k]), k
    last = tpl.tp_linear_logprobs_dlogits(H[s], E, y[s], rl["lse"], rl["entropy"], gr[s], gr[s], 1)
    assert torch.equal(d[s], last) and last.any()
