"""Log-probabilities and entropy without the logits matrix, and their gradient,
on the GPU against the fp64 oracle.

The GEMM adds h products in fp32, at most h/16 roundings of partial sums of
size ~10 or less: below 1e-3 of a logit for h <= 4096 (in chunks of 1024, whose
sums are added in fp32, less), and the log-probability
and entropy follow the logits one to one, so the bar is TOL_XENT relative to
values of 8 or more, as for the cross-entropy without the logits.  The bf16
gradient has the bf16 bar.
"""
import math
import time

import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
import tp_inputs
from oracle import tp_oracle as O
from tests.gpu_helpers import TOL_BF16, TOL_XENT, assert_close, f64, guarded

pytestmark = pytest.mark.gpu


def _inputs(T, v, h, seed):
    inp = tp_inputs.vocab_inputs(T, v, h, e_std=1.6 / math.sqrt(h), seed=seed)
    return inp["H"], inp["E"], inp["targets"]


def _check_fwd(r, ref):
    for k in ("logprob", "entropy", "lse"):
        got, want = f64(r[k]), ref[k]
        assert np.array_equal(np.isnan(got), np.isnan(want)), k
        ok = ~np.isnan(want)
        assert np.all(np.abs(got[ok] - want[ok]) <= TOL_XENT * np.maximum(np.abs(want[ok]), 4.0)), k


SHAPES = [(1, 2048, 64, 8), (300, 1000, 256, 4), (16, 2048, 64, 8), (200, 136, 512, 2),
          (513, 4096, 328, 1), (3, 50304, 1600, 4), (130, 8, 8, 1), (513, 20000, 2056, 1)]


@pytest.mark.parametrize("T,v,h,N", SHAPES)
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_forward_and_gradient(T, v, h, N, scale):
    H, E, y = _inputs(T, v, h, seed=T)
    st = tpl.new_status()
    Hd, Ed, yd = H.cuda(), E.cuda(), y.cuda()
    bufs, guards = {}, []
    for k in ("logprob", "entropy", "lse"):
        bufs[k], g = guarded((T,), torch.float32)
        guards.append(g)
    r = tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, N, scale=scale, dev_status=st, **bufs)
    for g in guards:
        g.check()
    L = O.logits(H, E)
    _check_fwd(r, O.logprobs(L, y, scale))
    gen = torch.Generator().manual_seed(1)
    dlp, de = torch.randn(T, generator=gen), 0.2 * torch.randn(T, generator=gen)
    if T > 2:
        dlp[1], de[1] = 0.0, 0.0
    out, guard = guarded((T, v), torch.bfloat16)
    for a, b in ((dlp, de), (dlp, None), (None, de)):
        tpl.tp_linear_logprobs_dlogits(Hd, Ed, yd, r["lse"], r["entropy"],
                                       None if a is None else a.cuda(),
                                       None if b is None else b.cuda(), N, scale=scale, dlogits=out,
                                       dev_status=st)
        guard.check("dlogits")
        want = O.logprobs_bwd(L, y, a, b, scale)
        assert_close("dlogits", out, want, TOL_BF16)
        if T > 2:
            assert not out[1].any()
    assert int(st.item()) == 0


@pytest.mark.parametrize("h", [1024, 1032, 2056, 3080])
@pytest.mark.parametrize("T,v", [(5, 1000), (300, 2056)])
def test_hidden_sizes_around_the_accumulation_chunk(T, v, h):
    H, E, y = _inputs(T, v, h, seed=h)
    Hd, Ed, yd = H.cuda(), E.cuda(), y.cuda()
    r = tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, 1)
    L = O.logits(H, E)
    _check_fwd(r, O.logprobs(L, y))
    g = torch.linspace(-1.0, 1.0, T)
    d = tpl.tp_linear_logprobs_dlogits(Hd, Ed, yd, r["lse"], r["entropy"], g.cuda(), g.cuda(), 1)
    assert_close("dlogits", d, O.logprobs_bwd(L, y, g, g), TOL_BF16)


@pytest.mark.parametrize("T", [1, 2, 3])
@pytest.mark.parametrize("v,h", [(1, 8), (31, 16), (33, 264), (1003, 1608), (50257, 512), (70, 8192)])
def test_one_and_two_tokens(T, v, h):
    """Slices that end inside the table, rows of H shorter than a warp's reach,
    every output alone, a target outside the vocabulary."""
    H, E, y = _inputs(T, v, h, seed=v + h)
    Hd, Ed, yd = H.cuda(), E.cuda(), y.cuda()
    ref = O.logprobs(O.logits(H, E), y, 1.25)
    bufs, guards = {}, []
    for k in ("logprob", "entropy", "lse"):
        bufs[k], g = guarded((T,), torch.float32)
        guards.append(g)
    st = tpl.new_status()
    need = tpl.tp_workspace_bytes(tpl.OP_LINEAR_LOGPROBS, T, h, v, 1)
    ws, g = guarded((need,), torch.uint8, fill=0xFF)
    guards.append(g)
    r = tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, 1, scale=1.25, ws=ws, dev_status=st, **bufs)
    for g in guards:
        g.check()
    _check_fwd(r, ref)
    assert int(st.item()) == 0
    again = tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, 1, scale=1.25)
    for k in bufs:
        assert torch.equal(r[k], again[k]), k
    bare = tpl.tp_linear_logprobs_fwd(Hd, Ed, None, 1, scale=1.25)
    assert torch.equal(bare["lse"], r["lse"]) and torch.equal(bare["entropy"], r["entropy"])
    yd[T - 1] = v
    bad = tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, 1, scale=1.25, dev_status=st)
    assert int(st.item()) == tpl.DEVERR_RANGE
    assert torch.isnan(bad["logprob"][T - 1]) and torch.equal(bad["lse"], r["lse"])
    assert torch.equal(bad["logprob"][:T - 1], r["logprob"][:T - 1])


def test_one_token_with_infinite_and_nan_logits():
    H = torch.ones(1, 64).bfloat16()
    E = (torch.randn(100, 64, generator=torch.Generator().manual_seed(4)) * 0.1).bfloat16()
    y = torch.tensor([7])
    E[40, 3] = -math.inf                          # a token of probability 0
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E.cuda(), y.cuda(), 1)
    _check_fwd(r, O.logprobs(O.logits(H, E), y))
    E[41, 5] = math.nan
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E.cuda(), y.cuda(), 1)
    for k in ("logprob", "entropy", "lse"):
        assert torch.isnan(r[k]).all(), k


def test_long_sums_of_one_sign():
    """Logits of 16 as 65536 positive products.  Within a chunk of 1024 the
    tensor core adds 64 times and truncates by at most 2^-22 of the sum so far;
    64 chunk sums are added in fp32 (2^-24 of the sum each); lse adds a few
    roundings of its 21.  One chain of 4096 truncations would be off by about
    4096·(1/2)·2^-24.5 = 8.6e-5 of the logits, 1.4e-3."""
    T, v, h = 16, 136, 65536
    gen = torch.Generator().manual_seed(3)
    H = (0.5 + torch.rand(T, h, generator=gen)).bfloat16()
    E = ((0.5 + torch.rand(v, h, generator=gen)) * (16.0 / h)).bfloat16()
    y = torch.randint(0, v, (T,), generator=gen)
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E.cuda(), y.cuda(), 1)
    z = H.double().numpy() @ E.double().numpy().T
    ref = O.logprobs(z, y)
    tol = z.max() * (64 * 2.0**-22 + 64 * 2.0**-24) + 8 * 21 * 2.0**-24
    assert np.all(np.abs(f64(r["lse"]) - ref["lse"]) <= tol)
    assert np.all(np.abs(f64(r["logprob"]) - ref["logprob"]) <= 2 * tol)


def test_forward_of_an_odd_vocabulary_without_targets():
    H, E, _ = _inputs(70, 1003, 64, seed=5)
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E.cuda(), None, 1)
    ref = O.logprobs(O.logits(H, E))
    assert r["logprob"] is None
    for k in ("entropy", "lse"):
        assert np.all(np.abs(f64(r[k]) - ref[k]) <= TOL_XENT * np.maximum(np.abs(ref[k]), 4.0))


def test_bad_targets_and_padded_rows():
    T, v = 40, 520
    H, E, y = _inputs(T, v, 64, seed=6)
    y = y.clone()
    y[3], y[7] = -1, v
    st = tpl.new_status()
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E.cuda(), y.cuda(), 2, dev_status=st)
    L = O.logits(H, E)
    _check_fwd(r, O.logprobs(L, y))
    assert int(st.item()) == tpl.DEVERR_RANGE
    g = torch.ones(T)
    g[7] = 0.0                                   # padded: zero, not flagged
    st = tpl.new_status()
    d = tpl.tp_linear_logprobs_dlogits(H.cuda(), E.cuda(), y.cuda(), r["lse"], None, g.cuda(), None,
                                       2, dev_status=st)
    assert int(st.item()) == tpl.DEVERR_RANGE
    assert torch.isnan(d[3]).all() and not d[7].any()
    g[3] = 0.0
    st = tpl.new_status()
    d = tpl.tp_linear_logprobs_dlogits(H.cuda(), E.cuda(), y.cuda(), r["lse"], None, g.cuda(), None,
                                       2, dev_status=st)
    assert int(st.item()) == 0
    assert_close("dlogits", d, O.logprobs_bwd(L, y, g, None), TOL_BF16)


def test_policy_step_matches_the_path_through_the_logits():
    """Hidden states to log-probabilities, the gradient at the logits and the
    output layer's backward: without the logits matrix, and through it."""
    T, v, h = 160, 4096, 256
    H, E, y = (a.cuda() for a in _inputs(T, v, h, seed=7))
    adv = torch.randn(T, generator=torch.Generator().manual_seed(3)).cuda() / T
    de = torch.full((T,), -0.01 / T, device="cuda")
    a = tpl.tp_linear_logprobs_fwd(H, E, y, 4, scale=1.25)
    da = tpl.tp_linear_logprobs_dlogits(H, E, y, a["lse"], a["entropy"], adv, de, 4, scale=1.25)
    L = tpl.tp_logits_fwd(H, E, 4)
    b = tpl.vp_logprobs_fwd(L, y, 4, scale=1.25)
    db = tpl.vp_logprobs_bwd(L, y, b["lse"], b["entropy"], adv, de, 4, scale=1.25)
    for k in ("logprob", "entropy", "lse"):
        # the same accumulators, summed in another order: 2·B of 4096 columns and roundings
        assert float((a[k] - b[k]).abs().max()) < 1e-4, k
    ga, gb = tpl.tp_logits_bwd(da, H, E, 4), tpl.tp_logits_bwd(db, H, E, 4)
    for p, q in zip(ga, gb):
        assert_close("gradient", p, f64(q), TOL_BF16)


def test_workspace_is_shared_by_two_captured_graphs_in_turn():
    T, v, h = 64, 1000, 128
    H, E, y = (a.cuda() for a in _inputs(T, v, h, seed=8))
    ws = torch.empty(tpl.tp_workspace_bytes(tpl.OP_LINEAR_LOGPROBS, T, h, v, 1), dtype=torch.uint8,
                     device="cuda")
    want = tpl.tp_linear_logprobs_fwd(H, E, y, 1)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = tpl.tp_linear_logprobs_fwd(H, E, y, 1, ws=ws)
        graphs.append((g, r))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, r in graphs:
        for k in want:
            assert torch.equal(r[k], want[k]), k


@pytest.mark.parametrize("tile", ["2x256", "1x256", "2x256t", "1x128"])
@pytest.mark.parametrize("unit,kblock", [(0, 1), (0, 20), (1, 16), (1, 33)])
def test_a_stalled_producer_times_out_and_the_next_call_is_right(tile, unit, kblock, monkeypatch):
    """The GEMM's bounded waits between the chunks of K (36 k-blocks of 64, 16 to a
    chunk) end by their limit and leave the context usable.  The tile shapes
    that these epilogues do not take fall back to one that they do."""
    monkeypatch.setenv("TP_GEMM_TILE", tile)
    T, v, h = 300, 1024, 2304
    H, E, y = _inputs(T, v, h, seed=9)
    Hd, Ed, yd = H.cuda(), E.cuda(), y.cuda()
    L = O.logits(H, E)
    ref = O.logprobs(L, y)
    g = torch.ones(T)
    lse = torch.from_numpy(ref["lse"]).float().cuda()
    gd = g.cuda()
    torch.cuda.synchronize()
    for call in (lambda st: tpl.tp_linear_logprobs_fwd(Hd, Ed, yd, 1, dev_status=st),
                 lambda st: tpl.tp_linear_logprobs_dlogits(Hd, Ed, yd, lse, None, gd, None, 1,
                                                           dev_status=st)):
        st = tpl.new_status()
        tpl.tp_debug_stall_next_gemm(unit, kblock, wait_limit_us=50000)
        t0 = time.perf_counter()
        call(st)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 2.0
        assert int(st.item()) & tpl.DEVERR_TIMEOUT
        st = tpl.new_status()
        out = call(st)
        assert int(st.item()) == 0
        if isinstance(out, dict):
            _check_fwd(out, ref)
        else:
            assert_close("dlogits", out, O.logprobs_bwd(L, y, g, None), TOL_BF16)
