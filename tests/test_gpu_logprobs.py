"""Token log-probabilities, entropy, top alternatives and their gradient on the
GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
from oracle import tp_oracle as O
from tests.gpu_helpers import f64, guarded
from tests.logprob_helpers import (OUT, U, entropy_bound, logprob_bound, lse_bound, model_logits,
                                   p_rel, within)

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16
INF = float("inf")


def check_fwd(x, y, scale=1.0, top_k=0, N=1, finite_scale_rows=None):
    """Every output against the oracle, in guarded buffers; returns the outputs."""
    T, v = x.shape
    bufs, guards = {}, {}
    for name in ("logprob", "entropy", "lse"):
        bufs[name], guards[name] = guarded((T,), F32)
    if y is None:
        bufs.pop("logprob")
    if top_k:
        bufs["top_idx"], guards["top_idx"] = guarded((T, top_k), torch.int32, fill=-7)
        bufs["top_logprob"], guards["top_logprob"] = guarded((T, top_k), F32)
    st = tpl.new_status()
    r = tpl.vp_logprobs_fwd(x.cuda(), None if y is None else y.cuda(), N, scale=scale,
                            top_k=top_k, dev_status=st, **bufs)
    for name, g in guards.items():
        g.check(name)
    ref = O.logprobs(x, y, scale, top_k)
    L = f64(x)
    with np.errstate(invalid="ignore"):
        M = np.nanmax(np.where(np.isnan(L), -np.inf, L), axis=1)
        lse_ok = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
        Mf = np.where(np.isfinite(M), M, 0.0)
        within("lse", f64(r["lse"]), ref["lse"], lse_bound(v, Mf, lse_ok, scale))
        within("entropy", f64(r["entropy"]), ref["entropy"],
               entropy_bound(v, Mf, np.nan_to_num(ref["entropy"]), lse_ok, scale))
        if y is not None:
            lp = np.nan_to_num(ref["logprob"], neginf=0.0)
            within("logprob", f64(r["logprob"]), ref["logprob"],
                   logprob_bound(v, Mf, lp, lse_ok, scale))
        if top_k:
            assert np.array_equal(r["top_idx"].cpu().numpy(), ref["top_idx"])
            tl = np.nan_to_num(ref["top_logprob"], neginf=0.0)
            within("top_logprob", f64(r["top_logprob"]), ref["top_logprob"],
                   logprob_bound(v, Mf[:, None], tl, lse_ok[:, None], scale))
    bad = y is not None and bool(((y < 0) | (y >= v)).any())
    assert int(st.item()) == (tpl.DEVERR_RANGE if bad else 0)
    return r


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,v,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 8, 8), (2, 9, 0), (6, 15, 4),
                                   (3, 33, 20), (17, 300, 64), (9, 1000, 128), (2, 2048, 128),
                                   (33, 4099, 20), (5, 32003, 7), (1, 50304, 20), (64, 50257, 8),
                                   (3, 131073, 128), (700, 1025, 5)])
def test_forward(dtype, T, v, K):
    x, y = model_logits(T, v, dtype, seed=T + v)
    check_fwd(x, y, top_k=K)


@pytest.mark.parametrize("T", [1, 2, 40, 300, 1300, 2500])
def test_forward_every_split(T):
    """Few rows share a row between blocks, many do not."""
    x, y = model_logits(T, 20011, F32, seed=T)
    check_fwd(x, y, scale=0.5, top_k=13)
    check_fwd(x, None, scale=2.0)


@pytest.mark.parametrize("v,N", [(4096, 8), (1002, 3), (48, 16)])
def test_shards_do_not_change_a_bit(v, N):
    x, y = model_logits(37, v, F32, seed=3)
    a = check_fwd(x, y, top_k=9, N=N)
    b = check_fwd(x, y, top_k=9, N=1)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def special_rows(v):
    g = torch.Generator().manual_seed(11)
    base = torch.randn(v, generator=g)
    rows = {"random": base}
    few = torch.full((v,), -INF)
    few[torch.randperm(v, generator=g)[:3]] = torch.tensor([1.0, 1.0, -2.0])
    rows["all but three banned"] = few
    rows["one left"] = torch.full((v,), -INF).index_fill_(0, torch.tensor([v - 1]), 4.0)
    rows["half banned"] = base.masked_fill(torch.rand(v, generator=g) < 0.5, -INF)
    rows["lowest value masks"] = base.masked_fill(torch.rand(v, generator=g) < 0.9,
                                                  torch.finfo(F32).min)
    rows["all banned"] = torch.full((v,), -INF)
    rows["all lowest"] = torch.full((v,), torch.finfo(F32).min)
    rows["constant"] = torch.full((v,), 3.25)
    rows["zeros of both signs"] = torch.where(torch.rand(v, generator=g) < 0.5, 0.0, -0.0)
    rows["ascending"] = torch.linspace(-4, 4, v)
    rows["descending"] = torch.linspace(4, -4, v)
    rows["steps"] = (torch.arange(v) // 3).float() * 1e-3
    rows["many equal at the top"] = torch.where(torch.arange(v) % 3 == 0, 2.0, base.clamp(max=1.0))
    rows["top in one place"] = base.clamp(max=1.0) + (torch.arange(v) < 400).float() * 9
    rows["top in one lane"] = base.clamp(max=1.0) + (torch.arange(v) % 2048 < 4).float() * 9
    rows["equal pairs"] = torch.randn(v, generator=g).mul(8).round()
    rows["sawtooth"] = (torch.arange(v) % 16).float()
    rows["blocks of large"] = (torch.arange(v) % 2048 < 8).float() * 5 + 1e-4 * torch.rand(v, generator=g)
    rows["large offset"] = base + 3000.0
    rows["far apart"] = base * 300.0
    rows["one spike"] = base.index_fill(0, torch.tensor([v // 2]), 60.0)
    rows["nan"] = base.index_fill(0, torch.tensor([v // 3]), float("nan"))
    rows["all nan"] = torch.full((v,), float("nan"))
    rows["+inf"] = base.index_fill(0, torch.tensor([v // 3]), INF)
    return rows


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("v", [40, 5003, 50304])
@pytest.mark.parametrize("together", [True, False])
def test_special_rows(dtype, v, together):
    rows = special_rows(v)
    x = torch.stack(list(rows.values()))
    finite = x.isfinite()
    x = torch.where(finite, x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max), x).to(dtype)
    y = torch.randint(0, v, (x.shape[0],), generator=torch.Generator().manual_seed(2))
    names = list(rows)
    skip = [names.index("+inf")]              # lse is NaN or +inf there: checked below
    keep = [i for i in range(len(names)) if i not in skip]
    if together:                              # enough rows that no row is shared by blocks
        reps = 1300 // len(keep) + 1
        check_fwd(x[keep].repeat(reps, 1), y[keep].repeat(reps), top_k=20)
    else:
        check_fwd(x[keep], y[keep], top_k=33)
        for i in keep:
            check_fwd(x[i:i + 1], y[i:i + 1], top_k=40)
    r = tpl.vp_logprobs_fwd(x[skip].cuda(), y[skip].cuda(), 1, top_k=5)
    assert int(r["top_idx"][0, 0]) == v // 3
    assert not torch.isfinite(r["lse"]).any() and torch.isnan(r["entropy"]).all()


def test_bad_targets_flag_and_spare_the_rest():
    x, y = model_logits(9, 5000, F32, seed=1)
    y = y.clone()
    y[2], y[5], y[7] = -1, 5000, 1 << 40
    check_fwd(x, y, top_k=3)


def check_bwd(x, y, g, e, scale, grad_dtype, in_place=False):
    T, v = x.shape
    f = O.logprobs(x, None, scale)
    lse = torch.tensor(f["lse"], dtype=F32)
    ent = torch.tensor(f["entropy"], dtype=F32)
    st = tpl.new_status()
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    out, guard = guarded((T, v), grad_dtype)
    xd = x.cuda()
    if in_place:
        out.copy_(xd)
        xd = out
    d = tpl.vp_logprobs_bwd(xd, c(y), c(lse), c(ent), c(g), c(e), 1, scale=scale, dlogits=out,
                            dev_status=st)
    guard.check("dlogits")
    ref = O.logprobs_bwd(x, y, g, e, scale)
    gg = np.zeros(T) if g is None else f64(g)
    ee = np.zeros(T) if e is None else f64(e)
    z = scale * f64(x)
    with np.errstate(invalid="ignore"):
        lp = np.where(z == -np.inf, 0.0, z - f["lse"][:, None])
        p = np.exp(z - f["lse"][:, None])
        term = p * (np.abs(gg)[:, None] + np.abs(ee)[:, None] * (np.abs(lp) + np.abs(f["entropy"])[:, None]))
        zf = np.where(np.isfinite(z), z, 0.0)
        # the term's factors, then two roundings and the output's own
        bound = scale * (term * (p_rel(zf, f["lse"][:, None]) + 8 * U)
                         + np.abs(gg)[:, None] * 4 * U) + 1.01 * OUT[grad_dtype] * np.abs(ref)
        bound += scale * (np.abs(gg) + np.abs(ee) * 200)[:, None] * 2.0 ** -126   # flushed probabilities
        # the exponent's error counts a second time in the factor (log p + H)
        bound += scale * p * np.abs(ee)[:, None] * 8 * U * (np.abs(zf) + np.abs(f["lse"])[:, None]
                                                             + np.abs(f["entropy"])[:, None])
    within("dlogits", f64(d), ref, np.nan_to_num(bound))
    flagged = y is not None and g is not None and bool((((y < 0) | (y >= v)) & (g != 0)).any())
    assert int(st.item()) == (tpl.DEVERR_RANGE if flagged else 0)
    return d


@pytest.mark.parametrize("dtype,grad_dtype", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("T,v", [(1, 1), (3, 7), (5, 8), (2, 15), (33, 300), (17, 4099), (4, 50304),
                                 (3, 131073), (900, 515)])
def test_backward(dtype, grad_dtype, T, v):
    x, y = model_logits(T, v, dtype, seed=v)
    gen = torch.Generator().manual_seed(T)
    g, e = torch.randn(T, generator=gen), 0.3 * torch.randn(T, generator=gen)
    if T > 2:
        g[1], e[1] = 0.0, 0.0
        g[2] = 0.0
    check_bwd(x, y, g, e, 1.0, grad_dtype)
    check_bwd(x, y, g, None, 0.7, grad_dtype)
    check_bwd(x, None, None, e, 1.6, grad_dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("v", [4096, 4099])
def test_backward_in_place(dtype, v):
    x, y = model_logits(23, v, dtype, seed=9)
    g = torch.randn(23, generator=torch.Generator().manual_seed(1))
    a = check_bwd(x, y, g, -0.1 * g, 1.25, dtype, in_place=True)
    b = check_bwd(x, y, g, -0.1 * g, 1.25, dtype)
    assert torch.equal(a, b)


def test_backward_masks_padding_and_bad_targets():
    T, v = 8, 2051
    x, y = model_logits(T, v, F32, seed=4)
    x = x.masked_fill(torch.rand(T, v, generator=torch.Generator().manual_seed(5)) < 0.5, -INF)
    y = x.argmax(1)
    g, e = torch.ones(T), torch.full((T,), 0.5)
    x[3], g[3], e[3], y[3] = float("nan"), 0.0, 0.0, -100      # a padded row: nothing is read of it
    y[5] = v                                                    # flagged, NaN
    check_bwd(x, y, g, e, 1.0, F32)


def test_gradient_against_differences():
    """(f(x + δ) − f(x − δ)) / 2δ of the forward's own outputs.  δ = 2^-3: the
    forward is right to about 1e-6, so the quotient to 1e-5; the cubic term
    δ²/6·|f'''| stays below δ²/6·2 ≈ 5e-3 of the upstream size."""
    T, v = 1, 24
    x, y = model_logits(T, v, F32, seed=6, peak=1.0)
    g, e = torch.tensor([0.8]), torch.tensor([-0.6])
    xd, yd = x.cuda(), y.cuda()
    f = tpl.vp_logprobs_fwd(xd, yd, 1, scale=0.9)
    d = f64(tpl.vp_logprobs_bwd(xd, yd, f["lse"], f["entropy"], g.cuda(), e.cuda(), 1, scale=0.9,
                                grad_dtype=F32))[0]
    delta = 2.0 ** -3
    for j in range(v):
        q = []
        for sgn in (1, -1):
            xs = x.clone()
            xs[0, j] += sgn * delta
            r = tpl.vp_logprobs_fwd(xs.cuda(), yd, 1, scale=0.9)
            q.append(0.8 * float(r["logprob"]) - 0.6 * float(r["entropy"]))
        assert abs((q[0] - q[1]) / (2 * delta) - d[j]) < 6e-3


def test_repeatable_on_another_stream_and_in_graphs():
    """The same bits from a side stream and from replays of a captured forward
    and backward whose inputs change between replays."""
    x, y = model_logits(50, 9001, F32, seed=8)
    x2, y2 = model_logits(50, 9001, F32, seed=9)
    g = torch.randn(50, generator=torch.Generator().manual_seed(0)).cuda()
    xd, yd = x.cuda(), y.cuda()

    def both(xd, yd):
        f = tpl.vp_logprobs_fwd(xd, yd, 1, top_k=17)
        return [*f.values(), tpl.vp_logprobs_bwd(xd, yd, f["lse"], f["entropy"], g, -g, 1)]

    want, want2 = both(xd, yd), both(x2.cuda(), y2.cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(xd, yd)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        xs, ys = xd.clone(), yd.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both(xs, ys)
        graphs.append((graph, xs, ys, outs))
    for graph, *_ in graphs:
        graph.replay()
    graphs[1][1].copy_(x2)
    graphs[1][2].copy_(y2)
    graphs[1][0].replay()
    torch.cuda.synchronize()
    for a, b, c, d, w2 in zip(want, other, graphs[0][3], graphs[1][3], want2):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(d, w2)
