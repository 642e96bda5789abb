"""Distillation from a teacher's top entries on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
from oracle import tp_oracle as O
from tests.gpu_helpers import f64, guarded
from tests.logprob_helpers import OUT, U, lse_bound, model_logits, p_rel, sum_bound, within

pytestmark = pytest.mark.gpu

F32, BF, I32 = torch.float32, torch.bfloat16, torch.int32
INF = float("inf")


def entries(T, v, K, seed, renormalize=True, ragged=False, duplicates=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(v, generator=g)[:K] if v >= K else
                       torch.randint(0, v, (K,), generator=g) for _ in range(T)]).to(I32)
    if duplicates and K > 3:
        ids[:, K // 2] = ids[:, 0]
        ids[:, K - 1] = ids[:, 0]
    t = 2.0 * torch.randn(T, K, generator=g)
    if not renormalize:
        t = torch.log_softmax(t, 1) - 0.2
    if ragged:
        n = torch.randint(0, K + 1, (T, 1), generator=g)
        ids = torch.where(torch.arange(K) < n, ids, torch.full_like(ids, -1))
    return ids, t


def check(x, ids, t, grad_dtype=F32, renormalize=True, weight=None, scale=1.0, grad_scale=1.0, N=1,
          with_grad=True, in_place=False):
    T, v = x.shape
    K = ids.shape[1]
    bufs, guards = {}, {}
    for name, shape in (("loss", (T,)), ("lse", (T,)), ("loss_sum", (1,))):
        bufs[name], guards[name] = guarded(shape, F32)
    xd = x.cuda()
    if with_grad:
        bufs["dlogits"], guards["dlogits"] = guarded((T, v), grad_dtype)
        if in_place:
            bufs["dlogits"].copy_(xd)
            xd = bufs["dlogits"]
    st = tpl.new_status()
    r = tpl.vp_distill(xd, ids.cuda(), t.cuda(), N, renormalize=renormalize,
                       weight=None if weight is None else weight.cuda(), scale=scale,
                       grad_scale=grad_scale, with_grad=with_grad, dev_status=st, **bufs)
    for name, g in guards.items():
        g.check(name)
    ref = O.distill(x, ids, t, renormalize, weight, scale, grad_scale)
    L = f64(x)
    w = np.ones(T) if weight is None else f64(weight)
    with np.errstate(invalid="ignore", divide="ignore"):
        M = np.nanmax(np.where(np.isnan(L), -np.inf, L), axis=1)
        Mf = np.where(np.isfinite(M), M, 0.0)
        lse = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
        within("lse", f64(r["lse"]), ref["lse"], lse_bound(v, Mf, lse, scale))
        # teacher: |t| and its log-sum-exp enter the exponent, K terms the sums
        tt = np.where((ids.numpy() >= 0), f64(t), 0.0)
        tt = np.where(np.isfinite(tt), tt, 0.0)
        tmax = np.abs(tt).max(axis=1) + np.log(K) + 1
        rel_t = 4 * U * tmax * 2 + U * (K + 32)
        lq = scale * np.take_along_axis(L, np.clip(ids.numpy(), 0, v - 1).astype(np.int64), 1) - lse[:, None]
        lq = np.abs(np.where(np.isfinite(lq), lq, 0.0)).max(axis=1)
        size = ref["P"] * (tmax + lq + np.abs(lse - scale * Mf))
        b = np.abs(w) * (size * (2 * rel_t + 16 * U) + ref["P"] * (sum_bound(v) + K * 2 * U * (tmax + lq)))
        within("loss", f64(r["loss"]), ref["loss"], np.nan_to_num(b))
        if np.isfinite(ref["loss"]).all():
            within("loss_sum", f64(r["loss_sum"]), [ref["loss_sum"]],
                   [b.sum() + U * (T / 1024 + 12) * np.abs(ref["loss"]).sum()])
        if with_grad:
            z = scale * L
            q = np.exp(z - lse[:, None])
            zf = np.where(np.isfinite(z), z, 0.0)
            c = np.abs(grad_scale * w * scale)[:, None]
            bound = c * (ref["P"][:, None] * q * (p_rel(zf, lse[:, None]) + sum_bound(v) + rel_t[:, None]
                                                  + 8 * U))
            listed = np.zeros((T, v))
            for i in range(T):
                ok = (ids[i].numpy() >= 0) & (ids[i].numpy() < v)
                listed[i, ids[i].numpy()[ok]] = 1
            bound += c * listed * ref["P"][:, None] * (rel_t[:, None] + 8 * U)
            bound += 1.01 * OUT[grad_dtype] * np.abs(ref["dlogits"])
            bound += c * ref["P"][:, None] * 2.0 ** -125
            within("dlogits", f64(r["dlogits"]), ref["dlogits"], np.nan_to_num(bound))
    live = w != 0
    bad = bool((((ids < -1) | (ids >= v)).any(1).numpy() & live).any())
    assert int(st.item()) == (tpl.DEVERR_RANGE if bad else 0)
    return r


@pytest.mark.parametrize("dtype,grad_dtype", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
@pytest.mark.parametrize("T,v,K", [(1, 1, 1), (2, 7, 3), (3, 15, 20), (5, 300, 8), (40, 1000, 64),
                                   (3, 4099, 129), (17, 8192, 256), (4, 50304, 64), (2, 131073, 33),
                                   (600, 1030, 5)])
def test_loss_and_gradient(dtype, grad_dtype, T, v, K):
    x, _ = model_logits(T, v, dtype, seed=v + K)
    ids, t = entries(T, v, K, seed=K)
    check(x, ids, t, grad_dtype, grad_scale=1.0 / T)


@pytest.mark.parametrize("renormalize", [True, False])
def test_ragged_weighted_duplicates_and_temperature(renormalize):
    T, v, K = 60, 5003, 37
    x, _ = model_logits(T, v, BF, seed=1)
    ids, t = entries(T, v, K, 2, renormalize, ragged=True, duplicates=True)
    w = torch.rand(T, generator=torch.Generator().manual_seed(3))
    w[::5] = 0.0
    check(x, ids, t, BF, renormalize, w, scale=0.5, grad_scale=0.25, N=1)
    check(x, ids, t, F32, renormalize, w, scale=1.5, with_grad=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("v,T", [(200001, 3), (337920, 2), (20011, 1), (20011, 900)])
def test_large_vocabulary_and_many_rows(dtype, v, T):
    x, _ = model_logits(T, v, dtype, seed=v)
    ids, t = entries(T, v, 50, seed=5)
    check(x, ids, t, dtype)


def test_loss_alone_has_no_widest_row():
    x, _ = model_logits(3, 400003, F32, seed=3)
    ids, t = entries(3, 400003, 17, seed=6, ragged=True)
    check(x, ids, t, with_grad=False)


@pytest.mark.parametrize("v", [2000, 6600, 9000, 13000, 16700, 20600, 26000, 32003, 42000, 53001, 80000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_every_width_of_block(dtype, v):
    """More rows than resident blocks, so that every block turns its buffers
    over; odd widths, a token three times among the slots, some rows padded."""
    T = 450 if v < 30000 else 170
    x, _ = model_logits(T, v, dtype, seed=v)
    ids, t = entries(T, v, 9, seed=v, duplicates=True)
    w = torch.ones(T)
    w[::7] = 0.0
    check(x, ids, t, dtype, weight=w, grad_scale=1 / T)


@pytest.mark.parametrize("v,T", [(34003, 320), (66007, 160), (140001, 80), (200003, 60), (260003, 40),
                                 (50257, 20), (8203, 23), (8203, 13)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_every_number_of_blocks_to_a_row(dtype, v, T):
    """One to eight blocks (six and eight for the widest fp32 rows, and for few
    rows of any width), several rows to a block."""
    x, _ = model_logits(T, v, dtype, seed=v + T)
    ids, t = entries(T, v, 20, seed=v, duplicates=True)
    check(x, ids, t, dtype, grad_scale=1.0 / T)


@pytest.mark.parametrize("K", [31, 32, 33, 64, 65, 128, 129, 256])
def test_every_number_of_slots(K):
    """All slots one token, all of them different, and a few repeated far apart."""
    v, T = 4099, 6
    x, _ = model_logits(T, v, F32, seed=K)
    ids, t = entries(T, v, K, seed=K)
    ids[0] = 17
    ids[1, K - 1] = ids[1, 0]
    ids[2, 1::3] = ids[2, 0]
    ids[3, :] = torch.arange(K) * 2 + 1024 * (torch.arange(K) % 2).to(I32)
    check(x, ids, t, F32)
    check(x, ids, t, with_grad=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("v", [4096, 4099, 50257])
def test_in_place(dtype, v):
    x, _ = model_logits(11, v, dtype, seed=7)
    ids, t = entries(11, v, 40, seed=8, duplicates=True)
    a = check(x, ids, t, dtype, in_place=True)
    b = check(x, ids, t, dtype)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_rows_without_teacher_masked_rows_and_bad_ids():
    T, v, K = 9, 3001, 6
    x, _ = model_logits(T, v, F32, seed=9)
    ids, t = entries(T, v, K, seed=10)
    w = torch.ones(T)
    ids[0] = -1                                  # no slot at all
    x[0] = float("nan")                          # ... whatever the logits
    t[1] = -INF                                  # slots of probability zero only
    w[2] = 0.0
    ids[2, 3] = v + 5                            # a padded row is not looked at
    x[3, ids[3, 1]] = -INF                       # listed but banned: loss +inf
    ids[4, 2] = v                                # flagged, NaN
    ids[5, 0] = -2                               # flagged, NaN
    t[6, 2:] = -INF
    ids[7, 1] = -1
    t[7, 1] = float("nan")                       # the value of an empty slot is not read
    x[8, 100:2000] = -INF
    ids[8] = torch.tensor([0, 1, 2, 2500, 2500, 2600], dtype=I32)
    x0 = x.clone()
    x0[0] = 0.0                                  # the oracle's lse of row 0 is not compared
    r = check(x0, ids, t, F32, weight=w)
    assert float(r["loss"][3]) == INF
    st = tpl.new_status()
    r2 = tpl.vp_distill(x.cuda(), ids.cuda(), t.cuda(), 1, weight=w.cuda(), grad_dtype=F32,
                        dev_status=st)
    assert float(r2["loss"][0]) == 0.0 and not r2["dlogits"][0].any()
    assert torch.equal(r2["dlogits"][6:], r["dlogits"][6:])


def test_a_whole_one_hot_teacher_is_cross_entropy():
    """K = 1 with its one slot: the loss and gradient of vp_xent.  Both losses
    are M + log S − x_y of the same sums up to their bounds."""
    x, y = model_logits(70, 4096, F32, seed=12)
    a = tpl.vp_distill(x.cuda(), y.to(I32)[:, None].cuda(), torch.zeros(70, 1).cuda(), 8,
                       grad_scale=1 / 70, grad_dtype=F32)
    b = tpl.vp_xent(x.cuda(), y.cuda(), 8, grad_scale=1 / 70)
    tol = 4 * sum_bound(4096) + 64 * U
    assert float((a["loss"] - b["loss"]).abs().max()) < tol * 20
    assert float((a["dlogits"] - b["dlogits"]).abs().max()) < tol / 70


def test_gradient_against_differences():
    """Central differences of the loss, δ = 2^-3 (see the log-probabilities')."""
    v, K = 24, 5
    x, _ = model_logits(1, v, F32, seed=13, peak=1.0)
    ids, t = entries(1, v, K, seed=14, duplicates=True)
    c = [a.cuda() for a in (ids, t)]
    d = f64(tpl.vp_distill(x.cuda(), *c, 1, scale=0.9, grad_dtype=F32)["dlogits"])[0]
    for j in range(v):
        q = []
        for sgn in (1, -1):
            xs = x.clone()
            xs[0, j] += sgn * 2.0 ** -3
            q.append(float(tpl.vp_distill(xs.cuda(), *c, 1, scale=0.9, with_grad=False)["loss"]))
        assert abs((q[0] - q[1]) * 4 - d[j]) < 6e-3


def test_repeatable_on_another_stream_and_in_graphs():
    x, _ = model_logits(50, 9001, F32, seed=8)
    x2, _ = model_logits(50, 9001, F32, seed=9)
    ids, t = (a.cuda() for a in entries(50, 9001, 21, seed=1, duplicates=True))
    both = lambda x: list(tpl.vp_distill(x, ids, t, 1, grad_dtype=F32).values())  # noqa: E731
    xd = x.cuda()
    want, want2 = both(xd), both(x2.cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(xd)
        more = both(xd)
    beside = both(xd)                            # two calls at once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    xs = xd.clone()
    with torch.cuda.graph(graph):
        outs = both(xs)
    graph.replay()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    xs.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c, d, e, f, w2 in zip(want, other, more, beside, first, outs, want2):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
        assert torch.equal(a, e) and torch.equal(f, w2)


def test_teacher_pass_feeds_the_student_step():
    """The chain of a distillation step: hidden states to logits, the teacher's
    top entries, the student's loss and gradient, the output layer's backward.
    The student that equals the teacher has a loss of the teacher's missing
    mass only (renormalized against all of it) and a small gradient."""
    T, h, v, K = 48, 128, 2048, 64
    g = torch.Generator().manual_seed(2)
    H = torch.randn(T, h, generator=g).bfloat16().cuda()
    E = (torch.randn(v, h, generator=g) * 0.3).bfloat16().cuda()
    Es = (E.float() + 0.05 * torch.randn(v, h, generator=g).cuda()).bfloat16()
    teacher = tpl.vp_logprobs_fwd(tpl.tp_logits_fwd(H, E, 4), None, 4, top_k=K)
    student = tpl.tp_logits_fwd(H, Es, 4)
    check(student.cpu(), teacher["top_idx"].cpu(), teacher["top_logprob"].cpu(), BF,
          renormalize=False, grad_scale=1 / T, N=4)
    r = tpl.vp_distill(student, teacher["top_idx"], teacher["top_logprob"], 4, renormalize=False,
                       grad_scale=1 / T)
    dH, dE = tpl.tp_logits_bwd(r["dlogits"], H, Es, 4)
    d64 = f64(r["dlogits"])
    assert np.allclose(f64(dH), d64 @ f64(Es), rtol=2e-2, atol=2e-2 * np.abs(d64 @ f64(Es)).max())
    assert np.allclose(f64(dE), d64.T @ f64(H), rtol=1e-3, atol=1e-3 * np.abs(d64.T @ f64(H)).max())
    same = tpl.vp_distill(tpl.tp_logits_fwd(H, E, 4), teacher["top_idx"], teacher["top_logprob"], 4,
                          renormalize=False, with_grad=False)
    assert float(same["loss"].abs().max()) < 1e-4
