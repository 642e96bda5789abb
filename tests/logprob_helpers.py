"""Inputs and error bounds shared by the tests of the token log-probability
and distillation entry points.

The bounds are worked out from the arithmetic, element by element, before any
run.  U = 2^-24 is half a step of fp32, relative to the value.

 * S = Σ exp(scale·(x − M)): each term is off by at most 2^-22 (the hardware
   exponential) + 2·U·|z − sM| (rounding of the difference and of its
   product), and |d|·exp(−|d|) < 0.4, so a term of weight exp(d) adds at most
   U to the relative error; a thread adds at most v/128 + 8 terms in
   sequence, and a tree of at most 16 levels joins them.  Relative error of S:
   B = U·(v/128 + 32).
 * lse = sM + log S: B (log S) plus two roundings at its size, and sM's own.
 * entropy = log S − s·U/S: U's terms carry d on top of S's error.
 * a probability p = exp(z − lse): the exponent is off by U·(2|z| + 2|lse|)
   (the product, the difference, lse rounded to fp32), the exponential by
   2^-22.
"""
import numpy as np
import torch

U = 2.0 ** -24
OUT = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def sum_bound(v):
    return U * (v / 128 + 32)


def lse_bound(v, M, lse, scale):
    """|error| of lse (and, with |logprob| added by the caller, of logprob)."""
    return sum_bound(v) + 4 * U * (np.abs(scale * M) + np.abs(lse) + np.abs(lse - scale * M))


def logprob_bound(v, M, lp, lse, scale):
    return sum_bound(v) + 4 * U * (np.abs(lp) + np.abs(lse - scale * M))


def entropy_bound(v, M, ent, lse, scale):
    log_s = np.abs(lse - scale * M)
    return sum_bound(v) * (2 + 2 * (log_s + np.abs(ent))) + 8 * U * (log_s + np.abs(ent))


def p_rel(z, lse):
    """Relative error of exp(z − lse); a probability below 2^-126 may flush to 0."""
    return 2.0 ** -22 + 4 * U * (np.abs(z) + np.abs(lse)) + U


def within(name, got, ref, bound):
    """Every element within its bound; infinities and NaN in the same places."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bound = np.broadcast_to(np.asarray(bound, np.float64), ref.shape)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), f"{name}: inf"
    ok = np.isfinite(ref)
    if ok.any():
        over = np.abs(got[ok] - ref[ok]) - bound[ok]
        k = int(np.argmax(over))
        assert over[k] <= 0, (f"{name}: {got[ok][k]!r} for {ref[ok][k]!r}, off by "
                              f"{abs(got[ok][k] - ref[ok][k]):.3e}, bound {bound[ok][k]:.3e}")


def model_logits(T, v, dtype, seed, peak=9.0):
    """Rows with a broad body and a few tokens that stand out."""
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(T, v, generator=g)
    at = torch.randint(0, v, (T, min(v, 12)), generator=g)
    x.scatter_(1, at, 4.0 + peak * torch.rand(at.shape, generator=g))
    y = torch.where(torch.rand(T, generator=g) < 0.5, at[:, 0], torch.randint(0, v, (T,), generator=g))
    return x.to(dtype), y
