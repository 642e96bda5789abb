"""The entropy of rows with one dominant token, where it is small.

A row of one lane's elements: 0 in the first step, the top at z = 5 in the
second, and n tokens at z = −13 behind it; everything else is banned.  With
t = exp(−18) the entropy is log(1 + n·t) + 18·n·t/(1 + n·t), about n·2.9e-7.

Summed against the maximum, S starts at 1 and each of the n additions rounds it
by at most 2^-24; U is of the entropy's own size, and its n additions and terms
(2^-22 for the exponential, 2^-24 for a product) are off by n·2^-24 + 2^-21 of
it; the first token's 5·exp(−5) goes the same way.  log, the quotient and the
difference add roundings of the results' own size.  Bound:
(n + 16)·2^-24 + (n·2^-24 + 2^-20)·H.

Against a reference 5 below the maximum, U holds 5·exp(5) = 742, whose step is
2^-14: every term 13·exp(−13) = 0.48 steps is lost, 2.9e-5·n/148 = 2.0e-7·n in
all, more than three times that bound.
"""
import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
from oracle import tp_oracle as O
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("top_k", [0, 5])
def test_small_entropy_beside_an_earlier_maximum(dtype, scale, top_k):
    T, v = 320, 50304                              # one block of 128 threads to a row
    per_unit = 128 // torch.finfo(dtype).bits  # elements of 16 bytes
    unit = torch.arange(v // per_unit)
    x = torch.full((T, v), -INF)
    n = 0
    for t in range(T):
        lane = (37 * t) % 128
        mine = unit[unit % 128 == lane] * per_unit + 2 * (t % (per_unit // 2))
        x[t, mine[4:]] = -13.0                     # four units to a step
        x[t, mine[0]] = 0.0
        x[t, mine[4]] = 5.0
        n = max(n, len(mine) - 5)
    x /= scale                                     # exact
    ref = O.logprobs(x.to(dtype), None, scale)
    assert n > 40 and 0.03 < ref["entropy"].max() < 0.05     # exp(-5) of the first token
    r = tpl.vp_logprobs_fwd(x.to(dtype).cuda(), None, 1, scale=scale, top_k=top_k)
    H = ref["entropy"]
    bound = (n + 16) * 2.0**-24 + (n * 2.0**-24 + 2.0**-20) * H
    err = np.abs(f64(r["entropy"]) - H)
    assert (err <= bound).all(), (err.max(), bound.max())
