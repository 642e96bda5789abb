"""The entropy of long accumulations, which only chunks of K keep.

The tensor core's additions truncate, so a chain of them shrinks every positive
sum by a common factor 1 − η, and an entropy moves by η·Var(z).  Two tokens of
z = 8 as 65536 positive products and some 6000 tokens of z = 0 (rows of zeros, exact)
share the probability evenly: Var(z) = 16, H = 5.4.

In chunks of 1024 the tensor core adds 64 times and truncates by at most 2^-22 of
the sum so far; 64 chunk sums are added in fp32, 2^-24 of the sum each:
ε = 64·2^-22 + 64·2^-24 = 1.9e-5.  |dH| <= Σ p·|log p + H|·ε·z = ε/2·4·8 = 16·ε = 3.1e-4,
plus the sums' own bound of 7e-5.  One chain of 4096 truncations, of half a step
of 2^-23.5 on average, would be off by 8.6e-5·16 = 1.4e-3.
"""
import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
from oracle import tp_oracle as O
from tests.gpu_helpers import f64
from tests.logprob_helpers import entropy_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [16, 200])
def test_entropy_of_long_sums_of_one_sign(T):
    v, h = 5960, 65536
    gen = torch.Generator().manual_seed(4)
    H = (0.5 + torch.rand(T, h, generator=gen)).bfloat16()
    rows = ((0.5 + torch.rand(2, h, generator=gen)) * (8.0 / h)).bfloat16()
    at = torch.tensor([300, 4001])
    E = torch.zeros(v, h, dtype=torch.bfloat16, device="cuda")
    E[at.cuda()] = rows.cuda()
    z = np.zeros((T, v))
    z[:, at.numpy()] = H.double().numpy() @ rows.double().numpy().T
    ref = O.logprobs(z)
    r = tpl.tp_linear_logprobs_fwd(H.cuda(), E, None, 1)
    lp = z - ref["lse"][:, None]
    eps = 64 * 2.0**-22 + 64 * 2.0**-24
    from_z = eps * (np.exp(lp) * np.abs(lp + ref["entropy"][:, None]) * z).sum(1)
    assert 5.0 < ref["entropy"].min() and 2.5e-4 < from_z.min() and from_z.max() < 3.5e-4
    bound = 1.01 * from_z + entropy_bound(v, z.max(1), ref["entropy"], ref["lse"], 1.0)
    err = np.abs(f64(r["entropy"]) - ref["entropy"])
    assert (err <= bound).all(), (err.max(), bound.min())
