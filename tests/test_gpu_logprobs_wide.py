"""Top alternatives of rows so wide that a block notes one maximum for several
steps: widths just above, just below and between those where the number of steps
to a group doubles (32·2^k steps of 512 units of a block), on one, two, four and
eight blocks to a row, with rows that start at every alignment.

Some thirty rows of every kind are repeated over the batch, so that each stands
at several alignments and the oracle sees it once.
"""
import numpy as np
import pytest
import torch

import linear_layers_b200 as tpl
from oracle import tp_oracle as O
from tests.gpu_helpers import f64, guarded
from tests.logprob_helpers import entropy_bound, logprob_bound, lse_bound, model_logits, within
from tests.test_gpu_logprobs import special_rows

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16

# rows to a launch that give one, two, four and eight blocks a row
T1, T2, T4, T8 = 300, 150, 75, 40
WIDE = [
    # one step fewer in the rows that start inside a unit
    (F32, T1, 65541), (F32, T1, 65542), (F32, T1, 131077), (F32, T1, 262149),
    (BF, T1, 131081), (BF, T1, 131085), (BF, T1, 262153),
    # one step fewer in the row's last block
    (F32, T2, 131076), (F32, T2, 131078), (F32, T2, 131081), (F32, T2, 262150),
    (F32, T4, 262148), (F32, T4, 262155), (F32, T8, 524293), (BF, T2, 262155), (BF, T4, 524299),
    # as many in every block, on both sides of a doubling
    (F32, T1, 65536), (F32, T1, 65548), (BF, T1, 131072), (BF, T1, 131096), (F32, T2, 131200),
    # several steps to a group, away from the doublings
    (F32, T1, 200003), (BF, T1, 200001), (F32, T2, 300007), (BF, 4, 1048613),
]


@pytest.mark.parametrize("dtype,T,v", WIDE)
def test_wide_rows(dtype, T, v):
    rows = special_rows(v)
    rows.pop("+inf")                                  # lse is NaN or +inf there
    x = torch.stack([*rows.values(), *model_logits(4, v, F32, seed=v)[0]])
    lo, hi = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.where(x.isfinite(), x.clamp(lo, hi), x).to(dtype)
    n = x.shape[0]
    assert n % 2 and n % 7                            # a row comes at every alignment
    y = torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(T))
    at = (torch.arange(T) * 7) % n
    seen = np.unique(at.numpy())                      # a small batch leaves rows out
    part = O.logprobs(x[seen], y[seen], 1.0, 128)
    back = np.searchsorted(seen, at.numpy())
    ref = {k: a[back] for k, a in part.items()}
    L = f64(x[seen])
    M = np.max(np.where(np.isnan(L), -np.inf, L), axis=1)[back]
    M = np.where(np.isfinite(M), M, 0.0)
    lse = np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0)
    xd, yd = x.cuda()[at.cuda()], y[at].cuda()
    for K in (1, 40, 128):
        bufs, guards = {}, {}
        for name, shape, dt, fill in (("logprob", (T,), F32, 7.0), ("entropy", (T,), F32, 7.0),
                                      ("lse", (T,), F32, 7.0), ("top_idx", (T, K), torch.int32, -7),
                                      ("top_logprob", (T, K), F32, 7.0)):
            bufs[name], guards[name] = guarded(shape, dt, fill=fill)
        st = tpl.new_status()
        r = tpl.vp_logprobs_fwd(xd, yd, 1, top_k=K, dev_status=st, **bufs)
        for name, g in guards.items():
            g.check(name)
        assert int(st.item()) == 0
        assert np.array_equal(r["top_idx"].cpu().numpy(), ref["top_idx"][:, :K])
        within("lse", f64(r["lse"]), ref["lse"], lse_bound(v, M, lse, 1.0))
        within("entropy", f64(r["entropy"]), ref["entropy"],
               entropy_bound(v, M, np.nan_to_num(ref["entropy"]), lse, 1.0))
        lp = np.nan_to_num(ref["logprob"], neginf=0.0)
        within("logprob", f64(r["logprob"]), ref["logprob"], logprob_bound(v, M, lp, lse, 1.0))
        lp = np.nan_to_num(ref["top_logprob"][:, :K], neginf=0.0)
        within("top_logprob", f64(r["top_logprob"]), ref["top_logprob"][:, :K],
               logprob_bound(v, M[:, None], lp, lse[:, None], 1.0))
