"""The failure path of the distillation step: a copy that never comes.  The waits
for it run out, the call says so and ends a few limits later, with dozens of rows
a block still to go, and the context stays usable.  The injection only withholds
a copy: nothing faults, and every wait ends by its own limit."""
import pytest
import torch

import linear_layers_b200 as tpl
from linear_layers_b200 import build as tpbuild
from tests.gpu_helpers import guarded
from tests.logprob_helpers import model_logits

LIMIT = 0.05


def test_injection_argument_checks():
    tpbuild.build()
    with pytest.raises(tpl.TPError):
        tpl.tp_debug_stall_next_distill(-1)
    for us in (0, 10_000_001):
        with pytest.raises(tpl.TPError):
            tpl.tp_debug_stall_next_distill(0, wait_limit_us=us)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,v", [
    (torch.float32, 9000, 4099),        # several small blocks to an SM, one to a row
    (torch.bfloat16, 6000, 20011),      # one block a row
    (torch.float32, 3000, 50304),       # two, two rows ahead
    (torch.float32, 900, 200001),       # six, one row ahead
    (torch.bfloat16, 3000, 140001),
    (torch.float32, 9, 50304),          # few rows on eight
])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_copy_that_never_comes_ends_the_call(dtype, T, v, where):
    row = {"first": 0, "middle": T // 2, "last": T - 1}[where]
    base, _ = model_logits(8, v, dtype, seed=v)
    x = base.cuda()[torch.arange(T, device="cuda") % 8]
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, v, (T, 16), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn(T, 16, generator=g, device="cuda")
    want = tpl.vp_distill(x, ids, t, 1)
    out, guard = guarded((T, v), torch.bfloat16)
    loss, loss_guard = guarded((T,), torch.float32)
    st = tpl.new_status()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    tpl.tp_debug_stall_next_distill(row, wait_limit_us=int(LIMIT * 1e6))
    begin.record()
    tpl.vp_distill(x, ids, t, 1, dlogits=out, loss=loss, dev_status=st)
    end.record()
    torch.cuda.synchronize()
    took = begin.elapsed_time(end) * 1e-3
    assert int(st.item()) == tpl.DEVERR_TIMEOUT
    assert LIMIT <= took < 8 * LIMIT, took     # one block's wait, its peers', the copies'
    guard.check("dlogits")
    loss_guard.check("loss")
    assert torch.equal(loss[:row], want["loss"][:row])
    assert torch.equal(out[:row], want["dlogits"][:row])
    st = tpl.new_status()
    again = tpl.vp_distill(x, ids, t, 1, dlogits=out, dev_status=st)
    assert int(st.item()) == 0
    for k in ("loss", "loss_sum", "lse", "dlogits"):
        assert torch.equal(again[k], want[k]), k
