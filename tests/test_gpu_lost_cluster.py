"""The single launch without its cluster, as a profiler that replays cooperative launches runs it:
the loss is reported, nothing is computed in its place, and the next call is whole again."""
import pytest
import torch

import synth
from parity import to_torch_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["int8_absmax", "int4_absmax"])
@pytest.mark.parametrize("d,T", [(256, 64), (1920, 200)])
def test_a_lost_cluster_is_reported(act, d, T):
    import w4a8_ptq_linear_b200 as oq
    N = 256
    plan = oq.Plan(d, d & -d, 1, seed=1, act=act)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=2.0, heavy_frac=0.0, seed=T))
    w = oq.prepare_weights(plan, to_torch_bf16(synth.make_w(N, d)))
    want = oq.linear_fused(plan, x, *w)
    assert oq.device_status()[0] == oq.OQ_OK
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    oq.debug_drop_cluster()
    oq.linear_fused(plan, x, *w, out=out)
    st, code = oq.device_status()
    assert st == oq.OQ_ERR_CUDA and code >> 63 == 1
    assert b"cluster" in oq.lib().oq_last_error()
    assert bool((out == 7).all())                  # nothing in the result's place
    assert oq.device_status()[0] == oq.OQ_OK       # cleared
    assert torch.equal(oq.linear_fused(plan, x, *w, out=out), want)
    assert oq.device_status()[0] == oq.OQ_OK
    plan.close()
