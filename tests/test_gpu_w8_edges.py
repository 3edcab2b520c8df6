"""The INT8 layer and the attention input where other tests do not reach: every size of head that a
cluster of blocks forms, operands on 16-byte boundaries, which way the heads are formed, a token
alone and among others, calls on another stream than the current one.

Tolerances of formed heads: those of the projection's test (test_gpu_heads), the layer's float64
value from its own codes and the float32 error of both steps."""
import pytest
import torch

import synth
from parity import to_torch_bf16
from test_gpu_heads import _check, _make, _project, _ref
from test_gpu_w8 import _check_bf16, _exact_acc, _inputs

pytestmark = pytest.mark.gpu


def _oq():
    import w4a8_ptq_linear_b200 as oq
    return oq


def _ok(oq):
    torch.cuda.synchronize()
    st, code = oq.device_status()
    assert st == 0, hex(code)


def _formed(y, plan, x, w, ws, w1, bias, m, D, Hq, Hk, pos):
    """Query and key heads of one sequence against float64."""
    oq = _oq()
    T = x.shape[0]
    a, sa, mean, _ = oq.rotate_quantize(plan, x)
    A = (a.double() @ w.double().T) * sa.double()[:, None] * ws.double()[None, :]
    M = mean.double()[:, None] * w1.double()[None, :]
    full, terms = A + M + bias.double(), A.abs() + M.abs() + bias.double().abs()
    nq = Hq * D
    for c0, H, i in ((0, Hq, 0), (nq, Hk, 1)):
        z, tz = (v[:, c0:c0 + H * D].view(1, T, H, D) for v in (full, terms))
        ref, bound = _ref(z, m, i, pos[None])
        zc = z - z.mean(-1, keepdim=True) if m["norm"] == "layer" else z
        r = ((zc.square().mean(-1, keepdim=True) + m["eps"]).rsqrt() if m["norm"] != "none"
             else torch.ones_like(z[..., :1]))
        e = 4.1 * 2.0 ** -24 * tz.amax(-1, keepdim=True)
        stretch = r * m["w"][i].double().abs().max() * e * (2 + zc.abs().amax(-1, keepdim=True) * r)
        _check(y[:, c0:c0 + H * D].view(1, T, H, D), ref, bound + 2 * stretch)


@pytest.mark.parametrize("D", range(16, 129, 16))
@pytest.mark.parametrize("norm,rope", [("layer", "halves"), ("rms", "pairs"), ("none", "halves")])
def test_heads_of_every_cluster(D, norm, rope):
    # up to 16 tokens the D / 16 blocks of a head are a cluster: of one to eight blocks
    oq = _oq()
    d, Hq, Hk = 512, 3, 2
    N = (Hq + Hk + 1) * D
    for T in (1, 8, 9, 16):
        plan, x, (w, ws, w1), bias = _project(T, d, N, True, 8, seed=T)
        h, m = _make(D, Hq, Hk, norm, rope, D, seed=D, n_pos=64)
        pos = torch.randint(-1, 64, (T,), device="cuda", dtype=torch.int32)
        y = oq.linear_qkv(plan, h, x, w, ws, w1, bias, positions=pos)
        assert torch.equal(y[:, (Hq + Hk) * D:], oq.linear_w8a8(plan, x, w, ws, w1, bias)[:, (Hq + Hk) * D:])
        _formed(y, plan, x, w, ws, w1, bias, m, D, Hq, Hk, pos)
        plan.close()
    _ok(oq)
