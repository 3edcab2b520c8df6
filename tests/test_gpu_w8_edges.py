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


def _off16(shape, dtype):
    """A contiguous tensor whose base is a multiple of 16 bytes, not of 32."""
    n = torch.Size(shape).numel()
    pad = 16 // torch.empty((), dtype=dtype).element_size()
    t = torch.empty(n + pad, dtype=dtype, device="cuda")[pad:].view(shape)
    assert t.data_ptr() % 32 == 16
    return t


def _moved(t):
    return _off16(t.shape, t.dtype).copy_(t)


@pytest.mark.parametrize("T", [1, 9, 20, 32, 40, 200, 300, 600])
@pytest.mark.parametrize("K,N", [(416, 208), (4096, 144)])
def test_operands_on_16_byte_boundaries(T, K, N):
    # codes, weights and result may lie on any multiple of 16 bytes: each alone and all together
    oq = _oq()
    a, w, sa, sw, mean, w1, bias = _inputs(T, K, N, T + K, lo=-128)
    acc = _exact_acc(a, w)
    want = oq.gemm_w8a8(a, sa, w, sw, mean=mean, w_rowsum=w1, bias=bias)
    _check_bf16(want, acc, sa, sw, mean, w1, bias)
    for ma, mw, mo in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)]:
        ai, wi = _moved(a) if ma else a, _moved(w) if mw else w
        y = _off16((T, N), torch.bfloat16) if mo else None
        s = _off16((T, N), torch.int32) if mo else None
        y = oq.gemm_w8a8(ai, sa, wi, sw, mean=mean, w_rowsum=w1, bias=bias, out=y)
        s = oq.gemm_w8a8(ai, sa, wi, sw, out_kind=oq.OUT_ACC, out=s)
        assert torch.equal(y, want) and torch.equal(s.double(), acc)
    _ok(oq)


@pytest.mark.parametrize("T", [3, 12, 60, 220, 400])
@pytest.mark.parametrize("D,rope", [(64, "halves"), (64, "pairs"), (80, "halves"), (256, "pairs")])
def test_projection_on_16_byte_boundaries(T, D, rope):
    oq = _oq()
    d, Hq, Hk = 512, 3, 2
    N = (Hq + Hk + 1) * D
    plan, x, (w, ws, w1), bias = _project(T, d, N, True, 8, seed=T)
    h, _ = _make(D, Hq, Hk, "layer", rope, D, n_pos=512)
    want = oq.linear_qkv(plan, h, x, w, ws, w1, bias)
    out = _off16((T, N), torch.bfloat16)
    assert torch.equal(oq.linear_qkv(plan, h, _moved(x), _moved(w), ws, w1, bias, out=out), want)
    _ok(oq)
    plan.close()


@pytest.mark.parametrize("D,rot", [(16, 16), (48, 48), (64, 48), (64, 64), (80, 80), (96, 96),
                                   (112, 96), (128, 128), (144, 128), (192, 192), (256, 256)])
def test_which_heads_the_projection_forms(D, rot):
    # what the GEMM does not form goes through float32 columns in the workspace, which therefore
    # tells the two ways apart; both against float64
    oq = _oq()
    d, Hq, Hk = 256, 2, 1
    N = (Hq + Hk + 1) * D
    h, m = _make(D, Hq, Hk, "rms", "halves", rot, seed=D, n_pos=1024)

    def columns(T):
        formed = (D <= 128 if T <= 16 else 128 % D == 0 if T <= 256
                  else D % 32 == 0 and rot % 32 == 0)
        return 0 if formed else (T * (Hq + Hk) * D * 4 + 255) // 256 * 256

    for T in (4, 60, 220, 400):
        plan, x, (w, ws, w1), bias = _project(T, d, N, True, 8, seed=T)
        need = oq.lib().oq_linear_qkv_workspace_bytes(plan.handle, h._ref, 1, T, N)
        assert need == plan.workspace_bytes(T) + max(columns(T), columns(min(T, 256)))
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        # exactly what this number of tokens takes
        room = torch.empty(plan.workspace_bytes(T) + columns(T), dtype=torch.uint8, device="cuda")
        y = oq.linear_qkv(plan, h, x, w, ws, w1, bias, workspace=room)
        _formed(y, plan, x, w, ws, w1, bias, m, D, Hq, Hk, pos)
        if columns(T):
            with pytest.raises(oq.OQError, match="too small"):
                oq.linear_qkv(plan, h, x, w, ws, w1, bias, workspace=room[:-256])
        plan.close()
    _ok(oq)


@pytest.mark.parametrize("D,norm,rope", [(128, "rms", "halves"), (64, "layer", "pairs"), (96, "rms", "pairs")])
def test_a_token_alone_and_among_others(D, norm, rope):
    # values are the same bits; a normed head may differ in its last bits, since each way of forming
    # it adds the head's squares in another order: both lie within their bound of the same value
    oq = _oq()
    d, Hq, Hk, most = 1024, 4, 2, 300
    N, n = (Hq + 2 * Hk) * D, (Hq + Hk) * D
    plan, x, (w, ws, w1), bias = _project(most, d, N, True, 8, seed=D)
    h, m = _make(D, Hq, Hk, norm, rope, D, seed=D, n_pos=512)
    pos = torch.arange(most, device="cuda", dtype=torch.int32)
    for T in (1, 9, 16, 17, 64, 256, 300):
        for t0 in (0, most - T):
            args = (x[t0:t0 + T], w, ws, w1, bias)
            y = oq.linear_qkv(plan, h, *args, positions=pos[t0:t0 + T])
            assert torch.equal(y, oq.linear_qkv(plan, h, *args, positions=pos[t0:t0 + T]))
            assert torch.equal(y[:, n:], oq.linear_w8a8(plan, x, w, ws, w1, bias)[t0:t0 + T, n:])
            _formed(y, plan, *args, m, D, Hq, Hk, pos[t0:t0 + T])
    _ok(oq)
    plan.close()


@pytest.mark.parametrize("shapes", [[(80, 128, 512)] * 4, [(40, 256, 3840), (80, 128, 2048),
                                                           (150, 256, 1024), (256, 1024, 4096)]])
def test_splits_of_several_streams_share_the_sms(shapes):
    # clusters of several calls side by side, each with columns of its SMs' tensor memory
    oq = _oq()
    jobs = []
    for i, (T, K, N) in enumerate(shapes):
        a, w, sa, sw, _, _, _ = _inputs(T, K, N, i)
        jobs.append((a, sa, w, sw, oq.gemm_w8a8(a, sa, w, sw)))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[oq.gemm_w8a8(*j[:4], stream=st) for st, j in zip(streams, jobs)] for _ in range(50)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, j[4]) for ys in got for y, j in zip(ys, jobs))
    _ok(oq)


@pytest.mark.parametrize("T", [1, 60, 256, 400])
def test_int4_projection_captured_and_replayed(T):
    oq = _oq()
    d, D, Hq, Hk = 512, 64, 4, 2
    N = (Hq + 2 * Hk) * D
    plan, x, prep, bias = _project(T, d, N, True, 4, seed=T)
    h, _ = _make(D, Hq, Hk, "rms", "halves", D, n_pos=2048)
    xs = [x, (x.float() * 0.5 + 1).bfloat16()]
    ps = [torch.arange(T, dtype=torch.int32, device="cuda") + o for o in (3, 1000)]
    want = [oq.linear_qkv(plan, h, a, *prep, bias, positions=p) for a, p in zip(xs, ps)]
    xin, pos = x.clone(), ps[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = oq.linear_qkv(plan, h, xin, *prep, bias, positions=pos)
    for i in (0, 1, 1, 0):
        xin.copy_(xs[i])
        pos.copy_(ps[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    _ok(oq)
    plan.close()
