"""Calls on another stream than the current one (stream=): what they allocate belongs to the stream
that writes it, so that no block still in use on the current stream is handed to them.

The first test reads the allocator's own record; the second keeps the current stream busy with a
tensor that is freed before the call. Results are compared bit for bit with calls on one stream."""
import pytest
import torch

import synth
from parity import to_torch_bf16

pytestmark = pytest.mark.gpu

D = 64


def _oq():
    import w4a8_ptq_linear_b200 as oq
    return oq


def _calls(T):
    """name -> a function of stream= that gives the tensors the call allocated and returned."""
    oq = _oq()
    d, N = 512, 384
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
    w = to_torch_bf16(synth.make_w(N, d))
    p8 = oq.Plan(d, 512, 1, center=True)
    p4 = oq.Plan(d, 512, 1, center=True, act="int4_absmax")
    plm = oq.Plan(d, 512, 1, center=True, act="int8_lloydmax")
    p2 = oq.Plan(d, 512, 1, center=True, act="int2_percentile")
    w8, w4, g64 = oq.prepare_weights_w8(p8, w), oq.prepare_weights(p8, w), oq.prepare_weights_g64(p4, w)
    a8, s8, m8, _ = oq.rotate_quantize(p8, x)
    a4, s4, m4, _ = oq.rotate_quantize(p4, x)
    al, sl, ml, _ = oq.rotate_quantize(plm, x)
    a2, s2, m2, _ = oq.rotate_quantize(p2, x)
    angle = torch.arange(1024.0)[:, None] * 10000.0 ** (-torch.arange(0, D, 2) / D)
    h = oq.Heads(D, 3, 1, rope="halves", cos=angle.cos().cuda(), sin=angle.sin().cuda())
    q, k = (torch.randn(T, n, D, device="cuda").bfloat16() for n in (3, 1))
    kw = dict(mean=m8, w_rowsum=w4[2])
    return {
        "rotate_quantize": lambda s: oq.rotate_quantize(p8, x, rotated=True, stream=s),
        "prepare_weights": lambda s: oq.prepare_weights(p8, w, stream=s),
        "prepare_weights_g64": lambda s: oq.prepare_weights_g64(p4, w, stream=s),
        "prepare_weights_w8": lambda s: oq.prepare_weights_w8(p8, w, stream=s),
        "gemm_w4a8": lambda s: (oq.gemm_w4a8(a8, s8, w4[0], w4[1], stream=s, **kw),),
        "gemm_w4a4": lambda s: (oq.gemm_w4a4(p4, "int4_absmax", a4, s4, w4[0], w4[1], mean=m4,
                                             w_rowsum=w4[2], stream=s),),
        "gemm_w4a2": lambda s: (oq.gemm_w4a2(a2, s2, w4[0], w4[1], mean=m2, w_rowsum=w4[2], stream=s),),
        "gemm_w4a8_lloydmax": lambda s: (oq.gemm_w4a8_lloydmax(plm, al, sl, w4[0], w4[1], mean=ml,
                                                               w_rowsum=w4[2], stream=s),),
        "gemm_w4a4_g64": lambda s: (oq.gemm_w4a4_g64("int4_absmax", a4, s4, g64[0], g64[1], g64[2],
                                                     mean=m4, w_rowsum=g64[3], stream=s),),
        "gemm_w8a8": lambda s: (oq.gemm_w8a8(a8, s8, w8[0], w8[1], mean=m8, w_rowsum=w8[2], stream=s),),
        "linear": lambda s: (oq.linear(p8, x, *w4, stream=s),),
        "linear_g64": lambda s: (oq.linear_g64(p4, x, *g64, stream=s),),
        "linear_static_scratch": lambda s: (oq.linear_static_scratch(p8, x, *w4, stream=s),),
        "linear_w8a8": lambda s: (oq.linear_w8a8(p8, x, *w8, stream=s),),
        "qk_norm_rope": lambda s: oq.qk_norm_rope(h, q, k, stream=s),
        "linear_qkv": lambda s: (oq.linear_qkv(p8, h, x, *w8, stream=s),),
        "linear_qkv_int4": lambda s: (oq.linear_qkv(p8, h, x, *w4, stream=s),),
        **({"linear_fused": lambda s: (oq.linear_fused(p8, x, *w4, stream=s),)} if T <= 256 else {}),
    }


def _owner(t):
    """The stream whose pool holds a tensor."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment")


@pytest.mark.parametrize("T", [3, 300])
def test_results_belong_to_the_stream_that_writes_them(T):
    oq = _oq()
    calls = _calls(T)
    want = {n: f(None) for n, f in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for n, f in calls.items():
        got = f(side)
        side.synchronize()
        for g, w in zip(got, want[n]):
            assert (g is None) == (w is None), n
            if g is not None:
                assert torch.equal(g, w), n
                assert _owner(g) == side.cuda_stream, f"{n}: {tuple(g.shape)} of another stream's pool"
                assert _owner(w) != side.cuda_stream, n
    assert oq.device_status()[0] == 0


@pytest.mark.parametrize("T", [3, 300])
def test_a_tensor_freed_while_its_stream_reads_it_is_left_alone(T):
    # a block of every size that the call asks for, freed while the current stream still reads it
    oq = _oq()
    calls = _calls(T)
    want = {n: f(None) for n, f in calls.items()}
    side = torch.cuda.Stream()
    sizes = sorted({t.numel() * t.element_size() for ts in want.values() for t in ts if t is not None}
                   | {512 * T + 2048, 1 << 20})
    for n, f in calls.items():
        torch.cuda.synchronize()
        held = [torch.full((b,), 1, dtype=torch.uint8, device="cuda") for b in sizes for _ in range(3)]
        torch.cuda._sleep(20_000_000)              # about ten milliseconds
        sums = [h.sum(dtype=torch.int64) for h in held]
        lens = [h.numel() for h in held]
        del held
        got = f(side)
        side.synchronize()
        assert [int(s) for s in sums] == lens, n
        for g, w in zip(got, want[n]):
            assert g is None or torch.equal(g, w), n
    assert oq.device_status()[0] == 0
