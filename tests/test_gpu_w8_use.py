"""The INT8 layer and the attention input as a program runs them: weights replaced between calls,
several host threads, heads whose size the GEMM's epilogue does not form, whole attention inputs.

Tolerances: bit equality where two ways compute the same thing; the whole block against float64
within the layer's 8e-3 (relative, Frobenius)."""
import threading

import numpy as np
import pytest
import torch

import oracle
import synth
from parity import OUT_TOL, rel_fro, to_torch_bf16

pytestmark = pytest.mark.gpu


def _oq():
    import w4a8_ptq_linear_b200 as oq
    return oq


def _ok(oq):
    torch.cuda.synchronize()
    st, code = oq.device_status()
    assert st == 0, hex(code)


def _tables(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return a.cos().float().cuda(), a.sin().float().cuda()


@pytest.mark.parametrize("T", [1, 20, 90, 600])
def test_weights_replaced_right_before_the_call(T):
    # the GEMM may fetch weights while the tokens are rotated: never ones from before the call
    oq = _oq()
    d, N = 1024, 528
    plan = oq.Plan(d, 1024, 1, center=True)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
    g = torch.Generator(device="cuda").manual_seed(T)
    sets = []
    for _ in range(3):
        w = torch.randint(-127, 128, (N, d), generator=g, device="cuda").to(torch.int8)
        sets.append((w, torch.rand(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")))
    want = [oq.linear_w8a8(plan, x, *s) for s in sets]
    torch.cuda.synchronize()
    w, s, w1 = (t.clone() for t in sets[0])
    xs = x.clone()
    got = []
    for i in range(60):
        for dst, src in zip((w, s, w1), sets[i % 3]):
            dst.copy_(src)
        xs.copy_(x)
        got.append(oq.linear_w8a8(plan, xs, w, s, w1))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))
    _ok(oq)
    plan.close()


def test_host_threads_at_once():
    oq = _oq()
    d, N, D = 512, 768, 64
    cos, sin = _tables(256, D)
    jobs = []
    for i, T in enumerate((1, 30, 100, 400)):
        plan = oq.Plan(d, 512, 1, seed=i, center=True)
        x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=i))
        prep = oq.prepare_weights_w8(plan, to_torch_bf16(synth.make_w(N, d)))
        h = oq.Heads(D, 4, 4, norm="rms", rope="halves", cos=cos, sin=sin)
        pos = torch.arange(T, dtype=torch.int32, device="cuda") % 256
        want = oq.linear_qkv(plan, h, x, *prep, positions=pos)
        jobs.append((plan, h, x, prep, pos, want))
    torch.cuda.synchronize()
    bad = []

    def run(job):
        plan, h, x, prep, pos, want = job
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                y = oq.linear_qkv(plan, h, x, *prep, positions=pos)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want):
                    bad.append(x.shape[0])

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    _ok(oq)
    for j in jobs:
        j[0].close()


@pytest.mark.parametrize("D,rot", [(80, 80), (48, 48), (144, 128), (64, 48), (16, 16)])
@pytest.mark.parametrize("rope,norm", [("pairs", "rms"), ("halves", "layer")])
@pytest.mark.parametrize("T", [4, 60, 220, 700])
def test_heads_outside_the_epilogue(D, rot, rope, norm, T):
    # sizes that are no multiple of 32: the projection's float32 columns go through the head kernel.
    # Against the two separate calls, whose projection is rounded to bf16 in between. That rounding is off
    # by 2^-8 of each element at most, so by 2^-8 of the head's length, and the last rounding of
    # either side by as much: 3 * 2^-8 of the length in all (for a layer norm, where a head's mean is
    # small beside its spread, as it is here).
    oq = _oq()
    d, Hq, Hk = 512, 3, 2
    N = (Hq + Hk + 1) * D
    N += -N % 16
    plan = oq.Plan(d, 512, 1, center=True)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
    prep = oq.prepare_weights_w8(plan, to_torch_bf16(synth.make_w(N, d)))
    cos, sin = _tables(1024, rot)
    h = oq.Heads(D, Hq, Hk, norm=norm, rope=rope, cos=cos, sin=sin)
    y = oq.linear_qkv(plan, h, x, *prep)
    z = oq.linear_w8a8(plan, x, *prep)
    n = (Hq + Hk) * D
    assert torch.equal(y[:, n:], z[:, n:])
    heads = z[:, :n].unflatten(-1, (Hq + Hk, D))
    q, k = oq.qk_norm_rope(h, heads[:, :Hq], heads[:, Hq:])
    want = torch.cat([q, k], 1).double()
    got = y[:, :n].unflatten(-1, (Hq + Hk, D)).double()
    off = (got - want).norm(dim=-1) / want.norm(dim=-1).clamp_min(1e-30)
    assert bool(torch.isfinite(got).all()) and off.max().item() <= 3 * 2.0 ** -8
    _ok(oq)
    plan.close()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_rows_wider_than_the_two_token_kernel(T):
    # d > 8192: another rotate-quantize kernel, after which the GEMM does not begin early
    oq = _oq()
    d, N = 9216, 144
    plan = oq.Plan(d, 1024, 1, seed=1, center=True)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
    codes, s, w1 = oq.prepare_weights_w8(plan, to_torch_bf16(synth.make_w(N, d)))
    y = oq.linear_w8a8(plan, x, codes, s, w1)
    a, sa, mean, _ = oq.rotate_quantize(plan, x)
    assert torch.equal(y, oq.gemm_w8a8(a, sa, codes, s, mean=mean, w_rowsum=w1))
    acc = a.double() @ codes.double().T
    assert torch.equal(oq.gemm_w8a8(a, sa, codes, s, out_kind=oq.OUT_ACC).double(), acc)
    _ok(oq)
    plan.close()


@pytest.mark.parametrize("T", [2, 9, 13, 16, 17, 33, 257, 400])
@pytest.mark.parametrize("D,rope,norm", [(64, "halves", "rms"), (128, "pairs", "layer"),
                                         (96, "halves", "none")])
def test_projection_around_its_shapes(T, D, rope, norm):
    # whole and missing positions, weights and biases, on both sides of every change of shape; the
    # two separate calls round the projection to bf16 in between (3 * 2^-8 of a head's length, and its
    # bias; see test_heads_outside_the_epilogue)
    oq = _oq()
    d, Hq, Hk, rot = 384, 3, 1, D // 2
    N = (Hq + Hk + 2) * D
    plan = oq.Plan(d, 128, 2, seed=2, center=True)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
    prep = oq.prepare_weights_w8(plan, to_torch_bf16(synth.make_w(N, d)))
    g = torch.Generator(device="cuda").manual_seed(T)
    qw, kw, qb, kb = (torch.randn(D, generator=g, device="cuda") for _ in range(4))
    cos, sin = _tables(64, rot)
    h = oq.Heads(D, Hq, Hk, norm=norm, q_weight=qw, q_bias=qb, k_weight=kw, k_bias=kb, rope=rope,
                 cos=cos, sin=sin)
    pos = torch.randint(-2, 70, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[-1], pos[0] = 64, 63                         # the first past the table, the last in it
    y = oq.linear_qkv(plan, h, x, *prep, positions=pos).unflatten(-1, (-1, D))
    z = oq.linear_w8a8(plan, x, *prep).unflatten(-1, (-1, D))
    assert torch.equal(y[:, Hq + Hk:], z[:, Hq + Hk:])
    q, k = oq.qk_norm_rope(h, z[:, :Hq], z[:, Hq:Hq + Hk], positions=pos)
    want, got = torch.cat([q, k], 1).double(), y[:, :Hq + Hk].double()
    lost = pos >= 64
    assert bool(torch.isnan(got[lost][..., :rot]).all())
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    got, want = got.nan_to_num(), want.nan_to_num()
    # without the norm an element is as long as the layer's; the bias is not touched by the rounding
    length = want.norm(dim=-1) + torch.cat([qb.norm().expand(Hq), kb.norm().expand(Hk)])
    length = length + (z[:, :Hq + Hk].double() * torch.stack([qw] * Hq + [kw] * Hk)).norm(dim=-1) * (norm == "none")
    assert bool(((got - want).norm(dim=-1) <= 3 * 2.0 ** -8 * length).all())
    _ok(oq)
    plan.close()


@pytest.mark.parametrize("D,rot", [(64, 64), (80, 80), (256, 256)])
def test_one_workspace_for_every_number_of_tokens(D, rot):
    # sized for the most tokens, used for fewer
    oq = _oq()
    d, Hq, Hk = 256, 3, 2
    N = (Hq + 2 * Hk) * D
    plan = oq.Plan(d, 256, 2, center=True)
    prep = oq.prepare_weights_w8(plan, to_torch_bf16(synth.make_w(N, d)))
    cos, sin = _tables(512, rot)
    h = oq.Heads(D, Hq, Hk, rope="pairs", cos=cos, sin=sin)
    need = [oq.lib().oq_linear_qkv_workspace_bytes(plan.handle, h._ref, 1, T, N) for T in range(0, 520)]
    assert all(a <= b for a, b in zip(need, need[1:]))
    for most in (512, 256, 20):
        ws = torch.empty(need[most], dtype=torch.uint8, device="cuda")
        for T in (most, 300, 256, 100, 17, 16, 1):
            if T <= most:
                x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.0, seed=T))
                y = oq.linear_qkv(plan, h, x, *prep, workspace=ws)
                assert torch.equal(y, oq.linear_qkv(plan, h, x, *prep))
    _ok(oq)
    plan.close()


def test_many_tokens_of_one_small_head():
    oq = _oq()
    cos, sin = _tables(16, 16)
    h = oq.Heads(16, 1, 1, norm="rms", rope="pairs", cos=cos, sin=sin)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(300001, 1, 16, generator=g, device="cuda").bfloat16()
    pos = torch.full((300001,), 3, dtype=torch.int32, device="cuda")
    qo, ko = oq.qk_norm_rope(h, q, q, positions=pos)
    assert torch.equal(qo, ko)
    x = q.double()
    n = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    z = torch.view_as_complex(n.unflatten(-1, (8, 2))) * torch.complex(cos[3].double(), sin[3].double())
    ref = torch.view_as_real(z).flatten(-2)
    # 2^-8 of the value, and float32 steps: under 48 * 2^-24 of a normed magnitude of at most 4
    assert bool(((qo.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 4 * 48 * 2.0 ** -24).all())
    _ok(oq)


@pytest.mark.parametrize("B,S", [(1, 1), (4, 1), (1, 50), (2, 200), (1, 700)])
@pytest.mark.parametrize("bits", [8, 4])
def test_an_attention_input_against_the_oracle(B, S, bits):
    # weights prepared, tokens projected, heads formed, values passed on: the whole in float64
    oq = _oq()
    d, D, Hq, Hk, rot = 512, 64, 6, 2, 64
    N, T = (Hq + 2 * Hk) * D, B * S
    xb = synth.make_x(T, d, mean_var=3.0, heavy_frac=0.01, seed=S)
    wb, bb = synth.make_w(N, d), synth.make_bias(N, seed=2)
    plan = oq.Plan(d, 512, 1, seed=4, center=True)
    prep = (oq.prepare_weights_w8 if bits == 8 else oq.prepare_weights)(plan, to_torch_bf16(wb))
    g = torch.Generator(device="cuda").manual_seed(S)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    cos, sin = _tables(1024, rot)
    h = oq.Heads(D, Hq, Hk, norm="rms", q_weight=qw, k_weight=kw, rope="pairs", cos=cos, sin=sin)
    pos = torch.randint(-1, 1024, (B, S), generator=g, device="cuda", dtype=torch.int32)
    y = oq.linear_qkv(plan, h, to_torch_bf16(xb), *prep, to_torch_bf16(bb), positions=pos)
    _ok(oq)
    rp = oracle.rpbh_plan(d, 512, 1, 4)
    qa = oracle.quantize_activations(synth.bf16_to_f64(xb), rp, 512, "int8_absmax", True, None)
    wf = synth.bf16_to_f64(wb)
    wc, sw = oracle.absmax_quantize(oracle.rotate(wf, rp, 512), 127 if bits == 8 else 7, 1e-10)
    z = oracle.epilogue(oracle.gemm_int(qa["codes"], wc), qa["scale"], sw, qa["mean"], wf.sum(1),
                        synth.bf16_to_f64(bb)).reshape(T, -1, D)
    p = pos.cpu().numpy().reshape(T)
    turn = cos.cpu().numpy().astype(np.float64) + 1j * sin.cpu().numpy().astype(np.float64)
    turn = np.where(p[:, None] < 0, 1.0, turn[np.maximum(p, 0)])[:, None, :]
    for lo, hi, w in ((0, Hq, qw), (Hq, Hq + Hk, kw)):
        a = z[:, lo:hi]
        a = a / np.sqrt((a * a).mean(-1, keepdims=True) + 1e-6) * w.double().cpu().numpy()
        c = (a[..., 0::2] + 1j * a[..., 1::2]) * turn
        z[:, lo:hi] = np.stack([c.real, c.imag], -1).reshape(a.shape)
    assert rel_fro(y.float().cpu().numpy(), z.reshape(T, N)) <= OUT_TOL
    plan.close()


@pytest.mark.parametrize("bits", [8, 4])
def test_no_sequences(bits):
    # an empty batch gives an empty result, with and without positions
    oq = _oq()
    d, D = 256, 32
    plan = oq.Plan(d, 256, 1)
    prep = (oq.prepare_weights_w8 if bits == 8 else oq.prepare_weights)(
        plan, to_torch_bf16(synth.make_w(128, d)))
    cos, sin = _tables(16, D)
    h = oq.Heads(D, 2, 1, rope="halves", cos=cos, sin=sin)
    x = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((0, 5), dtype=torch.int32, device="cuda")
    for kw in ({}, {"positions": pos}, {"batch": 0}, {"batch": 3}, {"batch": 0, "positions": pos}):
        assert oq.linear_qkv(plan, h, x, *prep, **kw).shape == (0, 128)
    with pytest.raises(oq.OQError):
        oq.linear_qkv(plan, h, x.new_zeros((5, d)), *prep, positions=pos)
    with pytest.raises(oq.OQError):
        oq.linear_qkv(plan, h, x, *prep, batch=-1)
    _ok(oq)
    plan.close()
