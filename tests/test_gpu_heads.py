"""Head norms and position rotation on the GPU against float64, and the projection with them.

Error of one element in float32, before its rounding to bf16 (2^-8 relative). The norm's
reciprocal r comes from a sum over D elements: at most D + 8 roundings of 2^-24 relative, halved
by the root, plus the root's own 2 ulp; a layer norm subtracts a mean that is off by at most
D 2^-24 mean|x|; the weight, the bias and the two products and the sum of the rotation add
six more roundings. With E(x) = (D + 32) 2^-24 (r |w| (|x - m| + mean|x|) + |b|), a rotated element is off by at most
|c| E(u) + |s| E(v) <= 1.5 (E(u) + E(v)), |c| and |s| being float32 values of at most one.
"""
import numpy as np
import pytest
import torch

import synth
from parity import to_torch_bf16

pytestmark = pytest.mark.gpu


def _oq():
    import w4a8_ptq_linear_b200 as oq
    return oq


def _ok(oq):
    torch.cuda.synchronize()
    st, code = oq.device_status()
    assert st == 0, hex(code)


def _tables(n, rot, seed=0):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f + seed
    return a.cos().float().cuda(), a.sin().float().cuda()


def _make(D, Hq, Hk, norm, rope, rot, seed=0, n_pos=64, weights=True, biases=True, eps=1e-6):
    oq = _oq()
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = [torch.randn(D, generator=g, device="cuda") for _ in range(4)]
    qw, kw = (v[0], v[1]) if weights else (None, None)
    qb, kb = (v[2], v[3]) if biases else (None, None)
    cos, sin = _tables(n_pos, rot) if rope != "none" else (None, None)
    h = oq.Heads(D, Hq, Hk, norm=norm, eps=eps, q_weight=qw, q_bias=qb, k_weight=kw, k_bias=kb,
                 rope=rope, cos=cos, sin=sin)
    return h, dict(norm=norm, rope=rope, rot=rot, eps=eps, cos=cos, sin=sin, w=(qw, kw), b=(qb, kb))


def _ref(x, m, i, pos):
    """(float64 result, bound on the float32 error) of [B, S, H, D] heads; pos [B, S]."""
    x = x.double()
    D = x.shape[-1]
    one, zero = torch.ones_like(x[0, 0, 0]), torch.zeros_like(x[0, 0, 0])
    w = m["w"][i].double() if m["w"][i] is not None else one
    b = m["b"][i].double() if m["b"][i] is not None else zero
    spread = torch.zeros_like(x[..., :1])
    if m["norm"] == "layer":
        spread = x.abs().mean(-1, keepdim=True)
        x = x - x.mean(-1, keepdim=True)
    r = torch.ones_like(spread)
    if m["norm"] != "none":
        r = (x.square().mean(-1, keepdim=True) + m["eps"]).rsqrt()
    n = x * r * w + b
    E = (D + 32) * 2.0 ** -24 * (r * w.abs() * (x.abs() + spread) + b.abs())
    if m["rope"] == "none":
        return n, E
    rot, p = m["rot"], pos.long()
    idx = p.clamp(0, m["cos"].shape[0] - 1)
    cos, sin = (t.double()[idx][:, :, None, :] for t in (m["cos"], m["sin"]))
    u, v = ((n[..., 0:rot:2], n[..., 1:rot:2]) if m["rope"] == "pairs"
            else (n[..., :rot // 2], n[..., rot // 2:rot]))
    a, c = u * cos - v * sin, u * sin + v * cos
    out, bound = n.clone(), E.clone()
    sl = ((slice(0, rot, 2), slice(1, rot, 2)) if m["rope"] == "pairs"
          else (slice(0, rot // 2), slice(rot // 2, rot)))
    out[..., sl[0]], out[..., sl[1]] = a, c
    bound[..., sl[0]] = bound[..., sl[1]] = 1.5 * (E[..., sl[0]] + E[..., sl[1]])
    turn = (p >= 0)[:, :, None, None]
    out, bound = torch.where(turn, out, n), torch.where(turn, bound, E)
    return out, bound


def _check(y, ref, bound):
    bad = (y.double() - ref).abs() > 2.0 ** -8 * (ref.abs() + bound) + bound
    assert bool(torch.isfinite(y).all())
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"


def _heads(B, S, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(B, S, H, D, generator=g, device="cuda") + 0.3).bfloat16()


@pytest.mark.parametrize("norm", ["rms", "layer", "none"])
@pytest.mark.parametrize("rope", ["pairs", "halves", "none"])
@pytest.mark.parametrize("D,rot", [(16, 16), (32, 16), (48, 32), (64, 64), (80, 80), (96, 64),
                                   (112, 112), (128, 128), (128, 32), (144, 144), (192, 128),
                                   (240, 240), (256, 256)])
def test_norms_and_rotations(norm, rope, D, rot):
    oq = _oq()
    for B, S, Hq, Hk in [(1, 1, 1, 1), (2, 5, 3, 1), (3, 7, 8, 2), (1, 33, 5, 5)]:
        h, m = _make(D, Hq, Hk, norm, rope, rot, seed=D + S)
        q, k = _heads(B, S, Hq, D, 1), _heads(B, S, Hk, D, 2)
        pos = torch.randint(-1, 64, (B, S), device="cuda", dtype=torch.int32)
        pos[0, 0] = -1
        qo, ko = oq.qk_norm_rope(h, q, k, positions=pos)
        for y, x, i in ((qo, q, 0), (ko, k, 1)):
            _check(y, *_ref(x, m, i, pos))
    _ok(oq)


def test_default_positions_and_shared_positions():
    oq = _oq()
    h, m = _make(64, 4, 2, "rms", "halves", 64)
    q, k = _heads(3, 40, 4, 64, 3), _heads(3, 40, 2, 64, 4)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    want = oq.qk_norm_rope(h, q, k, positions=pos[None].repeat(3, 1))
    for got in (oq.qk_norm_rope(h, q, k), oq.qk_norm_rope(h, q, k, positions=pos)):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    flat = oq.qk_norm_rope(h, q[1], k[1])
    assert torch.equal(flat[0], want[0][1]) and torch.equal(flat[1], want[1][1])
    _check(want[0], *_ref(q, m, 0, pos[None].repeat(3, 1)))


def test_without_weights_and_only_one_side():
    oq = _oq()
    pos = torch.arange(9, device="cuda", dtype=torch.int32)[None]
    h, m = _make(96, 4, 0, "layer", "pairs", 32, weights=False, biases=False)
    q = _heads(1, 9, 4, 96, 5)
    qo, ko = oq.qk_norm_rope(h, q, None)
    assert ko is None
    _check(qo, *_ref(q, m, 0, pos))
    h, m = _make(96, 0, 4, "rms", "halves", 96, weights=True, biases=False)
    qo, ko = oq.qk_norm_rope(h, None, q)
    assert qo is None
    _check(ko, *_ref(q, m, 1, pos))
    _ok(oq)


@pytest.mark.parametrize("D,Hq,Hk", [(64, 6, 2), (128, 9, 3), (80, 5, 5)])
def test_strides_in_place_and_untouched_neighbours(D, Hq, Hk):
    oq = _oq()
    B, S = 2, 19
    h, m = _make(D, Hq, Hk, "rms", "halves", D)
    rows = _heads(B, S, Hq + 2 * Hk + 1, D, 6)       # queries, keys, values and one more head
    q, k = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hk]
    want = oq.qk_norm_rope(h, q.contiguous(), k.contiguous())
    # head-major outputs inside a larger buffer
    buf = torch.full((B, Hq + 2, S + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
    qo = buf[:, 1:1 + Hq, :S].transpose(1, 2)
    _, ko = oq.qk_norm_rope(h, q, k, q_out=qo)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert bool((buf[:, 0] == 9).all() and (buf[:, -1] == 9).all() and (buf[:, :, S] == 9).all())
    # in place in the packed rows: values and the spare head stay
    rest = rows[:, :, Hq + Hk:].clone()
    oq.qk_norm_rope(h, q, k, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rows[:, :, Hq + Hk:], rest)
    _ok(oq)


def test_a_broadcast_input():
    # one key row for every token of the batch (stride 0): read as often as needed
    oq = _oq()
    h, m = _make(64, 2, 2, "rms", "pairs", 64)
    q, k = _heads(2, 6, 2, 64, 7), _heads(1, 1, 2, 64, 8).expand(2, 6, 2, 64)
    _, ko = oq.qk_norm_rope(h, q, k)
    _check(ko, *_ref(k, m, 1, torch.arange(6, device="cuda")[None].repeat(2, 1)))


@pytest.mark.parametrize("rope", ["pairs", "halves"])
def test_positions_outside_the_table(rope):
    oq = _oq()
    h, m = _make(96, 3, 1, "rms", rope, 64, n_pos=16)
    q, k = _heads(1, 8, 3, 96, 9), _heads(1, 8, 1, 96, 10)
    pos = torch.tensor([0, 15, -1, -2 ** 31, 3, 16, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    for y, x, i in zip(oq.qk_norm_rope(h, q, k, positions=pos), (q, k), (0, 1)):
        inside = pos < 16
        ref, bound = _ref(x, m, i, pos[None])
        _check(y[:, inside], ref[:, inside], bound[:, inside])
        assert bool(torch.isnan(y[:, ~inside][..., :64]).all())       # rotated elements
        _check(y[:, ~inside][..., 64:], ref[:, ~inside][..., 64:], bound[:, ~inside][..., 64:])
    _ok(oq)


@pytest.mark.parametrize("norm", ["rms", "layer", "none"])
def test_infinities_nan_and_zeros_stay_in_their_head(norm):
    oq = _oq()
    h, m = _make(64, 4, 1, norm, "halves", 32)
    q, k = _heads(1, 6, 4, 64, 11), _heads(1, 6, 1, 64, 12)
    clean = oq.qk_norm_rope(h, q, k)[0]
    q2 = q.clone()
    q2[0, 1, 2, 5], q2[0, 3, 0, 60], q2[0, 4, 3] = float("inf"), float("nan"), 0
    y = oq.qk_norm_rope(h, q2, k)[0]
    touched = torch.zeros(1, 6, 4, dtype=torch.bool, device="cuda")
    touched[0, 1, 2] = touched[0, 3, 0] = touched[0, 4, 3] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert bool(torch.isnan(y[0, 3, 0, 60])) and not bool(torch.isfinite(y[0, 1, 2, 5]))
    if norm == "none":   # an element that is not rotated, or rotated elsewhere, keeps its value
        assert bool(torch.isfinite(y[0, 3, 0, :60]).all())
    # a head of zeros: eps keeps the norm finite, the bias is left
    _check(y[:, 4:5, 3:4], *_ref(q2[:, 4:5, 3:4], m, 0, torch.full((1, 1), 4, device="cuda")))


def test_large_values_do_not_overflow_the_type():
    # magnitudes of 2^40: their squares are within float32, the normed values ordinary
    oq = _oq()
    h, m = _make(128, 2, 2, "rms", "pairs", 128)
    q = (_heads(1, 4, 2, 128, 13).float() * 2.0 ** 40).bfloat16()
    pos = torch.arange(4, device="cuda")[None]
    _check(oq.qk_norm_rope(h, q, q.clone())[0], *_ref(q, m, 0, pos))


def test_offsets_past_32_bits():
    # the last token's row starts 2^32 + elements into a sparse buffer
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 9 GB")
    oq = _oq()
    h, m = _make(64, 1, 1, "rms", "pairs", 64)
    pitch = (1 << 31) + 64
    buf = torch.zeros(2 * pitch + 192, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((1, 3, 1, 64), (0, pitch, 64, 1))
    x = _heads(1, 3, 1, 64, 14)
    q.copy_(x)
    qo, _ = oq.qk_norm_rope(h, q, x, q_out=q)
    _check(qo, *_ref(x, m, 0, torch.arange(3, device="cuda")[None]))
    _ok(oq)


def test_refusals():
    oq = _oq()
    h, _ = _make(64, 4, 2, "rms", "pairs", 64)
    q, k = _heads(1, 4, 4, 64, 1), _heads(1, 4, 2, 64, 2)
    with pytest.raises(oq.OQError, match="expected"):
        oq.qk_norm_rope(h, q, q)
    with pytest.raises(oq.OQError, match="positions"):
        oq.qk_norm_rope(h, q, k, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(oq.OQError, match="positions"):
        oq.qk_norm_rope(h, q, k, positions=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(oq.OQError, match="multiples of 8"):
        oq.qk_norm_rope(h, _heads(1, 4, 4, 68, 1)[..., :64], k)
    with pytest.raises(oq.OQError, match="aligned"):
        oq.qk_norm_rope(h, _heads(1, 4, 5, 64, 1).view(1, 4, -1)[..., 4:260].unflatten(-1, (4, 64)), k)
    with pytest.raises(oq.OQError, match="repeats"):
        oq.qk_norm_rope(h, q, k, k_out=k[:, :1].expand(1, 4, 2, 64))
    with pytest.raises(oq.OQError, match="bfloat16"):
        oq.qk_norm_rope(h, q.float(), k)


# ---- the projection -----------------------------------------------------------------------------

def _project(T, d, N, center, bits, seed=0):
    oq = _oq()
    hb = min(d & -d, 1024)
    plan = oq.Plan(d, hb, 2 if hb < 512 else 1, seed=seed, center=center)
    x = to_torch_bf16(synth.make_x(T, d, mean_var=3.0, heavy_frac=0.01, seed=seed))
    w = to_torch_bf16(synth.make_w(N, d))
    prep = oq.prepare_weights_w8 if bits == 8 else oq.prepare_weights
    return plan, x, prep(plan, w), to_torch_bf16(synth.make_bias(N, seed=4))


@pytest.mark.parametrize("norm,rope", [("rms", "halves"), ("rms", "pairs"), ("layer", "pairs"),
                                       ("layer", "halves"), ("none", "pairs"), ("rms", "none")])
@pytest.mark.parametrize("D,rot,Hq,Hk,extra", [(128, 128, 4, 2, 256), (64, 64, 3, 3, 192),
                                               (128, 64, 3, 1, 0), (64, 32, 5, 1, 80),
                                               (96, 96, 2, 2, 192), (32, 32, 6, 2, 64),
                                               (256, 256, 2, 1, 256), (64, 64, 0, 3, 64)])
def test_projection_is_the_layer_then_the_heads(norm, rope, D, rot, Hq, Hk, extra):
    """INT8 weights: the layer's float64 value from its own codes, then the heads. One rounding
    to bf16 (2^-8) and the float32 error of both steps: the layer's, 4.1 * 2^-24 of its terms, is
    stretched by the norm's r |w| (and by the element's share of the head's sums: at most twice)
    and by the rotation."""
    oq = _oq()
    d, N = 512, (Hq + Hk) * D + extra
    for B, S in [(1, 1), (2, 4), (1, 40), (3, 67), (2, 150), (1, 700)]:
        T = B * S
        plan, x, (w, ws, w1), bias = _project(T, d, N, True, 8, seed=S)
        h, m = _make(D, Hq, Hk, norm, rope, rot, seed=S, n_pos=1024, eps=1e-6)
        pos = torch.randint(-1, 1024, (B, S), device="cuda", dtype=torch.int32)
        y = oq.linear_qkv(plan, h, x, w, ws, w1, bias, positions=pos)
        layer = oq.linear_w8a8(plan, x, w, ws, w1, bias)
        nq, nk = Hq * D, (Hq + Hk) * D
        assert torch.equal(y[:, nk:], layer[:, nk:]), "the other columns are the layer's"
        a, sa, mean, _ = oq.rotate_quantize(plan, x)
        A = (a.double() @ w.double().T) * sa.double()[:, None] * ws.double()[None, :]
        M = mean.double()[:, None] * w1.double()[None, :]
        full = A + M + bias.double()
        terms = A.abs() + M.abs() + bias.double().abs()
        for c0, c1, H, i in ((0, nq, Hq, 0), (nq, nk, Hk, 1)):
            if H == 0:
                continue
            z, tz = (v[:, c0:c1].view(B, S, H, D) for v in (full, terms))
            ref, bound = _ref(z, m, i, pos)
            zc = z - z.mean(-1, keepdim=True) if norm == "layer" else z
            r = ((zc.square().mean(-1, keepdim=True) + m["eps"]).rsqrt() if norm != "none"
                 else torch.ones_like(z[..., :1]))
            wgt = m["w"][i].double().abs().max()
            # the layer's error e in every element: through x r, and through the sums of the norm
            # (the head's mean, and r by the head's error against its root mean square)
            e = 4.1 * 2.0 ** -24 * tz.amax(-1, keepdim=True)
            stretch = r * wgt * e * (2 + zc.abs().amax(-1, keepdim=True) * r)
            got = y[:, c0:c1].view(B, S, H, D)
            _check(got, ref, bound + 2 * stretch)
        plan.close()
    _ok(oq)


@pytest.mark.parametrize("bits,act", [(4, "int8_absmax"), (4, "int4_absmax")])
@pytest.mark.parametrize("S", [1, 30, 300])
def test_int4_projection_is_its_two_calls(bits, act, S):
    oq = _oq()
    d, D, Hq, Hk = 512, 64, 4, 2
    N, B = (Hq + 2 * Hk) * D, 2
    plan = oq.Plan(d, 512, 1, seed=1, center=True, act=act)
    x = to_torch_bf16(synth.make_x(B * S, d, mean_var=3.0, heavy_frac=0.0, seed=S))
    w, ws, w1 = oq.prepare_weights(plan, to_torch_bf16(synth.make_w(N, d)))
    h, _ = _make(D, Hq, Hk, "layer", "pairs", D, n_pos=512)
    y = oq.linear_qkv(plan, h, x, w, ws, w1, batch=B)
    want = oq.linear(plan, x, w, ws, w1).view(B, S, Hq + 2 * Hk, D)
    q, k = want[:, :, :Hq], want[:, :, Hq:Hq + Hk]
    oq.qk_norm_rope(h, q, k, q_out=q, k_out=k)
    assert torch.equal(y.view_as(want), want)
    _ok(oq)
    plan.close()


def test_projection_refusals_and_no_tokens():
    oq = _oq()
    plan, x, (w, ws, w1), bias = _project(4, 256, 256, True, 8)
    h, _ = _make(64, 2, 1, "rms", "pairs", 64)
    with pytest.raises(oq.OQError, match="fewer than"):
        oq.linear_qkv(plan, h, x, w[:128].contiguous(), ws[:128].contiguous(), w1[:128].contiguous())
    with pytest.raises(oq.OQError, match="sequences"):
        oq.linear_qkv(plan, h, x, w, ws, w1, batch=3)
    with pytest.raises(oq.OQError, match="too small"):
        oq.linear_qkv(plan, h, x, w, ws, w1,
                      workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    plan4 = oq.Plan(256, 256, 2, center=True, act="int4_absmax")
    with pytest.raises(oq.OQError, match="INT8_ABSMAX"):
        oq.linear_qkv(plan4, h, x, w, ws, w1)
    assert oq.linear_qkv(plan, h, x[:0], w, ws, w1).shape == (0, 256)
    _ok(oq)
    plan.close()
    plan4.close()


@pytest.mark.parametrize("S", [1, 20, 300, 700])
def test_projection_captured_and_replayed(S):
    # an attention input as a serving loop runs it: captured once, replayed at new positions
    oq = _oq()
    d, D, Hq, Hk = 1920, 64, 6, 2
    N = (Hq + 2 * Hk) * D
    plan, x, (w, ws, w1), bias = _project(S, d, N, True, 8)
    h, _ = _make(D, Hq, Hk, "rms", "halves", D, n_pos=2048)
    pos = torch.zeros(S, dtype=torch.int32, device="cuda")
    xs = [x, (x.float() * 0.5 + 1).bfloat16()]
    ps = [torch.arange(S, dtype=torch.int32, device="cuda") + o for o in (3, 1000)]
    want = [oq.linear_qkv(plan, h, a, w, ws, w1, bias, positions=p) for a, p in zip(xs, ps)]
    xin = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = oq.linear_qkv(plan, h, xin, w, ws, w1, bias, positions=pos)
    for i in (0, 1, 1, 0):
        xin.copy_(xs[i])
        pos.copy_(ps[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
    _ok(oq)
    plan.close()
