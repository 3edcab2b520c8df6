"""INT8 weights on the GPU: preparation, the W8A8 GEMM in every size class, the layer.

The integer sums are compared exactly. A bf16 result y = A + B with A = alpha_t s_o acc and
B = mean_t w1_o + b_o is computed in float32 with at most four roundings on the way, each off by
2^-24 relative to a term no larger than |A| + |mean_t w1_o| + |b_o|, and rounded to bf16 once
(2^-8 relative): |y - exact| <= 2^-8 |y| + 4.1 * 2^-24 * (1 + 2^-8) * (|A| + |mean_t w1_o| + |b_o|).
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from parity import OUT_TOL, absmax_boundary_mask, compare_codes, rel_fro, to_torch_bf16

pytestmark = pytest.mark.gpu


def _oq():
    import w4a8_ptq_linear_b200 as oq
    return oq


def _ok(oq):
    torch.cuda.synchronize()
    st, code = oq.device_status()
    assert st == 0, hex(code)


def _inputs(T, K, N, seed, lo=-127):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a = torch.randint(lo, 128, (T, K), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(lo, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    return a, w, 0.01 + r(T).abs(), 0.01 + r(N).abs(), r(T), r(N), r(N).bfloat16()


def _exact_acc(a, w):
    return a.double() @ w.double().T


def _check_bf16(y, acc, sa, sw, mean, w1, bias):
    A = acc * sa.double()[:, None] * sw.double()[None, :]
    m = torch.zeros_like(A) if mean is None else mean.double()[:, None] * w1.double()[None, :]
    b = torch.zeros_like(A) if bias is None else bias.double()[None, :].expand_as(A)
    ref = A + m + b
    e = 4.1 * 2.0 ** -24 * (1 + 2.0 ** -8) * (A.abs() + m.abs() + b.abs())
    bad = (y.double() - ref).abs() > 2.0 ** -8 * ref.abs() + e
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}"


# one token to several tiles; around every size at which another shape of the kernel takes over
TOKENS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 64, 65, 96, 127, 128, 129, 200, 255, 256,
          257, 300, 511, 513, 1000]
WIDTHS = [(32, 16), (64, 48), (96, 272), (160, 128), (1920, 80), (2080, 1200), (4096, 320),
          (512, 2064)]


@pytest.mark.parametrize("K,N", WIDTHS)
def test_sums_and_results(K, N):
    oq = _oq()
    for T in TOKENS:
        a, w, sa, sw, mean, w1, bias = _inputs(T, K, N, 1000 * T + K + N, lo=-128)
        acc = _exact_acc(a, w)
        got = oq.gemm_w8a8(a, sa, w, sw, out_kind=oq.OUT_ACC)
        assert torch.equal(got.double(), acc), f"T={T}: sums differ"
        _check_bf16(oq.gemm_w8a8(a, sa, w, sw, mean=mean, w_rowsum=w1, bias=bias), acc, sa, sw,
                    mean, w1, bias)
        _check_bf16(oq.gemm_w8a8(a, sa, w, sw), acc, sa, sw, None, None, None)
        _check_bf16(oq.gemm_w8a8(a, sa, w, sw, bias=bias), acc, sa, sw, None, None, bias)
    _ok(oq)


@pytest.mark.parametrize("T", [1, 5, 16, 100, 256, 700])
def test_largest_sums_do_not_wrap(T):
    # every product 128 * 128 at the largest width: 2^29, within int32
    oq = _oq()
    K, N = 32768, 32
    a = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    s = torch.ones(max(T, N), device="cuda")
    got = oq.gemm_w8a8(a, s[:T], w, s[:N], out_kind=oq.OUT_ACC)
    want = torch.full((T, N), 128 * 128 * K, dtype=torch.int32, device="cuda")
    want[:, 1] = -128 * 127 * K
    assert torch.equal(got, want)
    _ok(oq)


@pytest.mark.parametrize("T,K,N", [(1, 4096, 12288), (16, 12288, 4096), (40, 4096, 12288),
                                   (256, 1920, 5760), (2100, 1920, 5760), (4099, 4096, 4096),
                                   (700, 30720, 1920)])
def test_layer_sizes(T, K, N):
    oq = _oq()
    a, w, sa, sw, mean, w1, bias = _inputs(T, K, N, T + K + N)
    acc = _exact_acc(a, w)
    assert torch.equal(oq.gemm_w8a8(a, sa, w, sw, out_kind=oq.OUT_ACC).double(), acc)
    _check_bf16(oq.gemm_w8a8(a, sa, w, sw, mean=mean, w_rowsum=w1, bias=bias), acc, sa, sw, mean,
                w1, bias)
    _ok(oq)


@pytest.mark.parametrize("T", [3, 24, 77, 300])
def test_neighbours_of_the_output_stay(T):
    # rows in front of and behind the output, and a token's result without the other tokens
    oq = _oq()
    K, N = 416, 208
    a, w, sa, sw, mean, w1, bias = _inputs(T, K, N, T)
    big = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    oq.gemm_w8a8(a, sa, w, sw, mean=mean, w_rowsum=w1, bias=bias, out=big[1:-1])
    assert bool((big[0] == 7).all()) and bool((big[-1] == 7).all())
    i = T // 2
    one = oq.gemm_w8a8(a[i:i + 1].clone(), sa[i:i + 1].clone(), w, sw, mean=mean[i:i + 1].clone(),
                       w_rowsum=w1, bias=bias)
    assert torch.equal(one[0], big[1 + i]), "a token's result depends on the batch"
    _ok(oq)


@pytest.mark.parametrize("d,h,rounds", [(256, 64, 1), (1920, 128, 2), (96, 32, 2), (9216, 1024, 1)])
def test_prepared_weights(d, h, rounds):
    oq = _oq()
    n = 48
    wb = synth.make_w(n, d)
    plan = oq.Plan(d, h, rounds, seed=3)
    codes, s, w1 = oq.prepare_weights_w8(plan, to_torch_bf16(wb))
    _ok(oq)
    w = synth.bf16_to_f64(wb)
    z = oracle.rotate(w, oracle.rpbh_plan(d, h, rounds, 3), h)
    want, sw = oracle.absmax_quantize(z, 127, 1e-10)
    off, _ = compare_codes(codes.cpu().numpy().astype(np.int64), want, absmax_boundary_mask(z, sw, 127))
    assert off == 0
    assert np.abs(s.cpu().numpy() / sw - 1).max() <= 1e-5
    # d float32 additions in some order: each off by at most 2^-24 of the sum of magnitudes
    assert np.all(np.abs(w1.cpu().numpy() - w.sum(1)) <= d * 2.0 ** -24 * np.abs(w).sum(1))
    plan.close()


@pytest.mark.parametrize("T", [1, 6, 33, 130, 700])
@pytest.mark.parametrize("d,h,rounds,center", [(256, 64, 2, False), (1920, 128, 2, True),
                                               (4096, 1024, 1, True), (288, 32, 2, True)])
def test_layer_is_its_two_steps_and_matches_the_oracle(T, d, h, rounds, center):
    oq = _oq()
    n = 272
    xb = synth.make_x(T, d, mean_var=3.0, heavy_frac=0.01, seed=T)
    wb, bb = synth.make_w(n, d), synth.make_bias(n, seed=9)
    x, bias = to_torch_bf16(xb), to_torch_bf16(bb)
    plan = oq.Plan(d, h, rounds, seed=1, center=center)
    codes, s, w1 = oq.prepare_weights_w8(plan, to_torch_bf16(wb))
    y = oq.linear_w8a8(plan, x, codes, s, w1, bias)
    a, sa, mean, _ = oq.rotate_quantize(plan, x)
    two = oq.gemm_w8a8(a, sa, codes, s, mean=mean, w_rowsum=w1, bias=bias)
    assert torch.equal(y, two)
    wide = torch.zeros(T, d + 24, dtype=torch.bfloat16, device="cuda")   # a row pitch of its own
    wide[:, :d] = x
    assert torch.equal(oq.linear_w8a8(plan, wide[:, :d], codes, s, w1, bias), two)
    _ok(oq)
    rp = oracle.rpbh_plan(d, h, rounds, 1)
    qa = oracle.quantize_activations(synth.bf16_to_f64(xb), rp, h, "int8_absmax", center, None)
    wc, sw = oracle.absmax_quantize(oracle.rotate(synth.bf16_to_f64(wb), rp, h), 127, 1e-10)
    ref = oracle.epilogue(oracle.gemm_int(qa["codes"], wc), qa["scale"], sw,
                          qa["mean"] if center else None, synth.bf16_to_f64(wb).sum(1),
                          synth.bf16_to_f64(bb))
    assert rel_fro(y.float().cpu().numpy(), ref) <= OUT_TOL
    plan.close()


def test_no_tokens():
    oq = _oq()
    plan = oq.Plan(256, 64, 1)
    codes = torch.zeros(32, 256, dtype=torch.int8, device="cuda")
    s = torch.ones(32, device="cuda")
    e = torch.empty(0, 256, device="cuda")
    assert oq.gemm_w8a8(e.to(torch.int8), s[:0], codes, s).shape == (0, 32)
    assert oq.linear_w8a8(plan, e.bfloat16(), codes, s).shape == (0, 32)
    _ok(oq)
    plan.close()


def test_refusals_of_the_layer():
    oq = _oq()
    plan4 = oq.Plan(256, 64, 1, act="int4_absmax")
    plan = oq.Plan(256, 64, 1, center=True)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros(32, 256, dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    with pytest.raises(oq.OQError, match="INT8_ABSMAX"):
        oq.linear_w8a8(plan4, x, w, s)
    with pytest.raises(oq.OQError, match="w_rowsum"):
        oq.linear_w8a8(plan, x, w, s)
    with pytest.raises(oq.OQError, match="too small"):
        oq.linear_w8a8(plan, x, w, s, s, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(oq.OQError, match="expected 32"):
        oq.linear_w8a8(plan, x, w, s[:16], s)
    with pytest.raises(oq.OQError, match="contiguous"):
        oq.gemm_w8a8(w[:, ::2], s, w[:, :128].contiguous(), s)
    with pytest.raises(oq.OQError, match="columns"):
        oq.gemm_w8a8(w[:, :128].contiguous(), s, w, s)
    plan.close()
    plan4.close()


@pytest.mark.parametrize("T", [1, 12, 200, 600])
def test_streams_and_graphs(T):
    # two streams at once, then a captured pair of calls replayed on new inputs
    oq = _oq()
    K, N = 1920, 1200
    plan = oq.Plan(K, 128, 2, seed=2, center=True)
    sets = []
    for i in range(2):
        _, w, _, sw, _, w1, bias = _inputs(T, K, N, 50 + i)
        x = to_torch_bf16(synth.make_x(T, K, mean_var=3.0, heavy_frac=0.0, seed=i))
        sets.append((x, w, sw, w1, bias))
    want = [oq.linear_w8a8(plan, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [None, None]
        for i, (st, s) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(st):
                got[i] = oq.linear_w8a8(plan, *s)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    x = sets[0][0].clone()
    ws = torch.empty(plan.workspace_bytes(T), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = [oq.linear_w8a8(plan, x, *s[1:], workspace=ws) for s in sets]
    for i in (0, 1, 0):
        x.copy_(sets[i][0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[i], want[i])
    _ok(oq)
    plan.close()
