"""Refusals of the INT8-weight layer and of the attention input, on the CPU: every bad argument
is refused before anything is launched, through the C ABI and through the binding."""
import ctypes

import pytest
import torch

import w4a8_ptq_linear_b200 as oq

A = 1 << 20            # an aligned address that nothing reads: every call below is refused
BAD = oq.OQ_ERR_INVALID_ARG
MIS = oq.OQ_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    from w4a8_ptq_linear_b200 import build
    build.build()
    return oq.lib()


def heads_struct(**kw):
    d = dict(head_dim=64, q_heads=4, k_heads=2, norm=1, rope=1, rot_dim=64, eps=1e-6, q_weight=A,
             q_bias=None, k_weight=A, k_bias=None, cos=A, sin=A, n_pos=16)
    d.update(kw)
    return oq._HeadsStruct(**d)


def gemm(lib, **kw):
    d = dict(a=A, a_scale=A, mean=None, w=A, w_scale=A, w1=None, bias=None, T=4, K=64, N=32, kind=0,
             out=A)
    d.update(kw)
    return lib.oq_gemm_w8a8(*d.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(K=0), BAD), (dict(K=48), BAD),
    (dict(K=32800), BAD), (dict(N=0), BAD), (dict(N=24), BAD), (dict(kind=2), BAD),
    (dict(a=None), BAD), (dict(a_scale=None), BAD), (dict(w=None), BAD), (dict(w_scale=None), BAD),
    (dict(out=None), BAD), (dict(mean=A), BAD), (dict(a=A + 8), MIS), (dict(w=A + 4), MIS),
    (dict(out=A + 2), MIS)])
def test_gemm_refuses(lib, kw, want):
    assert gemm(lib, **kw) == want
    assert lib.oq_last_error()


def test_gemm_without_tokens_launches_nothing(lib):
    assert gemm(lib, T=0, a=None, a_scale=None, out=None) == oq.OQ_OK


def test_layer_and_preparation_refuse_a_missing_plan(lib):
    assert lib.oq_prepare_weights_w8(None, A, 4, 64, A, A, A, None) == BAD
    assert lib.oq_linear_w8a8(None, A, 1, 64, A, A, A, None, 32, A, A, 1 << 20, None) == BAD
    h = heads_struct()
    assert lib.oq_linear_qkv(None, ctypes.addressof(h), A, 1, 1, 64, 1, A, A, A, None, 512, None,
                             0, A, A, 1 << 20, None) == BAD
    assert lib.oq_linear_qkv_workspace_bytes(None, ctypes.addressof(h), 1, 1, 512) == 0


def norm_rope(lib, h, batch=2, seq=3, q=A, qs=(4096, 256, 64), k=A, ks=(4096, 256, 64), pos=None,
              pbs=0, qo=A, qos=(4096, 256, 64), ko=A, kos=(4096, 256, 64)):
    s = [None if v is None else (ctypes.c_int64 * 3)(*v) for v in (qs, ks, qos, kos)]
    return lib.oq_qk_norm_rope(ctypes.addressof(h) if h is not None else None, batch, seq, q, s[0],
                               k, s[1], pos, pbs, qo, s[2], ko, s[3], None)


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=0), BAD), (dict(head_dim=72), BAD), (dict(head_dim=272), BAD),
    (dict(q_heads=-1), BAD), (dict(q_heads=0, k_heads=0), BAD), (dict(q_heads=65536), BAD),
    (dict(norm=3), BAD), (dict(norm=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(rope=3), BAD), (dict(rot_dim=0), BAD),
    (dict(rot_dim=24), BAD), (dict(rot_dim=80), BAD), (dict(cos=None), BAD), (dict(sin=None), BAD),
    (dict(n_pos=0), BAD), (dict(cos=A + 4), MIS), (dict(q_weight=A + 8), MIS),
    (dict(k_bias=A + 4), MIS)])
def test_heads_refuse(lib, kw, want):
    assert norm_rope(lib, heads_struct(**kw)) == want
    assert lib.oq_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), BAD), (dict(seq=-1), BAD), (dict(batch=1 << 20, seq=1 << 20), BAD),
    (dict(q=None), BAD), (dict(ko=None), BAD), (dict(qs=None), BAD), (dict(q=A + 8), MIS),
    (dict(ko=A + 2), MIS), (dict(qs=(4096, 260, 64)), MIS), (dict(kos=(4096, 256, 68)), MIS),
    (dict(ks=(-8, 256, 64)), BAD), (dict(qos=(4096, 256, 0)), BAD), (dict(kos=(0, 256, 64)), BAD),
    (dict(pos=A, pbs=-3), BAD), (dict(pos=A + 2), MIS)])
def test_placement_refused(lib, kw, want):
    assert norm_rope(lib, heads_struct(), **kw) == want


def test_no_heads_struct_and_no_tokens(lib):
    assert norm_rope(lib, None) == BAD
    none = dict(q=None, k=None, qo=None, ko=None)
    assert norm_rope(lib, heads_struct(), batch=0, **none) == oq.OQ_OK
    assert norm_rope(lib, heads_struct(), seq=0, **none) == oq.OQ_OK


def test_binding_refuses_host_tensors_and_types():
    a, w = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(32, 64, dtype=torch.int8)
    s = torch.ones(2)
    with pytest.raises(oq.OQError, match="current CUDA device"):
        oq.gemm_w8a8(a, s, w, torch.ones(32))
    with pytest.raises(oq.OQError, match="int8"):
        oq.gemm_w8a8(a.float(), s, w, torch.ones(32))
    with pytest.raises(oq.OQError, match="unknown norm"):
        oq.Heads(64, 4, 2, norm="batch")
    with pytest.raises(oq.OQError, match="current CUDA device"):
        oq.Heads(64, 4, 2, q_weight=torch.ones(64))
    with pytest.raises(oq.OQError, match="same shape"):
        oq.Heads(64, 4, 2, rope="pairs", cos=torch.ones(4, 32))
    h = oq.Heads(64, 4, 2)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(oq.OQError, match="missing"):
        oq.qk_norm_rope(h, None, q[:, :2])
    with pytest.raises(oq.OQError, match="current CUDA device"):
        oq.qk_norm_rope(h, q, q[:, :2])
    with pytest.raises(oq.OQError, match="expected"):
        oq.qk_norm_rope(h, q[:, :3], q[:, :2])
