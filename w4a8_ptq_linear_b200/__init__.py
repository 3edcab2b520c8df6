"""Python binding of the rotated, quantized linear layer's C ABI (include/oq.h).

This module only marshals arguments: it turns torch tensors into device pointers and the
current CUDA stream into a ``cudaStream_t``, allocates outputs with torch, and calls the
shared library ``lib/liboq.so``. Every step of the layer runs in the library's kernels.
There is no CPU fallback: if the library is missing, importing works but every compute
call raises ``OQError``.

The function names follow the C ABI: ``rotate_quantize``, ``prepare_weights``,
``gemm_w4a8``, ``gemm_w4a4``, ``gemm_w4a2``, ``linear`` (oq_rotate_quantize, oq_prepare_weights, ...).

``stream=`` runs a call on another stream than the current one. What the call allocates (results,
workspace) then belongs to that stream; as ever in torch, the caller orders the streams: the call's
stream behind whatever wrote its inputs, and other streams behind the call before they read its
results (``wait_stream``), with ``record_stream`` for a tensor that outlives its owner's stream.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "liboq.so")
# the bounds-checked build (python -m w4a8_ptq_linear_b200.build --checked)
LIB_CHECKED_PATH = os.path.join(_PKG, "lib", "liboq_checked.so")

OQ_OK, OQ_ERR_INVALID_ARG, OQ_ERR_UNSUPPORTED, OQ_ERR_MISALIGNED = 0, 1, 2, 3
OQ_ERR_CUDA, OQ_ERR_DEVICE_TIMEOUT, OQ_ERR_NOMEM = 4, 5, 6
ACT_KINDS = {"int8_absmax": 0, "int4_absmax": 1, "int4_lloydmax": 2, "int4_percentile": 3,
             "int4_lloydmax_width": 4, "int8_lloydmax": 5, "int2_percentile": 6}
OUT_BF16, OUT_ACC = 0, 1
NORMS = {"none": 0, "rms": 1, "layer": 2}
ROPES = {"none": 0, "pairs": 1, "halves": 2}
W_INT4, W_INT8 = 0, 1

# (name, restype, argtypes) of every exported entry point
_P, _I, _I64, _U64, _SZ, _D = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                               ctypes.c_size_t, ctypes.c_double)
SIGNATURES = [
    ("oq_status_string", ctypes.c_char_p, [_I]),
    ("oq_last_error", ctypes.c_char_p, []),
    ("oq_device_status", _I, [_I, ctypes.POINTER(_U64)]),
    ("oq_default_block", _I, [_I]),
    ("oq_default_rounds", _I, [_I]),
    ("oq_rpbh_tables", _I, [_I, _I, _U64, _P, _P]),
    ("oq_lloyd_max_codebook", _I, [_P, _P]),
    ("oq_lloyd_max_codebook_width", _I, [_I, _P, _P]),
    ("oq_lloyd_max_codebook_8bit", _I, [_P, _P]),
    ("oq_plan_create", _I, [ctypes.POINTER(_P), _I, _I, _I, _U64, _I, _I]),
    ("oq_plan_destroy", None, [_P]),
    ("oq_plan_get_rpbh", _I, [_P, _I, _P, _P]),
    ("oq_plan_get_codebook", _I, [_P, _I, _P, _P]),
    ("oq_rotate_quantize", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    ("oq_prepare_weights", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    ("oq_gemm_w4a8", _I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_gemm_w4a4", _I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_gemm_w4a2", _I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_gemm_w4a8_lloydmax", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_linear_workspace_bytes", _SZ, [_P, _I64]),
    ("oq_linear", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    ("oq_debug_wait_timeout", _I, [_U64, _P]),
    ("oq_prepare_weights_g64", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    ("oq_gemm_w4a4_g64", _I, [_I, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_linear_g64", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    ("oq_linear_fused", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    ("oq_linear_static_scratch", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P]),
    ("oq_prepare_weights_w8", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P]),
    ("oq_gemm_w8a8", _I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    ("oq_linear_w8a8", _I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    ("oq_qk_norm_rope", _I, [_P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P]),
    ("oq_linear_qkv_workspace_bytes", _SZ, [_P, _P, _I, _I64, _I64]),
    ("oq_linear_qkv", _I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _I64, _P, _I64, _P,
                           _P, _SZ, _P]),
    ("oq_mma_peak_loop", _I, [_I, _I64, _P, _P]),
    ("oq_debug_pair_layout", _I, [_I, _I, _U64, _P]),
    ("oq_debug_drop_cluster", _I, []),
]


class OQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_status_name(status)}: {msg}")
        self.status = status


_lib = None


def _status_name(s: int) -> str:
    names = {0: "OQ_OK", 1: "OQ_ERR_INVALID_ARG", 2: "OQ_ERR_UNSUPPORTED",
             3: "OQ_ERR_MISALIGNED", 4: "OQ_ERR_CUDA", 5: "OQ_ERR_DEVICE_TIMEOUT",
             6: "OQ_ERR_NOMEM"}
    return names.get(s, f"status {s}")


def load(path: str):
    """A ctypes handle on a build of the library at `path`, with every signature set."""
    if not os.path.exists(path):
        raise OQError(OQ_ERR_UNSUPPORTED,
                      f"{path} is not built: run python -m w4a8_ptq_linear_b200.build")
    L = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def lib():
    """The loaded ctypes library; raises OQError if it is not built."""
    global _lib
    if _lib is None:
        _lib = load(LIB_PATH)
    return _lib


class using:
    """Within the block, every call of this module goes to the library build `handle` (for
    example ``load(LIB_CHECKED_PATH)``); plans must be created and used inside one build."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        global _lib
        self.saved = lib()
        _lib = self.handle
        return self.handle

    def __exit__(self, *exc):
        global _lib
        _lib = self.saved


def _check(status: int):
    if status != OQ_OK:
        raise OQError(status, lib().oq_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _new(like, shape, dtype, stream):
    """A new tensor on like's device, from the allocator's pool of the stream that the call runs on:
    a block of another stream's pool may still be in use there, and would go back to that stream
    while this one writes it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def device_status(clear: bool = True):
    """(status, code) of the device error word; synchronizes the current device."""
    code = ctypes.c_uint64(0)
    st = lib().oq_device_status(1 if clear else 0, ctypes.byref(code))
    return st, code.value


def default_block(d: int) -> int:
    return lib().oq_default_block(d)


def default_rounds(h: int) -> int:
    return lib().oq_default_rounds(h)


def rpbh_tables(d: int, round_: int, seed: int):
    """Host RPBH tables of one round: (signs int8[d], perm int32[d])."""
    s = np.empty(d, np.int8)
    p = np.empty(d, np.int32)
    _check(lib().oq_rpbh_tables(d, round_, seed, s.ctypes.data, p.ctypes.data))
    return s, p


def lloyd_max_codebook():
    """The library's Newton-solved N(0,1) codebook: (centroids[16], thresholds[15])."""
    c = np.empty(16, np.float64)
    t = np.empty(15, np.float64)
    _check(lib().oq_lloyd_max_codebook(c.ctypes.data, t.ctypes.data))
    return c, t


def lloyd_max_codebook_8bit():
    """The library's Newton-solved 256-level N(0,1) codebook: (centroids, thresholds)."""
    c = np.empty(256, np.float64)
    t = np.empty(255, np.float64)
    _check(lib().oq_lloyd_max_codebook_8bit(c.ctypes.data, t.ctypes.data))
    return c, t


def lloyd_max_codebook_width(d: int):
    """The library's Newton-solved codebook of the width-d marginal: (centroids, thresholds)."""
    c = np.empty(16, np.float64)
    t = np.empty(15, np.float64)
    _check(lib().oq_lloyd_max_codebook_width(d, c.ctypes.data, t.ctypes.data))
    return c, t


@dataclass
class Plan:
    """An RPBH plan on the current CUDA device (oq_plan_create / oq_plan_destroy)."""
    d: int
    h: int
    rounds: int
    seed: int = 0
    center: bool = False
    act: str = "int8_absmax"

    def __post_init__(self):
        h = ctypes.c_void_p()
        _check(lib().oq_plan_create(ctypes.byref(h), self.d, self.h, self.rounds, self.seed,
                                    1 if self.center else 0, ACT_KINDS[self.act]))
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            lib().oq_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def rpbh(self, round_: int):
        s = np.empty(self.d, np.int8)
        p = np.empty(self.d, np.int32)
        _check(lib().oq_plan_get_rpbh(self._h, round_, s.ctypes.data, p.ctypes.data))
        return s, p

    def codebook(self):
        """The plan's Lloyd-Max codebook (oq_plan_get_codebook): (centroids, thresholds),
        16 or 256 levels by the plan's activation kind."""
        levels = 256 if self.act == "int8_lloydmax" else 16
        c = np.empty(levels, np.float64)
        t = np.empty(levels - 1, np.float64)
        _check(lib().oq_plan_get_codebook(self._h, levels, c.ctypes.data, t.ctypes.data))
        return c, t

    @property
    def packed(self) -> bool:
        return self.act not in ("int8_absmax", "int8_lloydmax")

    @property
    def code_row_bytes(self) -> int:
        """Bytes of one token's codes: d (8-bit kinds), d/2 (4-bit) or d/4 (2-bit)."""
        if not self.packed:
            return self.d
        return self.d // 4 if self.act == "int2_percentile" else self.d // 2

    def workspace_bytes(self, T: int) -> int:
        return int(lib().oq_linear_workspace_bytes(self._h, T))


def rotate_quantize(plan: Plan, x, *, codes=None, scale=None, mean=None, rotated=False,
                    stream=None):
    """oq_rotate_quantize on a bf16 [T, d] CUDA tensor.

    Returns (codes, scale, mean or None, rotated float32 [T, d] or None)."""
    import torch
    T, ldx = x.shape[0], x.stride(0)
    if codes is None:
        codes = _new(x, (T, plan.code_row_bytes),
                     torch.int8 if plan.act == "int8_absmax" else torch.uint8, stream)
    if scale is None:
        scale = _new(x, (T,), torch.float32, stream)
    if plan.center and mean is None:
        mean = _new(x, (T,), torch.float32, stream)
    rot = _new(x, (T, plan.d), torch.float32, stream) if rotated else None
    _check(lib().oq_rotate_quantize(plan.handle, _ptr(x), T, ldx, _ptr(codes), _ptr(scale),
                                    _ptr(mean) if plan.center else None, _ptr(rot),
                                    _stream(stream)))
    return codes, scale, (mean if plan.center else None), rot


def prepare_weights(plan: Plan, w, *, stream=None):
    """oq_prepare_weights on a bf16 [n_out, d] CUDA tensor: (w_packed, w_scale, w_rowsum)."""
    import torch
    n = w.shape[0]
    wp = _new(w, (n, plan.d // 2), torch.uint8, stream)
    ws = _new(w, (n,), torch.float32, stream)
    w1 = _new(w, (n,), torch.float32, stream)
    _check(lib().oq_prepare_weights(plan.handle, _ptr(w), n, w.stride(0), _ptr(wp), _ptr(ws),
                                    _ptr(w1), _stream(stream)))
    return wp, ws, w1


def _out(like, T, N, out_kind, acc_dtype, out, stream):
    import torch
    if out is not None:
        return out
    return _new(like, (T, N), torch.bfloat16 if out_kind == OUT_BF16 else acc_dtype, stream)


def gemm_w4a8(a, a_scale, w_packed, w_scale, *, mean=None, w_rowsum=None, bias=None,
              out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w4a8: int8 [T, K] codes x packed INT4 [N, K/2] weights."""
    import torch
    T, K = a.shape
    N = w_packed.shape[0]
    out = _out(a, T, N, out_kind, torch.int32, out, stream)
    _check(lib().oq_gemm_w4a8(_ptr(a), _ptr(a_scale), _ptr(mean), _ptr(w_packed), _ptr(w_scale),
                              _ptr(w_rowsum), _ptr(bias), T, K, N, out_kind, _ptr(out),
                              _stream(stream)))
    return out


def gemm_w4a4(plan, kind, a_packed, a_scale, w_packed, w_scale, *, mean=None, w_rowsum=None,
              bias=None, out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w4a4: packed 4-bit [T, K/2] codes (absmax or Lloyd-Max) x packed INT4."""
    import torch
    T, K = a_packed.shape[0], a_packed.shape[1] * 2
    N = w_packed.shape[0]
    acc_dt = torch.float32 if kind.startswith("int4_lloydmax") else torch.int32
    out = _out(a_packed, T, N, out_kind, acc_dt, out, stream)
    _check(lib().oq_gemm_w4a4(plan.handle if plan is not None else None, ACT_KINDS[kind],
                              _ptr(a_packed), _ptr(a_scale), _ptr(mean), _ptr(w_packed),
                              _ptr(w_scale), _ptr(w_rowsum), _ptr(bias), T, K, N, out_kind,
                              _ptr(out), _stream(stream)))
    return out


def gemm_w4a2(a_packed, a_scale, w_packed, w_scale, *, mean=None, w_rowsum=None, bias=None,
              out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w4a2: 2-bit codes [T, K/4] (four per byte) x packed INT4 [N, K/2] weights."""
    import torch
    T, K = a_packed.shape[0], a_packed.shape[1] * 4
    N = w_packed.shape[0]
    out = _out(a_packed, T, N, out_kind, torch.int32, out, stream)
    _check(lib().oq_gemm_w4a2(_ptr(a_packed), _ptr(a_scale), _ptr(mean), _ptr(w_packed),
                              _ptr(w_scale), _ptr(w_rowsum), _ptr(bias), T, K, N, out_kind,
                              _ptr(out), _stream(stream)))
    return out


def gemm_w4a8_lloydmax(plan, codes, sigma, w_packed, w_scale, *, mean=None, w_rowsum=None,
                       bias=None, out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w4a8_lloydmax: uint8 [T, K] 8-bit Lloyd-Max codes x packed INT4."""
    import torch
    T, K = codes.shape
    N = w_packed.shape[0]
    out = _out(codes, T, N, out_kind, torch.float32, out, stream)
    _check(lib().oq_gemm_w4a8_lloydmax(plan.handle, _ptr(codes), _ptr(sigma), _ptr(mean),
                                       _ptr(w_packed), _ptr(w_scale), _ptr(w_rowsum), _ptr(bias),
                                       T, K, N, out_kind, _ptr(out), _stream(stream)))
    return out


def linear(plan: Plan, x, w_packed, w_scale, w_rowsum=None, bias=None, *, workspace=None,
           out=None, stream=None):
    """oq_linear: the whole layer on a bf16 [T, d] CUDA tensor -> bf16 [T, N]."""
    import torch
    T = x.shape[0]
    N = w_packed.shape[0]
    need = plan.workspace_bytes(T)
    if workspace is None:
        workspace = _new(x, (max(need, 256),), torch.uint8, stream)
    if out is None:
        out = _new(x, (T, N), torch.bfloat16, stream)
    _check(lib().oq_linear(plan.handle, _ptr(x), T, x.stride(0), _ptr(w_packed), _ptr(w_scale),
                           _ptr(w_rowsum), _ptr(bias), N, _ptr(out), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def linear_fused(plan: Plan, x, w_packed, w_scale, w_rowsum=None, bias=None, *, workspace=None,
                 out=None, stream=None):
    """oq_linear_fused: the whole layer in one launch (T <= 256; INT8 absmax, INT4 absmax and
    INT4 percentile plans)."""
    import torch
    T = x.shape[0]
    N = w_packed.shape[0]
    need = plan.workspace_bytes(T)
    if workspace is None:
        workspace = _new(x, (max(need, 256),), torch.uint8, stream)
    if out is None:
        out = _new(x, (T, N), torch.bfloat16, stream)
    _check(lib().oq_linear_fused(plan.handle, _ptr(x), T, x.stride(0), _ptr(w_packed),
                                 _ptr(w_scale), _ptr(w_rowsum), _ptr(bias), N, _ptr(out),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)))
    return out


def prepare_weights_g64(plan: Plan, w, *, stream=None):
    """oq_prepare_weights_g64 on a bf16 [n_out, d] CUDA tensor: asymmetric INT4 groups of 64.

    Returns (w_packed uint8 [n, d/2]: Q - 8 nibbles in the GEMM layout, K order 0, 2, 1, 3
    inside every four columns; w_sz int32 [d/64, n] of fp16 (sigma, z) pairs; w_scale float32
    [n] (ones); w_rowsum float32 [n])."""
    import torch
    n = w.shape[0]
    wp = _new(w, (n, plan.d // 2), torch.uint8, stream)
    wsz = _new(w, (plan.d // 64, n), torch.int32, stream)
    ws = _new(w, (n,), torch.float32, stream)
    w1 = _new(w, (n,), torch.float32, stream)
    _check(lib().oq_prepare_weights_g64(plan.handle, _ptr(w), n, w.stride(0), _ptr(wp), _ptr(wsz),
                                        _ptr(ws), _ptr(w1), _stream(stream)))
    return wp, wsz, ws, w1


def gemm_w4a4_g64(kind, a_packed, a_scale, w_packed, w_sz, w_scale, *, mean=None, w_rowsum=None,
                  bias=None, out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w4a4_g64: packed INT4 [T, K/2] codes x asymmetric grouped INT4 weights."""
    import torch
    T, K = a_packed.shape[0], a_packed.shape[1] * 2
    N = w_packed.shape[0]
    out = _out(a_packed, T, N, out_kind, torch.float32, out, stream)
    _check(lib().oq_gemm_w4a4_g64(ACT_KINDS[kind], _ptr(a_packed), _ptr(a_scale), _ptr(mean),
                                  _ptr(w_packed), _ptr(w_sz), _ptr(w_scale), _ptr(w_rowsum),
                                  _ptr(bias), T, K, N, out_kind, _ptr(out), _stream(stream)))
    return out


def linear_g64(plan: Plan, x, w_packed, w_sz, w_scale, w_rowsum=None, bias=None, *,
               workspace=None, out=None, stream=None):
    """oq_linear_g64: the whole layer against asymmetric grouped weights -> bf16 [T, N]."""
    import torch
    T = x.shape[0]
    N = w_packed.shape[0]
    need = plan.workspace_bytes(T)
    if workspace is None:
        workspace = _new(x, (max(need, 256),), torch.uint8, stream)
    if out is None:
        out = _new(x, (T, N), torch.bfloat16, stream)
    _check(lib().oq_linear_g64(plan.handle, _ptr(x), T, x.stride(0), _ptr(w_packed), _ptr(w_sz),
                               _ptr(w_scale), _ptr(w_rowsum), _ptr(bias), N, _ptr(out),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream)))
    return out


def linear_static_scratch(plan: Plan, x, w_packed, w_scale, w_rowsum=None, bias=None, *,
                          out=None, stream=None):
    """oq_linear_static_scratch: the whole layer without a caller workspace.

    For callers that cannot allocate device scratch (plug-ins inside a framework that owns all
    device memory, or paths that may not call cudaMalloc). The scratch is a 16 MiB array inside
    the library, shared by every call on the device; calls that overlap on the GPU race on it.
    T is limited to what fits that array. Make the first call on a device before any capture.
    """
    import torch
    T = x.shape[0]
    N = w_packed.shape[0]
    if out is None:
        out = _new(x, (T, N), torch.bfloat16, stream)
    _check(lib().oq_linear_static_scratch(plan.handle, _ptr(x), T, x.stride(0), _ptr(w_packed),
                                          _ptr(w_scale), _ptr(w_rowsum), _ptr(bias), N,
                                          _ptr(out), _stream(stream)))
    return out


# ---- INT8 weights and the attention input -----------------------------------------------------
# These calls cost a few microseconds on the GPU where tokens are few, so their checks are one
# comparison to a property; what is wrong is worked out in _refuse.

def _refuse(t, name, dtype, shape=None):
    """OQError for a tensor the library could not read: another type or size, on the host or
    another device, elements that do not follow one another."""
    import torch
    what = f"{name}: {t.dtype} {tuple(t.shape)}"
    if t.dtype != dtype:
        raise OQError(OQ_ERR_INVALID_ARG, f"{what}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        want = f"{shape[0]} elements" if len(shape) == 1 else tuple(shape)
        raise OQError(OQ_ERR_INVALID_ARG, f"{what}, expected {want}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise OQError(OQ_ERR_INVALID_ARG, f"{what} on {t.device}, not the current CUDA device")
    raise OQError(OQ_ERR_INVALID_ARG, f"{what}: must be contiguous, strides {t.stride()}")


def _device():
    """Index of the current CUDA device; -2, where no tensor is, before CUDA is in use."""
    import torch
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _raw_stream(stream, dev):
    import torch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _need(t, name, dtype, shape, dev):
    """The device pointer of a contiguous tensor of this type and shape on device `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, shape)
    return t.data_ptr()


def _need_opt(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _need_rows(t, name, dtype, d, dev):
    """Pointer and row pitch of a [rows, d] tensor whose rows may lie apart."""
    if t.dim() != 2 or t.shape[1] != d:
        _refuse(t, name, dtype, ("rows", d))
    n, _ = t.shape
    pitch, step = t.stride()
    if t.dtype is not dtype or t.get_device() != dev or step != 1:
        _refuse(t, name, dtype)
    return t.data_ptr(), n, pitch if n > 1 else d


def _need_2d(t, name, dtype, dev):
    """Pointer and shape of a contiguous matrix."""
    if t.dim() != 2 or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, name, dtype, None if t.dim() == 2 else ("rows", "columns"))
    return t.data_ptr(), *t.shape


_LAYER_SIZES = 64   # numbers of tokens whose workspace size a plan remembers at most


def _layer_bytes(plan, T):
    """plan.workspace_bytes(T), without asking the library again for the T of the last calls."""
    kept = plan.__dict__.setdefault("_layer_bytes", {})
    need = kept.get(T)
    if need is None:
        if len(kept) >= _LAYER_SIZES:
            kept.clear()
        need = kept[T] = plan.workspace_bytes(T)
    return need


def _scratch(workspace, need, like, stream):
    """Pointer and size of the caller's workspace, or of one from torch's allocator; the tensor
    itself, to be kept until the call has been made."""
    import torch
    if workspace is None:
        workspace = _new(like, (max(need, 256),), torch.uint8, stream)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise OQError(OQ_ERR_INVALID_ARG, "workspace: must be contiguous, on the input's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def prepare_weights_w8(plan: Plan, w, *, stream=None):
    """oq_prepare_weights_w8 on a bf16 [n_out, d] CUDA tensor: (w_codes int8 [n_out, d],
    w_scale float32 [n_out], w_rowsum float32 [n_out])."""
    import torch
    dev = _device()
    wp, n, ldw = _need_rows(w, "w", torch.bfloat16, plan.d, dev)
    codes = _new(w, (n, plan.d), torch.int8, stream)
    ws = _new(w, (n,), torch.float32, stream)
    w1 = _new(w, (n,), torch.float32, stream)
    _check(lib().oq_prepare_weights_w8(plan.handle, wp, n, ldw, codes.data_ptr(), ws.data_ptr(),
                                       w1.data_ptr(), _raw_stream(stream, dev)))
    return codes, ws, w1


def gemm_w8a8(a, a_scale, w_codes, w_scale, *, mean=None, w_rowsum=None, bias=None,
              out_kind=OUT_BF16, out=None, stream=None):
    """oq_gemm_w8a8: int8 [T, K] codes x int8 [N, K] weights -> bf16 (or int32 sums) [T, N]."""
    import torch
    f32, dev = torch.float32, _device()
    ap, T, K = _need_2d(a, "a", torch.int8, dev)
    wp, N, Kw = _need_2d(w_codes, "w_codes", torch.int8, dev)
    if Kw != K:
        raise OQError(OQ_ERR_INVALID_ARG, f"a has {K} columns, w_codes {Kw}")
    dt = torch.bfloat16 if out_kind == OUT_BF16 else torch.int32
    if out is None:
        out = _new(a, (T, N), dt, stream)
    else:
        _need(out, "out", dt, (T, N), dev)
    _check(lib().oq_gemm_w8a8(
        ap, _need(a_scale, "a_scale", f32, (T,), dev), _need_opt(mean, "mean", f32, (T,), dev), wp,
        _need(w_scale, "w_scale", f32, (N,), dev), _need_opt(w_rowsum, "w_rowsum", f32, (N,), dev),
        _need_opt(bias, "bias", torch.bfloat16, (N,), dev), T, K, N, out_kind,
        out.data_ptr(), _raw_stream(stream, dev)))
    return out


def linear_w8a8(plan: Plan, x, w_codes, w_scale, w_rowsum=None, bias=None, *, workspace=None,
                out=None, stream=None):
    """oq_linear_w8a8: the whole layer against INT8 weights, bf16 [T, d] -> bf16 [T, N]."""
    import torch
    f32, bf16, dev = torch.float32, torch.bfloat16, _device()
    xp, T, ldx = _need_rows(x, "x", bf16, plan.d, dev)
    wp, N, Kw = _need_2d(w_codes, "w_codes", torch.int8, dev)
    if Kw != plan.d:
        raise OQError(OQ_ERR_INVALID_ARG, f"w_codes: {Kw} columns, plan d={plan.d}")
    if out is None:
        out = _new(x, (T, N), bf16, stream)
    else:
        _need(out, "out", bf16, (T, N), dev)
    ws, nbytes, keep = _scratch(workspace, _layer_bytes(plan, T), x, stream)
    _check(lib().oq_linear_w8a8(
        plan.handle, xp, T, ldx, wp, _need(w_scale, "w_scale", f32, (N,), dev),
        _need_opt(w_rowsum, "w_rowsum", f32, (N,), dev), _need_opt(bias, "bias", bf16, (N,), dev),
        N, out.data_ptr(), ws, nbytes, _raw_stream(stream, dev)))
    return out


class _HeadsStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("head_dim", "q_heads", "k_heads", "norm", "rope",
                                               "rot_dim")]
                + [("eps", ctypes.c_float)]
                + [(n, _P) for n in ("q_weight", "q_bias", "k_weight", "k_bias", "cos", "sin")]
                + [("n_pos", _I64)])


class Heads:
    """The query and key heads of an attention input (oq_heads): their norm ("none", "rms",
    "layer") with float32 [head_dim] weights and biases, and their rotation ("none", "pairs",
    "halves") with float32 [n_pos, rot_dim / 2] tables of cosines and sines. It keeps the
    tensors alive and can be used by any number of calls on the device it was made on."""

    def __init__(self, head_dim, q_heads, k_heads, *, norm="rms", eps=1e-6, q_weight=None,
                 q_bias=None, k_weight=None, k_bias=None, rope="none", cos=None, sin=None):
        import torch
        f32, dev = torch.float32, _device()
        if norm not in NORMS or rope not in ROPES:
            raise OQError(OQ_ERR_INVALID_ARG, f"unknown norm {norm!r} or rope {rope!r}")
        self.head_dim, self.q_heads, self.k_heads = head_dim, q_heads, k_heads
        self._keep = (q_weight, q_bias, k_weight, k_bias, cos, sin)
        vec = [_need_opt(t, n, f32, (head_dim,), dev) for t, n in
               ((q_weight, "q_weight"), (q_bias, "q_bias"), (k_weight, "k_weight"),
                (k_bias, "k_bias"))]
        tab, rot, n_pos = [None, None], 0, 0
        if rope != "none":
            if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
                raise OQError(OQ_ERR_INVALID_ARG, "cos and sin: two tables of the same shape")
            tab = [_need(t, n, f32, cos.shape, dev) for t, n in ((cos, "cos"), (sin, "sin"))]
            n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        self.device = dev if any(vec + tab) else None   # without tensors: any
        self._s = _HeadsStruct(head_dim, q_heads, k_heads, NORMS[norm], ROPES[rope], rot, eps,
                               *vec, *tab, n_pos)
        self._ref = ctypes.addressof(self._s)

    def _check_device(self, dev):
        if self.device not in (None, dev):
            raise OQError(OQ_ERR_INVALID_ARG, f"heads belong to device {self.device}, current "
                                              f"device is {dev}")


_Strides = _I64 * 12


def _head_rows(t, name, shape, dev):
    """(pointer, batch, token and head stride) of a bf16 [S, heads, D] or [B, S, heads, D] view
    of this shape, elements contiguous."""
    import torch
    if (t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != dev
            or t.stride(-1) != 1):
        _refuse(t, name, torch.bfloat16, shape)
    st = t.stride()
    return t.data_ptr(), (st[:3] if len(st) == 4 else (0, st[0], st[1]))


def _positions(positions, B, S, dev):
    """(pointer, batch stride) of int32 [S] or [B, S] positions."""
    import torch
    if positions is None:
        return None, 0
    one = positions.dim() == 1
    return (_need(positions, "positions", torch.int32, (S,) if one else (B, S), dev),
            0 if one else S)


def qk_norm_rope(heads: Heads, q, k, *, positions=None, q_out=None, k_out=None, stream=None):
    """oq_qk_norm_rope on bf16 [S, heads, head_dim] or [B, S, heads, head_dim] tensors (any
    strides with contiguous elements; None where there are no such heads). positions: int32 [S]
    or [B, S], default 0..S-1; a negative one leaves its token unrotated. Returns (q_out, k_out),
    new contiguous tensors unless given; an output may be its input."""
    import torch
    dev = _device()
    heads._check_device(dev)
    first = q if q is not None else k
    if first is None:
        raise OQError(OQ_ERR_INVALID_ARG, "neither q nor k given")
    lead = tuple(first.shape[:-2])
    if len(lead) not in (1, 2):
        _refuse(first, "q" if q is not None else "k", torch.bfloat16, ("[B,] S", "heads", "D"))
    at, strides = [], ()
    for t, o, name, n in ((q, q_out, "q", heads.q_heads), (k, k_out, "k", heads.k_heads)):
        if t is None:
            if n or o is not None:
                raise OQError(OQ_ERR_INVALID_ARG, f"{name}: missing, with {n} heads")
            at += (None, None, None)
            strides += (0, 0, 0, 0, 0, 0)
            continue
        D = heads.head_dim
        shape = (*lead, n, D)
        ptr, st = _head_rows(t, name, shape, dev)
        if o is None:
            o = _new(t, shape, torch.bfloat16, stream)
            optr, ost = o.data_ptr(), (lead[-1] * n * D, n * D, D)
        else:
            optr, ost = _head_rows(o, name + "_out", shape, dev)
        at += (ptr, optr, o)
        strides += (*st, *ost)
    B, S = lead if len(lead) == 2 else (1, lead[0])
    pos, pbs = _positions(positions, B, S, dev)
    table = _Strides(*strides)                   # q, q_out, k, k_out, three strides each
    s = ctypes.addressof(table)
    _check(lib().oq_qk_norm_rope(heads._ref, B, S, at[0], s, at[3], s + 48, pos, pbs, at[1], s + 24,
                                 at[4], s + 72, _raw_stream(stream, dev)))
    return at[2], at[5]


def linear_qkv(plan: Plan, heads: Heads, x, w, w_scale, w_rowsum=None, bias=None, *, batch=1,
               positions=None, workspace=None, out=None, stream=None):
    """oq_linear_qkv: the projection of bf16 [batch * S, d] tokens to [batch * S, N] rows of
    query heads, key heads (both normed and rotated) and the remaining columns (values). w: int8
    [N, d] of prepare_weights_w8, or uint8 [N, d/2] of prepare_weights. positions: int32 [S] or
    [batch, S], as for qk_norm_rope; a [B, S] tensor also sets the batch."""
    import torch
    f32, bf16, dev = torch.float32, torch.bfloat16, _device()
    heads._check_device(dev)
    xp, T, ldx = _need_rows(x, "x", bf16, plan.d, dev)
    w8 = w.dtype is torch.int8
    wp, N, Kw = _need_2d(w, "w", torch.int8 if w8 else torch.uint8, dev)
    if Kw != (plan.d if w8 else plan.d // 2):
        raise OQError(OQ_ERR_INVALID_ARG, f"w: {Kw} columns for plan d={plan.d}")
    if positions is not None and positions.dim() == 2:
        batch = positions.shape[0]
    if batch < 0 or (T % batch if batch else T):
        raise OQError(OQ_ERR_INVALID_ARG, f"{T} tokens are not {batch} sequences of one length")
    S = T // batch if batch else 0 if positions is None else positions.shape[-1]
    pos, pbs = _positions(positions, batch, S, dev)
    if out is None:
        out = _new(x, (T, N), bf16, stream)
    else:
        _need(out, "out", bf16, (T, N), dev)
    L, kind = lib(), W_INT8 if w8 else W_INT4
    need = L.oq_linear_qkv_workspace_bytes(plan.handle, heads._ref, kind, T, N)
    ws, nbytes, keep = _scratch(workspace, need, x, stream)
    _check(L.oq_linear_qkv(
        plan.handle, heads._ref, xp, batch, S, ldx, kind, wp,
        _need(w_scale, "w_scale", f32, (N,), dev), _need_opt(w_rowsum, "w_rowsum", f32, (N,), dev),
        _need_opt(bias, "bias", bf16, (N,), dev), N, pos, pbs, out.data_ptr(), ws,
        nbytes, _raw_stream(stream, dev)))
    return out


def mma_peak_loop(kind: str, iters: int, stream=None) -> int:
    """oq_mma_peak_loop: launches the tensor-core peak loop (kind "i8", "f16", or "i8_serial":
    each group of four MMAs waited for before the next) on the stream; returns the number of
    CTA pairs, from which the operation count follows."""
    pairs = ctypes.c_int(0)
    _check(lib().oq_mma_peak_loop({"i8": 0, "f16": 1, "i8_serial": 2}[kind], iters,
                                  ctypes.byref(pairs), _stream(stream)))
    return pairs.value


def debug_pair_layout(d: int, h: int, seed: int = 0):
    """oq_debug_pair_layout: the word of every channel in the two-token kernel's
    interleaved row (int32[d])."""
    w = np.empty(d, np.int32)
    _check(lib().oq_debug_pair_layout(d, h, seed, w.ctypes.data))
    return w


def debug_wait_timeout(timeout_ns: int, stream=None):
    """Launch a kernel whose bounded wait must give up (tests the error path)."""
    _check(lib().oq_debug_wait_timeout(timeout_ns, _stream(stream)))


def debug_drop_cluster():
    """oq_debug_drop_cluster: this thread's next single launch goes out without its cluster."""
    _check(lib().oq_debug_drop_cluster())
