"""ctypes binding of ``libqvla.so`` (the C ABI declared in ``include/qvla.h``).

Argument marshalling only: every function here validates Python-side types,
allocates output tensors with PyTorch (device memory is PyTorch's job) and calls
the C entry point of the same name.  No step of the layer's arithmetic runs in
Python.  Importing this module loads the library and raises ImportError when it
has not been built (``python -m w4a4_post_quantization_zigzag_b200.build``).
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import (POINTER, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_uint32,
                    c_void_p)
from typing import Optional, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqvla.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m w4a4_post_quantization_zigzag_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)


def _check_stamp():
    """The loaded library must be the build of the sources next to it."""
    from . import build as _build
    _lib.qvla_source_hash.restype = ctypes.c_char_p
    have = _lib.qvla_source_hash().decode()
    want = _build.source_hash()
    if have != want:
        raise ImportError(f"{LIB_PATH} was built from other sources (stamp {have[:12]}, "
                          f"sources {want[:12]}): rebuild it with "
                          "`python -m w4a4_post_quantization_zigzag_b200.build`")


_check_stamp()

QVLA_OK = 0
QVLA_ERR_ARG = 1
QVLA_ERR_SHAPE = 2
QVLA_ERR_ALIGN = 3
QVLA_ERR_STEP_RANGE = 4
QVLA_ERR_UNSUPPORTED = 5
QVLA_ERR_CUDA = 6
QVLA_ERR_DEVICE_FLAG = 7
QVLA_ERR_WORKSPACE = 8

QVLA_DTYPE_F32 = 0
QVLA_DTYPE_BF16 = 1
QVLA_SCALE_DYNAMIC = 0
QVLA_SCALE_TABLE = 1

QVLA_DEVERR_STEP_RANGE = 0x1
QVLA_DEVERR_TIMEOUT = 0x2
QVLA_DEVERR_TMEM = 0x4
QVLA_DEVERR_CACHE_RANGE = 0x8

# Every symbol include/qvla.h declares.
EXPORTED = (
    "qvla_status_str", "qvla_abi_version", "qvla_read_error_word", "qvla_packed_sizes",
    "qvla_pack_weights", "qvla_rotate_weights_f32", "qvla_quant_pack_weights_f32",
    "qvla_rotate_quant_act", "qvla_rotate_act_f32", "qvla_quant_act_f32", "qvla_w4a4_gemm",
    "qvla_w4a4_gemm_s32", "qvla_rotate_quant_act_batched", "qvla_w4a4_gemm_batched",
    "qvla_rotate_quant_workspace_bytes", "qvla_rotate_quant_act_noalloc",
    "qvla_pack_weights_hadamard", "qvla_pack_weights_w8", "qvla_rotate_quant_act_a8",
    "qvla_rotate_quant_a8_workspace_bytes", "qvla_w8a8_gemm", "qvla_w8a8_gemm_s32",
    "qvla_gptq_quantize_host", "qvla_pack_weights_gptq", "qvla_gptq_hessian_host",
    "qvla_selftest_wait_timeout", "qvla_source_hash", "qvla_rotate_quant_act_a8_batched",
    "qvla_w8a8_gemm_batched", "qvla_pack_weights_w4g", "qvla_w4a16_gemv", "qvla_rope_table",
    "qvla_qk_norm_rope", "qvla_paged_attn_decode", "qvla_paged_attn_workspace_bytes",
)

QVLA_NOALLOC_SCRATCH_BYTES = 16 << 20


class qvla_packed_linear(ctypes.Structure):
    _fields_ = [("N", c_int32), ("K", c_int32), ("block", c_int32),
                ("perm", c_void_p), ("rot", c_void_p), ("rot_tc", c_void_p), ("wq", c_void_p),
                ("w_scale", c_void_p), ("bias", c_void_p)]


class qvla_linear_problem(ctypes.Structure):
    _fields_ = [("L", POINTER(qvla_packed_linear)), ("x", c_void_p), ("xdt", c_int32),
                ("M", c_int32), ("ldx", c_int32), ("mode", c_int32), ("table", c_void_p),
                ("T", c_int32), ("Lcount", c_int32), ("step_dev", c_void_p),
                ("step_host", c_int32), ("layer", c_int32), ("xq", c_void_p), ("s_x", c_void_p),
                ("y", c_void_p), ("ldy", c_int32), ("workspace", c_void_p),
                ("ws_bytes", c_size_t), ("xq8", c_void_p)]


class qvla_group_linear(ctypes.Structure):
    _fields_ = [("N", c_int32), ("K", c_int32), ("group", c_int32), ("sdt", c_int32),
                ("wq", c_void_p), ("w_scale", c_void_p), ("w_zero", c_void_p), ("bias", c_void_p)]


class qvla_kv_cache(ctypes.Structure):
    _fields_ = [("pages", c_int32), ("page_size", c_int32), ("heads", c_int32), ("dim", c_int32),
                ("bits", c_int32), ("k", c_void_p), ("v", c_void_p), ("page_stride", c_int64),
                ("token_stride", c_int64), ("head_stride", c_int64), ("k_scale", c_void_p),
                ("v_scale", c_void_p), ("s_page_stride", c_int64), ("s_token_stride", c_int64),
                ("s_head_stride", c_int64)]


_P = POINTER(qvla_packed_linear)
_PP = POINTER(qvla_linear_problem)
_sig = {
    "qvla_status_str": (ctypes.c_char_p, [c_int]),
    "qvla_abi_version": (c_int, []),
    "qvla_source_hash": (ctypes.c_char_p, []),
    "qvla_read_error_word": (c_int, [POINTER(c_uint32), c_int]),
    "qvla_selftest_wait_timeout": (c_int, [ctypes.c_uint64, c_void_p]),
    "qvla_packed_sizes": (c_int, [c_int, c_int, c_int, POINTER(c_size_t), POINTER(c_size_t),
                                  POINTER(c_size_t), POINTER(c_size_t)]),
    "qvla_pack_weights": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                  c_void_p]),
    "qvla_pack_weights_hadamard": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p,
                                           c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                           c_void_p]),
    "qvla_pack_weights_w8": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                     c_void_p]),
    "qvla_gptq_hessian_host": (c_int, [c_void_p, c_int, c_int, c_void_p]),
    "qvla_gptq_quantize_host": (c_int, [c_void_p, c_int, c_int, c_void_p, ctypes.c_double,
                                        c_void_p, c_void_p, c_void_p]),
    "qvla_pack_weights_gptq": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_int, c_int,
                                       ctypes.c_double, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                       c_void_p, c_size_t, c_void_p]),
    "qvla_rotate_quant_act_a8": (c_int, [c_void_p, c_int, c_int, c_int, _P, c_void_p, c_void_p,
                                         c_void_p, c_size_t, c_void_p]),
    "qvla_rotate_quant_a8_workspace_bytes": (c_int, [c_int, c_int, POINTER(c_size_t)]),
    "qvla_w8a8_gemm": (c_int, [c_void_p, c_void_p, c_int, _P, c_void_p, c_int, c_void_p]),
    "qvla_w8a8_gemm_s32": (c_int, [c_void_p, c_int, _P, c_void_p, c_void_p]),
    "qvla_rotate_weights_f32": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p,
                                        c_void_p, c_void_p]),
    "qvla_quant_pack_weights_f32": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p,
                                            c_void_p]),
    "qvla_rotate_quant_act": (c_int, [c_void_p, c_int, c_int, c_int, _P, c_int, c_void_p, c_int,
                                      c_int, c_void_p, c_int, c_int, c_void_p, c_void_p,
                                      c_void_p, c_size_t, c_void_p]),
    "qvla_rotate_quant_workspace_bytes": (c_int, [c_int, c_int, c_int, c_int, POINTER(c_size_t)]),
    "qvla_rotate_quant_act_noalloc": (c_int, [c_void_p, c_int, c_int, c_int, _P, c_int, c_void_p,
                                              c_int, c_int, c_void_p, c_int, c_int, c_void_p,
                                              c_void_p, c_void_p]),
    "qvla_rotate_act_f32": (c_int, [c_void_p, c_int, c_int, c_int, _P, c_void_p, c_void_p]),
    "qvla_quant_act_f32": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_int, c_int,
                                   c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "qvla_w4a4_gemm": (c_int, [c_void_p, c_void_p, c_int, _P, c_void_p, c_int, c_int, c_void_p]),
    "qvla_w4a4_gemm_s32": (c_int, [c_void_p, c_int, _P, c_void_p, c_int, c_void_p]),
    "qvla_rotate_quant_act_batched": (c_int, [_PP, c_int, c_void_p]),
    "qvla_w4a4_gemm_batched": (c_int, [_PP, c_int, c_int, c_void_p]),
    "qvla_rotate_quant_act_a8_batched": (c_int, [_PP, c_int, c_void_p]),
    "qvla_w8a8_gemm_batched": (c_int, [_PP, c_int, c_void_p]),
    "qvla_pack_weights_w4g": (c_int, [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                      c_void_p, c_void_p]),
    "qvla_w4a16_gemv": (c_int, [c_void_p, c_int, c_int, c_int, POINTER(qvla_group_linear),
                                c_void_p, c_int, c_int, c_void_p]),
    "qvla_rope_table": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p]),
    "qvla_qk_norm_rope": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                  c_int, c_int, c_int, c_void_p, c_void_p, c_float, c_void_p,
                                  c_int, c_int, c_int, c_void_p, POINTER(qvla_kv_cache), c_void_p,
                                  c_void_p, c_int, c_void_p, c_int, c_void_p]),
    "qvla_paged_attn_decode": (c_int, [c_void_p, c_int, c_int, c_int, c_int,
                                       POINTER(qvla_kv_cache), c_void_p, c_int, c_void_p, c_float,
                                       c_int, c_int, c_void_p, c_int, c_void_p, c_void_p, c_size_t,
                                       c_void_p]),
    "qvla_paged_attn_workspace_bytes": (c_int, [c_int, c_int, c_int, POINTER(c_size_t)]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class QvlaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {qvla_status_str(code)} (status {code})")


def qvla_status_str(code: int) -> str:
    return _lib.qvla_status_str(code).decode()


def qvla_abi_version() -> int:
    return _lib.qvla_abi_version()


def qvla_source_hash() -> str:
    return _lib.qvla_source_hash().decode()


def _check(rc: int, where: str):
    if rc != QVLA_OK:
        raise QvlaError(rc, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream) -> c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return c_void_p(stream.cuda_stream)
    return c_void_p(int(stream))


def qvla_read_error_word(clear: bool = True) -> int:
    v = c_uint32(0)
    _check(_lib.qvla_read_error_word(ctypes.byref(v), int(clear)), "qvla_read_error_word")
    return int(v.value)


def qvla_selftest_wait_timeout(limit_ns: int = 50_000, stream=None):
    """Launch the failure-path self-test: a wait that nothing ends, bounded
    by limit_ns; the error word then holds QVLA_DEVERR_TIMEOUT."""
    _check(_lib.qvla_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "qvla_selftest_wait_timeout")


def qvla_packed_sizes(N: int, K: int, block: int) -> Tuple[int, int, int, int]:
    """(wq_bytes, rot_bytes, rot_tc_bytes, workspace_bytes)."""
    a, b, t, c = c_size_t(), c_size_t(), c_size_t(), c_size_t()
    _check(_lib.qvla_packed_sizes(N, K, block, ctypes.byref(a), ctypes.byref(b), ctypes.byref(t),
                                  ctypes.byref(c)), "qvla_packed_sizes")
    return a.value, b.value, t.value, c.value


class PackedLinear:
    """Device buffers of one packed linear plus the C struct that points at them."""

    def __init__(self, N, K, block, perm, rot, wq, w_scale, bias=None, rot_tc=None):
        self.N, self.K, self.block = int(N), int(K), int(block)
        self.perm, self.rot, self.wq, self.w_scale, self.bias = perm, rot, wq, w_scale, bias
        self.rot_tc = rot_tc
        self._s = qvla_packed_linear(self.N, self.K, self.block, perm.data_ptr(),
                                     rot.data_ptr() if rot is not None else None,
                                     rot_tc.data_ptr() if rot_tc is not None else None,
                                     wq.data_ptr(), w_scale.data_ptr(),
                                     bias.data_ptr() if bias is not None else None)

    @property
    def struct(self):
        return ctypes.byref(self._s)

    def device_bytes(self) -> int:
        n = sum(t.numel() * t.element_size() for t in (self.perm, self.rot, self.wq, self.w_scale)
                if t is not None)
        n += self.rot_tc.numel() * 2 if self.rot_tc is not None else 0
        return n + (self.bias.numel() * 4 if self.bias is not None else 0)


def qvla_pack_weights(W: torch.Tensor, block: int, bias: Optional[torch.Tensor] = None,
                      perm_in: Optional[np.ndarray] = None, rsvd_in: Optional[np.ndarray] = None,
                      stream=None) -> PackedLinear:
    """W: cuda fp32 [N, K].  perm_in: host int32 [K]; rsvd_in: host float64 [nb, b, b]."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    wq_b, rot_b, tc_b, ws_b = qvla_packed_sizes(N, K, block)
    dev = W.device
    perm = torch.empty(K, dtype=torch.int32, device=dev)
    rot = torch.empty(rot_b // 4, dtype=torch.float32, device=dev)
    rot_tc = torch.empty(tc_b // 2, dtype=torch.int16, device=dev) if tc_b else None
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device=dev)
    s_w = torch.empty(N, dtype=torch.float32, device=dev)
    ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    p_in = r_in = None
    if perm_in is not None:
        perm_in = np.ascontiguousarray(perm_in, dtype=np.int32)
        assert perm_in.shape == (K,)
        p_in = perm_in.ctypes.data_as(c_void_p)
    if rsvd_in is not None:
        rsvd_in = np.ascontiguousarray(rsvd_in, dtype=np.float64)
        assert rsvd_in.shape == (K // block, block, block)
        r_in = rsvd_in.ctypes.data_as(c_void_p)
    _check(_lib.qvla_pack_weights(_ptr(W), N, K, block, p_in, r_in, _ptr(perm), _ptr(rot),
                                  _ptr(rot_tc), _ptr(wq), _ptr(s_w), _ptr(ws), ws_b,
                                  _stream(stream)), "qvla_pack_weights")
    if bias is not None:
        assert bias.is_cuda and bias.dtype == torch.float32 and bias.shape == (N,)
        bias = bias.contiguous()
    return PackedLinear(N, K, block, perm, rot.view(K // block, block, block), wq, s_w, bias,
                        rot_tc=rot_tc)


def qvla_pack_weights_hadamard(W: torch.Tensor, block: int, bias: Optional[torch.Tensor] = None,
                               perm_in: Optional[np.ndarray] = None, image: bool = True,
                               stream=None) -> PackedLinear:
    """Hadamard-only pack (R_SVD = I): rot = None; with `image` (blocks 64 /
    128) the tensor-core image of R_B = H_b, else rot_tc = None."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    wq_b, _, tc_b, ws_b = qvla_packed_sizes(N, K, block)
    dev = W.device
    rot_tc = torch.empty(tc_b // 2, dtype=torch.int16, device=dev) if (tc_b and image) else None
    perm = torch.empty(K, dtype=torch.int32, device=dev)
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device=dev)
    s_w = torch.empty(N, dtype=torch.float32, device=dev)
    ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    p_in = None
    if perm_in is not None:
        perm_in = np.ascontiguousarray(perm_in, dtype=np.int32)
        assert perm_in.shape == (K,)
        p_in = perm_in.ctypes.data_as(c_void_p)
    _check(_lib.qvla_pack_weights_hadamard(_ptr(W), N, K, block, p_in, _ptr(perm),
                                           _ptr(rot_tc), _ptr(wq), _ptr(s_w), _ptr(ws), ws_b,
                                           _stream(stream)),
           "qvla_pack_weights_hadamard")
    if bias is not None:
        assert bias.is_cuda and bias.dtype == torch.float32 and bias.shape == (N,)
        bias = bias.contiguous()
    return PackedLinear(N, K, block, perm, None, wq, s_w, bias, rot_tc=rot_tc)


def _host_f64(a, shape):
    if a is None:
        return None, None
    a = np.ascontiguousarray(a, dtype=np.float64)
    assert a.shape == shape
    return a, a.ctypes.data_as(c_void_p)


def qvla_gptq_hessian_host(xr: np.ndarray) -> np.ndarray:
    """H = X'^T X' (fp64 [K, K]) of host fp32 rotated calibration rows [T, K]."""
    xr = np.ascontiguousarray(xr, dtype=np.float32)
    T, K = xr.shape
    H = np.empty((K, K), np.float64)
    _check(_lib.qvla_gptq_hessian_host(xr.ctypes.data_as(c_void_p), T, K,
                                       H.ctypes.data_as(c_void_p)), "qvla_gptq_hessian_host")
    return H


def qvla_gptq_quantize_host(Wr: np.ndarray, H: Optional[np.ndarray] = None, damp: float = 0.05,
                            U: Optional[np.ndarray] = None):
    """GPTQ codes of host fp32 rotated weights Wr [N, K]; returns (int8 [N, K], fp32 [N])."""
    Wr = np.ascontiguousarray(Wr, dtype=np.float32)
    N, K = Wr.shape
    H, h_p = _host_f64(H, (K, K))
    U, u_p = _host_f64(U, (K, K))
    q = np.empty((N, K), np.int8)
    s = np.empty(N, np.float32)
    _check(_lib.qvla_gptq_quantize_host(Wr.ctypes.data_as(c_void_p), N, K, h_p, float(damp), u_p,
                                        q.ctypes.data_as(c_void_p), s.ctypes.data_as(c_void_p)),
           "qvla_gptq_quantize_host")
    return q, s


def qvla_pack_weights_gptq(W: torch.Tensor, block: int, x_cal: Optional[torch.Tensor] = None,
                           damp: float = 0.05, bias: Optional[torch.Tensor] = None,
                           perm_in: Optional[np.ndarray] = None,
                           rsvd_in: Optional[np.ndarray] = None, U: Optional[np.ndarray] = None,
                           stream=None) -> PackedLinear:
    """As qvla_pack_weights, with GPTQ weight codes (calibration rows x_cal [T, K] on the device,
    fp32 or bf16, or a given inverse-Hessian factor U)."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    wq_b, rot_b, tc_b, ws_b = qvla_packed_sizes(N, K, block)
    dev = W.device
    perm = torch.empty(K, dtype=torch.int32, device=dev)
    rot = torch.empty(rot_b // 4, dtype=torch.float32, device=dev)
    rot_tc = torch.empty(tc_b // 2, dtype=torch.int16, device=dev) if tc_b else None
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device=dev)
    s_w = torch.empty(N, dtype=torch.float32, device=dev)
    ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    p_in = None
    if perm_in is not None:
        perm_in = np.ascontiguousarray(perm_in, dtype=np.int32)
        assert perm_in.shape == (K,)
        p_in = perm_in.ctypes.data_as(c_void_p)
    rsvd_in, r_in = _host_f64(rsvd_in, (K // block, block, block))
    U, u_p = _host_f64(U, (K, K))
    T, xdt, cal, cal_b = 0, QVLA_DTYPE_F32, None, 0
    if x_cal is not None:
        assert x_cal.is_cuda and x_cal.is_contiguous() and x_cal.dim() == 2 and x_cal.shape[1] == K
        xdt = _dtype_code(x_cal)
        T = x_cal.shape[0]
        cal = torch.empty(T * K, dtype=torch.float32, device=dev)
        cal_b = T * K * 4
    _check(_lib.qvla_pack_weights_gptq(_ptr(W), N, K, block, _ptr(x_cal), xdt, T, float(damp),
                                       p_in, r_in, u_p, _ptr(perm), _ptr(rot), _ptr(rot_tc),
                                       _ptr(wq), _ptr(s_w), _ptr(ws), ws_b, _ptr(cal), cal_b,
                                       _stream(stream)), "qvla_pack_weights_gptq")
    if bias is not None:
        assert bias.is_cuda and bias.dtype == torch.float32 and bias.shape == (N,)
        bias = bias.contiguous()
    return PackedLinear(N, K, block, perm, rot.view(K // block, block, block), wq, s_w, bias,
                        rot_tc=rot_tc)


def qvla_pack_weights_w8(W: torch.Tensor, block: int, bias: Optional[torch.Tensor] = None,
                         perm_in: Optional[np.ndarray] = None,
                         rsvd_in: Optional[np.ndarray] = None, image: bool = True,
                         stream=None) -> PackedLinear:
    """W8A8 variant: the same P and R (and, with `image`, the tensor-core image
    of R_B for blocks 64 / 128), int8 weight codes wq [N, K]."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    _, rot_b, tc_b, ws_b = qvla_packed_sizes(N, K, block)
    dev = W.device
    rot_tc = torch.empty(tc_b // 2, dtype=torch.int16, device=dev) if (tc_b and image) else None
    perm = torch.empty(K, dtype=torch.int32, device=dev)
    rot = torch.empty(rot_b // 4, dtype=torch.float32, device=dev)
    wq = torch.empty(N, K, dtype=torch.int8, device=dev)
    s_w = torch.empty(N, dtype=torch.float32, device=dev)
    ws = torch.empty(ws_b, dtype=torch.uint8, device=dev)
    p_in = r_in = None
    if perm_in is not None:
        perm_in = np.ascontiguousarray(perm_in, dtype=np.int32)
        assert perm_in.shape == (K,)
        p_in = perm_in.ctypes.data_as(c_void_p)
    if rsvd_in is not None:
        rsvd_in = np.ascontiguousarray(rsvd_in, dtype=np.float64)
        assert rsvd_in.shape == (K // block, block, block)
        r_in = rsvd_in.ctypes.data_as(c_void_p)
    _check(_lib.qvla_pack_weights_w8(_ptr(W), N, K, block, p_in, r_in, _ptr(perm), _ptr(rot),
                                     _ptr(rot_tc), _ptr(wq), _ptr(s_w), _ptr(ws), ws_b,
                                     _stream(stream)),
           "qvla_pack_weights_w8")
    if bias is not None:
        assert bias.is_cuda and bias.dtype == torch.float32 and bias.shape == (N,)
        bias = bias.contiguous()
    return PackedLinear(N, K, block, perm, rot.view(K // block, block, block), wq, s_w, bias,
                        rot_tc=rot_tc)


def qvla_rotate_quant_a8_workspace_bytes(M: int, K: int) -> int:
    b = c_size_t()
    _check(_lib.qvla_rotate_quant_a8_workspace_bytes(M, K, ctypes.byref(b)),
           "qvla_rotate_quant_a8_workspace_bytes")
    return b.value


def qvla_rotate_quant_act_a8(x: torch.Tensor, L: PackedLinear,
                             xq8: Optional[torch.Tensor] = None,
                             s_x: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """8-bit per-token dynamic codes xq8 [M, K] int8 and s_x [M]."""
    M = x.shape[0]
    if xq8 is None:
        xq8 = torch.empty(M, L.K, dtype=torch.int8, device=x.device)
    if s_x is None:
        s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(qvla_rotate_quant_a8_workspace_bytes(M, L.K), 16),
                                dtype=torch.uint8, device=x.device)
    _check(_lib.qvla_rotate_quant_act_a8(_ptr(x), _dtype_code(x), M, x.stride(0), L.struct,
                                         _ptr(xq8), _ptr(s_x), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream)), "qvla_rotate_quant_act_a8")
    return xq8, s_x


def qvla_w8a8_gemm(xq8: torch.Tensor, s_x: torch.Tensor, L: PackedLinear,
                   y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M = xq8.shape[0]
    if y is None:
        y = torch.empty(M, L.N, dtype=torch.bfloat16, device=xq8.device)
    _check(_lib.qvla_w8a8_gemm(_ptr(xq8), _ptr(s_x), M, L.struct, _ptr(y), y.stride(0),
                               _stream(stream)), "qvla_w8a8_gemm")
    return y


def qvla_w8a8_gemm_s32(xq8: torch.Tensor, L: PackedLinear, stream=None) -> torch.Tensor:
    M = xq8.shape[0]
    acc = torch.empty(M, L.N, dtype=torch.int32, device=xq8.device)
    _check(_lib.qvla_w8a8_gemm_s32(_ptr(xq8), M, L.struct, _ptr(acc), _stream(stream)),
           "qvla_w8a8_gemm_s32")
    return acc


def qvla_rotate_weights_f32(W: torch.Tensor, block: int, perm: torch.Tensor,
                            rsvd64: torch.Tensor, stream=None) -> torch.Tensor:
    N, K = W.shape
    Wr = torch.empty(N, K, dtype=torch.float32, device=W.device)
    _check(_lib.qvla_rotate_weights_f32(_ptr(W), N, K, block, _ptr(perm), _ptr(rsvd64), _ptr(Wr),
                                        _stream(stream)), "qvla_rotate_weights_f32")
    return Wr


def qvla_quant_pack_weights_f32(Wr: torch.Tensor, stream=None):
    N, K = Wr.shape
    wq = torch.empty(N, K // 2, dtype=torch.uint8, device=Wr.device)
    s_w = torch.empty(N, dtype=torch.float32, device=Wr.device)
    _check(_lib.qvla_quant_pack_weights_f32(_ptr(Wr), N, K, _ptr(wq), _ptr(s_w), _stream(stream)),
           "qvla_quant_pack_weights_f32")
    return wq, s_w


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return QVLA_DTYPE_BF16
    if x.dtype == torch.float32:
        return QVLA_DTYPE_F32
    raise TypeError(f"unsupported activation dtype {x.dtype}")


def _expect(t: torch.Tensor, dtype, shape, device, name: str):
    """Caller-given buffers: the kernels write exactly this shape, densely."""
    if (t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device
            or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def _expect_rows(x: torch.Tensor, K: int, name: str = "x"):
    """Token rows [M, K] with unit stride along K (any row pitch)."""
    if x.dim() != 2 or x.shape[1] != K or (x.numel() and x.stride(1) != 1):
        raise ValueError(f"{name}: expected [M, {K}] rows with unit stride along K, "
                         f"got shape {tuple(x.shape)} strides {tuple(x.stride())}")


def _step_args(step):
    """int -> checked on the host; cuda int32 tensor -> read on the device."""
    if step is None:
        return None, 0
    if isinstance(step, torch.Tensor):
        assert step.is_cuda and step.dtype == torch.int32
        return _ptr(step), 0
    return None, int(step)


def qvla_rotate_quant_workspace_bytes(M: int, K: int, block: int, dtype=torch.bfloat16) -> int:
    b = c_size_t()
    code = QVLA_DTYPE_BF16 if dtype == torch.bfloat16 else QVLA_DTYPE_F32
    _check(_lib.qvla_rotate_quant_workspace_bytes(M, K, block, code, ctypes.byref(b)),
           "qvla_rotate_quant_workspace_bytes")
    return b.value


def qvla_rotate_quant_act(x: torch.Tensor, L: PackedLinear, mode: int = QVLA_SCALE_DYNAMIC,
                          table: Optional[torch.Tensor] = None, step=None, layer: int = 0,
                          xq: Optional[torch.Tensor] = None, s_x: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """workspace: optional uint8 device scratch of qvla_rotate_quant_workspace_bytes() bytes."""
    _expect_rows(x, L.K)
    M = x.shape[0]
    if xq is None:
        xq = torch.empty(M, L.K // 2, dtype=torch.uint8, device=x.device)
    if s_x is None:
        s_x = torch.empty(M, dtype=torch.float32, device=x.device)
    _expect(xq, torch.uint8, (M, L.K // 2), x.device, "xq")
    _expect(s_x, torch.float32, (M,), x.device, "s_x")
    T, Lc = (table.shape if table is not None else (0, 0))
    sd, sh = _step_args(step)
    ws_n = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.qvla_rotate_quant_act(_ptr(x), _dtype_code(x), M, x.stride(0), L.struct, mode,
                                      _ptr(table), T, Lc, sd, sh, layer, _ptr(xq), _ptr(s_x),
                                      _ptr(workspace), ws_n, _stream(stream)),
           "qvla_rotate_quant_act")
    return xq, s_x


def qvla_rotate_quant_act_noalloc(x: torch.Tensor, L: PackedLinear, xq: torch.Tensor,
                                  s_x: torch.Tensor, mode: int = QVLA_SCALE_DYNAMIC,
                                  table: Optional[torch.Tensor] = None, step=None,
                                  layer: int = 0, stream=None):
    """qvla_rotate_quant_act for callers that cannot allocate device memory:
    the outputs are given, and the scratch is the library's fixed per-device
    array (at most QVLA_NOALLOC_SCRATCH_BYTES).  Calls that may overlap on the
    GPU race on that array."""
    _expect_rows(x, L.K)
    M = x.shape[0]
    _expect(xq, torch.uint8, (M, L.K // 2), x.device, "xq")
    _expect(s_x, torch.float32, (M,), x.device, "s_x")
    T, Lc = (table.shape if table is not None else (0, 0))
    sd, sh = _step_args(step)
    _check(_lib.qvla_rotate_quant_act_noalloc(_ptr(x), _dtype_code(x), M, x.stride(0), L.struct,
                                              mode, _ptr(table), T, Lc, sd, sh, layer, _ptr(xq),
                                              _ptr(s_x), _stream(stream)),
           "qvla_rotate_quant_act_noalloc")
    return xq, s_x


def qvla_rotate_act_f32(x: torch.Tensor, L: PackedLinear, stream=None) -> torch.Tensor:
    M = x.shape[0]
    xr = torch.empty(M, L.K, dtype=torch.float32, device=x.device)
    _check(_lib.qvla_rotate_act_f32(_ptr(x), _dtype_code(x), M, x.stride(0), L.struct, _ptr(xr),
                                    _stream(stream)), "qvla_rotate_act_f32")
    return xr


def qvla_quant_act_f32(xr: torch.Tensor, mode: int = QVLA_SCALE_DYNAMIC,
                       table: Optional[torch.Tensor] = None, step=None, layer: int = 0,
                       stream=None):
    M, K = xr.shape
    xq = torch.empty(M, K // 2, dtype=torch.uint8, device=xr.device)
    s_x = torch.empty(M, dtype=torch.float32, device=xr.device)
    T, Lc = (table.shape if table is not None else (0, 0))
    sd, sh = _step_args(step)
    _check(_lib.qvla_quant_act_f32(_ptr(xr), M, K, mode, _ptr(table), T, Lc, sd, sh, layer,
                                   _ptr(xq), _ptr(s_x), _stream(stream)), "qvla_quant_act_f32")
    return xq, s_x


def qvla_w4a4_gemm(xq: torch.Tensor, s_x: torch.Tensor, L: PackedLinear, split_k: int = 0,
                   y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    M = xq.shape[0]
    if y is None:
        y = torch.empty(M, L.N, dtype=torch.bfloat16, device=xq.device)
    _check(_lib.qvla_w4a4_gemm(_ptr(xq), _ptr(s_x), M, L.struct, _ptr(y), y.stride(0), split_k,
                               _stream(stream)), "qvla_w4a4_gemm")
    return y


def qvla_w4a4_gemm_s32(xq: torch.Tensor, L: PackedLinear, split_k: int = 0,
                       stream=None) -> torch.Tensor:
    M = xq.shape[0]
    acc = torch.empty(M, L.N, dtype=torch.int32, device=xq.device)
    _check(_lib.qvla_w4a4_gemm_s32(_ptr(xq), M, L.struct, _ptr(acc), split_k, _stream(stream)),
           "qvla_w4a4_gemm_s32")
    return acc


def from_host_packed(wq: np.ndarray, s_w: np.ndarray, perm: np.ndarray, rsvd: np.ndarray,
                     bias: Optional[np.ndarray] = None, device="cuda") -> PackedLinear:
    """Uploads host arrays into a PackedLinear (e.g. to run the GEMM on given codes)."""
    N, Kh = wq.shape
    K = 2 * Kh
    block = rsvd.shape[-1]
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).to(device)
    return PackedLinear(N, K, block, t(perm, np.int32), t(rsvd, np.float32), t(wq, np.uint8),
                        t(s_w, np.float32), None if bias is None else t(bias, np.float32))


class LinearProblem:
    """One independent linear of a batched call; keeps its tensors alive."""

    def __init__(self, L: PackedLinear, x: Optional[torch.Tensor] = None,
                 mode: int = QVLA_SCALE_DYNAMIC, table: Optional[torch.Tensor] = None,
                 step=None, layer: int = 0, xq: Optional[torch.Tensor] = None,
                 s_x: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, xq8=None):
        """xq8: the int8 image of the codes that the batched rotate-quantise
        writes and the batched GEMM reads (a device int8 [M, K] tensor, or
        True to allocate one); None leaves the GEMM to unpack xq."""
        M = x.shape[0] if x is not None else xq.shape[0]
        dev = (x if x is not None else xq).device
        if x is not None:
            _expect_rows(x, L.K)
        self.L, self.x, self.table, self.step = L, x, table, step
        self.xq = xq if xq is not None else torch.empty(M, L.K // 2, dtype=torch.uint8, device=dev)
        self.s_x = s_x if s_x is not None else torch.empty(M, dtype=torch.float32, device=dev)
        self.y = y if y is not None else torch.empty(M, L.N, dtype=torch.bfloat16, device=dev)
        if xq8 is True:
            xq8 = torch.empty(M, L.K, dtype=torch.int8, device=dev)
        self.xq8 = xq8
        _expect(self.xq, torch.uint8, (M, L.K // 2), dev, "xq")
        _expect(self.s_x, torch.float32, (M,), dev, "s_x")
        if xq8 is not None:
            _expect(xq8, torch.int8, (M, L.K), dev, "xq8")
        if self.y.dim() != 2 or tuple(self.y.shape) != (M, L.N) or self.y.stride(1) != 1 \
                or self.y.dtype != torch.bfloat16:
            raise ValueError(f"y: expected bf16 [{M}, {L.N}] rows with unit stride")
        T, Lc = (table.shape if table is not None else (0, 0))
        sd, sh = _step_args(step)
        self.c = qvla_linear_problem(
            ctypes.pointer(L._s), x.data_ptr() if x is not None else None,
            _dtype_code(x) if x is not None else QVLA_DTYPE_BF16, M,
            x.stride(0) if x is not None else L.K, mode,
            table.data_ptr() if table is not None else None, T, Lc,
            sd.value if sd is not None else None, sh, layer, self.xq.data_ptr(),
            self.s_x.data_ptr(), self.y.data_ptr(), self.y.stride(0),
            workspace.data_ptr() if workspace is not None else None,
            workspace.numel() * workspace.element_size() if workspace is not None else 0,
            xq8.data_ptr() if xq8 is not None else None)
        self.workspace = workspace


def _problem_array(problems):
    arr = (qvla_linear_problem * len(problems))(*[p.c for p in problems])
    return arr


def qvla_rotate_quant_act_batched(problems, stream=None):
    arr = _problem_array(problems)
    _check(_lib.qvla_rotate_quant_act_batched(arr, len(problems), _stream(stream)),
           "qvla_rotate_quant_act_batched")


def qvla_w4a4_gemm_batched(problems, split_k: int = 0, stream=None):
    arr = _problem_array(problems)
    _check(_lib.qvla_w4a4_gemm_batched(arr, len(problems), split_k, _stream(stream)),
           "qvla_w4a4_gemm_batched")


def qvla_rotate_quant_act_a8_batched(problems, stream=None):
    """8-bit activation codes of W8A8 linears: each problem's xq8 (int8
    [M, K]) receives the codes themselves and s_x the per-token scales; each
    problem needs a workspace (qvla_rotate_quant_a8_workspace_bytes)."""
    arr = _problem_array(problems)
    _check(_lib.qvla_rotate_quant_act_a8_batched(arr, len(problems), _stream(stream)),
           "qvla_rotate_quant_act_a8_batched")


def qvla_w8a8_gemm_batched(problems, stream=None):
    """W8A8 GEMMs of the problems (xq8 holds 8-bit codes, L a W8 pack)."""
    arr = _problem_array(problems)
    _check(_lib.qvla_w8a8_gemm_batched(arr, len(problems), _stream(stream)),
           "qvla_w8a8_gemm_batched")


# --------------------------------------------------------------------------
# Operators around the linears of a decode step
# --------------------------------------------------------------------------

def _launch(fn, where: str, device: int, stream, *args):
    """fn(*args, stream) with `device` current; by default on its current stream."""
    if device < 0:
        raise ValueError(f"{where}: the tensors must be on a CUDA device")
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _launch(fn, where, device, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = fn(*args, stream)
    if rc != QVLA_OK:
        raise QvlaError(rc, where)


def _empty(shape, dtype, device, stream, like: Optional[torch.Tensor] = None) -> torch.Tensor:
    """An output or scratch tensor whose memory belongs to the stream the
    kernel runs on, so that its earlier and later uses there are in order.
    like: a tensor of this shape, type and place, if there is one."""
    if stream is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _expect_on(t: torch.Tensor, dtype, shape, device: int, name: str):
    """A dense tensor of exactly this type and shape on CUDA device `device`."""
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != device
            or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on cuda:{device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")


def qvla_pack_weights_w4g(W: torch.Tensor, group: int = 128, zero_points: bool = False,
                          scale_dtype=torch.float32, stream=None):
    """4-bit codes of W (cuda fp32 [N, K]) with one scale per `group` inputs:
    (wq uint8 [N, K/2], w_scale [N, K/group], w_zero uint8 [N, K/group] or None)."""
    if W.dim() != 2:
        raise ValueError(f"W: expected [N, K], got shape {tuple(W.shape)}")
    N, K = W.shape
    dev = W.get_device()
    _expect_on(W, torch.float32, (N, K), dev, "W")
    _expect_int32("W", N | K)
    if group <= 0 or K % group:
        raise QvlaError(QVLA_ERR_SHAPE, "qvla_pack_weights_w4g")
    wq = _empty((N, K // 2), torch.uint8, W.device, stream)
    scale = _empty((N, K // group), scale_dtype, W.device, stream)
    zero = _empty((N, K // group), torch.uint8, W.device, stream) if zero_points else None
    _launch(_lib.qvla_pack_weights_w4g, "qvla_pack_weights_w4g", dev, stream, W.data_ptr(), N, K,
            group, _dtype_code(scale), wq.data_ptr(), scale.data_ptr(),
            None if zero is None else zero.data_ptr())
    return wq, scale, zero


def qvla_w4a16_gemv(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                    w_zero: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, out_dtype=None,
                    stream=None) -> torch.Tensor:
    """y [M, N] = x W^T + bias for few rows x (bf16 or fp32 [M, K]) and the
    group-quantised weights of qvla_pack_weights_w4g(); y has out_dtype
    (default: x's)."""
    N, Kh = wq.shape
    K, groups = 2 * Kh, w_scale.shape[-1]
    dev, dt = x.get_device(), out_dtype or x.dtype
    _expect_rows(x, K)
    _expect_on(wq, torch.uint8, (N, Kh), dev, "wq")
    _expect_on(w_scale, w_scale.dtype, (N, groups), dev, "w_scale")
    if groups == 0 or K % groups:
        raise ValueError(f"w_scale: {groups} groups do not divide {K} inputs")
    if w_zero is not None:
        _expect_on(w_zero, torch.uint8, (N, groups), dev, "w_zero")
    if bias is not None:
        _expect_on(bias, torch.float32, (N,), dev, "bias")
    M = x.shape[0]
    ldx = x.stride(0) if M > 1 else K
    _expect_int32("x", M | N | K | ldx)
    pitch = (N + 7) // 8 * 8              # rows whose pitch is a multiple of 16 bytes
    if y is None:
        y = _empty((M, pitch), dt, x.device, stream)
        if N != pitch:
            y = y[:, :N]
    elif (y.shape != (M, N) or y.get_device() != dev or (y.stride(1) != 1 and y.numel())
          or (out_dtype is not None and y.dtype is not dt)):
        raise ValueError(f"y: expected {dt} [{M}, {N}] rows with unit stride on {x.device}")
    ldy = y.stride(0) if M > 1 else pitch
    _expect_int32("y", ldy)
    L = qvla_group_linear(N, K, K // groups, _dtype_code(w_scale), wq.data_ptr(),
                          w_scale.data_ptr(), _address(w_zero), _address(bias))
    _launch(_lib.qvla_w4a16_gemv, "qvla_w4a16_gemv", dev, stream, x.data_ptr(), _dtype_code(x), M,
            ldx, L, y.data_ptr(), _dtype_code(y), ldy)
    return y


def qvla_rope_table(inv_freq, P: int, device="cuda", stream=None) -> torch.Tensor:
    """fp32 [P, 2 * len(inv_freq)]: cosines, then sines, of p * inv_freq for
    positions p < P (inv_freq: host float64, one entry per pair)."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if f.ndim != 1:
        raise ValueError("inv_freq: expected one frequency per pair")
    _expect_int32("qvla_rope_table", P)
    table = _empty((P, 2 * f.shape[0]), torch.float32, torch.device(device), stream)
    _launch(_lib.qvla_rope_table, "qvla_rope_table", table.get_device(), stream,
            f.ctypes.data_as(c_void_p), f.shape[0], P, table.data_ptr())
    return table


def _expect_int32(where: str, bits: int):
    """bits: sizes, or their bitwise or, that the C call takes as 32-bit integers."""
    if bits >> 31:
        raise QvlaError(QVLA_ERR_SHAPE, where)


def _head_rows(x: torch.Tensor, shape, device: int, dtype, name: str) -> int:
    """The row pitch of [rows, heads, dim] whose heads lie one after the other."""
    st = x.stride()
    if (x.shape != shape or x.dtype is not dtype or x.get_device() != device
            or ((st[2] != 1 or (st[1] != shape[2] and shape[1] > 1)) and x.numel())):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} rows on cuda:{device} with the "
                         f"heads one after the other, got {x.dtype} {tuple(x.shape)} with strides "
                         f"{tuple(st)} on {x.device}")
    pitch = st[0] if shape[0] > 1 else shape[1] * shape[2]
    _expect_int32(name, shape[0] | shape[1] | shape[2] | pitch)
    return pitch


def _kv_struct(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale, v_scale, device: int):
    """The C cache of [pages, page_size, heads, dim] views in any memory order
    (bf16, or int8 with fp32 scales [pages, page_size, heads])."""
    shape, st, dt = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or st[3] != 1:
        raise ValueError("k_cache: expected [pages, page_size, heads, dim] with unit stride "
                         f"along dim, got shape {tuple(shape)} strides {tuple(st)}")
    if v_cache.shape != shape or v_cache.stride() != st or v_cache.dtype is not dt:
        raise ValueError("v_cache: expected the shape, strides and type of k_cache")
    _expect_int32("k_cache", shape[0] | shape[1] | shape[2] | shape[3])
    if k_cache.get_device() != device or v_cache.get_device() != device:
        raise ValueError(f"k_cache, v_cache: expected them on cuda:{device}")
    if dt is torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale, v_scale: a bf16 cache has none")
        return qvla_kv_cache(*shape, 16, k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1],
                             st[2])
    if dt is not torch.int8:
        raise TypeError(f"unsupported cache dtype {dt}")
    for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if (s is None or s.dtype is not torch.float32 or s.shape != shape[:3]
                or s.get_device() != device):
            raise ValueError(f"{name}: expected fp32 {tuple(shape[:3])} on cuda:{device}")
    ss = k_scale.stride()
    if v_scale.stride() != ss:
        raise ValueError("v_scale: expected the strides of k_scale")
    return qvla_kv_cache(*shape, 8, k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2],
                         k_scale.data_ptr(), v_scale.data_ptr(), ss[0], ss[1], ss[2])


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def qvla_qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                      v: Optional[torch.Tensor] = None, q_norm: Optional[torch.Tensor] = None,
                      k_norm: Optional[torch.Tensor] = None,
                      rope_table: Optional[torch.Tensor] = None,
                      positions: Optional[torch.Tensor] = None,
                      slots: Optional[torch.Tensor] = None,
                      k_cache: Optional[torch.Tensor] = None,
                      v_cache: Optional[torch.Tensor] = None, k_scale=None, v_scale=None,
                      eps: float = 1e-6, interleaved: bool = False,
                      q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                      stream=None):
    """RMS norm of the heads of q [T, Hq, D] and k [T, Hkv, D], position
    rotation by rope_table (qvla_rope_table()) at `positions`, and k and v
    written to the cache slots `slots` (negative: not written).  Returns
    q_out; without a cache (q_out, k_out).  q_out / k_out may be q / k."""
    one = q if q is not None else k
    if one is None or one.dim() != 3:
        raise ValueError("q, k: expected [T, heads, D] rows, at least one of them")
    T, _, D = one.shape
    dt, dev = one.dtype, one.get_device()
    Hq = Hkv = ldq = ldk = ldv = ldqo = ldko = P = rot = 0
    if q is not None:
        shape = q.shape
        ldq, Hq = _head_rows(q, shape, dev, dt, "q"), shape[1]
        if q_out is None:
            q_out = _empty(shape, dt, q.device, stream, q)
        ldqo = _head_rows(q_out, shape, dev, dt, "q_out")
    if k is not None:
        if k.dim() != 3:
            raise ValueError(f"k: expected [{T}, heads, {D}], got {tuple(k.shape)}")
        shape = (T, k.shape[1], D)
        ldk, Hkv = _head_rows(k, shape, dev, dt, "k"), shape[1]
        if k_out is None and k_cache is None:
            k_out = _empty(shape, dt, k.device, stream, k)
        if k_out is not None:
            ldko = _head_rows(k_out, shape, dev, dt, "k_out")
    if q_norm is not None:
        _expect_on(q_norm, torch.float32, (D,), dev, "q_norm")
    if k_norm is not None:
        _expect_on(k_norm, torch.float32, (D,), dev, "k_norm")
    if rope_table is not None:
        if positions is None or rope_table.dim() != 2:
            raise ValueError("rope_table: expected [positions, rot], and the tokens' positions")
        P, rot = rope_table.shape
        _expect_int32("rope_table", P)
        _expect_on(rope_table, torch.float32, (P, rot), dev, "rope_table")
        _expect_on(positions, torch.int32, (T,), dev, "positions")
    cache = None
    if k_cache is not None:
        if k is None or v is None or slots is None or v_cache is None:
            raise ValueError("a cache needs k, v, slots and v_cache")
        ldv = _head_rows(v, (T, Hkv, D), dev, dt, "v")
        _expect_on(slots, torch.int32, (T,), dev, "slots")
        cache = _kv_struct(k_cache, v_cache, k_scale, v_scale, dev)
    _launch(_lib.qvla_qk_norm_rope, "qvla_qk_norm_rope", dev, stream, _address(q), _address(k),
            _address(v), _dtype_code(one), T, Hq, Hkv, D, ldq, ldk, ldv, _address(q_norm),
            _address(k_norm), eps, _address(rope_table), P, rot, int(interleaved),
            _address(positions), cache, _address(slots), _address(q_out), ldqo, _address(k_out),
            ldko)
    return q_out if cache is not None else (q_out, k_out)


@functools.lru_cache(maxsize=256)
def qvla_paged_attn_workspace_bytes(Hq: int, heads: int, dim: int) -> int:
    b = c_size_t()
    _check(_lib.qvla_paged_attn_workspace_bytes(Hq, heads, dim, ctypes.byref(b)),
           "qvla_paged_attn_workspace_bytes")
    return b.value


def qvla_paged_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           page_table: torch.Tensor, seq_lens: torch.Tensor,
                           scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                           k_scale=None, v_scale=None, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence, q [B, Hq, D], over the paged
    cache; scale defaults to D ** -0.5.  lse: optional fp32 [B, Hq] output.
    workspace: uint8 device scratch of qvla_paged_attn_workspace_bytes()
    (allocated per call when None)."""
    if q.dim() != 3:
        raise ValueError(f"q: expected [B, heads, D], got {tuple(q.shape)}")
    shape, dt, dev = q.shape, q.dtype, q.get_device()
    B, Hq, D = shape
    ldq = _head_rows(q, shape, dev, dt, "q")
    cache = _kv_struct(k_cache, v_cache, k_scale, v_scale, dev)
    if cache.dim != D:
        raise ValueError(f"k_cache: expected dim {D}, got {cache.dim}")
    _expect_on(seq_lens, torch.int32, (B,), dev, "seq_lens")
    max_pages = page_table.shape[-1]
    _expect_int32("window, sinks, max_pages", window | sinks | max_pages)
    _expect_on(page_table, torch.int32, (B, max_pages), dev, "page_table")
    if out is None:
        out = _empty(shape, dt, q.device, stream, q)
    ldo = _head_rows(out, shape, dev, dt, "out")
    if lse is not None:
        _expect_on(lse, torch.float32, (B, Hq), dev, "lse")
    if workspace is None:
        ws_bytes = qvla_paged_attn_workspace_bytes(Hq, cache.heads, D)
        workspace = _empty(ws_bytes, torch.uint8, q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on cuda:{dev}")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _launch(_lib.qvla_paged_attn_decode, "qvla_paged_attn_decode", dev, stream, q.data_ptr(),
            _dtype_code(q), B, Hq, ldq, cache, page_table.data_ptr(), max_pages,
            seq_lens.data_ptr(), D ** -0.5 if scale is None else scale, window, sinks,
            out.data_ptr(), ldo, _address(lse), workspace.data_ptr(), ws_bytes)
    return out
