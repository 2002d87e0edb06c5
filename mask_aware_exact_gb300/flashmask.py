"""Thin ctypes binding over libflashmask.so (include/flashmask.h).

Argument marshalling only: each function checks dtypes, devices and
contiguity of the torch tensors it is given, passes their device pointers and
the current CUDA stream to the C entry point of the same name, and raises on a
non-OK status. Every step of the computation runs in the library's kernels;
there is no fallback path. If the library is missing the import of the
binding still works but the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflashmask.so")

FM_OK, FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA, FM_ERR_TIMEOUT, FM_ERR_WORKSPACE = range(6)
FM_ERR_PAGE = 6
FM_TILE = 128
FM_PAGE = 64
FM_BF16, FM_F16, FM_F32 = range(3)
FM_TILE_NONE, FM_TILE_PARTIAL, FM_TILE_FULL = 0, 1, 2


class _FmMask(ctypes.Structure):
    _fields_ = [("lts", ctypes.c_void_p), ("lte", ctypes.c_void_p), ("uts", ctypes.c_void_p),
                ("ute", ctypes.c_void_p), ("Hm", ctypes.c_int), ("causal", ctypes.c_int)]


class FmWsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("status", "minmax", "labels", "labels_t", "row_count", "row_list", "row_order",
                 "col_count", "col_list", "col_order", "lse2", "delta", "dq_accum", "kv_part",
                 "kv_sync", "total")]


class FmFp8Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("fwd_total", "q8", "k8", "vt8", "qscale", "kscale", "vscale", "total")]


class _FmHeads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("H", ctypes.c_int),
                ("xs", ctypes.c_int64 * 3), ("ys", ctypes.c_int64 * 3)]


class _FmCache(ctypes.Structure):
    _fields_ = [("k8", ctypes.c_void_p), ("v8", ctypes.c_void_p), ("kscale", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("pages", ctypes.c_int), ("Hk", ctypes.c_int),
                ("d", ctypes.c_int)]


EXPORTED = ("flashmask_workspace_bytes", "flashmask_workspace_layout", "flashmask_classify",
            "flashmask_fwd", "flashmask_bwd", "flashmask_bwd_preprocess", "flashmask_bwd_main",
            "flashmask_bwd_finalize", "flashmask_fwd_noalloc", "flashmask_host_workspace_bytes",
            "flashmask_fwd_bwd_host", "flashmask_localize", "flashmask_selftest_timeout",
            "flashmask_fwd_fp8_workspace_bytes", "flashmask_fwd_fp8_layout", "flashmask_fwd_fp8",
            "flashmask_check_status", "flashmask_status_string", "flashmask_rope",
            "flashmask_cache_workspace_bytes", "flashmask_cache_append", "flashmask_fwd_cache")

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads the library (once) and declares the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with mask_aware_exact_gb300.build.build()")
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.flashmask_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.flashmask_workspace_bytes.restype = sz
    L.flashmask_workspace_layout.argtypes = [i, i, i, i, i, i, ctypes.POINTER(FmWsLayout)]
    L.flashmask_workspace_layout.restype = i
    L.flashmask_classify.argtypes = [ctypes.POINTER(_FmMask), i, i, vp, sz, vp]
    L.flashmask_classify.restype = i
    L.flashmask_fwd.argtypes = [vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp, vp, vp, sz,
                                i, vp]
    L.flashmask_fwd.restype = i
    L.flashmask_bwd.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp,
                                vp, vp, vp, sz, i, vp]
    L.flashmask_bwd.restype = i
    L.flashmask_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, i, vp, sz, vp]
    L.flashmask_bwd_preprocess.restype = i
    L.flashmask_bwd_main.argtypes = [vp, vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp, vp,
                                     vp, sz, vp]
    L.flashmask_bwd_main.restype = i
    L.flashmask_bwd_finalize.argtypes = [i, i, i, i, i, f, vp, vp, sz, vp]
    L.flashmask_bwd_finalize.restype = i
    L.flashmask_fwd_noalloc.argtypes = [vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp, vp,
                                        vp]
    L.flashmask_fwd_noalloc.restype = i
    L.flashmask_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    L.flashmask_fwd_fp8_workspace_bytes.restype = sz
    L.flashmask_fwd_fp8_layout.argtypes = [i, i, i, i, ctypes.POINTER(FmFp8Layout)]
    L.flashmask_fwd_fp8_layout.restype = i
    L.flashmask_fwd_fp8.argtypes = [vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp, vp, vp,
                                    sz, i, vp]
    L.flashmask_fwd_fp8.restype = i
    L.flashmask_host_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.flashmask_host_workspace_bytes.restype = sz
    L.flashmask_fwd_bwd_host.argtypes = [vp, vp, vp, vp, ctypes.POINTER(_FmMask), i, i, i, i, f, vp,
                                         vp, vp, vp, vp, vp, sz, i, vp]
    L.flashmask_fwd_bwd_host.restype = i
    L.flashmask_localize.argtypes = [ctypes.POINTER(_FmMask), i, i, i, i, vp, vp, vp, vp, vp, vp]
    L.flashmask_localize.restype = i
    L.flashmask_selftest_timeout.argtypes = [vp, sz, ctypes.c_longlong, i, vp]
    L.flashmask_selftest_timeout.restype = i
    L.flashmask_check_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
    L.flashmask_check_status.restype = i
    L.flashmask_status_string.argtypes = [i]
    L.flashmask_status_string.restype = ctypes.c_char_p
    L.flashmask_rope.argtypes = [vp, i, vp, ctypes.c_int64, vp, i, i, i, i, i, i, f, i, vp]
    L.flashmask_rope.restype = i
    L.flashmask_cache_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.flashmask_cache_workspace_bytes.restype = sz
    L.flashmask_cache_append.argtypes = [ctypes.POINTER(_FmCache), vp, i, vp, vp, vp, vp, vp, vp,
                                         i, i, vp, sz, vp]
    L.flashmask_cache_append.restype = i
    L.flashmask_fwd_cache.argtypes = [vp, vp, ctypes.POINTER(_FmCache), vp, i, vp, vp,
                                      ctypes.POINTER(_FmMask), i, i, i, f, vp, vp, vp, vp, sz, vp]
    L.flashmask_fwd_cache.restype = i
    _lib = L
    return L


class FlashMaskError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = load().flashmask_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status != FM_OK:
        raise FlashMaskError(status, where)


def _stream_ptr(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


@dataclass
class DeviceMask:
    """Boundary vectors on the device (int32 [B, Hm, N]) plus Hm and the causal flag."""

    lts: torch.Tensor
    lte: torch.Tensor
    uts: torch.Tensor | None
    ute: torch.Tensor | None
    causal: bool

    @property
    def Hm(self) -> int:
        return self.lts.shape[1]

    @staticmethod
    def from_spec(spec, device="cuda") -> "DeviceMask":
        t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(device)
        return DeviceMask(t(spec.lts), t(spec.lte), t(spec.uts), t(spec.ute), bool(spec.causal))

    def c_struct(self) -> _FmMask:
        for v in (self.lts, self.lte, self.uts, self.ute):
            if v is not None:
                if v.dtype != torch.int32 or not v.is_cuda or not v.is_contiguous():
                    raise ValueError("mask vectors must be contiguous int32 CUDA tensors")
        p = lambda v: None if v is None else v.data_ptr()
        return _FmMask(p(self.lts), p(self.lte), p(self.uts), p(self.ute), self.Hm, int(self.causal))


def _bf16(x: torch.Tensor, name: str):
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 4:
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, H, N, d]")


def flashmask_workspace_bytes(B, H, Hm, N, d, for_bwd=True) -> int:
    return int(load().flashmask_workspace_bytes(B, H, Hm, N, d, int(bool(for_bwd))))


def flashmask_workspace_layout(B, H, Hm, N, d, for_bwd=True) -> FmWsLayout:
    out = FmWsLayout()
    _check(load().flashmask_workspace_layout(B, H, Hm, N, d, int(bool(for_bwd)), ctypes.byref(out)),
           "flashmask_workspace_layout")
    return out


def alloc_workspace(B, H, Hm, N, d, for_bwd=True, device="cuda") -> torch.Tensor:
    n = flashmask_workspace_bytes(B, H, Hm, N, d, for_bwd)
    if n == 0:
        raise FlashMaskError(FM_ERR_UNSUPPORTED, "flashmask_workspace_bytes")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def flashmask_classify(mask: DeviceMask, B: int, N: int, ws: torch.Tensor, stream=None):
    m = mask.c_struct()
    _check(load().flashmask_classify(ctypes.byref(m), B, N, ws.data_ptr(), ws.numel(),
                                     _stream_ptr(stream)), "flashmask_classify")


def flashmask_fwd(q, k, v, mask: DeviceMask, ws, scale=None, o=None, lse=None, ws_classified=False,
                  stream=None):
    """Returns (O bf16 [B,H,N,d], LSE fp32 [B,H,N])."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _bf16(t, n)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    m = mask.c_struct()
    _check(load().flashmask_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(m), B, H, N,
                                d, scale, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                int(bool(ws_classified)), _stream_ptr(stream)), "flashmask_fwd")
    return o, lse


def flashmask_fwd_fp8_workspace_bytes(B, H, Hm, N) -> int:
    return load().flashmask_fwd_fp8_workspace_bytes(B, H, Hm, N)


def flashmask_fwd_fp8_layout(B, H, Hm, N) -> FmFp8Layout:
    out = FmFp8Layout()
    _check(load().flashmask_fwd_fp8_layout(B, H, Hm, N, ctypes.byref(out)),
           "flashmask_fwd_fp8_layout")
    return out


def read_fp8_operands(ws, B, H, Hm, N):
    """The e4m3 operands and scales the last FP8 forward left in `ws`, as torch
    tensors on its device: q8, k8 uint8 [B,H,N,128], vt8 uint8 [B,H,128,Npad],
    qscale, kscale fp32 [B,H,Tr], vscale fp32 [B,H]."""
    L = flashmask_fwd_fp8_layout(B, H, Hm, N)
    Tr = (N + 127) // 128
    Npad = 128 * Tr

    def part(off, n):
        return ws[off:off + n]
    q8 = part(L.q8, B * H * N * 128).view(B, H, N, 128)
    k8 = part(L.k8, B * H * N * 128).view(B, H, N, 128)
    vt8 = part(L.vt8, B * H * 128 * Npad).view(B, H, 128, Npad)
    qs = part(L.qscale, B * H * Tr * 4).view(torch.float32).view(B, H, Tr)
    ks = part(L.kscale, B * H * Tr * 4).view(torch.float32).view(B, H, Tr)
    vs = part(L.vscale, B * H * 4).view(torch.float32).view(B, H)
    return q8, k8, vt8, qs, ks, vs


def alloc_fp8_workspace(B, H, Hm, N, device="cuda") -> torch.Tensor:
    n = flashmask_fwd_fp8_workspace_bytes(B, H, Hm, N)
    if n == 0:
        raise FlashMaskError(FM_ERR_UNSUPPORTED, "flashmask_fwd_fp8_workspace_bytes")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def flashmask_fwd_fp8(q, k, v, mask: DeviceMask, ws, scale=None, o=None, lse=None,
                      ws_classified=False, stream=None):
    """FP8 (e4m3) forward of bf16 Q, K, V with d = 128; returns (O bf16, LSE fp32)
    like flashmask_fwd. `ws` comes from alloc_fp8_workspace."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _bf16(t, n)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    m = mask.c_struct()
    _check(load().flashmask_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(m), B, H,
                                    N, d, scale, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                    ws.numel(), int(bool(ws_classified)), _stream_ptr(stream)),
           "flashmask_fwd_fp8")
    return o, lse


def flashmask_bwd(q, k, v, o, lse, do, mask: DeviceMask, ws, scale=None, dq=None, dk=None, dv=None,
                  ws_classified=False, stream=None):
    """Returns (dQ, dK, dV) bf16 [B,H,N,d]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _bf16(t, n)
    if lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    m = mask.c_struct()
    _check(load().flashmask_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                lse.data_ptr(), do.data_ptr(), ctypes.byref(m), B, H, N, d, scale,
                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(),
                                ws.numel(), int(bool(ws_classified)), _stream_ptr(stream)),
           "flashmask_bwd")
    return dq, dk, dv


def flashmask_bwd_preprocess(o, lse, do, Hm: int, ws, stream=None):
    _bf16(o, "o")
    _bf16(do, "do")
    B, H, N, d = o.shape
    _check(load().flashmask_bwd_preprocess(o.data_ptr(), lse.data_ptr(), do.data_ptr(), B, H, Hm, N,
                                           d, ws.data_ptr(), ws.numel(), _stream_ptr(stream)),
           "flashmask_bwd_preprocess")


def flashmask_bwd_main(q, k, v, do, mask: DeviceMask, ws, dk, dv, scale=None, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (do, "do"), (dk, "dk"), (dv, "dv")):
        _bf16(t, n)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    m = mask.c_struct()
    _check(load().flashmask_bwd_main(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                                     ctypes.byref(m), B, H, N, d, scale, dk.data_ptr(),
                                     dv.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _stream_ptr(stream)), "flashmask_bwd_main")


def flashmask_bwd_finalize(dq, Hm: int, ws, scale=None, stream=None):
    _bf16(dq, "dq")
    B, H, N, d = dq.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    _check(load().flashmask_bwd_finalize(B, H, Hm, N, d, scale, dq.data_ptr(), ws.data_ptr(),
                                         ws.numel(), _stream_ptr(stream)), "flashmask_bwd_finalize")


def flashmask_check_status(ws: torch.Tensor, stream=None) -> tuple[int, int]:
    """(status, failure site) after synchronising the stream; clears the word."""
    detail = ctypes.c_int(0)
    st = load().flashmask_check_status(ws.data_ptr(), _stream_ptr(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def flashmask_status_string(status: int) -> str:
    return load().flashmask_status_string(status).decode()


def read_classification(ws: torch.Tensor, B: int, Hm: int, N: int) -> dict:
    """Copies the classification regions of a workspace to host numpy arrays."""
    L = flashmask_workspace_layout(B, Hm, Hm, N, 64, False)
    Tr = Tc = (N + FM_TILE - 1) // FM_TILE
    h = ws[:L.total].cpu().numpy()

    def region(off, count, dtype, shape):
        return h[off:off + count * np.dtype(dtype).itemsize].view(dtype).reshape(shape).copy()

    return {
        "minmax": region(L.minmax, B * Hm * Tc * 8, np.int32, (B, Hm, Tc, 8)),
        "labels": region(L.labels, B * Hm * Tr * Tc, np.uint8, (B, Hm, Tr, Tc)),
        "labels_t": region(L.labels_t, B * Hm * Tc * Tr, np.uint8, (B, Hm, Tc, Tr)),
        "row_count": region(L.row_count, B * Hm * Tr, np.int32, (B, Hm, Tr)),
        "row_list": region(L.row_list, B * Hm * Tr * Tc, np.int32, (B, Hm, Tr, Tc)),
        "row_order": region(L.row_order, B * Hm * Tr, np.int32, (B, Hm, Tr)),
        "col_count": region(L.col_count, B * Hm * Tc, np.int32, (B, Hm, Tc)),
        "col_list": region(L.col_list, B * Hm * Tc * Tr, np.int32, (B, Hm, Tc, Tr)),
        "col_order": region(L.col_order, B * Hm * Tc, np.int32, (B, Hm, Tc)),
    }


def flashmask_fwd_noalloc(q, k, v, mask: DeviceMask, o, lse, scale=None, stream=None):
    """Forward into caller-provided O and LSE with no workspace and no allocation.

    The tables live in the library's fixed scratch array, so calls that may
    overlap on the GPU must be serialised by the caller, and the first call on
    a device must come before any stream capture. Shapes whose tables do not fit
    raise FlashMaskError with FM_ERR_WORKSPACE."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _bf16(t, n)
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    m = mask.c_struct()
    _check(load().flashmask_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(m),
                                        B, H, N, d, scale, o.data_ptr(), lse.data_ptr(),
                                        _stream_ptr(stream)), "flashmask_fwd_noalloc")
    return o, lse


# ---------------------------------------------------------------- host buffers
@dataclass
class HostMask:
    """Boundary vectors in host memory (contiguous int32 [B, Hm, N] CPU tensors,
    page-locked when made by from_spec) plus the causal flag."""

    lts: torch.Tensor
    lte: torch.Tensor
    uts: torch.Tensor | None
    ute: torch.Tensor | None
    causal: bool

    @property
    def Hm(self) -> int:
        return self.lts.shape[1]

    @staticmethod
    def from_spec(spec, pin=True) -> "HostMask":
        def t(a):
            if a is None:
                return None
            x = torch.from_numpy(np.ascontiguousarray(a, np.int32))
            return x.pin_memory() if pin else x
        return HostMask(t(spec.lts), t(spec.lte), t(spec.uts), t(spec.ute), bool(spec.causal))

    def c_struct(self) -> _FmMask:
        for v in (self.lts, self.lte, self.uts, self.ute):
            if v is not None:
                if v.dtype != torch.int32 or v.is_cuda or not v.is_contiguous():
                    raise ValueError("host mask vectors must be contiguous int32 CPU tensors")
        p = lambda v: None if v is None else v.data_ptr()
        return _FmMask(p(self.lts), p(self.lte), p(self.uts), p(self.ute), self.Hm, int(self.causal))


def flashmask_host_workspace_bytes(B, H, Hm, N, d, chunk_heads) -> int:
    return int(load().flashmask_host_workspace_bytes(B, H, Hm, N, d, chunk_heads))


def alloc_host_workspace(B, H, Hm, N, d, chunk_heads, device="cuda") -> torch.Tensor:
    n = flashmask_host_workspace_bytes(B, H, Hm, N, d, chunk_heads)
    if n == 0:
        raise FlashMaskError(FM_ERR_UNSUPPORTED, "flashmask_host_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def flashmask_fwd_bwd_host(q, k, v, do, mask: HostMask, dev_ws, chunk_heads, scale=None,
                           out=None, stream=None):
    """Forward and backward between host tensors (bf16 [B,H,N,d], page-locked for
    the copies to overlap). Returns (O, LSE, dQ, dK, dV) on the host; `out` may
    hold preallocated host tensors in that order. Blocks until the results are
    in host memory."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (do, "do")):
        if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous bf16 CPU tensor")
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        pin = q.is_pinned()
        mk = lambda shape, dt: torch.empty(shape, dtype=dt, pin_memory=pin)
        out = (mk(q.shape, torch.bfloat16), mk((B, H, N), torch.float32), mk(q.shape, torch.bfloat16),
               mk(q.shape, torch.bfloat16), mk(q.shape, torch.bfloat16))
    o, lse, dq, dk, dv = out
    m = mask.c_struct()
    _check(load().flashmask_fwd_bwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                                         ctypes.byref(m), B, H, N, d, scale, o.data_ptr(),
                                         lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                         dev_ws.data_ptr(), dev_ws.numel(), int(chunk_heads),
                                         _stream_ptr(stream)), "flashmask_fwd_bwd_host")
    return o, lse, dq, dk, dv


def flashmask_localize(mask: DeviceMask, B: int, N: int, row0: int, rows: int, stream=None):
    """Boundary vectors of the local problem of a rank holding query rows
    [row0, row0 + rows): returns (DeviceMask with causal=False, inexact flag as
    a bool). Synchronises the stream to read the flag."""
    dev = mask.lts.device
    shape = (B, mask.Hm, N)
    out = [torch.empty(shape, dtype=torch.int32, device=dev) for _ in range(4)]
    flag = torch.zeros(1, dtype=torch.int32, device=dev)
    m = mask.c_struct()
    _check(load().flashmask_localize(ctypes.byref(m), B, N, int(row0), int(rows), out[0].data_ptr(),
                                     out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                                     flag.data_ptr(), _stream_ptr(stream)), "flashmask_localize")
    return DeviceMask(out[0], out[1], out[2], out[3], False), bool(flag.item())


def flashmask_selftest_timeout(ws: torch.Tensor, limit_ns: int, ctas: int = 1, stream=None):
    """Queues the bounded-wait self-test (see include/flashmask.h)."""
    _check(load().flashmask_selftest_timeout(ws.data_ptr(), ws.numel(), int(limit_ns), int(ctas),
                                             _stream_ptr(stream)), "flashmask_selftest_timeout")


# ---------------------------------------------------------------- rotary positions
_ROPE_DTYPES = {torch.bfloat16: FM_BF16, torch.float16: FM_F16, torch.float32: FM_F32}
_STRIDES = struct.Struct("@3q")
_HEADS = struct.Struct("@PPi6q")  # an _FmHeads: x, y, H, strides of x and y
assert _HEADS.size == ctypes.sizeof(_FmHeads)


def _launch(index, stream, tensors, call):
    """call(raw stream) on device `index`: on `stream`, or on that device's current
    one. With a stream of its own the call's outputs are allocated for that stream
    and its inputs are kept until it has passed the call."""
    if stream is None:
        if index == torch._C._cuda_getDevice():
            return call(torch._C._cuda_getCurrentRawStream(index))
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index))
    if stream.device.index != index:
        raise ValueError("stream and tensors must be on the same device")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _want(t, name, dtype, index, shape):
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{index}")


def _rows(t, name, dtype, index):
    """Strides of a [B, H, N, d] tensor with any but a contiguous last dimension's."""
    st = t.stride()
    if t.dtype is not dtype or t.get_device() != index or index < 0 or len(st) != 4 or \
            (st[3] != 1 and t.shape[3] != 1):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [B, H, N, d] with a contiguous last "
                         f"dimension, on the same device as the others")
    return st


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original: int = 8192, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Frequencies (fp64 [rot_dim / 2], radians per position) and the factor on the
    rotated values for flashmask_rope. Pair i turns by base^(-2 i / rot_dim) a
    position. scaling: "none"; "linear" divides every frequency by `factor`;
    "parts" keeps pairs that turn at least `fast` times within `original`
    positions, divides those that turn at most `slow` times by `factor`, mixes
    the two linearly between, and multiplies the rotated values by
    0.1 ln(factor) + 1."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and not negative")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    f = base ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / max(rot_dim, 1))
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        keep = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling != "none":
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.from_numpy(f).to(device), mscale


def _rope(q, k, freqs, positions, interleaved, mscale, out, stream, inverse, where):
    dtype = q.dtype
    code = _ROPE_DTYPES.get(dtype)
    if code is None:
        raise ValueError("q must be bf16, fp16 or fp32")
    index = q.get_device()
    sq, sk = _rows(q, "q", dtype, index), None
    B, Hq, N, d = q.shape
    if k is not None:
        sk = _rows(k, "k", dtype, index)
        Bk, Hk, Nk, dk = k.shape
        if Bk != B or Nk != N or dk != d:
            raise ValueError("q and k must share B, N and d")
    n = freqs.numel()
    _want(freqs, "freqs", torch.float64, index, (n,))
    if 2 * n > d:
        raise ValueError("freqs must be [rot_dim / 2] with rot_dim <= d")
    pos, pos_stride = None, 0
    if positions is not None:
        sp, tp = positions.shape, positions.stride()
        if positions.dtype is not torch.int32 or positions.get_device() != index or \
                len(sp) != 2 or sp[1] != N or (sp[0] != 1 and sp[0] != B) or (N > 1 and tp[1] != 1):
            raise ValueError(f"positions must be int32 [{B}, {N}] or [1, {N}] on cuda:{index}, rows "
                             "contiguous")
        pos = positions.data_ptr()
        pos_stride = tp[0] if sp[0] > 1 else 0
    yq = yk = tq = tk = None
    if out is not None:
        yq, yk = out[0], (out[1] if k is not None else None)
        tq = _rows(yq, "out", dtype, index)
        if yk is not None:
            tk = _rows(yk, "out", dtype, index)
        if yq.shape != q.shape or (k is not None and yk.shape != k.shape):
            raise ValueError("out must have the shapes of q and k")

    def call(raw):
        oq, ok, uq, uk = yq, yk, tq, tk
        if oq is None:
            device = q.device
            oq, uq = torch.empty((B, Hq, N, d), dtype=dtype, device=device), (Hq * N * d, N * d, d)
            if k is not None:
                ok, uk = torch.empty((B, Hk, N, d), dtype=dtype, device=device), (Hk * N * d, N * d, d)
        if B * N * d > 0:
            heads = _HEADS.pack(q.data_ptr(), oq.data_ptr(), Hq, *sq[:3], *uq[:3])
            if k is not None:
                heads += _HEADS.pack(k.data_ptr(), ok.data_ptr(), Hk, *sk[:3], *uk[:3])
            st = _lib.flashmask_rope(heads, 1 if k is None else 2, pos, pos_stride, freqs.data_ptr(), B, N,
                                     d, 2 * n, bool(interleaved), code, mscale, inverse, raw)
            if st:
                raise FlashMaskError(st, where)
        return oq, ok

    if _lib is None:
        load()
    return _launch(index, stream, () if stream is None else (q, k, freqs, positions, yq, yk), call)


def flashmask_rope(q, k, freqs, positions=None, interleaved=False, mscale=1.0, out=None,
                   stream=None):
    """Q and K [B, H, N, d] (bf16, fp16 or fp32; any strides with a contiguous last
    dimension; k may be None) with the first 2 * len(freqs) elements of every
    head rotated by their token's position; returns (Q', K'). freqs and mscale
    as rope_frequencies gives them. positions: int32 [B, N] or [1, N] (None:
    token n sits at n). out: a pair to write into, (q, k) itself to rotate in
    place."""
    return _rope(q, k, freqs, positions, interleaved, mscale, out, stream, 0, "flashmask_rope")


def flashmask_rope_bwd(dq, dk, freqs, positions=None, interleaved=False, mscale=1.0, out=None,
                       stream=None):
    """Gradients of flashmask_rope's inputs from those of its outputs, same arguments."""
    return _rope(dq, dk, freqs, positions, interleaved, mscale, out, stream, 1,
                 "flashmask_rope_bwd")


# ---------------------------------------------------------------- 8-bit paged cache
@dataclass(frozen=True)
class KVCache:
    """Keys and values as e4m3 codes in pages of FM_PAGE tokens with one scale per
    page and head: k8 [pages, Hk, 64, d], v8 [pages, Hk, d, 64] (float8_e4m3fn,
    V transposed, no NaN codes in it), kscale, vscale fp32 [pages, Hk] (finite, not
    negative). Its tensors are checked at its first use, and again if one of them has
    changed its place, shape, layout or type since (set_, resize_, .data)."""

    k8: torch.Tensor
    v8: torch.Tensor
    kscale: torch.Tensor
    vscale: torch.Tensor

    @staticmethod
    def empty(pages: int, Hk: int, d: int, device="cuda") -> "KVCache":
        f8 = dict(dtype=torch.float8_e4m3fn, device=device)
        return KVCache(torch.zeros((pages, Hk, FM_PAGE, d), **f8),
                       torch.zeros((pages, Hk, d, FM_PAGE), **f8),
                       torch.ones((pages, Hk), device=device), torch.ones((pages, Hk), device=device))

    @property
    def tensors(self):
        return self.k8, self.v8, self.kscale, self.vscale

    @property
    def _handle(self):
        """(C struct, Hk, d, device index)"""
        k8, v8, ks, vs = self.k8, self.v8, self.kscale, self.vscale
        at = (k8.data_ptr(), v8.data_ptr(), ks.data_ptr(), vs.data_ptr(), k8.shape, v8.shape, ks.shape,
              vs.shape, k8.is_contiguous(), v8.is_contiguous(), ks.is_contiguous(), vs.is_contiguous(),
              k8.dtype, v8.dtype, ks.dtype, vs.dtype)
        made = self.__dict__.get("_made")
        if made is None or made[0] != at:
            made = at, self._check()
            object.__setattr__(self, "_made", made)
        return made[1]

    def _check(self):
        k8 = self.k8
        index = k8.get_device()
        if k8.dim() != 4 or k8.shape[2] != FM_PAGE or index < 0:
            raise ValueError("k8 must be a CUDA tensor [pages, Hk, 64, d]")
        pages, Hk, _, d = k8.shape
        _want(k8, "k8", torch.float8_e4m3fn, index, k8.shape)
        _want(self.v8, "v8", torch.float8_e4m3fn, index, (pages, Hk, d, FM_PAGE))
        _want(self.kscale, "kscale", torch.float32, index, (pages, Hk))
        _want(self.vscale, "vscale", torch.float32, index, (pages, Hk))
        return _FmCache(k8.data_ptr(), self.v8.data_ptr(), self.kscale.data_ptr(),
                        self.vscale.data_ptr(), pages, Hk, d), Hk, d, index

    def c_struct(self) -> _FmCache:
        return self._handle[0]


def flashmask_cache_workspace_bytes(B, H, Hk, N, d, max_pages) -> int:
    return int(load().flashmask_cache_workspace_bytes(B, H, Hk, N, d, max_pages))


def alloc_cache_workspace(B, H, Hk, N, d, max_pages, device="cuda") -> torch.Tensor:
    """Zeroed workspace of flashmask_cache_append and flashmask_fwd_cache."""
    n = flashmask_cache_workspace_bytes(B, H, Hk, N, d, max_pages)
    if n == 0:
        raise FlashMaskError(FM_ERR_UNSUPPORTED, "flashmask_cache_workspace_bytes")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def _per_sequence(t, name, B, index):
    if t is None:
        return None
    _want(t, name, torch.int32, index, (B,))
    return t.data_ptr()


def _page_table(t, B, index):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("page_table must be int32 [B, max_pages]")
    _want(t, "page_table", torch.int32, index, (B, shape[1]))
    return shape[1]


def flashmask_cache_append(cache: KVCache, page_table, k, v, start, ws, count=None, stream=None):
    """Writes K and V (bf16 [B, Hk, N, d], last dimension contiguous) behind the
    start[b] tokens that sequence b holds; count[b] <= N of its rows are real.
    page_table int32 [B, max_pages]; start, count int32 [B]. See
    include/flashmask.h for scales and rounding."""
    c, Hk, d, index = cache._handle
    ks, vs = _rows(k, "k", torch.bfloat16, index), _rows(v, "v", torch.bfloat16, index)
    shape = k.shape
    B, heads, N, width = shape
    if v.shape != shape or heads != Hk or width != d:
        raise ValueError("k and v must be [B, Hk, N, d] with the cache's Hk and d")
    max_pages = _page_table(page_table, B, index)
    st, ct = _per_sequence(start, "start", B, index), _per_sequence(count, "count", B, index)
    ws_bytes = ws.numel()
    _want(ws, "ws", torch.uint8, index, (ws_bytes,))

    def call(raw):
        code = load().flashmask_cache_append(c, page_table.data_ptr(), max_pages, k.data_ptr(),
                                             _STRIDES.pack(*ks[:3]), v.data_ptr(),
                                             _STRIDES.pack(*vs[:3]), st, ct, B, N, ws.data_ptr(),
                                             ws_bytes, raw)
        if code:
            raise FlashMaskError(code, "flashmask_cache_append")

    _launch(index, stream, () if stream is None else (*cache.tensors, page_table, k, v, start, count, ws),
            call)


def flashmask_fwd_cache(q, cache: KVCache, page_table, lens, ws, mask: DeviceMask | None = None,
                        q_lens=None, scale=None, o=None, lse=None, stream=None):
    """Attention of the N query tokens of each sequence (q bf16 [B, H, N, d], last
    dimension contiguous) over its lens[b] cached tokens, the query tokens' own
    among them; q_lens[b] <= N of its rows are real. mask: causal when None,
    else a DeviceMask whose vectors are [B, Hm, 64 * max_pages] (lts and lte may
    be None). Returns (O bf16 like q, LSE fp32 [B, H, N]); rows behind q_lens[b]
    of `o` and `lse` are left as they were."""
    c, _, d, index = cache._handle
    qs = _rows(q, "q", torch.bfloat16, index)
    shape = q.shape
    B, H, N, width = shape
    if width != d:
        raise ValueError("q must have the cache's d")
    max_pages = _page_table(page_table, B, index)
    ln, ql = _per_sequence(lens, "lens", B, index), _per_sequence(q_lens, "q_lens", B, index)
    ws_bytes = ws.numel()
    _want(ws, "ws", torch.uint8, index, (ws_bytes,))
    vectors, m = (), None
    if mask is not None:
        vectors = (mask.lts, mask.lte, mask.uts, mask.ute)
        Hm, ptrs = 1, []
        for t in vectors:
            if t is not None:
                Hm = t.shape[1] if t.dim() == 3 else -1
        for t in vectors:
            if t is not None:
                _want(t, "mask vectors", torch.int32, index, (B, Hm, max_pages * FM_PAGE))
            ptrs.append(None if t is None else t.data_ptr())
        m = _FmMask(*ptrs, Hm, bool(mask.causal))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    os = (H * N * d, N * d, d)
    if o is not None:
        os = _rows(o, "o", torch.bfloat16, index)
        if o.shape != shape:
            raise ValueError("o must have q's shape")
    if lse is not None:
        _want(lse, "lse", torch.float32, index, (B, H, N))

    def call(raw):
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device) if o is None else o
        norm = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
        code = load().flashmask_fwd_cache(q.data_ptr(), _STRIDES.pack(*qs[:3]), c,
                                          page_table.data_ptr(), max_pages, ln, ql, m, B, H, N, scale,
                                          out.data_ptr(), _STRIDES.pack(*os[:3]), norm.data_ptr(),
                                          ws.data_ptr(), ws_bytes, raw)
        if code:
            raise FlashMaskError(code, "flashmask_fwd_cache")
        return out, norm

    return _launch(index, stream, () if stream is None else
                   (q, *cache.tensors, page_table, lens, q_lens, ws, o, lse, *vectors), call)
