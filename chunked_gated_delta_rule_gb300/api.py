"""ctypes binding of ``include/gdr.h``: argument marshalling only.

Every step of the forward and backward passes runs in the CUDA library; these
functions pass tensor pointers, sizes and the current CUDA stream across the
C ABI.  If the library has not been built (``__graft_entry__.build()``),
every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional

import torch

from . import build as _build

GDR_F32, GDR_BF16, GDR_F16, GDR_E4M3, GDR_I8 = 0, 1, 2, 3, 4


class gdr_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("K", ctypes.c_int64), ("V", ctypes.c_int64), ("N", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("max_len", ctypes.c_int64),
                ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2),
                ("v_stride", ctypes.c_int64 * 2), ("o_stride", ctypes.c_int64 * 2)]


class gdr_plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("bv", ctypes.c_int32),
                ("n_segments", ctypes.c_int32), ("compose", ctypes.c_int32)]


class gdr_options(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("force_path", ctypes.c_int32),
                ("force_bv", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
                ("events", ctypes.c_void_p), ("max_launches", ctypes.c_int32),
                ("launch_ids", ctypes.c_void_p), ("n_launches", ctypes.c_void_p),
                ("grid_limit", ctypes.c_int32)]


class gdr_paged_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dtype", ctypes.c_int32),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3)]


# Diagnostic entry points declared in include/gdr_selftest.h.
SELFTEST_EXPORTS = ("gdr_selftest_umma", "gdr_selftest_tma", "gdr_selftest_inverse",
                    "gdr_selftest_timeout")

class gdr_conv_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("C", ctypes.c_int64),
                ("W", ctypes.c_int64), ("N", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("max_len", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]


class gdr_scan_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("C", ctypes.c_int64),
                ("S", ctypes.c_int64), ("G", ctypes.c_int64), ("N", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("softplus", ctypes.c_int32), ("max_len", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("z_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64 * 2), ("c_stride", ctypes.c_int64 * 2)]


class gdr_scan_tensors(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")]


class gdr_scan_grads(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz",
                                                     "ddt_bias", "dh0")]


class gdr_norm_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("group", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("sum_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]


# Every symbol include/gdr.h declares.
EXPORTS = ("gdr_chunk_fwd", "gdr_chunk_fwd_ex", "gdr_chunk_fwd_host", "gdr_chunk_fwd_noalloc",
           "gdr_workspace_size", "gdr_plan_query", "gdr_recurrent_fwd", "gdr_kernel_name", "gdr_error_string",
           "gdr_release_cached", "gdr_version", "gdr_chunk_bwd", "gdr_bwd_workspace_size",
           "gdr_cache_write", "gdr_cache_read", "gdr_paged_attn", "gdr_attn_workspace_size",
           "gdr_short_conv_fwd", "gdr_short_conv_bwd", "gdr_short_conv_bwd_workspace_size",
           "gdr_selective_scan_fwd", "gdr_selective_scan_bwd", "gdr_selective_scan_workspace_size",
           "gdr_selective_scan_bwd_workspace_size", "gdr_rms_norm_fwd", "gdr_rms_norm_bwd",
           "gdr_rms_norm_bwd_workspace_size")

_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def load_library():
    """Open ``libgdr.so``.  Raises if it has not been built: there is no
    fallback implementation."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is missing; build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        vp, i32p = ctypes.c_void_p, ctypes.c_void_p
        dims_p = ctypes.POINTER(gdr_dims)
        fwd_args = [dims_p, vp, vp, vp, vp, vp, i32p, vp, vp, vp, ctypes.c_int]
        lib.gdr_chunk_fwd.argtypes = fwd_args + [vp]
        lib.gdr_chunk_fwd.restype = ctypes.c_int
        lib.gdr_chunk_fwd_ex.argtypes = fwd_args + [ctypes.POINTER(gdr_options), vp]
        lib.gdr_chunk_fwd_ex.restype = ctypes.c_int
        lib.gdr_chunk_fwd_host.argtypes = fwd_args + [vp]
        lib.gdr_chunk_fwd_host.restype = ctypes.c_int
        lib.gdr_chunk_fwd_noalloc.argtypes = fwd_args + [vp]
        lib.gdr_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.gdr_recurrent_fwd.argtypes = [dims_p, vp, vp, vp, vp, vp, i32p, vp, ctypes.c_int64,
                                          i32p, vp, vp, vp]
        lib.gdr_recurrent_fwd.restype = ctypes.c_int
        lib.gdr_chunk_bwd.argtypes = [dims_p, vp, vp, vp, vp, vp, i32p, vp, vp, vp, vp, vp, vp,
                                      vp, vp, vp, ctypes.c_int, ctypes.POINTER(gdr_options), vp]
        lib.gdr_chunk_bwd.restype = ctypes.c_int
        lib.gdr_bwd_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
        lib.gdr_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdr_workspace_size.argtypes = [dims_p, ctypes.c_int, ctypes.c_int]
        lib.gdr_workspace_size.restype = ctypes.c_size_t
        lib.gdr_plan_query.argtypes = [dims_p, ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(gdr_plan)]
        lib.gdr_plan_query.restype = ctypes.c_int
        lib.gdr_kernel_name.argtypes = [ctypes.c_int]
        lib.gdr_kernel_name.restype = ctypes.c_char_p
        lib.gdr_error_string.argtypes = [ctypes.c_int]
        lib.gdr_error_string.restype = ctypes.c_char_p
        lib.gdr_selftest_umma.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, vp, vp]
        lib.gdr_selftest_umma.restype = ctypes.c_int
        lib.gdr_selftest_tma.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp]
        lib.gdr_selftest_tma.restype = ctypes.c_int
        lib.gdr_selftest_timeout.argtypes = [vp, ctypes.c_uint64, vp, vp]
        lib.gdr_selftest_timeout.restype = ctypes.c_int
        lib.gdr_selftest_inverse.argtypes = [vp, vp, vp]
        lib.gdr_selftest_inverse.restype = ctypes.c_int
        cache_p = ctypes.POINTER(gdr_paged_cache)
        for name in ("gdr_cache_write", "gdr_cache_read"):
            getattr(lib, name).argtypes = [dims_p, cache_p, vp, vp, i32p, vp, vp]
            getattr(lib, name).restype = ctypes.c_int
        lib.gdr_paged_attn.argtypes = [dims_p, cache_p, vp, i32p, vp, vp, ctypes.c_int,
                                       ctypes.c_int64, ctypes.POINTER(gdr_options), vp]
        lib.gdr_paged_attn.restype = ctypes.c_int
        lib.gdr_attn_workspace_size.argtypes = [dims_p, cache_p]
        lib.gdr_attn_workspace_size.restype = ctypes.c_size_t
        opt_p, i64 = ctypes.POINTER(gdr_options), ctypes.c_int64
        conv_p, norm_p = ctypes.POINTER(gdr_conv_dims), ctypes.POINTER(gdr_norm_dims)
        scan_p, in_p = ctypes.POINTER(gdr_scan_dims), ctypes.POINTER(gdr_scan_tensors)
        for name, args in (
                ("gdr_short_conv_fwd", [conv_p, vp, vp, vp, i32p, vp, vp, i64, i32p, vp]),
                ("gdr_short_conv_bwd", [conv_p, vp, vp, vp, i32p, vp, vp, vp, vp, vp, vp, vp]),
                ("gdr_selective_scan_fwd", [scan_p, in_p, i32p, vp, vp, i64, i32p, vp, ctypes.c_int]),
                ("gdr_selective_scan_bwd", [scan_p, in_p, i32p, vp, vp, vp,
                                            ctypes.POINTER(gdr_scan_grads)]),
                ("gdr_rms_norm_fwd", [norm_p, vp, vp, vp, vp, vp, vp]),
                ("gdr_rms_norm_bwd", [norm_p, vp, vp, vp, vp, vp, vp])):
            getattr(lib, name).argtypes = args + [opt_p, vp]
            getattr(lib, name).restype = ctypes.c_int
        for name, args in (("gdr_short_conv_bwd_workspace_size", [conv_p]),
                           ("gdr_selective_scan_workspace_size", [scan_p, ctypes.c_int]),
                           ("gdr_selective_scan_bwd_workspace_size", [scan_p]),
                           ("gdr_rms_norm_bwd_workspace_size", [norm_p])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_size_t
        lib.gdr_release_cached.argtypes = []
        lib.gdr_release_cached.restype = ctypes.c_int
        lib.gdr_version.argtypes = []
        lib.gdr_version.restype = ctypes.c_int
        _lib = lib
        return lib


class GdrError(RuntimeError):
    def __init__(self, code: int):
        msg = load_library().gdr_error_string(code).decode()
        super().__init__(f"gdr error {code}: {msg}")
        self.code = code


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return GDR_F32
    if t == torch.bfloat16:
        return GDR_BF16
    if t == torch.float16:
        return GDR_F16
    raise TypeError(f"unsupported dtype {t}: q, k, v must be float32, bfloat16 or float16")


GDR_SEQLENS_I64 = 1  # gdr_dims.flags: cu_seqlens holds int64 offsets
GDR_STATE_VK = 2     # gdr_dims.flags: h0 / ht / state pool are S [.., V, K]


def make_dims(B, T, H, K, V, N=0, dtype=GDR_BF16, flags=0, max_len=0) -> gdr_dims:
    return gdr_dims(B, T, H, K, V, N, dtype, flags, max_len)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _row_strides(t):
    """(token, head) element strides of a [B, T, H, D] tensor, or (0, 0)
    when it is contiguous.  The last dimension must be contiguous and B, T
    must flatten into one token dimension."""
    if t.is_contiguous():
        return (0, 0)
    B, T = t.shape[0], t.shape[1]
    if t.stride(-1) != 1 or (B > 1 and t.stride(0) != T * t.stride(1)):
        raise ValueError("q, k, v and o need a contiguous last dimension and batch rows "
                         "T token strides apart")
    return (t.stride(1), t.stride(2))


def _dims_of(q, v, cu_seqlens, state_layout="kv", max_seqlen=None, k=None, o=None) -> gdr_dims:
    """Sizes and flags: int64 cu_seqlens sets GDR_SEQLENS_I64; state_layout
    "vk" (states as S, [.., V, K]) sets GDR_STATE_VK; ``max_seqlen`` (the
    longest sequence's token count, a planning hint; None = unknown) goes
    to gdr_dims.max_len; the token / head strides of q, k, v, o (views of a
    larger tensor) go to the stride fields."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    N = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    if state_layout not in ("kv", "vk"):
        raise ValueError(f"state_layout must be 'kv' or 'vk', got {state_layout!r}")
    flags = (GDR_SEQLENS_I64 if cu_seqlens is not None and cu_seqlens.dtype == torch.int64
             else 0) | (GDR_STATE_VK if state_layout == "vk" else 0)
    dims = make_dims(B, T, H, K, V, N, _dtype_code(q.dtype), flags,
                     0 if max_seqlen is None else int(max_seqlen))
    for name, t in (("q_stride", q), ("k_stride", k), ("v_stride", v), ("o_stride", o)):
        if t is not None:
            getattr(dims, name)[:] = _row_strides(t)
    return dims


def _state_dims(dims, state_layout):
    return (dims.V, dims.K) if state_layout == "vk" else (dims.K, dims.V)


def _check_cu(t, device=None):
    if t is not None and t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"cu_seqlens must be int32 or int64, got {t.dtype}")
    _check("cu_seqlens", t, None, device)


def _check(name, t, dtype, device=None, strided=False):
    """dtype / device checks; contiguous unless ``strided`` (q, k, v, o of
    the device entry points, whose token and head strides go to the
    library)."""
    if t is None:
        return
    if strided:
        _row_strides(t)
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


class LaunchTimer:
    """Caller-side CUDA events for the per-launch timing hook of
    gdr_chunk_fwd_ex (benchmarks).  After a call, ``ids[:count]`` are the
    kernel ids launched and ``elapsed_ms(i)`` the duration of launch i once
    the stream has been synchronised."""

    def __init__(self, max_launches=16):
        self.max = max_launches
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_launches)]
        for e in self.events:  # torch creates the CUDA event on first record
            e.record()
        torch.cuda.current_stream().synchronize()
        self._handles = (ctypes.c_void_p * (2 * max_launches))(
            *[ctypes.c_void_p(e.cuda_event) for e in self.events])
        self._ids = (ctypes.c_int32 * max_launches)()
        self._count = ctypes.c_int32(0)

    @property
    def count(self):
        return int(self._count.value)

    @property
    def ids(self):
        return [int(self._ids[i]) for i in range(min(self.count, self.max))]

    def elapsed_ms(self, i):
        return self.events[2 * i].elapsed_time(self.events[2 * i + 1])


def gdr_chunk_fwd(q, k, v, g, beta=None, cu_seqlens=None, h0=None, *, n_segments=0,
                  state_layout="kv", max_seqlen=None,
                  output_final_state=True, o=None, ht=None, scale=0.0, force_path=0,
                  force_bv=0, workspace=None, status=None, stream=None, timer=None,
                  grid_limit=0):
    """Forward pass on CUDA tensors (layouts of include/gdr.h).  Returns
    ``(o, ht)``; ``ht`` is None unless ``output_final_state``.  Work is
    enqueued on ``stream`` (default: torch's current stream) and not
    synchronised.  ``max_seqlen`` is the longest sequence's token count when
    the caller knows it (a planning hint: cu_seqlens stays on the device).
    ``timer`` (a :class:`LaunchTimer`) records events around every kernel
    launch; ``grid_limit`` caps the CTAs of the persistent kernels."""
    lib = load_library()
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("gdr_chunk_fwd takes CUDA tensors; use gdr_chunk_fwd_host for host buffers")
    _check("q", q, None, dev, strided=True)
    for name, t in (("k", k), ("v", v)):
        _check(name, t, q.dtype, dev, strided=True)
    _check("g", g, torch.float32, dev)
    _check("beta", beta, torch.float32, dev)
    _check_cu(cu_seqlens, dev)
    _check("h0", h0, torch.float32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _check("o", o, q.dtype, dev, strided=True)
    dims = _dims_of(q, v, cu_seqlens, state_layout, max_seqlen, k=k, o=o)
    nseq = dims.N if dims.N else dims.B
    if ht is None and output_final_state:
        ht = torch.empty(nseq, dims.H, *_state_dims(dims, state_layout), dtype=torch.float32,
                         device=dev)
    _check("ht", ht, torch.float32, dev)
    opt = gdr_options(float(scale), int(force_path), int(force_bv),
                      None if workspace is None else workspace.data_ptr(),
                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                      None if status is None else status.data_ptr())
    opt.grid_limit = int(grid_limit)
    if timer is not None:
        opt.events = ctypes.cast(timer._handles, ctypes.c_void_p)
        opt.max_launches = timer.max
        opt.launch_ids = ctypes.cast(timer._ids, ctypes.c_void_p)
        opt.n_launches = ctypes.cast(ctypes.pointer(timer._count), ctypes.c_void_p)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = lib.gdr_chunk_fwd_ex(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                  _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                                  int(n_segments), ctypes.byref(opt),
                                  ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return o, ht


def gdr_chunk_bwd(q, k, v, g, beta, do, cu_seqlens=None, h0=None, dht=None, *, n_segments=0,
                  state_layout="kv", want_dh0=True, scale=0.0, workspace=None, status=None,
                  dq=None, dk=None, dv=None, dg=None, dbeta=None, dh0=None, stream=None,
                  timer=None, force_path=0, grid_limit=0):
    """Backward pass on CUDA tensors: the gradients of ``<do, o> + <dht, ht>``
    for the forward pass on the same inputs.  Returns ``(dq, dk, dv, dg,
    dbeta, dh0)``: dq, dk, dv in the input dtype, the rest float32; ``dbeta``
    is None in the beta-free mode and ``dh0`` None unless ``want_dh0``.  Work
    is enqueued on ``stream`` (default: torch's current stream).
    ``force_path`` 1 takes the CUDA-core route (FP32 arithmetic), 2 the
    tensor-core route (BF16, K = V = 128, delta rule, serial), 0 the plan's."""
    lib = load_library()
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("gdr_chunk_bwd takes CUDA tensors")
    _check("q", q, None, dev, strided=True)
    for name, t in (("k", k), ("v", v)):
        _check(name, t, q.dtype, dev, strided=True)
    _check("do", do, q.dtype, dev)
    if do.shape != v.shape:
        raise ValueError("do must have v's shape")
    _check("g", g, torch.float32, dev)
    _check("beta", beta, torch.float32, dev)
    _check_cu(cu_seqlens, dev)
    _check("h0", h0, torch.float32, dev)
    _check("dht", dht, torch.float32, dev)
    dims = _dims_of(q, v, cu_seqlens, state_layout, k=k)
    nseq = dims.N if dims.N else dims.B
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev) if dk is None else dk
    dv = torch.empty(v.shape, dtype=q.dtype, device=dev) if dv is None else dv
    dg = torch.empty(g.shape, dtype=torch.float32, device=dev) if dg is None else dg
    if beta is not None and dbeta is None:
        dbeta = torch.empty(beta.shape, dtype=torch.float32, device=dev)
    if want_dh0 and dh0 is None:
        dh0 = torch.empty(nseq, dims.H, *_state_dims(dims, state_layout), dtype=torch.float32,
                          device=dev)
    for name, t, dt in (("dq", dq, q.dtype), ("dk", dk, q.dtype), ("dv", dv, q.dtype),
                        ("dg", dg, torch.float32), ("dbeta", dbeta, torch.float32),
                        ("dh0", dh0, torch.float32)):
        _check(name, t, dt, dev)
    opt = gdr_options(float(scale), int(force_path), 0,
                      None if workspace is None else workspace.data_ptr(),
                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                      None if status is None else status.data_ptr())
    opt.grid_limit = int(grid_limit)
    if timer is not None:
        opt.events = ctypes.cast(timer._handles, ctypes.c_void_p)
        opt.max_launches = timer.max
        opt.launch_ids = ctypes.cast(timer._ids, ctypes.c_void_p)
        opt.n_launches = ctypes.cast(ctypes.pointer(timer._count), ctypes.c_void_p)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = lib.gdr_chunk_bwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(do), _ptr(dht),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0),
                               int(n_segments), ctypes.byref(opt),
                               ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return dq, dk, dv, dg, dbeta, dh0


def gdr_bwd_workspace_size(B, T, H, K, V, N=0, dtype=GDR_BF16, beta_free=False, flags=0,
                           n_segments=0) -> int:
    return int(load_library().gdr_bwd_workspace_size(
        ctypes.byref(make_dims(B, T, H, K, V, N, dtype, flags)), int(beta_free),
        int(n_segments)))


def gdr_recurrent_fwd(q, k, v, g, beta=None, cu_seqlens=None, *, state, state_indices=None,
                      state_layout="kv",
                      o=None, status=None, stream=None):
    """Per-token recurrence from rows of the state pool ``state`` ([P, H, K,
    V] float32, updated in place): sequence n starts from row
    ``state_indices[n]`` (row n if None) and writes its final state back
    there.  Returns ``o``.  Work is enqueued on ``stream`` and not
    synchronised."""
    lib = load_library()
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("gdr_recurrent_fwd takes CUDA tensors")
    _check("q", q, None, dev, strided=True)
    for name, t in (("k", k), ("v", v)):
        _check(name, t, q.dtype, dev, strided=True)
    _check("g", g, torch.float32, dev)
    _check("beta", beta, torch.float32, dev)
    _check_cu(cu_seqlens, dev)
    _check("state", state, torch.float32, dev)
    _check("state_indices", state_indices, torch.int32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _check("o", o, q.dtype, dev, strided=True)
    dims = _dims_of(q, v, cu_seqlens, state_layout, k=k, o=o)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = lib.gdr_recurrent_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                   _ptr(beta), _ptr(cu_seqlens), _ptr(state),
                                   ctypes.c_int64(state.shape[0]), _ptr(state_indices), _ptr(o),
                                   _ptr(status), ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return o


_CACHE_DTYPES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16, torch.float16: GDR_F16,
                 torch.float8_e4m3fn: GDR_E4M3, torch.int8: GDR_I8}


def _on(index, **tensors):
    """Every given tensor lies on CUDA device ``index``, contiguous, and has the
    dtype it is paired with (None: any)."""
    for name, (t, dtype) in tensors.items():
        if t is None:
            continue
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _cache_of(k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, nseq, index):
    """The C struct of a paged cache; sizes, types and devices checked."""
    dtype = k_cache.dtype
    fmt = _CACHE_DTYPES.get(dtype)
    if fmt is None or v_cache.dtype is not dtype:
        raise TypeError("k_cache and v_cache must share a dtype: float32, bfloat16, float16, "
                        f"float8_e4m3fn or int8, got {dtype} and {v_cache.dtype}")
    shape, v_shape, t_shape = k_cache.shape, v_cache.shape, page_table.shape
    if len(shape) != 4 or len(v_shape) != 4:
        raise ValueError("k_cache and v_cache must be [pages, page size, heads, K] and [.., V]")
    P, page, H, _ = shape
    if v_shape[0] != P or v_shape[1] != page or v_shape[2] != H:
        raise ValueError("k_cache and v_cache must share pages, page size and heads")
    if k_scale is None:
        if fmt >= GDR_E4M3 or v_scale is not None:
            raise ValueError("k_scale and v_scale belong to an 8-bit cache, both of them")
        ks = vs = None
    else:
        if fmt < GDR_E4M3 or v_scale is None:
            raise ValueError("k_scale and v_scale belong to an 8-bit cache, both of them")
        _on(index, k_scale=(k_scale, torch.float32), v_scale=(v_scale, torch.float32))
        if k_scale.shape != (P, H, page) or v_scale.shape != (P, H, page):
            raise ValueError("k_scale and v_scale must be [pages, heads, page size]")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    if page_table.dtype is not torch.int32 or kv_lens.dtype is not torch.int32:
        raise TypeError("page_table and kv_lens must be int32")
    if not (index == k_cache.get_device() == v_cache.get_device() == page_table.get_device()
            == kv_lens.get_device()):
        raise ValueError(f"the caches, page_table and kv_lens must be on cuda:{index}")
    if not (page_table.is_contiguous() and kv_lens.is_contiguous()):
        raise ValueError("page_table and kv_lens must be contiguous")
    if len(t_shape) != 2 or t_shape[0] != nseq or kv_lens.shape != (nseq,):
        raise ValueError("page_table must be [sequences, pages a sequence], kv_lens [sequences]")
    c = gdr_paged_cache(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, page_table.data_ptr(),
                        kv_lens.data_ptr(), P, page, t_shape[1], H, fmt)
    if not k_cache.is_contiguous():
        c.k_stride[:] = _page_strides(k_cache)
    if not v_cache.is_contiguous():
        c.v_stride[:] = _page_strides(v_cache)
    return c


def _page_strides(t):
    if t.stride(-1) != 1 or min(t.stride()) < 1:
        raise ValueError("k_cache and v_cache need a contiguous last dimension")
    return t.stride()[:3]


def _paged_dims(B, T, H, K, V, cu_seqlens, dtype, index, max_seqlen=None):
    """gdr_dims of a call on a paged cache, and its number of sequences."""
    if cu_seqlens is None:
        n, flags = 0, 0
    else:
        if cu_seqlens.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
        _on(index, cu_seqlens=(cu_seqlens, None))
        n = cu_seqlens.numel() - 1
        flags = GDR_SEQLENS_I64 if cu_seqlens.dtype == torch.int64 else 0
    return gdr_dims(B, T, H, K, V, n, _dtype_code(dtype), flags,
                    0 if max_seqlen is None else int(max_seqlen)), B if cu_seqlens is None else n


def _set_strides(field, t):
    if not t.is_contiguous():
        field[:] = _row_strides(t)


def _paged_call(fn, index, stream, *args):
    """Calls a library function on ``stream`` (default: the current one)."""
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:  # torch holds a tensor there: it is initialised
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        raise GdrError(rc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_status(status, index):
    """The status word is written on the device."""
    if status is not None:
        _on(index, status=(status, torch.int32))
        if status.numel() < 1:
            raise ValueError("status must have an element")


def gdr_cache_write(k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, *,
                    k_scale=None, v_scale=None, status=None, stream=None):
    """Stores the new tokens' ``k`` [B, T, H, K] and ``v`` [B, T, H, V] in the
    paged cache ``k_cache`` [P, page size, H, K], ``v_cache`` [.., V], in place.
    ``kv_lens`` [N] counts each sequence's tokens including the new ones: token
    i of the L new ones goes to position ``kv_lens[n] - L + i``, slot ``position
    % page size`` of page ``page_table[n, position // page size]``.  A cache of
    k's dtype holds the rows as they are; a float8_e4m3fn or int8 cache holds
    them quantised, with a scale for each (token, head) row in ``k_scale`` and
    ``v_scale`` [P, H, page size] (float32)."""
    lib = load_library()
    index = k.get_device()
    if index < 0:
        raise ValueError("gdr_cache_write takes CUDA tensors")
    if v.get_device() != index or v.dtype != k.dtype:
        raise ValueError("k and v must share a device and a dtype")
    _check_status(status, index)
    if v.shape[:-1] != k.shape[:-1] or k_cache.shape[2:] != k.shape[2:] or \
            v_cache.shape[-1] != v.shape[-1]:
        raise ValueError("k, v and the caches must agree in tokens, heads and widths")
    dims, nseq = _paged_dims(*k.shape, v.shape[3], cu_seqlens, k.dtype, index)
    _set_strides(dims.k_stride, k)
    _set_strides(dims.v_stride, v)
    cache = _cache_of(k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, nseq, index)
    _paged_call(lib.gdr_cache_write, index, stream, dims, cache, k.data_ptr(), v.data_ptr(),
                _addr(cu_seqlens), _addr(status))


def gdr_cache_read(k_cache, v_cache, page_table, kv_lens, T, cu_seqlens=None, *, k_scale=None,
                   v_scale=None, dtype=None, k=None, v=None, status=None, stream=None):
    """What the paged cache holds for the last tokens of every sequence, as
    ``(k, v)`` [B, T, H, K] and [B, T, H, V]: ``T`` tokens of each sequence, or
    with ``cu_seqlens`` the packed lengths (T their sum, B = 1).  ``dtype`` is
    the cache's own unless that is an 8-bit format (then bfloat16 by default);
    ``k`` and ``v`` may be given to write into."""
    lib = load_library()
    index = k_cache.get_device()
    if index < 0:
        raise ValueError("gdr_cache_read takes CUDA tensors")
    _check_status(status, index)
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [pages, page size, heads, K] and [.., V]")
    B = kv_lens.numel() if cu_seqlens is None else 1
    if dtype is None:
        dtype = k.dtype if k is not None else (
            k_cache.dtype if k_cache.element_size() > 1 else torch.bfloat16)
    H, K, V = k_cache.shape[2], k_cache.shape[3], v_cache.shape[3]
    for name, t, D in (("k", k, K), ("v", v, V)):
        if t is not None and (t.get_device() != index or t.dtype != dtype or
                              t.shape != (B, T, H, D)):
            raise ValueError(f"{name} must be {[B, T, H, D]}, {dtype}, on cuda:{index}")
    if k is None:
        k = torch.empty((B, T, H, K), dtype=dtype, device=k_cache.device)
    if v is None:
        v = (torch.empty_like(k) if V == K and k.is_contiguous()
             else torch.empty((B, T, H, V), dtype=dtype, device=k_cache.device))
    dims, nseq = _paged_dims(B, T, H, K, V, cu_seqlens, dtype, index)
    _set_strides(dims.k_stride, k)
    _set_strides(dims.v_stride, v)
    cache = _cache_of(k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, nseq, index)
    _paged_call(lib.gdr_cache_read, index, stream, dims, cache, k.data_ptr(), v.data_ptr(),
                _addr(cu_seqlens), _addr(status))
    return k, v


def gdr_paged_attn(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, *, k_scale=None,
                   v_scale=None, causal=True, window=0, scale=0.0, max_seqlen=None, o=None,
                   lse=None, force_path=0, grid_limit=0, workspace=None, status=None,
                   stream=None, timer=None):
    """Softmax attention of the new tokens ``q`` [B, T, Hq, K] over the paged
    cache (laid out as for :func:`gdr_cache_write`, which put the new tokens'
    own keys and values there).  Token i, at position p, sees the positions
    below ``kv_lens[n]``, up to p when ``causal`` and above ``p - window`` when
    ``window`` > 0; Hq is a multiple of the cache's heads.  Returns ``(o,
    lse)``: o [B, T, Hq, V] in q's dtype and the log of the softmax's
    denominator [B, T, Hq] (float32); a row that sees nothing has o = 0 and lse
    = -inf.  ``max_seqlen`` is the most new tokens of a sequence when the
    caller knows it (a planning hint).  ``workspace`` may hold the call's scratch
    (:func:`gdr_attn_workspace_size` bytes, 256-byte aligned).  Work is enqueued on
    ``stream`` (default: the current one) and not synchronised."""
    lib = load_library()
    index = q.get_device()
    if index < 0:
        raise ValueError("gdr_paged_attn takes CUDA tensors")
    _check_status(status, index)
    _on(index, workspace=(workspace, None))
    shape, k_shape, v_shape = q.shape, k_cache.shape, v_cache.shape
    if len(shape) != 4 or len(k_shape) != 4 or len(v_shape) != 4 or shape[3] != k_shape[3]:
        raise ValueError("q must be [B, T, heads, K], the caches [pages, page size, heads, K or V]")
    B, T, H, K = shape
    V = v_shape[3]
    if o is None:
        o = torch.empty_like(q) if V == K and q.is_contiguous() else q.new_empty((B, T, H, V))
    elif o.shape != (B, T, H, V) or o.dtype != q.dtype or o.get_device() != index:
        raise ValueError(f"o must be {[B, T, H, V]}, {q.dtype}, on cuda:{index}")
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    else:
        _on(index, lse=(lse, torch.float32))
        if lse.shape != (B, T, H):
            raise ValueError("lse must be [B, T, heads]")
    dims, nseq = _paged_dims(B, T, H, K, V, cu_seqlens, q.dtype, index, max_seqlen)
    _set_strides(dims.q_stride, q)
    _set_strides(dims.o_stride, o)
    cache = _cache_of(k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, nseq, index)
    if cache.dtype < GDR_E4M3 and k_cache.dtype != q.dtype:
        raise TypeError(f"the caches must be {q.dtype} or an 8-bit format, got {k_cache.dtype}")
    opt = None
    if scale or force_path or grid_limit or workspace is not None or status is not None or timer:
        opt = gdr_options(float(scale), int(force_path), 0, _addr(workspace),
                          0 if workspace is None else workspace.numel() * workspace.element_size(),
                          _addr(status))
        opt.grid_limit = int(grid_limit)
        if timer is not None:
            opt.events = ctypes.cast(timer._handles, ctypes.c_void_p)
            opt.max_launches = timer.max
            opt.launch_ids = ctypes.cast(timer._ids, ctypes.c_void_p)
            opt.n_launches = ctypes.cast(ctypes.pointer(timer._count), ctypes.c_void_p)
    _paged_call(lib.gdr_paged_attn, index, stream, dims, cache, q.data_ptr(), _addr(cu_seqlens),
                o.data_ptr(), lse.data_ptr(), 1 if causal else 0, int(window), opt)
    return o, lse


def gdr_attn_workspace_size(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens=None, *,
                            k_scale=None, v_scale=None) -> int:
    """Bytes of device scratch that :func:`gdr_paged_attn` needs for these tensors,
    whatever its route."""
    index = q.get_device()
    if index < 0:
        raise ValueError("gdr_attn_workspace_size takes CUDA tensors")
    dims, nseq = _paged_dims(*q.shape, v_cache.shape[3], cu_seqlens, q.dtype, index)
    cache = _cache_of(k_cache, v_cache, page_table, kv_lens, k_scale, v_scale, nseq, index)
    with torch.cuda.device(index):
        return int(load_library().gdr_attn_workspace_size(ctypes.byref(dims), ctypes.byref(cache)))


def gdr_chunk_fwd_host(q, k, v, g, beta=None, cu_seqlens=None, h0=None, *, n_segments=0,
                       state_layout="kv",
                       output_final_state=True, o=None, ht=None, stream=None):
    """Forward pass on HOST (CPU) tensors through ``gdr_chunk_fwd_host``: the
    library copies inputs in, runs, copies o / ht out and synchronises.
    Pinned tensors give asynchronous copies."""
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta),
                    ("cu_seqlens", cu_seqlens), ("h0", h0)):
        if t is not None and t.device.type != "cpu":
            raise ValueError(f"{name} must be a host tensor")
    _check("k", k, q.dtype)
    _check("v", v, q.dtype)
    _check("g", g, torch.float32)
    _check("beta", beta, torch.float32)
    _check_cu(cu_seqlens)
    _check("h0", h0, torch.float32)
    dims = _dims_of(q, v, cu_seqlens, state_layout)
    nseq = dims.N if dims.N else dims.B
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype)
    if ht is None and output_final_state:
        ht = torch.empty(nseq, dims.H, *_state_dims(dims, state_layout), dtype=torch.float32)
    if stream is None:
        stream = torch.cuda.current_stream()
    rc = lib.gdr_chunk_fwd_host(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                                int(n_segments), ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return o, ht


NOALLOC_SCRATCH_BYTES = 64 << 20


def gdr_chunk_fwd_noalloc(q, k, v, g, beta=None, cu_seqlens=None, h0=None, *, n_segments=0,
                          state_layout="kv", max_seqlen=None,
                          output_final_state=True, o=None, ht=None, stream=None):
    """Forward pass through ``gdr_chunk_fwd_noalloc``: the library uses a
    fixed 64 MiB device array as scratch and allocates nothing, for callers
    that must not allocate device memory during the call.  ``o`` and ``ht``
    should be passed in by such callers (this wrapper creates them with
    torch only when they are omitted).  Calls that overlap on the GPU share
    the one scratch array and must be ordered by the caller; the first call
    on a device should happen outside CUDA graph capture."""
    lib = load_library()
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("gdr_chunk_fwd_noalloc takes CUDA tensors")
    _check("q", q, None, dev, strided=True)
    for name, t in (("k", k), ("v", v)):
        _check(name, t, q.dtype, dev, strided=True)
    _check("g", g, torch.float32, dev)
    _check("beta", beta, torch.float32, dev)
    _check_cu(cu_seqlens, dev)
    _check("h0", h0, torch.float32, dev)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    _check("o", o, q.dtype, dev, strided=True)
    dims = _dims_of(q, v, cu_seqlens, state_layout, max_seqlen, k=k, o=o)
    nseq = dims.N if dims.N else dims.B
    if ht is None and output_final_state:
        ht = torch.empty(nseq, dims.H, *_state_dims(dims, state_layout), dtype=torch.float32,
                         device=dev)
    _check("ht", ht, torch.float32, dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = lib.gdr_chunk_fwd_noalloc(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                       _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht),
                                       int(n_segments), ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return o, ht


def gdr_workspace_size(B, T, H, K, V, N=0, dtype=GDR_BF16, beta_free=False, n_segments=0,
                       max_len=0) -> int:
    return int(load_library().gdr_workspace_size(
        ctypes.byref(make_dims(B, T, H, K, V, N, dtype, max_len=max_len)), int(bool(beta_free)),
        int(n_segments)))


def gdr_plan_query(B, T, H, K, V, N=0, dtype=GDR_BF16, beta_free=False, n_segments=0,
                   max_len=0) -> dict:
    plan = gdr_plan()
    rc = load_library().gdr_plan_query(ctypes.byref(make_dims(B, T, H, K, V, N, dtype,
                                                              max_len=max_len)),
                                       int(bool(beta_free)), int(n_segments), ctypes.byref(plan))
    if rc != 0:
        raise GdrError(rc)
    return dict(path=plan.path, bv=plan.bv, n_segments=plan.n_segments, compose=plan.compose)


def gdr_selftest_umma(A, B, a_mn, b_mn, status=None):
    """D = A @ B^T (A [128, Kd], B [N, Kd] BF16 CUDA tensors) computed by one
    tcgen05 MMA chain with the given operand layouts; returns D (FP32)."""
    N, Kd = B.shape
    D = torch.full((A.shape[0], N), float("nan"), dtype=torch.float32, device=A.device)
    rc = load_library().gdr_selftest_umma(_ptr(A), _ptr(B), _ptr(D), N, Kd, int(a_mn), int(b_mn),
                                          _ptr(status),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return D


def gdr_selftest_tma(src, t0, h, k0, status=None):
    """One 64x64 box of src [T, H, K] (BF16 CUDA) through TMA + the swizzle
    address map; returns the [64, 64] box."""
    T, H, K = src.shape
    out = torch.full((64, 64), float("nan"), dtype=torch.bfloat16, device=src.device)
    rc = load_library().gdr_selftest_tma(_ptr(src), T, H, K, int(t0), int(h), int(k0), _ptr(out),
                                         _ptr(status),
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return out


def gdr_selftest_inverse(A):
    """(I + tril(A, -1))^-1 for a 64x64 FP32 CUDA tensor, by the device routine
    of the tensor-core path."""
    A = A.contiguous()
    T = torch.full_like(A, float("nan"))
    rc = load_library().gdr_selftest_inverse(_ptr(A), _ptr(T),
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    return T


def gdr_selftest_timeout(limit_ns=1_000_000):
    """Runs the bounded-wait failure path once; returns (status, done)."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    done = torch.zeros(1, dtype=torch.int32, device="cuda")
    rc = load_library().gdr_selftest_timeout(_ptr(status), int(limit_ns), _ptr(done),
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if rc != 0:
        raise GdrError(rc)
    torch.cuda.synchronize()
    return int(status.item()), int(done.item())


def gdr_kernel_name(kid: int) -> str:
    return load_library().gdr_kernel_name(int(kid)).decode()


def gdr_error_string(code: int) -> str:
    return load_library().gdr_error_string(int(code)).decode()


def gdr_release_cached() -> None:
    """Return the device memory the library keeps between calls (its
    stream-ordered scratch pools) to the driver."""
    rc = load_library().gdr_release_cached()
    if rc != 0:
        raise GdrError(rc)


def gdr_version() -> int:
    return int(load_library().gdr_version())
