"""ctypes binding of the operators of a state-space layer (``include/gdr.h``): short
convolution, selective scan and root-mean-square norm.  Argument marshalling only."""
from __future__ import annotations

import ctypes

import torch

from .api import (GDR_E4M3, GDR_I8, GDR_SEQLENS_I64, _addr, _check_status, _dtype_code, _on,
                  _paged_call, gdr_conv_dims, gdr_norm_dims, gdr_options, gdr_scan_dims,
                  gdr_scan_grads, gdr_scan_tensors, load_library)


def _index_of(name, x):
    index = x.get_device()
    if index < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    return index


def _like(index, dtype, shape, **tensors):
    """Every given tensor lies on CUDA device ``index`` and has this dtype and shape."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _token_stride(name, t):
    """Elements from one token of [B, T, C] to the next, 0 when contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    B, T, C = t.shape
    step = t.stride(1) if T > 1 else t.stride(0) if B > 1 else C
    if (C > 1 and t.stride(2) != 1) or (B > 1 and T > 1 and t.stride(0) != T * step) or step < 1:
        raise ValueError(f"{name} needs contiguous channels and batch rows T token strides apart")
    return step


def _group_strides(name, t):
    """Token and group strides of [B, T, G, S], (0, 0) when contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return (0, 0)
    B, T, G, S = t.shape
    step = t.stride(1) if T > 1 else t.stride(0) if B > 1 else G * S
    group = t.stride(2) if G > 1 else S
    if (S > 1 and t.stride(3) != 1) or (B > 1 and T > 1 and t.stride(0) != T * step) or \
            min(step, group) < 1:
        raise ValueError(f"{name} needs contiguous states and batch rows T token strides apart")
    return (step, group)


def _seqs(B, cu_seqlens, index):
    """(N, flags, sequences) of a call."""
    if cu_seqlens is None:
        return 0, 0, B
    if cu_seqlens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
    _on(index, cu_seqlens=(cu_seqlens, None))
    n = cu_seqlens.numel() - 1
    return n, GDR_SEQLENS_I64 if cu_seqlens.dtype == torch.int64 else 0, n


def _options(index, workspace, status, timer):
    _check_status(status, index)
    if workspace is None and status is None and timer is None:
        return None
    _on(index, workspace=(workspace, None))
    opt = gdr_options(workspace=_addr(workspace), status=_addr(status),
                      workspace_bytes=0 if workspace is None
                      else workspace.numel() * workspace.element_size())
    if timer is not None:
        opt.events = ctypes.cast(timer._handles, ctypes.c_void_p)
        opt.max_launches = timer.max
        opt.launch_ids = ctypes.cast(timer._ids, ctypes.c_void_p)
        opt.n_launches = ctypes.cast(ctypes.pointer(timer._count), ctypes.c_void_p)
    return opt


def _call(fn, index, stream, tensors, *args):
    """The library's call; the memory of ``tensors`` is not handed out again before ``stream``
    is through with them, whatever stream they were made on."""
    _paged_call(fn, index, stream, *args)
    if stream is not None:
        for t in tensors:
            if t is not None and t.numel():
                t.record_stream(stream)


def _states(index, nseq, tail, dtype, h0, ht, state, state_indices, want, device):
    """(h0, ht, rows) of a call that goes on from ``h0`` [N, ...] or moves the pool ``state`` on in
    place."""
    if state is not None:
        if h0 is not None or ht is not None:
            raise ValueError("state is read and written in place: h0 and ht do not go with it")
        _like(index, dtype, (state.shape[0],) + tail, state=state)
        _on(index, state=(state, None), state_indices=(state_indices, torch.int32))
        if state_indices is not None and state_indices.shape != (nseq,):
            raise ValueError(f"state_indices must be [{nseq}], got {list(state_indices.shape)}")
        if state_indices is None and state.shape[0] < nseq:
            raise ValueError(f"state must have a row for each of {nseq} sequences")
        return state, state, state.shape[0]
    if state_indices is not None:
        raise ValueError("state_indices belong to state")
    if ht is None and want:
        ht = torch.empty((nseq,) + tail, dtype=dtype, device=device)
    _like(index, dtype, (nseq,) + tail, h0=h0, ht=ht)
    _on(index, h0=(h0, None), ht=(ht, None))
    return h0, ht, nseq


def _weight_code(name, t, dtype):
    if t.dtype != dtype and t.dtype != torch.float32:
        raise TypeError(f"{name} must be {dtype} or float32, got {t.dtype}")
    return _dtype_code(t.dtype)


_ACTIVATIONS = {None: 0, "silu": 1}


def _conv_dims(x, weight, bias, cu_seqlens, activation, max_seqlen, index):
    if x.dim() != 3 or weight.dim() != 2 or weight.shape[0] != x.shape[2]:
        raise ValueError("x must be [B, T, C], weight [C, W]")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    B, T, C = x.shape
    wd = _weight_code("weight", weight, x.dtype)
    _on(index, weight=(weight, None))
    _like(index, weight.dtype, (C,), bias=bias)
    _on(index, bias=(bias, None))
    n, flags, nseq = _seqs(B, cu_seqlens, index)
    return gdr_conv_dims(B, T, C, weight.shape[1], n, _dtype_code(x.dtype), flags, wd,
                         _ACTIVATIONS[activation], 0 if max_seqlen is None else int(max_seqlen),
                         _token_stride("x", x)), nseq


def gdr_short_conv_fwd(x, weight, bias=None, cu_seqlens=None, h0=None, *, activation="silu",
                       state=None, state_indices=None, output_final_state=False, max_seqlen=None,
                       y=None, ht=None, status=None, stream=None, timer=None):
    """Causal convolution of ``x`` [B, T, C] (a view with a token stride will do) along each
    sequence with a filter of W = 2 to 4 taps a channel, ``weight`` [C, W] and ``bias`` [C] (x's
    dtype or float32), and SiLU behind it.  A sequence's inputs before its first token are its row
    of ``h0`` [N, W - 1, C] (zeros if None), oldest first; ``ht`` gets those before the token that
    will follow.  With ``state`` [P, W - 1, C] the rows ``state_indices`` (row n if None) of a
    pool take the place of both, in place.  Returns ``(y, ht)``; ht is ``state``, or None unless
    wanted.  ``max_seqlen`` is a planning hint, as everywhere.  Work is enqueued on ``stream``
    (default: the current one) and not synchronised."""
    lib = load_library()
    index = _index_of("gdr_short_conv_fwd", x)
    dims, nseq = _conv_dims(x, weight, bias, cu_seqlens, activation, max_seqlen, index)
    opt = _options(index, None, status, timer)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(index, x.dtype, x.shape, y=y)
        dims.y_stride = _token_stride("y", y)
    h0, ht, rows = _states(index, nseq, (dims.W - 1, dims.C), x.dtype, h0, ht, state,
                           state_indices, output_final_state, x.device)
    _call(lib.gdr_short_conv_fwd, index, stream,
          (x, weight, bias, cu_seqlens, h0, ht, state_indices, y), dims, x.data_ptr(),
          weight.data_ptr(), _addr(bias), _addr(cu_seqlens), _addr(h0), _addr(ht), rows,
          _addr(state_indices), y.data_ptr(), opt)
    return y, ht


def gdr_short_conv_bwd(x, weight, dy, bias=None, cu_seqlens=None, h0=None, dht=None, *,
                       activation="silu", want_dh0=False, max_seqlen=None, workspace=None,
                       status=None, stream=None, timer=None):
    """Gradients of ``<dy, y> + <dht, ht>`` for :func:`gdr_short_conv_fwd` on the same inputs:
    ``(dx, dweight, dbias, dh0)``, dx and dh0 in x's dtype, dweight and dbias float32; dbias is None
    without a bias, dh0 unless ``want_dh0``."""
    lib = load_library()
    index = _index_of("gdr_short_conv_bwd", x)
    dims, nseq = _conv_dims(x, weight, bias, cu_seqlens, activation, max_seqlen, index)
    opt = _options(index, workspace, status, timer)
    _like(index, x.dtype, x.shape, dy=dy)
    dims.y_stride = _token_stride("dy", dy)
    tail = (nseq, dims.W - 1, dims.C)
    _like(index, x.dtype, tail, h0=h0, dht=dht)
    _on(index, h0=(h0, None), dht=(dht, None))
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
    db = None if bias is None else torch.empty(x.shape[2], device=x.device)
    dh0 = torch.empty(tail, dtype=x.dtype, device=x.device) if want_dh0 else None
    _call(lib.gdr_short_conv_bwd, index, stream,
          (x, weight, dy, bias, cu_seqlens, h0, dht, dx, dw, db, dh0, workspace), dims,
          x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(cu_seqlens), _addr(h0),
          dy.data_ptr(), _addr(dht), dx.data_ptr(), dw.data_ptr(), _addr(db), _addr(dh0), opt)
    return dx, dw, db, dh0


def _scan_dims(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, softplus, max_seqlen, index):
    if x.dim() != 3 or A.dim() != 2 or A.shape[0] != x.shape[2] or B.dim() != 4 or \
            B.shape[:2] != x.shape[:2] or B.shape[3] != A.shape[1]:
        raise ValueError("x must be [B, T, C], A [C, S], B and C [B, T, groups, S]")
    nb, T, ch = x.shape
    _like(index, x.dtype, x.shape, dt=dt, z=z)
    _like(index, x.dtype, B.shape, B=B, C=C)
    _like(index, torch.float32, (ch,), D=D, dt_bias=dt_bias)
    _on(index, A=(A, torch.float32), D=(D, None), dt_bias=(dt_bias, None))
    n, flags, nseq = _seqs(nb, cu_seqlens, index)
    dims = gdr_scan_dims(nb, T, ch, A.shape[1], B.shape[2], n, _dtype_code(x.dtype), flags,
                         1 if softplus else 0, 0 if max_seqlen is None else int(max_seqlen),
                         _token_stride("x", x), _token_stride("dt", dt),
                         0 if z is None else _token_stride("z", z))
    dims.b_stride[:] = _group_strides("B", B)
    dims.c_stride[:] = _group_strides("C", C)
    return dims, nseq, gdr_scan_tensors(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                        C.data_ptr(), _addr(D), _addr(z), _addr(dt_bias))


def gdr_selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, cu_seqlens=None, h0=None,
                           *, softplus=True, state=None, state_indices=None,
                           output_final_state=True, max_seqlen=None, n_segments=0, y=None, ht=None,
                           workspace=None, status=None, stream=None, timer=None):
    """Selective state-space scan of ``x`` [B, T, C] along each sequence: with d = softplus(dt +
    dt_bias) (d = dt + dt_bias unless ``softplus``), h = exp(d A) h + d x B, y = (<C, h> + D x)
    silu(z).  ``dt`` and ``z`` are like x, ``A`` [C, S] float32 with S up to 64, ``B`` and ``C``
    [B, T, G, S] like x (channel c is in group c // (C / G)), ``D`` and ``dt_bias`` [C] float32; x,
    dt, z, B and C may be views with token strides.  The states [N, C, S] float32 come from ``h0``
    and go to ``ht``, or are rows ``state_indices`` of the pool ``state`` [P, C, S], in place, as for
    :func:`gdr_short_conv_fwd`.  ``n_segments`` as in ``gdr_chunk_fwd``: 0 plans, 1 runs the
    sequences whole, more cuts them.  Returns ``(y, ht)``; ht is ``state``, or None unless
    ``output_final_state``."""
    lib = load_library()
    index = _index_of("gdr_selective_scan_fwd", x)
    dims, nseq, tensors = _scan_dims(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, softplus,
                                     max_seqlen, index)
    opt = _options(index, workspace, status, timer)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _like(index, x.dtype, x.shape, y=y)
        dims.y_stride = _token_stride("y", y)
    h0, ht, rows = _states(index, nseq, (dims.C, dims.S), torch.float32, h0, ht, state,
                           state_indices, output_final_state, x.device)
    _call(lib.gdr_selective_scan_fwd, index, stream,
          (x, dt, A, B, C, D, z, dt_bias, cu_seqlens, h0, ht, state_indices, y, workspace), dims,
          tensors, _addr(cu_seqlens), _addr(h0), _addr(ht), rows, _addr(state_indices),
          y.data_ptr(), int(n_segments), opt)
    return y, ht


def gdr_selective_scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, cu_seqlens=None,
                           h0=None, dht=None, *, softplus=True, want_dh0=False, max_seqlen=None,
                           workspace=None, status=None, stream=None, timer=None):
    """Gradients of ``<dy, y> + <dht, ht>`` for :func:`gdr_selective_scan_fwd` on the same
    inputs: ``(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)``, each in its input's dtype; None for
    an input that is None, dh0 unless ``want_dh0``."""
    lib = load_library()
    index = _index_of("gdr_selective_scan_bwd", x)
    dims, nseq, tensors = _scan_dims(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, softplus,
                                     max_seqlen, index)
    opt = _options(index, workspace, status, timer)
    _like(index, x.dtype, x.shape, dy=dy)
    dims.y_stride = _token_stride("dy", dy)
    _like(index, torch.float32, (nseq, dims.C, dims.S), h0=h0, dht=dht)
    _on(index, h0=(h0, None), dht=(dht, None))

    def new(like):
        return None if like is None else torch.empty(like.shape, dtype=like.dtype, device=x.device)

    dh0 = torch.empty((nseq, dims.C, dims.S), device=x.device) if want_dh0 else None
    out = (new(x), new(dt), new(A), new(B), new(C), new(D), new(z), new(dt_bias), dh0)
    grads = gdr_scan_grads(*(_addr(t) for t in out))
    _call(lib.gdr_selective_scan_bwd, index, stream,
          (x, dt, A, B, C, dy, D, z, dt_bias, cu_seqlens, h0, dht, workspace) + out, dims, tensors,
          _addr(cu_seqlens), _addr(h0), dy.data_ptr(), _addr(dht), grads, opt)
    return out


_OUT_DTYPES = {torch.float8_e4m3fn: GDR_E4M3, torch.int8: GDR_I8}


def _row_stride(name, t):
    """Elements from one row of [..., D] to the next, 0 when contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    shape, strides = t.shape, t.stride()
    if shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name} needs a contiguous last dimension")
    step, need = None, None
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if step is None:
            step = need = s
        elif s != need:
            raise ValueError(f"{name}: rows must lie at one stride")
        need *= n
    return shape[-1] if step is None else step


def gdr_rms_norm_fwd(x, weight=None, residual=None, *, eps=1e-6, dtype=None, group=0, y=None,
                     residual_out=None, scale=None, stream=None, timer=None):
    """Root-mean-square norm of the rows ``x`` [..., D], D up to 16384: with r = x + residual
    (rounded to x's dtype), y = r / sqrt(mean(r^2) + eps) * weight.  ``weight`` [D] is of x's dtype
    or float32.  ``dtype`` float8_e4m3fn or int8 quantises y, with a float32 scale for each row
    (``scale`` [...]) or, with ``group`` 128, for each 128 columns ([..., ceil(D / 128)]), as
    :func:`gdr_cache_write` does.  Returns ``(y, r, scale)``; r is None without a residual, scale
    unless y is quantised.  ``residual_out`` may be the residual or x itself, ``y`` x (in place)."""
    lib = load_library()
    index = _index_of("gdr_rms_norm_fwd", x)
    D = x.shape[-1]
    code = _dtype_code(x.dtype)
    if dtype is None or dtype == x.dtype:
        out, out_code = x.dtype, code
    elif dtype in _OUT_DTYPES:
        out, out_code = dtype, _OUT_DTYPES[dtype]
    else:
        raise TypeError(f"dtype must be {x.dtype}, float8_e4m3fn or int8, got {dtype}")
    if group and (out_code < GDR_E4M3 or group != 128):
        raise ValueError("group is 0, or 128 where y is quantised")
    wd = code if weight is None else _weight_code("weight", weight, x.dtype)
    if weight is not None:
        _like(index, weight.dtype, (D,), weight=weight)
        _on(index, weight=(weight, None))
    _like(index, x.dtype, x.shape, residual=residual, residual_out=residual_out)
    if y is None:
        y = torch.empty(x.shape, dtype=out, device=x.device)
    else:
        _like(index, out, x.shape, y=y)
    if residual is not None and residual_out is None:
        residual_out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif residual is None and residual_out is not None:
        raise ValueError("residual_out belongs to a residual")
    if out_code >= GDR_E4M3:
        want = x.shape[:-1] + ((D + 127) // 128,) if group else x.shape[:-1]
        if scale is None:
            scale = torch.empty(want, device=x.device)
        _like(index, torch.float32, want, scale=scale)
        _on(index, scale=(scale, None))
    elif scale is not None:
        raise ValueError("scale belongs to a quantised y")
    dims = gdr_norm_dims(x.numel() // D if D else 0, D, code, wd, out_code, int(group), float(eps),
                         _row_stride("x", x), 0, 0, _row_stride("y", y))
    if residual is not None:
        dims.residual_stride = _row_stride("residual", residual)
        dims.sum_stride = _row_stride("residual_out", residual_out)
    _call(lib.gdr_rms_norm_fwd, index, stream, (x, residual, weight, residual_out, y, scale), dims,
          x.data_ptr(), _addr(residual), _addr(weight), _addr(residual_out), y.data_ptr(),
          _addr(scale), _options(index, None, None, timer))
    return y, residual_out, scale


def gdr_rms_norm_bwd(dy, r, weight=None, dr=None, *, eps=1e-6, workspace=None, stream=None,
                     timer=None):
    """Gradients of ``<dy, y> + <dr, r>`` for :func:`gdr_rms_norm_fwd` (y of x's dtype), from ``r``
    (its r, or its x without a residual): ``(dx, dweight)``; dx is the gradient of x and of the
    residual alike, dweight float32 (None without a weight)."""
    lib = load_library()
    index = _index_of("gdr_rms_norm_bwd", r)
    D, code = r.shape[-1], _dtype_code(r.dtype)
    _like(index, r.dtype, r.shape, dy=dy, dr=dr)
    wd = code if weight is None else _weight_code("weight", weight, r.dtype)
    if weight is not None:
        _like(index, weight.dtype, (D,), weight=weight)
        _on(index, weight=(weight, None))
    opt = _options(index, workspace, None, timer)
    dx = torch.empty(r.shape, dtype=r.dtype, device=r.device)
    dw = None if weight is None else torch.empty(D, device=r.device)
    dims = gdr_norm_dims(r.numel() // D if D else 0, D, code, wd, code, 0, float(eps),
                         _row_stride("r", r), 0 if dr is None else _row_stride("dr", dr), 0,
                         _row_stride("dy", dy))
    _call(lib.gdr_rms_norm_bwd, index, stream, (dy, r, weight, dr, dx, dw, workspace), dims,
          r.data_ptr(), _addr(weight), dy.data_ptr(), _addr(dr), dx.data_ptr(), _addr(dw), opt)
    return dx, dw


def gdr_short_conv_bwd_workspace_size(B, T, C, W, N=0, dtype=torch.bfloat16) -> int:
    """Bytes of scratch that :func:`gdr_short_conv_bwd` needs."""
    code = _dtype_code(dtype)
    return int(load_library().gdr_short_conv_bwd_workspace_size(
        gdr_conv_dims(B, T, C, W, N, code, 0, code)))


def gdr_selective_scan_workspace_size(B, T, C, S, groups=1, N=0, dtype=torch.bfloat16,
                                      max_seqlen=0, n_segments=0, backward=False) -> int:
    """Bytes of scratch that :func:`gdr_selective_scan_fwd`, or with ``backward``
    :func:`gdr_selective_scan_bwd`, needs."""
    dims = gdr_scan_dims(B, T, C, S, groups, N, _dtype_code(dtype), 0, 1, max_seqlen)
    lib = load_library()
    if backward:
        return int(lib.gdr_selective_scan_bwd_workspace_size(dims))
    return int(lib.gdr_selective_scan_workspace_size(dims, int(n_segments)))


def gdr_rms_norm_bwd_workspace_size(rows, D, dtype=torch.bfloat16) -> int:
    """Bytes of scratch that :func:`gdr_rms_norm_bwd` needs."""
    code = _dtype_code(dtype)
    return int(load_library().gdr_rms_norm_bwd_workspace_size(
        gdr_norm_dims(rows, D, code, code, code)))
