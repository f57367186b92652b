"""ctypes binding of the operators of a state-space layer (``include/gdr.h``): short
convolution, selective scan and root-mean-square norm.  Argument marshalling only."""
from __future__ import annotations

import ctypes

import torch

from .api import (GDR_BF16, GDR_E4M3, GDR_F16, GDR_F32, GDR_I8, GDR_SEQLENS_I64, GdrError,
                  _check_status, _dtype_code, _on, gdr_conv_dims, gdr_norm_dims, gdr_options,
                  gdr_scan_dims, gdr_scan_grads, gdr_scan_tensors, load_library)

# A decode step's time is the time of its calls, most of it here: so what is usually right is
# tested in line, and a function that names what is wrong is called only where something is.

_CODES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16, torch.float16: GDR_F16}
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _refuse(index, dtype, shape, **tensors):
    """Raises for the first tensor that is not on CUDA device ``index``, of this dtype and shape."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _like(index, dtype, shape, name, t, contiguous=False):
    """The tensor's address, None without one: it lies on CUDA device ``index`` and has this dtype
    and shape."""
    if t is None:
        return None
    if t.get_device() != index or t.dtype is not dtype or t.shape != shape:
        _refuse(index, dtype, shape, **{name: t})
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """A new tensor that a call on ``stream`` (None: the current one) writes.  Its memory is that
    stream's: what the current one has let go may still be in use there, which ``stream`` does not
    wait for.  The current stream, where the caller goes on, may use it and let it go as its own."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if t.numel():
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _new(like, stream):
    """A contiguous tensor of the same shape, type and device, for a call on ``stream``."""
    if stream is None and like.is_contiguous():
        return torch.empty_like(like)  # the quickest of torch's ways
    return _empty(like.shape, like.dtype, like.device, stream)


def _stride(name, t):
    """Elements from one token of [B, T, C] to the next, 0 when contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    B, T, C = t.shape
    b, step, c = t.stride()
    if T == 1:
        step = b if B > 1 else C
    if (C > 1 and c != 1) or (B > 1 and T > 1 and b != T * step) or step < 1:
        raise ValueError(f"{name} needs contiguous channels and batch rows T token strides apart")
    return step


def _group_strides(name, t):
    """Token and group strides of [B, T, G, S], None when contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return None
    B, T, G, S = t.shape
    b, step, group, c = t.stride()
    if T == 1:
        step = b if B > 1 else G * S
    if G == 1:
        group = S
    if (S > 1 and c != 1) or (B > 1 and T > 1 and b != T * step) or min(step, group) < 1:
        raise ValueError(f"{name} needs contiguous states and batch rows T token strides apart")
    return (step, group)


def _seqs(B, cu_seqlens, index):
    """(N, flags, sequences, address of the offsets) of a call."""
    if cu_seqlens is None:
        return 0, 0, B, None
    wide = cu_seqlens.dtype is torch.int64
    if not wide and cu_seqlens.dtype is not torch.int32:
        raise TypeError(f"cu_seqlens must be int32 or int64, got {cu_seqlens.dtype}")
    n = cu_seqlens.numel() - 1
    return (n, GDR_SEQLENS_I64 if wide else 0, n,
            _like(index, cu_seqlens.dtype, (n + 1,), "cu_seqlens", cu_seqlens, True))


def _options(index, workspace, status, timer):
    if workspace is None and status is None and timer is None:
        return None
    _check_status(status, index)
    _on(index, workspace=(workspace, None))
    opt = gdr_options(workspace=None if workspace is None else workspace.data_ptr(),
                      status=None if status is None else status.data_ptr(),
                      workspace_bytes=0 if workspace is None
                      else workspace.numel() * workspace.element_size())
    if timer is not None:
        opt.events = ctypes.cast(timer._handles, ctypes.c_void_p)
        opt.max_launches = timer.max
        opt.launch_ids = ctypes.cast(timer._ids, ctypes.c_void_p)
        opt.n_launches = ctypes.cast(ctypes.pointer(timer._count), ctypes.c_void_p)
    return opt


def _call(fn, index, stream, tensors, *args):
    """The library's call on ``stream`` (default: the current one).  The memory of ``tensors`` is
    not handed out again before ``stream`` is through with them, whatever stream they were made
    on."""
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:  # torch holds a tensor there: it is initialised
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != 0:
        raise GdrError(rc)
    if stream is not None:
        for t in tensors:
            if t is not None and t.numel():
                t.record_stream(stream)


def _states(index, nseq, tail, dtype, h0, ht, state, state_indices, want, x, stream):
    """(ht, rows, addresses of h0, ht and the indices) of a call that goes on from ``h0`` [N, ...],
    or moves the pool ``state`` on in place."""
    if state is not None:
        if h0 is not None or ht is not None:
            raise ValueError("state is read and written in place: h0 and ht do not go with it")
        rows = state.shape[0]
        p = _like(index, dtype, (rows,) + tail, "state", state, True)
        if state_indices is None and rows < nseq:
            raise ValueError(f"state must have a row for each of {nseq} sequences")
        return state, rows, p, p, _like(index, torch.int32, (nseq,), "state_indices",
                                        state_indices, True)
    if state_indices is not None:
        raise ValueError("state_indices belong to state")
    shape = (nseq,) + tail
    if ht is None and want:
        ht = _empty(shape, dtype, x.device, stream)
    return (ht, nseq, _like(index, dtype, shape, "h0", h0, True),
            _like(index, dtype, shape, "ht", ht, True), None)


def _weight(index, dtype, shape, t, name="weight"):
    """(type, address) of a parameter of x's dtype or float32."""
    wt = t.dtype
    if wt is not dtype and wt is not torch.float32:
        raise TypeError(f"{name} must be {dtype} or float32, got {wt}")
    return _CODES[wt], _like(index, wt, shape, name, t, True)


_ACTIVATIONS = {None: 0, "silu": 1}


def _conv_call(name, x, weight, bias, cu_seqlens, activation, max_seqlen):
    """What both directions of the convolution share: (index, gdr_conv_dims, sequences, addresses
    of weight, bias and offsets)."""
    index, dtype = x.get_device(), x.dtype
    if index < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [B, T, C], weight [C, W]")
    B, T, C = x.shape
    W = weight.shape[1]
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    wd, w = _weight(index, dtype, (C, W), weight)
    n, flags, nseq, cu = _seqs(B, cu_seqlens, index)
    return index, gdr_conv_dims(B, T, C, W, n, _dtype_code(dtype), flags, wd, _ACTIVATIONS[activation],
                                0 if max_seqlen is None else max_seqlen, _stride("x", x)), nseq, w, \
        _like(index, weight.dtype, (C,), "bias", bias, True), cu


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
    (default: the current one) and not synchronised; outputs made here are then in memory of
    ``stream``, which is also kept for what the current stream has to do when they are let go."""
    lib = load_library()
    index, dims, nseq, w, b, cu = _conv_call("gdr_short_conv_fwd", x, weight, bias, cu_seqlens,
                                             activation, max_seqlen)
    opt = _options(index, None, status, timer)
    if y is None:
        y = _new(x, stream)
    else:
        _like(index, x.dtype, x.shape, "y", y)
        dims.y_stride = _stride("y", y)
    ht, rows, p0, pt, idx = _states(index, nseq, (weight.shape[1] - 1, x.shape[2]), x.dtype, h0, ht,
                                    state, state_indices, output_final_state, x, stream)
    _call(lib.gdr_short_conv_fwd, index, stream,
          (x, weight, bias, cu_seqlens, h0, ht, state_indices, y, status), dims, x.data_ptr(), w, b,
          cu, p0, pt, rows, idx, y.data_ptr(), opt)
    return y, ht


def gdr_short_conv_bwd(x, weight, dy, bias=None, cu_seqlens=None, h0=None, dht=None, *,
                       activation="silu", want_dh0=False, max_seqlen=None, workspace=None,
                       status=None, stream=None, timer=None):
    """Gradients of ``<dy, y> + <dht, ht>`` for :func:`gdr_short_conv_fwd` on the same inputs:
    ``(dx, dweight, dbias, dh0)``, dx and dh0 in x's dtype, dweight and dbias float32; dbias is None
    without a bias, dh0 unless ``want_dh0``."""
    lib = load_library()
    index, dims, nseq, w, b, cu = _conv_call("gdr_short_conv_bwd", x, weight, bias, cu_seqlens,
                                             activation, max_seqlen)
    opt = _options(index, workspace, status, timer)
    g = _like(index, x.dtype, x.shape, "dy", dy)
    dims.y_stride = _stride("dy", dy)
    tail = (nseq, weight.shape[1] - 1, x.shape[2])
    p0 = _like(index, x.dtype, tail, "h0", h0, True)
    gt = _like(index, x.dtype, tail, "dht", dht, True)
    dx = _new(x, stream)
    dw = _empty(weight.shape, torch.float32, x.device, stream)
    db = None if bias is None else _empty(bias.shape, torch.float32, x.device, stream)
    dh0 = _empty(tail, x.dtype, x.device, stream) if want_dh0 else None
    _call(lib.gdr_short_conv_bwd, index, stream,
          (x, weight, dy, bias, cu_seqlens, h0, dht, dx, dw, db, dh0, workspace, status), dims,
          x.data_ptr(), w, b, cu, p0, g, gt, dx.data_ptr(), dw.data_ptr(),
          None if db is None else db.data_ptr(), None if dh0 is None else dh0.data_ptr(), opt)
    return dx, dw, db, dh0


def _scan_call(name, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, softplus, max_seqlen):
    """What both directions of the scan share: (index, gdr_scan_dims, sequences, gdr_scan_tensors,
    address of the offsets)."""
    index, dtype = x.get_device(), x.dtype
    if index < 0:
        raise ValueError(f"{name} takes CUDA tensors")
    if x.dim() != 3 or A.dim() != 2 or B.dim() != 4:
        raise ValueError("x must be [B, T, C], A [C, S], B and C [B, T, groups, S]")
    shape = x.shape
    nb, T, ch = shape
    S, G = A.shape[1], B.shape[2]
    vec, bc = (ch,), (nb, T, G, S)
    n, flags, nseq, cu = _seqs(nb, cu_seqlens, index)
    tensors = gdr_scan_tensors(
        x.data_ptr(), _like(index, dtype, shape, "dt", dt),
        _like(index, torch.float32, (ch, S), "A", A, True), _like(index, dtype, bc, "B", B),
        _like(index, dtype, bc, "C", C), _like(index, torch.float32, vec, "D", D, True),
        _like(index, dtype, shape, "z", z), _like(index, torch.float32, vec, "dt_bias", dt_bias, True))
    dims = gdr_scan_dims(nb, T, ch, S, G, n, _dtype_code(dtype), flags, 1 if softplus else 0,
                         0 if max_seqlen is None else max_seqlen, _stride("x", x), _stride("dt", dt),
                         0 if z is None else _stride("z", z))
    strides = _group_strides("B", B)
    if strides:
        dims.b_stride[:] = strides
    strides = _group_strides("C", C)
    if strides:
        dims.c_stride[:] = strides
    return index, dims, nseq, tensors, cu


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
    index, dims, nseq, tensors, cu = _scan_call("gdr_selective_scan_fwd", x, dt, A, B, C, D, z,
                                                dt_bias, cu_seqlens, softplus, max_seqlen)
    opt = _options(index, workspace, status, timer)
    if y is None:
        y = _new(x, stream)
    else:
        _like(index, x.dtype, x.shape, "y", y)
        dims.y_stride = _stride("y", y)
    ht, rows, p0, pt, idx = _states(index, nseq, (x.shape[2], A.shape[1]), torch.float32, h0, ht,
                                    state, state_indices, output_final_state, x, stream)
    _call(lib.gdr_selective_scan_fwd, index, stream,
          (x, dt, A, B, C, D, z, dt_bias, cu_seqlens, h0, ht, state_indices, y, workspace, status),
          dims, tensors, cu, p0, pt, rows, idx, y.data_ptr(), n_segments, opt)
    return y, ht


def gdr_selective_scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, cu_seqlens=None,
                           h0=None, dht=None, *, softplus=True, want_dh0=False, max_seqlen=None,
                           workspace=None, status=None, stream=None, timer=None):
    """Gradients of ``<dy, y> + <dht, ht>`` for :func:`gdr_selective_scan_fwd` on the same
    inputs: ``(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)``, each in its input's dtype; None for
    an input that is None, dh0 unless ``want_dh0``."""
    lib = load_library()
    index, dims, nseq, tensors, cu = _scan_call("gdr_selective_scan_bwd", x, dt, A, B, C, D, z,
                                                dt_bias, cu_seqlens, softplus, max_seqlen)
    opt = _options(index, workspace, status, timer)
    g = _like(index, x.dtype, x.shape, "dy", dy)
    dims.y_stride = _stride("dy", dy)
    shape = (nseq, x.shape[2], A.shape[1])
    p0 = _like(index, torch.float32, shape, "h0", h0, True)
    gt = _like(index, torch.float32, shape, "dht", dht, True)

    def new(like):
        return None if like is None else _new(like, stream)

    dh0 = _empty(shape, torch.float32, x.device, stream) if want_dh0 else None
    out = (new(x), new(dt), new(A), new(B), new(C), new(D), new(z), new(dt_bias), dh0)
    grads = gdr_scan_grads(*[None if t is None else t.data_ptr() for t in out])
    _call(lib.gdr_selective_scan_bwd, index, stream,
          (x, dt, A, B, C, dy, D, z, dt_bias, cu_seqlens, h0, dht, workspace, status) + out, dims,
          tensors, cu, p0, g, gt, grads, opt)
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
        if s != need or step < 1:  # 0: a broadcast row, which is one row and not as many as there are
            raise ValueError(f"{name}: rows must lie at one stride, and not in one place")
        need *= n
    return shape[-1] if step is None else step


def gdr_rms_norm_fwd(x, weight=None, residual=None, *, eps=1e-6, dtype=None, group=0, y=None,
                     residual_out=None, scale=None, stream=None, timer=None):
    """Root-mean-square norm of the rows ``x`` [..., D], D up to 16384: with r = x + residual
    (rounded to x's dtype), y = r / sqrt(mean(r^2) + eps) * weight.  ``weight`` [D] is of x's dtype
    or float32.  ``dtype`` float8_e4m3fn or int8 quantises y, with a float32 scale for each row
    (``scale`` [...]) or, with ``group`` 128, for each 128 columns ([..., ceil(D / 128)]), as
    :func:`gdr_cache_write` does.  Returns ``(y, r, scale)``; r is None without a residual, scale
    unless y is quantised.  ``residual_out`` may be the residual or x itself, ``y`` x (in place).
    Rows may be slices of wider ones; one row broadcast to many is refused."""
    lib = load_library()
    index, own, shape = x.get_device(), x.dtype, x.shape
    if index < 0:
        raise ValueError("gdr_rms_norm_fwd takes CUDA tensors")
    code, D = _dtype_code(own), shape[-1]
    if dtype is None or dtype is own:
        out, out_code = own, code
    elif dtype in _OUT_DTYPES:
        out, out_code = dtype, _OUT_DTYPES[dtype]
    else:
        raise TypeError(f"dtype must be {own}, float8_e4m3fn or int8, got {dtype}")
    if group and (out is own or group != 128):
        raise ValueError("group is 0, or 128 where y is quantised")
    wd, w = (code, None) if weight is None else _weight(index, own, (D,), weight)
    if y is None:
        y = _new(x, stream) if out is own else _empty(shape, out, x.device, stream)
        ys = 0
    else:
        _like(index, out, shape, "y", y)
        ys = _row_stride("y", y)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out belongs to a residual")
        pr = po = None
        rs = os = 0
    else:
        pr = _like(index, own, shape, "residual", residual)
        rs = _row_stride("residual", residual)
        if residual_out is None:
            residual_out = _new(x, stream)
        po = _like(index, own, shape, "residual_out", residual_out)
        os = _row_stride("residual_out", residual_out)
    ps = None
    if out is not own:
        want = shape[:-1] + ((D + 127) // 128,) if group else shape[:-1]
        if scale is None:
            scale = _empty(want, torch.float32, x.device, stream)
        ps = _like(index, torch.float32, want, "scale", scale, True)
    elif scale is not None:
        raise ValueError("scale belongs to a quantised y")
    dims = gdr_norm_dims(x.numel() // D if D else 0, D, code, wd, out_code, group, eps,
                         _row_stride("x", x), rs, os, ys)
    _call(lib.gdr_rms_norm_fwd, index, stream, (x, residual, weight, residual_out, y, scale), dims,
          x.data_ptr(), pr, w, po, y.data_ptr(), ps, _options(index, None, None, timer))
    return y, residual_out, scale


def gdr_rms_norm_bwd(dy, r, weight=None, dr=None, *, eps=1e-6, workspace=None, stream=None,
                     timer=None):
    """Gradients of ``<dy, y> + <dr, r>`` for :func:`gdr_rms_norm_fwd` (y of x's dtype), from ``r``
    (its r, or its x without a residual): ``(dx, dweight)``; dx is the gradient of x and of the
    residual alike, dweight float32 (None without a weight)."""
    lib = load_library()
    index, dtype, shape = r.get_device(), r.dtype, r.shape
    if index < 0:
        raise ValueError("gdr_rms_norm_bwd takes CUDA tensors")
    code, D = _dtype_code(dtype), shape[-1]
    wd, w = (code, None) if weight is None else _weight(index, dtype, (D,), weight)
    g, gr = _like(index, dtype, shape, "dy", dy), _like(index, dtype, shape, "dr", dr)
    opt = _options(index, workspace, None, timer)
    dx = _new(r, stream)
    dw = None if weight is None else _empty((D,), torch.float32, r.device, stream)
    dims = gdr_norm_dims(r.numel() // D if D else 0, D, code, wd, code, 0, eps, _row_stride("r", r),
                         0 if dr is None else _row_stride("dr", dr), 0, _row_stride("dy", dy))
    _call(lib.gdr_rms_norm_bwd, index, stream, (dy, r, weight, dr, dx, dw, workspace), dims,
          r.data_ptr(), w, g, gr, dx.data_ptr(), None if dw is None else dw.data_ptr(), opt)
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
