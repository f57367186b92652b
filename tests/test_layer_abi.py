"""The entry points of the short convolution, the selective scan and the norm on the CPU:
arguments that are refused before any work, scratch sizes, and the binding's checks.  No compute
call is made."""
import ctypes

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from chunked_gated_delta_rule_gb300 import api

BF16, F32, F16, E4M3, I8 = api.GDR_BF16, api.GDR_F32, api.GDR_F16, api.GDR_E4M3, api.GDR_I8


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_delta_rule_gb300 import build
    build.build()
    return pkg.load_library()


def _p(x):
    return None if x is None else ctypes.c_void_p(0x10000 * x)


def _with(struct, **kw):
    for name, x in kw.items():
        if isinstance(x, tuple):
            getattr(struct, name)[:] = x
        else:
            setattr(struct, name, x)
    return struct


def conv(**kw):
    return _with(api.gdr_conv_dims(1, 64, 128, 4, 0, BF16, 0, BF16, 1), **kw)


def scan(**kw):
    return _with(api.gdr_scan_dims(1, 64, 128, 16, 1, 0, BF16, 0, 1), **kw)


def norm(**kw):
    return _with(api.gdr_norm_dims(64, 128, BF16, BF16, BF16, 0, 1e-6), **kw)


def conv_fwd(lib, d, x=1, w=2, b=None, cu=None, h0=None, ht=None, rows=0, idx=None, y=3, opt=None):
    return lib.gdr_short_conv_fwd(d, _p(x), _p(w), _p(b), _p(cu), _p(h0), _p(ht), rows, _p(idx), _p(y),
                                  opt, None)


def conv_bwd(lib, d, x=1, w=2, b=None, cu=None, dy=3, dx=4, dw=5, db=None, opt=None):
    return lib.gdr_short_conv_bwd(d, _p(x), _p(w), _p(b), _p(cu), None, _p(dy), None, _p(dx), _p(dw), _p(db),
                                  None, opt, None)


BAD_CONV = [(dict(B=0), -1), (dict(T=-1), -1), (dict(C=0), -1), (dict(W=1), -1), (dict(W=5), -2),
            (dict(dtype=E4M3), -1), (dict(weight_dtype=F16), -1), (dict(activation=2), -1),
            (dict(flags=2), -1), (dict(N=-1), -1), (dict(B=2, N=2), -1), (dict(max_len=-1), -1),
            (dict(x_stride=-8), -1), (dict(y_stride=64), -1), (dict(T=1 << 31), -2),
            (dict(C=1 << 30), -2), (dict(N=2), -1)]


@pytest.mark.parametrize("bad,code", BAD_CONV, ids=str)
def test_bad_convolutions(lib, bad, code):
    assert conv_fwd(lib, conv(**bad)) == code
    assert conv_bwd(lib, conv(**bad)) == code


def test_bad_convolution_calls(lib):
    ok = conv()
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(cu=9), dict(h0=4, rows=0), dict(ht=4),
               dict(idx=5)):
        assert conv_fwd(lib, ok, **kw) == -1, kw
    assert conv_fwd(lib, conv(B=3), h0=4, ht=4, rows=2) == -1       # row n for 3 sequences
    for kw in (dict(x=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(cu=9),
               dict(db=6)):
        assert conv_bwd(lib, ok, **kw) == -1, kw
    for opt in (api.gdr_options(1.0), api.gdr_options(0.0, 1), api.gdr_options(0.0, 0, 16)):
        assert conv_fwd(lib, ok, opt=opt) == -1 and conv_bwd(lib, ok, opt=opt) == -1
    assert conv_bwd(lib, ok, opt=_with(api.gdr_options(), workspace=0x1000000, workspace_bytes=16)) == -6
    assert conv_bwd(lib, ok, opt=_with(api.gdr_options(), workspace=0x1000010, workspace_bytes=1 << 30)) == -1


def scan_in(**kw):
    t = api.gdr_scan_tensors(*(0x10000 * i for i in range(1, 9)))
    return _with(t, **kw)


def scan_fwd(lib, d, t=None, cu=None, h0=None, ht=None, rows=0, idx=None, y=9, segments=0, opt=None):
    return lib.gdr_selective_scan_fwd(d, t or scan_in(), _p(cu), _p(h0), _p(ht), rows, _p(idx), _p(y),
                                      segments, opt, None)


def scan_bwd(lib, d, t=None, cu=None, dy=9, opt=None, **kw):
    g = _with(api.gdr_scan_grads(*(0x100000 * i for i in range(1, 10))), **kw)
    return lib.gdr_selective_scan_bwd(d, t or scan_in(), _p(cu), None, _p(dy), None, g, opt, None)


BAD_SCAN = [(dict(B=0), -1), (dict(T=-1), -1), (dict(C=0), -1), (dict(S=0), -1), (dict(S=65), -2),
            (dict(G=0), -1), (dict(G=3), -1), (dict(dtype=I8), -1), (dict(softplus=2), -1),
            (dict(N=-1), -1), (dict(B=2, N=2), -1), (dict(N=2), -1), (dict(max_len=-1), -1),
            (dict(dt_stride=-1), -1), (dict(y_stride=100), -1), (dict(b_stride=(16, 0)), -1),
            (dict(c_stride=(0, 16)), -1), (dict(T=1 << 31), -2), (dict(C=1 << 27), -2)]


@pytest.mark.parametrize("bad,code", BAD_SCAN, ids=str)
def test_bad_scans(lib, bad, code):
    assert scan_fwd(lib, scan(**bad)) == code
    assert scan_bwd(lib, scan(**bad)) == code
    if bad != dict(N=2):  # which lacks but its offsets
        assert lib.gdr_selective_scan_bwd_workspace_size(scan(**bad)) == 0


def test_bad_scan_calls(lib):
    ok = scan()
    for name in ("x", "dt", "A", "B", "C"):
        assert scan_fwd(lib, ok, scan_in(**{name: None})) == -1, name
        assert scan_bwd(lib, ok, scan_in(**{name: None})) == -1, name
    for kw in (dict(y=None), dict(cu=9), dict(h0=4, rows=0), dict(idx=5), dict(segments=-1)):
        assert scan_fwd(lib, ok, **kw) == -1, kw
    for kw in (dict(dy=None), dict(cu=9), dict(dx=None), dict(ddt=None), dict(dA=None), dict(dB=None),
               dict(dC=None), dict(dz=None)):
        assert scan_bwd(lib, ok, **kw) == -1, kw
    # gradients of what is not there
    for name, grad in (("D", "dD"), ("z", "dz"), ("dt_bias", "ddt_bias")):
        assert scan_bwd(lib, ok, scan_in(**{name: None})) == -1, grad
    assert scan_bwd(lib, ok, opt=_with(api.gdr_options(), workspace=0x1000000, workspace_bytes=256)) == -6
    assert scan_fwd(lib, ok, opt=api.gdr_options(2.0)) == -1


def norm_fwd(lib, d, x=1, res=None, w=2, out=None, y=3, scale=None, opt=None):
    return lib.gdr_rms_norm_fwd(d, _p(x), _p(res), _p(w), _p(out), _p(y), _p(scale), opt, None)


def test_bad_norms(lib):
    for bad, code in ((dict(rows=-1), -1), (dict(D=0), -1), (dict(D=16385), -2), (dict(dtype=I8), -1),
                      (dict(weight_dtype=F16), -1), (dict(out_dtype=F32), -1), (dict(eps=-1.0), -1),
                      (dict(eps=float("nan")), -1), (dict(group=128), -1), (dict(x_stride=64), -1),
                      (dict(sum_stride=-1), -1)):
        assert norm_fwd(lib, norm(**bad)) == code, bad
        assert lib.gdr_rms_norm_bwd(norm(**bad), _p(1), _p(2), _p(3), None, _p(4), _p(5), None, None) == code, bad
    ok, q = norm(), norm(out_dtype=E4M3)
    for kw in (dict(x=None), dict(y=None), dict(res=4), dict(out=4), dict(scale=5)):
        assert norm_fwd(lib, ok, **kw) == -1, kw
    assert norm_fwd(lib, q) == -1                                    # a scale is wanted
    assert norm_fwd(lib, ok, res=4, out=3, y=3) == -1                # two outputs in one place
    assert norm_fwd(lib, q, y=1, scale=5) == -1                      # 8 bits over rows to be read
    assert norm_fwd(lib, q, res=4, out=6, y=4, scale=5) == -1
    assert norm_fwd(lib, norm(out_dtype=E4M3, group=64), scale=5) == -1
    bwd = lambda d, r=1, w=2, dy=3, dx=4, dw=5, opt=None: lib.gdr_rms_norm_bwd(  # noqa: E731
        d, _p(r), _p(w), _p(dy), None, _p(dx), _p(dw), opt, None)
    for kw in (dict(r=None), dict(dy=None), dict(dx=None), dict(w=None)):
        assert bwd(ok, **kw) == -1, kw
    assert bwd(q) == -1
    assert bwd(ok, opt=_with(api.gdr_options(), workspace=0x1000000, workspace_bytes=16)) == -6


def test_outputs_in_the_place_of_inputs(lib):
    assert conv_fwd(lib, conv(), y=1) == -1
    assert conv_bwd(lib, conv(), dx=1) == -1 and conv_bwd(lib, conv(), dx=3) == -1
    ins = scan_in()
    for name in ("x", "dt", "z", "B", "C"):
        assert scan_fwd(lib, scan(), y=getattr(ins, name) // 0x10000) == -1, name
        for out in ("dx", "ddt", "dB", "dC", "dz"):
            assert scan_bwd(lib, scan(), **{out: getattr(ins, name)}) == -1, (name, out)
    assert scan_bwd(lib, scan(), dx=0x10000 * 9) == -1               # dy
    # rows of the norm at another stride
    assert norm_fwd(lib, norm(x_stride=256), y=1) == -1
    assert norm_fwd(lib, norm(sum_stride=256), res=4, out=4) == -1
    assert norm_fwd(lib, norm(sum_stride=256), res=4, out=1) == -1
    assert norm_fwd(lib, norm(y_stride=256), res=4, out=6, y=4) == -1


def test_scratch_sizes(lib):
    from chunked_gated_delta_rule_gb300 import layer
    conv_ws = layer.gdr_short_conv_bwd_workspace_size
    assert 0 < conv_ws(1, 1000, 512, 4) and conv_ws(1, 1000, 512, 5) == 0
    assert conv_ws(1, 0, 512, 4) == 0                                # no tokens, no sums
    size = layer.gdr_selective_scan_workspace_size
    assert size(1, 16384, 2048, 16) > 0                              # one long sequence is cut
    assert size(64, 256, 2048, 16) == 0                              # many are run whole
    assert size(1, 16384, 2048, 16, n_segments=1) == 0
    back = size(1, 16384, 2048, 16, backward=True)
    assert back > 2 * (16384 // 64) * 2048 * 16 * 4
    assert size(1, 32768, 2048, 16, backward=True) > back
    assert size(1, 100, 2048, 65) == 0
    assert layer.gdr_rms_norm_bwd_workspace_size(1000, 512) >= 512 * 4
    assert layer.gdr_rms_norm_bwd_workspace_size(1000, 20000) == 0


def test_binding_rejects_host_tensors():
    x, w = torch.zeros(1, 8, 32), torch.zeros(32, 4)
    A, bc = torch.zeros(32, 16), torch.zeros(1, 8, 1, 16)
    for call in (lambda: pkg.gdr_short_conv_fwd(x, w), lambda: pkg.gdr_short_conv_bwd(x, w, x),
                 lambda: pkg.gdr_selective_scan_fwd(x, x, A, bc, bc),
                 lambda: pkg.gdr_selective_scan_bwd(x, x, A, bc, bc, x),
                 lambda: pkg.gdr_rms_norm_fwd(x), lambda: pkg.gdr_rms_norm_bwd(x, x),
                 lambda: pkg.short_conv(x, w), lambda: pkg.rms_norm(x)):
        with pytest.raises(ValueError):
            call()


def test_kernel_names():
    names = [pkg.gdr_kernel_name(i) for i in range(39, 56)]
    assert "?" not in names and len(set(names)) == len(names)
    assert pkg.gdr_kernel_name(56) == "?"
