"""The paged cache's entry points on the CPU: arguments that are refused
before any work, and the binding's checks.  No compute call is made."""
import ctypes

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from chunked_gated_delta_rule_gb300 import api


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_delta_rule_gb300 import build
    build.build()
    return pkg.load_library()


def _cache(dtype=api.GDR_BF16, H=2, **kw):
    c = api.gdr_paged_cache(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 10, 16, 4, H, dtype)
    for name, x in kw.items():
        if isinstance(x, tuple):
            getattr(c, name)[:] = x
        else:
            setattr(c, name, x)
    return c


def _p(x):
    return None if x is None else ctypes.c_void_p(0x10000 * x)


def _attn(lib, dims, cache, q=1, o=2, cu=None, window=0, opt=None):
    return lib.gdr_paged_attn(ctypes.byref(dims), None if cache is None else ctypes.byref(cache),
                              _p(q), _p(cu), _p(o), None, 1, window,
                              None if opt is None else ctypes.byref(opt), None)


def _rows(lib, name, dims, cache, k=1, v=2, cu=None):
    return getattr(lib, name)(ctypes.byref(dims), None if cache is None else ctypes.byref(cache),
                              _p(k), _p(v), _p(cu), None, None)


BAD_CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(page_table=None), -1), (dict(kv_lens=None), -1),
    (dict(n_pages=0), -1), (dict(page_size=0), -1), (dict(max_pages=0), -1), (dict(H=0), -1),
    (dict(dtype=api.GDR_F16), -1), (dict(dtype=7), -1),
    (dict(dtype=api.GDR_E4M3, k_scale=None), -1), (dict(dtype=api.GDR_I8, v_scale=None), -1),
    (dict(k_stride=(64, 0, 8)), -1), (dict(v_stride=(64, -1, 8)), -1),
    (dict(n_pages=1 << 31), -2), (dict(page_size=1 << 20, max_pages=1 << 12), -2),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad, code):
    dims = api.make_dims(1, 8, 2, 64, 64)
    assert _attn(lib, dims, _cache(**bad)) == code
    for name in ("gdr_cache_write", "gdr_cache_read"):
        assert _rows(lib, name, dims, _cache(**bad)) == code


def test_bad_calls(lib):
    ok, c = api.make_dims(1, 8, 4, 64, 64), _cache()
    assert _attn(lib, ok, None) == -1
    assert _attn(lib, ok, c, q=None) == -1 and _attn(lib, ok, c, o=None) == -1
    assert _attn(lib, ok, c, cu=3) == -1                                   # cu without N
    assert _attn(lib, api.make_dims(1, 8, 4, 64, 64, N=2), c) == -1        # N without cu
    assert _attn(lib, ok, c, window=-1) == -1
    assert _attn(lib, api.make_dims(1, 8, 3, 64, 64), c) == -1             # 3 heads over 2
    assert _attn(lib, api.make_dims(1, 8, 4, 60, 64), c) == -2             # K % 16
    assert _attn(lib, api.make_dims(1, 8, 4, 64, 512), c) == -2            # V > 256
    for opt in (api.gdr_options(float("nan")), api.gdr_options(-1.0),
                api.gdr_options(0.0, 4), api.gdr_options(0.0, -1), api.gdr_options(0.0, 0, 32)):
        assert _attn(lib, ok, c, opt=opt) == -1
    lim = api.gdr_options()
    lim.grid_limit = -1
    assert _attn(lib, ok, c, opt=lim) == -1
    bad_o = api.make_dims(1, 8, 4, 64, 64)
    bad_o.o_stride[:] = (64, 32)                                           # rows overlap
    assert _attn(lib, bad_o, c) == -1
    two = api.make_dims(1, 8, 2, 64, 64)
    for name in ("gdr_cache_write", "gdr_cache_read"):
        assert _rows(lib, name, two, c, k=None) == -1 and _rows(lib, name, two, c, v=None) == -1
        assert _rows(lib, name, ok, c) == -1                               # 4 heads into 2
        assert _rows(lib, name, two, c, cu=3) == -1
    over = api.make_dims(1, 8, 2, 64, 64)
    over.v_stride[:] = (32, 64)                                            # outputs overlap
    assert _rows(lib, "gdr_cache_read", over, c) == -1
    over.v_stride[:] = (0, 0)
    over.k_stride[:] = (32, 64)
    assert _rows(lib, "gdr_cache_read", over, c) == -1


def test_empty_calls_do_nothing(lib):
    c = _cache()
    assert _attn(lib, api.make_dims(1, 0, 4, 64, 64), c) == 0
    for name in ("gdr_cache_write", "gdr_cache_read"):
        assert _rows(lib, name, api.make_dims(1, 0, 2, 64, 64), c) == 0


def test_workspace_size(lib):
    dims, c = api.make_dims(1, 8, 4, 128, 128), _cache()
    assert lib.gdr_attn_workspace_size(ctypes.byref(dims), ctypes.byref(c)) > 0
    assert lib.gdr_attn_workspace_size(ctypes.byref(dims), ctypes.byref(_cache(dtype=9))) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkg.gdr_cache_write(x, x, c, c, table, lens)
    with pytest.raises(ValueError):
        pkg.gdr_cache_read(c, c, table, lens, 4)
    with pytest.raises(ValueError):
        pkg.gdr_paged_attn(x, c, c, table, lens)


def test_binding_checks_caches():
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    good = dict(k_cache=c, v_cache=c, page_table=table, kv_lens=lens, k_scale=None, v_scale=None,
                nseq=1, index=-1)
    api._cache_of(**good)
    scale = torch.zeros(3, 2, 16)
    for bad, err in ((dict(v_cache=c.float()), TypeError), (dict(k_cache=c.double()), TypeError),
                     (dict(k_cache=c[0]), ValueError), (dict(v_cache=c[:2]), ValueError),
                     (dict(k_cache=c.transpose(2, 3)), ValueError),
                     (dict(k_scale=scale, v_scale=scale), ValueError),
                     (dict(k_cache=c.to(torch.int8), v_cache=c.to(torch.int8)), ValueError),
                     (dict(k_cache=c.to(torch.int8), v_cache=c.to(torch.int8), k_scale=scale,
                           v_scale=scale[:, :, :8].contiguous()), ValueError),
                     (dict(page_table=table.long()), TypeError),
                     (dict(page_table=table[0]), ValueError), (dict(nseq=2), ValueError),
                     (dict(kv_lens=lens.float()), TypeError)):
        with pytest.raises(err):
            api._cache_of(**{**good, **bad})


def test_empty_tensors_need_no_address(lib):
    """A tensor without elements has none."""
    c = _cache()
    assert _attn(lib, api.make_dims(1, 0, 4, 64, 64), c, q=None, o=None) == 0
    assert _attn(lib, api.make_dims(1, 0, 4, 64, 64, N=2), c, q=None, o=None, cu=3) == 0
    assert _attn(lib, api.make_dims(1, 0, 3, 64, 64), c, q=None, o=None) == -1  # 3 heads over 2
    for name in ("gdr_cache_write", "gdr_cache_read"):
        assert _rows(lib, name, api.make_dims(1, 0, 2, 64, 64), c, k=None, v=None) == 0
        assert _rows(lib, name, api.make_dims(1, 0, 2, 64, 64), None, k=None, v=None) == -1


def test_attention_refuses_positions_that_steps_would_pass(lib):
    """A step's positions are 32-bit numbers too, up to 127 past the last: tables
    of more than 2^31 - 1024 positions are refused."""
    dims = api.make_dims(1, 8, 2, 64, 64)
    for page, pages in ((1, (1 << 31) - 1), (16, (1 << 27) - 1), ((1 << 31) - 1, 1)):
        assert _attn(lib, dims, _cache(page_size=page, max_pages=pages)) == -2
