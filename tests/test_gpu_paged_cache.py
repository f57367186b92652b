"""The paged cache on the GPU: writing (quantising) and reading back against
the 64-bit forms; untouched slots keep their bits."""
import math

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from paged_ref import CACHE, IO, Batch, quantise

pytestmark = pytest.mark.gpu


def _write(b, k, v, kc, vc, ks, vs, status=None, cu="own"):
    pkg.gdr_cache_write(k, v, kc, vc, b.on("table"), b.on("lens"),
                        (None if b.dense else b.on("cu")) if isinstance(cu, str) else cu,
                        k_scale=ks, v_scale=vs, status=status)


def _expected(b):
    """Cache contents after the write, on the CPU: values as float64 / raw."""
    kc, vc = b.kc.clone(), b.vc.clone()
    ks, vs = (None if s is None else s.clone() for s in (b.ks, b.vs))
    t = 0
    k, v = b.k.reshape(-1, b.Hk, b.K), b.v.reshape(-1, b.Hk, b.V)
    for i, (a, n) in enumerate(zip(b.q_lens, b.kv_lens)):
        for j in range(a):
            p = n - a + j
            if p >= 0:
                page, slot = int(b.table[i, p // b.page]), p % b.page
                for x, c, s in ((k[t + j], kc, ks), (v[t + j], vc, vs)):
                    if s is None:
                        c[page, slot] = x
                    else:
                        q, sc = quantise(x, b.fmt)
                        c[page, slot] = q.float().to(CACHE[b.fmt])
                        s[page, :, slot] = sc
        t += a
    return kc, vc, ks, vs


def _same(a, b):
    """Bit equality, NaN equal to NaN."""
    a, b = a.cpu(), b.cpu()
    if a.dtype == torch.float8_e4m3fn:
        a, b = a.view(torch.uint8), b.view(torch.uint8)
        return bool((a == b).all())
    return torch.equal(a.nan_to_num(nan=12345.0) if a.is_floating_point() else a,
                       b.nan_to_num(nan=12345.0) if b.is_floating_point() else b)


LENS = [([1], [1]), ([5, 0, 17, 1], [5, 3, 40, 33]), ([64, 3], [64, 130]), ([40, 7], [33, 7])]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_write_then_read(dtype, fmt, lens):
    b = Batch(*lens, K=64, V=112, heads=3, kv_heads=3, page=12, dtype=dtype, fmt=fmt)
    kc, vc, ks, vs = (b.on(x) for x in ("kc", "vc", "ks", "vs"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _write(b, b.on("k"), b.on("v"), kc, vc, ks, vs, status)
    ekc, evc, eks, evs = _expected(b)
    assert int(status) == 0
    assert _same(kc, ekc) and _same(vc, evc)
    if fmt != "same":
        assert _same(ks, eks) and _same(vs, evs)
    k, v = pkg.gdr_cache_read(kc, vc, b.on("table"), b.on("lens"), b.T, b.on("cu"), k_scale=ks,
                              v_scale=vs, dtype=IO[dtype], status=status)
    assert int(status) == 0
    t = 0
    for i, (a, n) in enumerate(zip(b.q_lens, b.kv_lens)):
        for j in range(a):
            p = n - a + j
            for got, src in ((k, b.k), (v, b.v)):
                x = src[0, t + j]
                if p < 0:
                    want = torch.zeros_like(x)
                elif fmt == "same":
                    want = x
                else:
                    q, s = quantise(x, fmt)
                    want = (q.float() * s[..., None]).to(IO[dtype])
                assert _same(got[0, t + j], want), (i, j)
        t += a


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_without_a_scale(fmt):
    """Zero rows, a row of the type's smallest values, rows with NaN or
    infinities, a row of the largest ones."""
    b = Batch([6], [6], K=32, kv_heads=1, heads=1, dtype="bf16", fmt=fmt)
    b.k[0, 0] = 0
    b.k[0, 1] = 2.0 ** -133  # BF16's smallest subnormal: the scale underflows
    b.k[0, 2, 0, 5] = math.nan
    b.k[0, 3, 0, 31] = math.inf
    b.k[0, 4] = torch.finfo(torch.bfloat16).max
    kc, vc, ks, vs = (b.on(x) for x in ("kc", "vc", "ks", "vs"))
    _write(b, b.on("k"), b.on("v"), kc, vc, ks, vs)
    k, _ = pkg.gdr_cache_read(kc, vc, b.on("table"), b.on("lens"), 6, b.on("cu"), k_scale=ks,
                              v_scale=vs)
    k = k.cpu().float()
    assert (k[0, 0] == 0).all()
    assert k[0, 1].abs().max() <= 2.0 ** -130
    assert k[0, 2].isnan().all() and k[0, 3].isnan().all()
    # the scale is rounded: within a unit of BF16 of the largest value
    assert (k[0, 4] / torch.finfo(torch.bfloat16).max - 1).abs().max() <= 2.0 ** -8
    ekc, _, eks, _ = _expected(b)
    assert _same(kc, ekc) and _same(ks, eks)


@pytest.mark.parametrize("offset", [0, 1])
def test_strided_rows_and_pages(offset):
    """k and v as slices of one projection, head-major pages, keys and values
    side by side; ``offset`` one element off a 16-byte boundary."""
    b = Batch([9, 20], [25, 20], K=64, heads=4, kv_heads=2, page=8, dtype="bf16", fmt="same")
    fused = torch.randn(1, b.T, 3, 2, 64 + 8).to(torch.bfloat16).cuda()
    k, v = fused[:, :, 1, :, offset:offset + 64], fused[:, :, 2, :, offset:offset + 64]
    pages = torch.zeros(b.n_pages, 2, b.Hk, b.page, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = pages[:, 0].transpose(1, 2), pages[:, 1].transpose(1, 2)
    _write(b, k, v, kc, vc, None, None)
    ref_k, ref_v = torch.zeros_like(kc).contiguous(), torch.zeros_like(vc).contiguous()
    _write(b, k.contiguous(), v.contiguous(), ref_k, ref_v, None, None)
    assert torch.equal(kc, ref_k) and torch.equal(vc, ref_v)
    out = torch.zeros(1, b.T, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    pkg.gdr_cache_read(kc, vc, b.on("table"), b.on("lens"), b.T, b.on("cu"), k=out[:, :, 0],
                       v=out[:, :, 1])
    assert torch.equal(out[:, :, 0], k) and torch.equal(out[:, :, 1], v)


def test_dense_rows_and_int64_offsets():
    b = Batch([3, 3], [10, 4], K=128, dtype="f16", fmt="int8", dense=True)
    c1 = [b.on(x) for x in ("kc", "vc", "ks", "vs")]
    c2 = [x.clone() for x in c1]
    _write(b, b.on("k"), b.on("v"), *c1)
    flat = [x.reshape(1, 6, b.Hk, -1) for x in (b.on("k"), b.on("v"))]
    _write(b, *flat, *c2, cu=b.on("cu").long())
    for x, y in zip(c1, c2):
        assert _same(x, y)


def test_bad_tables_touch_nothing_and_are_reported():
    """A page outside the cache, a length past the table: reported, and only
    the tokens concerned are skipped."""
    b = Batch([4, 4], [4, 4], K=32, page=4, dtype="bf16")
    kc, vc = b.on("kc").nan_to_num(), b.on("vc").nan_to_num()
    before = kc.clone()
    for table, lens in (([[b.n_pages], [0]], [4, 4]), ([[-1], [0]], [4, 4]),
                        ([[1], [0]], [2 ** 30, 4])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kc.copy_(before)
        pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc,
                            torch.tensor(table, dtype=torch.int32).cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), b.on("cu"), status=status)
        assert int(status) == -7
        assert torch.equal(kc[0], b.k[0, 4:].cuda())
        assert torch.equal(kc[1:], before[1:])


def test_bad_offsets_are_reported():
    b = Batch([4, 4], [4, 4], K=32, page=4, dtype="bf16")
    kc, vc = b.on("kc").nan_to_num(), b.on("vc").nan_to_num()
    for cu in ([0, 9, 8], [0, 4, 100], [3, 4, 8]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc, b.on("table"), b.on("lens"),
                            torch.tensor(cu, dtype=torch.int32).cuda(), status=status)
        assert int(status) == -5


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: its last pages are written and read
    at their own places."""
    page, H, D = 128, 8, 128
    n_pages = (1 << 32) // (page * H * D) + 3
    kc = torch.zeros(n_pages, page, H, D, dtype=torch.int8, device="cuda")
    vc = torch.zeros(n_pages, page, H, D, dtype=torch.int8, device="cuda")
    ks = torch.zeros(n_pages, H, page, device="cuda")
    vs = torch.zeros(n_pages, H, page, device="cuda")
    table = torch.tensor([[n_pages - 1, n_pages // 2 + 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(1, 200, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    pkg.gdr_cache_write(k, v, kc, vc, table, lens, k_scale=ks, v_scale=vs)
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        q, sc = quantise(x[0].cpu(), "int8")
        got = torch.cat([c[n_pages - 1], c[n_pages // 2 + 1][:72]]).cpu()
        assert torch.equal(got.double(), q)
        assert torch.equal(torch.cat([s[n_pages - 1].T, s[n_pages // 2 + 1].T[:72]]).cpu(), sc)
        for low in (0, 1, 2):
            assert not bool(c[low].any())
