"""Attention over the paged cache on the GPU against the 64-bit form, on every
route that takes the case."""
import math

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from paged_ref import Batch, check

pytestmark = pytest.mark.gpu

ROUTES = [1, 2, 3]

# (new tokens, cached tokens with them): one token, none, odd chunks, a chunk
# longer than the cache (its first rows see nothing), pages ending in tiles
LENS = {
    "one": ([1], [1]),
    "mixed": ([3, 0, 1, 70, 5], [3, 9, 131, 200, 0]),
    "short": ([20, 2], [13, 64]),
    "long": ([130], [700]),
}


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype,fmt", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                       ("bf16", "int8"), ("f16", "e4m3"), ("f16", "int8")])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("heads,kv_heads,K,page", [(4, 2, 128, 16), (6, 2, 64, 24)])
def test_types_and_lengths(route, dtype, fmt, lens, heads, kv_heads, K, page):
    b = Batch(*LENS[lens], heads=heads, kv_heads=kv_heads, K=K, page=page, dtype=dtype, fmt=fmt)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {dtype} {fmt} {lens}")


@pytest.mark.parametrize("fmt", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("K,V", [(16, 16), (48, 208), (256, 256), (128, 64)])
def test_fp32_and_other_widths(fmt, K, V):
    b = Batch([3, 40], [50, 40], heads=3, kv_heads=1, K=K, V=V, dtype="f32", fmt=fmt, page=5)
    check(b, *b.run(), *b.attention(), label=f"f32 {fmt} {K} {V}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 37, 1000])
def test_masks(route, causal, window):
    b = Batch([1, 60, 9], [333, 150, 5], heads=8, kv_heads=2, dtype="bf16", page=32)
    check(b, *b.run(force_path=route, causal=causal, window=window),
          *b.attention(causal, window), label=f"{route} {causal} {window}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", ["same", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (16, 1), (32, 1), (12, 4), (16, 16)])
def test_shared_heads(route, fmt, heads, kv_heads):
    b = Batch([1, 6], [300, 50], heads=heads, kv_heads=kv_heads, dtype="bf16", fmt=fmt, page=16)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {heads}/{kv_heads}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("q_len", [1, 4, 64])
def test_long_axis(route, q_len):
    """Few rows over a long context: the axis is split and joined."""
    b = Batch([q_len], [5003], heads=4, kv_heads=1, dtype="bf16", page=64)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {q_len}")


@pytest.mark.parametrize("route", ROUTES)
def test_many_sequences(route):
    """More sequences than threads, most of them short, some empty."""
    kv = [(37 * i) % 90 for i in range(700)]
    q = [min(k, 1 + i % 2) for i, k in enumerate(kv)]
    b = Batch(q, kv, heads=2, kv_heads=1, K=64, dtype="f16", page=16)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("size", [0.01, 30.0])
def test_sharp_and_flat_softmax(route, size):
    """Scores so far apart that one key takes a row, and nearly equal ones,
    with the largest at either end of the axis."""
    b = Batch([40], [400], heads=2, kv_heads=1, dtype="bf16", page=16)
    b.q = (b.q * size).to(b.q.dtype)
    order = torch.arange(400)
    for sign in (1, -1):
        grow = torch.exp(sign * 0.004 * (order - 200).float())
        pages = b.table[0, order // b.page].long()
        b.kc[pages, order % b.page] = (b.kc[pages, order % b.page].float() *
                                       grow[:, None, None]).to(b.kc.dtype)
        check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {size} {sign}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["same", "e4m3", "int8"])
def test_uneven_query_rows(route, dtype, fmt):
    """One column 2^6 times the others, rows near the least and the largest
    magnitudes, rows of zeros: the same bounds."""
    b = Batch([70], [300], heads=4, kv_heads=1, dtype=dtype, fmt=fmt, page=16)
    b.q[:, 0::5, :, 9] *= 64
    b.q[:, 0::5] /= 16
    b.q[:, 1::5] *= 2.0 ** (-120 if dtype == "bf16" else -20)
    b.q[:, 2::5] = 0
    o, lse = b.run(force_path=route)
    check(b, o, lse, *b.attention(), label=f"{route} {dtype} {fmt}")
    b.q[:, 3, 1, 7], b.q[:, 4, 2, 7], b.q[:, 8, 3, 0] = math.nan, math.inf, -math.inf
    bad, _ = b.run(force_path=route)
    rows = [(3, 1), (4, 2), (8, 3)]
    for t, h in rows:
        assert bad[t, h].isnan().all() or not torch.isfinite(bad[t, h]).all()
    keep = torch.ones(70, 4, dtype=torch.bool)
    for t, h in rows:
        keep[t, h] = False
    assert torch.equal(bad.cpu()[keep], o.cpu()[keep])


@pytest.mark.parametrize("route", ROUTES)
def test_masked_places_never_reach_a_row(route):
    """NaN and infinities at positions that only later rows see: the rows
    before them are exact, the rows that see them are not finite."""
    b = Batch([50], [150], heads=2, kv_heads=1, dtype="bf16", page=16)
    ref_o, ref_lse = b.attention()
    at = 120  # token 20 of the call
    page, slot = int(b.table[0, at // 16]), at % 16
    b.vc[page, slot, 0, 3] = math.inf
    b.vc[page, slot, 0, 7] = math.nan
    o, lse = b.run(force_path=route)
    check(b, o[:20], lse[:20], ref_o[:20], ref_lse[:20], label="before")
    assert not torch.isfinite(o[20:, :, 3]).any() and o[20:, :, 7].isnan().all()
    keep = [d for d in range(128) if d not in (3, 7)]
    assert torch.isfinite(o[20:][..., keep]).all()
    b.kc[page, slot, 0, 3] = math.nan
    o, lse = b.run(force_path=route)
    check(b, o[:20], lse[:20], ref_o[:20], ref_lse[:20], label="before, key")
    assert o[20:].isnan().all() and lse[20:].isnan().all()


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_rows_without_a_scale(route, dtype, fmt):
    """8-bit rows stored without a scale (they held a NaN): the rows that see
    them are NaN, the others exact; scales that differ by 2^40 between tokens,
    and rows of zeros."""
    b = Batch([50], [150], heads=2, kv_heads=1, dtype=dtype, fmt=fmt, page=16)
    tokens = torch.arange(150)
    pages, slots = b.table[0, tokens // 16].long(), tokens % 16
    b.vs[pages, 0, slots] *= 2.0 ** ((tokens % 5) * -10).float()
    b.vs[pages[7:9], 0, slots[7:9]] = 0
    b.ks[pages[9], 0, slots[9]] = 0
    ref_o, ref_lse = b.attention()
    for which in ("vs", "ks"):
        keep = getattr(b, which).clone()
        getattr(b, which)[pages[120], 0, slots[120]] = math.nan
        o, lse = b.run(force_path=route)
        check(b, o[:20], lse[:20], ref_o[:20], ref_lse[:20], label=f"{which} before")
        assert o[20:].isnan().all()
        setattr(b, which, keep)
    check(b, *b.run(force_path=route), ref_o, ref_lse, label="all")


@pytest.mark.parametrize("route", ROUTES)
def test_strides_layouts_and_outputs(route):
    """q a slice of a fused projection, o a slice of a wider tensor, head-major
    pages; bits equal to the contiguous call's."""
    b = Batch([9, 1, 33], [90, 64, 33], heads=4, kv_heads=2, dtype="bf16", page=16)
    o, lse = b.run(force_path=route)
    fused = torch.zeros(1, b.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, :, 2:6] = b.on("q")
    wide = torch.zeros(1, b.T, 4, 256, dtype=torch.bfloat16, device="cuda")
    kc, vc = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (b.on("kc"), b.on("vc")))
    o2, lse2 = b.run(force_path=route, q=fused[:, :, 2:6], o=wide[..., 128:], kc=kc, vc=vc)
    assert torch.equal(o, o2.reshape(o.shape)) and torch.equal(lse, lse2)
    assert (wide[..., :128] == 0).all()


def test_misaligned_views_take_a_route():
    """Bases and strides off 16-byte boundaries."""
    b = Batch([9, 33], [90, 33], heads=4, kv_heads=2, dtype="bf16", page=16)
    q = torch.zeros(1, b.T, 4, 129, dtype=torch.bfloat16, device="cuda")
    q[..., 1:] = b.on("q")
    kc = torch.zeros(b.n_pages, 16, 2, 129, dtype=torch.bfloat16, device="cuda")
    kc[..., 1:] = b.on("kc")
    ref = b.attention()
    check(b, *b.run(q=q[..., 1:]), *ref, label="q")
    check(b, *b.run(kc=kc[..., 1:]), *ref, label="k")
    o = torch.zeros(1, b.T, 4, 131, dtype=torch.bfloat16, device="cuda")[..., 3:]
    check(b, *b.run(o=o), *ref, label="o")


@pytest.mark.parametrize("route", ROUTES)
def test_repeats_grids_streams_and_graphs(route):
    b = Batch([5, 130, 1], [900, 400, 1500], heads=8, kv_heads=2, dtype="bf16", page=16)
    args = [b.on(x) for x in ("q", "kc", "vc", "table", "lens", "cu")]
    o, lse = b.run(force_path=route)
    o2, lse2 = b.run(force_path=route)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ref = b.attention()
    for limit in (1, 7):  # another split of the axis: another order of sums
        check(b, *b.run(force_path=route, grid_limit=limit), *ref, label=f"grid {limit}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, lse3 = pkg.gdr_paged_attn(*args, force_path=route, stream=side)
    side.synchronize()
    assert torch.equal(o, o3.reshape(o.shape))
    out = torch.zeros_like(o3), torch.zeros_like(lse3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            pkg.gdr_paged_attn(*args, force_path=route, o=out[0], lse=out[1])
    for _ in range(2):
        out[0].zero_()
        out[1].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out[0].reshape(o.shape)) and torch.equal(lse, out[1].reshape(lse.shape))


@pytest.mark.parametrize("route", ROUTES)
def test_dense_rows_hints_and_scale(route):
    b = Batch([2, 2, 2], [100, 2, 0], heads=4, kv_heads=4, dtype="f16", page=16, dense=True)
    check(b, *b.run(force_path=route, scale=0.3), *b.attention(scale=0.3), label="scale")
    b = Batch([1, 90], [40, 90], heads=4, kv_heads=2, dtype="bf16", page=16)
    ref = b.attention()
    for hint in (None, 1, 90, 10 ** 6):  # a hint steers, it never decides
        check(b, *b.run(force_path=route, max_seqlen=hint), *ref, label=f"hint {hint}")


@pytest.mark.parametrize("route", ROUTES)
def test_bad_tables_are_reported(route):
    b = Batch([4, 4], [30, 30], heads=2, kv_heads=1, dtype="bf16", page=16)
    ref_o, ref_lse = b.attention()
    for table, lens, code in (([[10 ** 6, -3], None], [30, 30], -7), (None, [-5, 30], -7),
                              (None, [10 ** 9, 30], -7)):
        tb = b.table.clone()
        if table:
            tb[0] = torch.tensor(table[0], dtype=torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = pkg.gdr_paged_attn(b.on("q"), b.on("kc"), b.on("vc"), tb.cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(), b.on("cu"),
                                    force_path=route, status=status)
        assert int(status) == code
        check(b, o[0, 4:], lse[0, 4:], ref_o[4:], ref_lse[4:], label=str(code))
    for cu in ([0, 9, 8], [0, 4, 100], [-4, 4, 8]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkg.gdr_paged_attn(b.on("q"), b.on("kc"), b.on("vc"), b.on("table"), b.on("lens"),
                           torch.tensor(cu, dtype=torch.int32).cuda(), force_path=route,
                           status=status)
        assert int(status) == -5, cu


@pytest.mark.parametrize("route", ROUTES)
def test_offsets_past_32_bits(route):
    """Pages past the 2^31st element of the cache."""
    page, H, D = 128, 8, 128
    n_pages = (1 << 31) // (page * H * D) + 3
    b = Batch([3], [200], heads=8, kv_heads=8, dtype="bf16", page=page)
    kc = torch.zeros(n_pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(n_pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32)
    for c, src in ((kc, b.kc), (vc, b.vc)):
        for i in range(2):
            c[int(far[0, i])] = src[int(b.table[0, i])].cuda()
    ref = b.attention()
    b.table = far
    check(b, *b.run(force_path=route, kc=kc, vc=vc), *ref, label="far pages")
