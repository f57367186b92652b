"""The paged cache and the attention over it at their edges: what a row must not
see, scales and queries of very different size, tables that do not fit, empty
calls, load paths of odd pages.  Bounds are those of paged_ref.py."""
import math

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from paged_ref import Batch, check

pytestmark = pytest.mark.gpu

ROUTES = [1, 2, 3]


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype,fmt", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                       ("f16", "int8")])
@pytest.mark.parametrize("q_len,heads", [(1, 4), (1, 32), (2, 32), (4, 4)])
def test_positions_that_left_the_window(route, dtype, fmt, q_len, heads):
    """NaN and infinities in the first page below the window, which is loaded
    with it: a tile whose rows all see the same positions too."""
    b = Batch([q_len], [150], heads=heads, kv_heads=2, dtype=dtype, fmt=fmt, page=64)
    first = 150 - q_len - 36  # what the first token sees
    for at, bad in ((first - 1, math.nan), (first - 3, math.inf), (first - 40, math.nan)):
        page, slot = int(b.table[0, at // 64]), at % 64
        if fmt == "same":
            b.vc[page, slot, :, 5:90] = bad
            b.kc[page, slot, :, 5:90] = bad
        else:
            b.vs[page, :, slot] = math.nan
            b.ks[page, :, slot] = math.nan
    check(b, *b.run(force_path=route, window=37), *b.attention(window=37),
          label=f"{route} {dtype} {fmt} {q_len} {heads}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,K", [("e4m3", 128), ("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("bits", [8, 16, 20, 24, 30, 60])
def test_one_value_far_larger_than_the_others(route, dtype, fmt, K, bits):
    """A value 2^bits times the others: of a later token, of one below the
    window, of one with next to no weight.  The rows that do not take it keep
    their own values."""
    b = Batch([50], [150], heads=2, kv_heads=1, K=K, dtype=dtype, fmt=fmt, page=16)

    def place(at):
        return int(b.table[0, at // 16]), 0, at % 16

    vs, kc, ks = b.vs.clone(), b.kc.clone(), b.ks.clone()
    most = float(vs.nan_to_num().max()) * (127 if fmt == "int8" else 448)
    big = min(2.0 ** bits, torch.finfo(b.q.dtype).max / (4 * most))  # the output fits its type
    b.vs[place(149)] *= big
    check(b, *b.run(force_path=route), *b.attention(), label=f"later {bits}")
    b.vs = vs.clone()
    b.vs[place(75)] *= big
    ref_o, ref_lse = b.attention(window=40)
    check(b, *b.run(force_path=route, window=40), ref_o, ref_lse, label=f"window {bits}")
    # queries above 0, a key of equal and very negative columns
    b.vs = vs.clone()
    b.vs[place(90)] *= big
    b.q = b.q.abs()
    page, _, slot = place(90)
    b.kc[page, slot, 0] = torch.full((K,), -120.0).to(kc.dtype)
    b.ks[place(90)] = 0.5
    ref_o, ref_lse = b.attention()
    assert float(ref_o.abs().max()) < 100  # the value takes no part
    check(b, *b.run(force_path=route), ref_o, ref_lse, label=f"weightless {bits}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt,K", [("e4m3", 128), ("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("bits", [6, 9, 10, 12, 14])
def test_outlier_channel_of_the_queries(route, dtype, fmt, K, bits):
    """One channel of the queries 2^bits, where the keys do not vary: it adds the
    same to every score, and the softmax is that of the other channels."""
    b = Batch([70], [300], heads=4, kv_heads=1, K=K, dtype=dtype, fmt=fmt, page=16)
    g = torch.Generator().manual_seed(7)
    size = 60.0 if fmt == "e4m3" else 20.0
    b.kc = (size * torch.randn(b.kc.shape, generator=g)).clamp(-120, 120)
    b.kc = (b.kc if fmt == "e4m3" else b.kc.round()).to(b.vc.dtype)
    b.kc[..., 9] = torch.full(b.kc.shape[:-1], 32.0).to(b.kc.dtype)
    b.ks[:] = 1 / size
    b.q[..., 9] = 2.0 ** bits
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {dtype} {fmt} {K} {bits}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("cu,held", [([3, 7, 8], [(3, 7), (7, 8)]), ([0, 4, 6], [(0, 4), (4, 6)]),
                                     ([0, 6, 2, 8], None),
                                     ([0, 4, 100], [(0, 4)]), ([-4, 4, 8], [(4, 8)]), ([0, 9, 8], [])])
def test_tokens_that_no_sequence_holds(route, cu, held):
    """Offsets that do not run from 0 to T: reported; the tokens of sequences
    that are within T get their results, the others o = 0 and lse = -inf."""
    b = Batch([8], [30], heads=2, kv_heads=1, dtype="bf16", page=16)
    table = b.table.repeat(len(cu) - 1, 1).cuda()
    lens = torch.full((len(cu) - 1,), 30, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((1, 8, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 8, 2), math.nan, device="cuda")
    pkg.gdr_paged_attn(b.on("q"), b.on("kc"), b.on("vc"), table, lens,
                       torch.tensor(cu, dtype=torch.int32, device="cuda"), force_path=route,
                       status=status, o=o, lse=lse)
    assert int(status) == -5
    if held is None:  # sequences that overlap: in any order
        return
    loose = torch.ones(8, dtype=torch.bool)
    for t0, t1 in held:
        part = Batch([t1 - t0], [30], heads=2, kv_heads=1, dtype="bf16", page=16)
        part.table, part.kc, part.vc, part.q = b.table, b.kc, b.vc, b.q[:, t0:t1]
        check(part, o[0, t0:t1], lse[0, t0:t1], *part.attention(), label=f"{cu} {t0}")
        loose[t0:t1] = False
    assert (o[0].cpu()[loose] == 0).all() and (lse[0].cpu()[loose] == -math.inf).all()


@pytest.mark.parametrize("cu,held", [([3, 7, 8], [3, 4, 5, 6, 7]), ([0, 4, 6], [0, 1, 2, 3, 4, 5]),
                                     ([0, 4, 100], [0, 1, 2, 3]), ([-4, 4, 8], [4, 5, 6, 7]),
                                     ([0, 9, 8], []), ([0, 6, 2, 8], None)])
def test_cache_rows_that_no_sequence_holds(cu, held):
    """The same tables: such tokens are not stored and read as zeros."""
    n = len(cu) - 1
    b = Batch([8], [8], heads=1, kv_heads=1, K=32, page=8, dtype="bf16")
    kc, vc = (torch.full((n, 8, 1, 32), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.full((n,), 8, dtype=torch.int32, device="cuda")
    cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc, table, lens, cu_dev, status=status[:1])
    k, v = pkg.gdr_cache_read(kc, vc, table, lens, 8, cu_dev, status=status[1:])
    assert status.tolist() == [-5, -5]
    if held is None:
        return
    for got, cache, x in ((k, kc, b.k), (v, vc, b.v)):
        want, pages = torch.zeros_like(x), torch.full((n, 8, 1, 32), 7.0, dtype=torch.bfloat16)
        for t in held:
            seq = max(i for i in range(n) if cu[i] <= t < cu[i + 1])
            want[0, t] = x[0, t]
            pages[seq, 8 - (cu[seq + 1] - t)] = x[0, t]
        assert torch.equal(got.cpu(), want) and torch.equal(cache.cpu(), pages)


@pytest.mark.parametrize("length,stands_for", [(-5, 0), (65, 64), (1 << 30, 64), (-(1 << 31), 0)])
def test_lengths_outside_the_table(length, stands_for):
    """Reported; the sequence's tokens are neither stored nor read, the attention
    takes the nearest length inside; the other sequence is untouched by it."""
    b = Batch([4, 4], [64, 30], heads=2, kv_heads=1, K=64, page=16, dtype="bf16")
    cu, table = b.on("cu"), b.on("table")
    kc, vc = b.on("kc").nan_to_num(0.5), b.on("vc").nan_to_num(0.5)
    before = kc.clone(), vc.clone()
    lens, near = (torch.tensor([x, 30], dtype=torch.int32, device="cuda") for x in (length, stands_for))
    status = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc, table, lens, cu, status=status[:1])
    at = torch.arange(26, 30)
    for c, old, x in ((kc, before[0], b.k), (vc, before[1], b.v)):
        want = old.cpu()
        want[b.table[1, at // 16].long(), at % 16] = x[0, 4:]
        assert torch.equal(c.cpu(), want)
    k, v = pkg.gdr_cache_read(kc, vc, table, lens, 8, cu, status=status[1:2])
    for got, x in ((k, b.k), (v, b.v)):
        assert (got[0, :4] == 0).all() and torch.equal(got[0, 4:].cpu(), x[0, 4:])
    for route in ROUTES:
        status[2] = 0
        o, lse = pkg.gdr_paged_attn(b.on("q"), kc, vc, table, lens, cu, status=status[2:],
                                    force_path=route)
        assert status.tolist() == [-7, -7, -7]
        o2, lse2 = pkg.gdr_paged_attn(b.on("q"), kc, vc, table, near, cu, force_path=route)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("packed", [True, False])
def test_calls_without_tokens(packed):
    """A step with no new tokens: nothing to do, and no error."""
    b = Batch([3, 2], [30, 20], heads=4, kv_heads=2, K=64, dtype="bf16", page=16)
    kc, vc = b.on("kc"), b.on("vc")
    lead = (1, 0) if packed else (2, 0)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda") if packed else None
    k = torch.empty(*lead, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(*lead, 4, 64, dtype=torch.bfloat16, device="cuda")
    pkg.gdr_cache_write(k, k, kc, vc, b.on("table"), b.on("lens"), cu)
    k2, v2 = pkg.gdr_cache_read(kc, vc, b.on("table"), b.on("lens"), 0, cu)
    o, lse = pkg.gdr_paged_attn(q, kc, vc, b.on("table"), b.on("lens"), cu)
    torch.cuda.synchronize()
    assert k2.shape == v2.shape == (*lead, 2, 64)
    assert o.shape == q.shape and lse.shape == q.shape[:-1]
    assert torch.equal(kc.nan_to_num(), b.on("kc").nan_to_num())


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt,K", [("e4m3", 128), ("int8", 128), ("int8", 64)])
@pytest.mark.parametrize("bits", [-40, 0, 40])
@pytest.mark.parametrize("spread", [False, True])
def test_rows_of_zeros_keep_their_weight(route, fmt, K, bits, spread):
    """Values of zeros (their scale is 0) beside values of about 2^bits, some of
    them 2^-20 of that: they take their part of the softmax's sum."""
    b = Batch([50], [150], heads=2, kv_heads=1, K=K, dtype="bf16", fmt=fmt, page=16)
    b.vs *= 2.0 ** bits
    at = torch.arange(150)
    pages, slots = b.table[0, at // 16].long(), at % 16
    if spread:
        b.vs[pages[1::3], 0, slots[1::3]] *= 2.0 ** -20
    b.vs[pages[::2], 0, slots[::2]] = 0
    b.vc[pages[::2], slots[::2]] = torch.zeros(K).to(b.vc.dtype)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {fmt} {K} {bits} {spread}")


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt,K", [("e4m3", 128), ("int8", 128), ("int8", 64)])
@pytest.mark.parametrize("some", [False, True])
def test_values_near_the_least_magnitudes(route, fmt, K, some):
    """Scales of values about 2^-110 (BF16 goes down to 2^-133): of all tokens,
    or of all but a few whose weight is nothing beside the others'."""
    b = Batch([50], [150], heads=2, kv_heads=1, K=K, dtype="bf16", fmt=fmt, page=16)
    b.vs *= 2.0 ** -103
    if some:
        b.q = b.q.abs()
        for at in (40, 90):
            page, slot = int(b.table[0, at // 16]), at % 16
            b.vs[page, 0, slot] = 1e-30
            b.kc[page, slot, 0] = torch.full((K,), -120.0).to(b.kc.dtype)
            b.ks[page, 0, slot] = 0.5
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {fmt} {K} {some}")


@pytest.mark.parametrize("route", [1, 3, 0])
@pytest.mark.parametrize("dtype,fmt", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                       ("bf16", "int8"), ("f16", "e4m3"), ("f16", "int8")])
@pytest.mark.parametrize("page,K", [(1, 128), (5, 64), (12, 128), (4, 64)])
def test_pages_that_no_box_fits(route, dtype, fmt, page, K):
    """Pages of no multiple of 8 slots: gathered row by row."""
    b = Batch([3, 0, 1, 70, 5], [3, 9, 131, 200, 0], heads=4, kv_heads=2, K=K, page=page,
              dtype=dtype, fmt=fmt)
    check(b, *b.run(force_path=route), *b.attention(), label=f"{route} {dtype} {fmt} {page}")
    check(b, *b.run(force_path=route, window=33), *b.attention(window=33), label="window")
    with pytest.raises(pkg.GdrError):  # boxes of 8 slots at least
        b.run(force_path=2)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("K", [64, 128])
def test_scales_off_16_bytes(fmt, K):
    b = Batch([1, 20], [131, 200], heads=4, kv_heads=2, K=K, page=16, dtype="bf16", fmt=fmt)
    ref = b.attention()
    for name in ("ks", "vs"):
        keep = getattr(b, name)
        flat = torch.zeros(keep.numel() + 1, device="cuda")
        flat[1:] = keep.reshape(-1).cuda()
        moved = flat[1:].view(keep.shape)
        setattr(b, name, moved)
        b_on = b.on
        b.on = lambda n, m=moved, f=b_on, name=name: m if n == name else f(n)
        for route in (0, 1, 3):
            check(b, *b.run(force_path=route), *ref, label=f"{name} {route}")
        b.on = b_on
        setattr(b, name, keep)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("K,V", [(16, 16), (48, 208), (256, 256), (128, 64), (64, 128)])
def test_other_widths_in_16_bits(dtype, fmt, K, V):
    b = Batch([3, 40, 1], [50, 40, 300], heads=4, kv_heads=2, K=K, V=V, dtype=dtype, fmt=fmt,
              page=16)
    check(b, *b.run(), *b.attention(), label=f"{dtype} {fmt} {K} {V}")


def test_status_and_workspace_must_be_on_the_device():
    b = Batch([3], [30], heads=2, kv_heads=1, K=64, dtype="bf16", page=16)
    args = [b.on(x) for x in ("kc", "vc", "table", "lens")]
    host = torch.zeros(1, dtype=torch.int32)
    for bad in (host, host.cuda().long()):
        with pytest.raises((ValueError, TypeError)):
            pkg.gdr_paged_attn(b.on("q"), *args, b.on("cu"), status=bad)
        with pytest.raises((ValueError, TypeError)):
            pkg.gdr_cache_write(b.on("k"), b.on("v"), *args, b.on("cu"), status=bad)
        with pytest.raises((ValueError, TypeError)):
            pkg.gdr_cache_read(*args, 3, b.on("cu"), status=bad)
    with pytest.raises(ValueError):
        pkg.gdr_paged_attn(b.on("q"), *args, b.on("cu"),
                           workspace=torch.zeros(1 << 24, dtype=torch.uint8))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("fmt", ["same", "e4m3"])
def test_workspace_of_the_caller(route, fmt):
    """The bits of the call that takes its own scratch, and nothing written past
    the size that the library asks for."""
    b = Batch([5, 130, 1], [900, 400, 1500], heads=8, kv_heads=2, dtype="bf16", fmt=fmt, page=16)
    need = pkg.gdr_attn_workspace_size(*(b.on(x) for x in ("q", "kc", "vc", "table", "lens", "cu")),
                                       k_scale=b.on("ks"), v_scale=b.on("vs"))
    o, lse = b.run(force_path=route)
    room = torch.full((need + 256,), 91, dtype=torch.uint8, device="cuda")
    o2, lse2 = b.run(force_path=route, workspace=room[:need])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (room[need:] == 91).all()
    if route > 1:
        with pytest.raises(pkg.GdrError):
            b.run(force_path=route, workspace=room[:256])
        with pytest.raises(pkg.GdrError):
            b.run(force_path=route, workspace=room[16:need + 16])


@pytest.mark.parametrize("fmt,most", [("int8", 127.0), ("e4m3", 448.0)])
def test_rows_whose_scale_is_rounded_far(fmt, most):
    """FP32 rows so small that their scale is a few of the type's smallest
    units: quotients past the format's largest value are its largest value."""
    b = Batch([40], [40], heads=1, kv_heads=1, K=32, page=16, dtype="f32", fmt=fmt)
    units = 1 + 23 * torch.arange(40, dtype=torch.float64)  # of 2^-149
    b.k[0] = (units[:, None, None] * torch.linspace(-1, 1, 32, dtype=torch.float64)
              ).round().mul(2.0 ** -149).float()
    kc, vc, ks, vs = (b.on(x) for x in ("kc", "vc", "ks", "vs"))
    pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc, b.on("table"), b.on("lens"), b.on("cu"),
                        k_scale=ks, v_scale=vs)
    at = torch.arange(40)
    pages, slots = b.table[0, at // 16].long(), at % 16
    got, scale = kc.cpu().float()[pages, slots, 0].double(), ks.cpu()[pages, 0, slots].double()
    assert float(got.abs().max()) == most
    x = b.k[0, :, 0].double()
    want = torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros_like(x)).clamp(-most, most)
    step = 1.0 if fmt == "int8" else 32.0
    assert ((got - want).abs() <= step / 2).all() and (got * want >= 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_zeros_keep_their_sign(dtype):
    """E4M3 has a zero of either sign, and -0 / s is -0."""
    b = Batch([20], [20], heads=1, kv_heads=1, K=32, page=16, dtype=dtype, fmt="e4m3")
    b.k[0, ::2, 0, 3] = -0.0
    b.k[0, 1::2, 0, 3] = 0.0
    kc, vc, ks, vs = (b.on(x) for x in ("kc", "vc", "ks", "vs"))
    pkg.gdr_cache_write(b.on("k"), b.on("v"), kc, vc, b.on("table"), b.on("lens"), b.on("cu"),
                        k_scale=ks, v_scale=vs)
    at = torch.arange(20)
    got = kc.cpu().view(torch.uint8)[b.table[0, at // 16].long(), at % 16, 0, 3]
    assert got.tolist() == [128, 0] * 10
    k, _ = pkg.gdr_cache_read(kc, vc, b.on("table"), b.on("lens"), 20, b.on("cu"), k_scale=ks,
                              v_scale=vs, dtype=b.k.dtype)
    assert torch.equal(torch.signbit(k[0, :, 0, 3]).cpu(), torch.arange(20) % 2 == 0)
