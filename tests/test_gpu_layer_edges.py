"""The operators of a state-space layer on the GPU where they can go wrong beside their values:
rows in one place, values of FP32's least units, other streams, strided gradients."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import close, rms_norm, selective_scan

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def test_norm_of_broadcast_rows():
    """One row in the place of many is refused wherever it comes in, or would be written; as many
    rows of the same values are not."""
    one, w, full = randn(64), randn(64, seed=1), randn(8, 64, seed=2)
    for rows in (one.expand(8, 64), one.expand(2, 4, 64)):
        like = full.reshape(rows.shape)
        for call in (lambda: gdr.gdr_rms_norm_fwd(rows, w), lambda: gdr.rms_norm(rows, w),
                     lambda: gdr.gdr_rms_norm_fwd(like, w, rows), lambda: gdr.rms_norm(like, w, rows),
                     lambda: gdr.gdr_rms_norm_fwd(like, w, y=rows),
                     lambda: gdr.gdr_rms_norm_fwd(like, w, like, residual_out=rows),
                     lambda: gdr.gdr_rms_norm_fwd(rows, w, dtype=torch.int8),
                     lambda: gdr.gdr_rms_norm_bwd(rows, like, w), lambda: gdr.gdr_rms_norm_bwd(like, rows, w),
                     lambda: gdr.gdr_rms_norm_bwd(like, like, w, rows)):
            with pytest.raises(ValueError):
                call()
        y, _, _ = gdr.gdr_rms_norm_fwd(rows.contiguous(), w)
        close("y", y, rms_norm(rows.cpu().double(), w.cpu().double(), 1e-6))
    # a gradient that comes in broadcast, as that of a sum over rows does
    x = full.clone().requires_grad_()
    gdr.rms_norm(x, w)[0].sum().backward()
    dx, _ = gdr.gdr_rms_norm_bwd(torch.ones_like(full), full, w)
    assert torch.equal(x.grad, dx)


FMT = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


@pytest.mark.parametrize("fmt", FMT.values(), ids=FMT.keys())
@pytest.mark.parametrize("D,group", [(128, 0), (256, 128), (7, 0), (1002, 0), (1002, 128), (2048, 0), (2048, 128)])
def test_eight_bits_of_least_units(fmt, D, group):
    """Rows of a few of FP32's least units, whose scale is rounded by up to a third: no value
    passes the format's largest, none changes its sign, and the bytes are the cache's."""
    rows = 96
    x = randn(rows, D, seed=3).double().cpu()
    x = (x * 2.0 ** torch.linspace(-150.0, -118.0, rows).double()[:, None]).float().cuda()
    units = torch.tensor([1, 2, 63, 64, 95, 127, 190, 191, 317, 318, 444, 1000]) * 2.0 ** -149
    x[:12] = (units[:, None] * torch.linspace(-1.0, 1.0, D)).cuda()
    x[:12, 0] = -units.cuda()
    # 1 under the root: y is x
    y, _, _ = gdr.gdr_rms_norm_fwd(x, None, eps=1.0)
    assert torch.equal(y, x) and (x != 0).any(1)[:12].all()
    q, _, scale = gdr.gdr_rms_norm_fwd(x, None, eps=1.0, dtype=fmt, group=group)
    top = 448.0 if fmt is FMT["e4m3"] else 127.0
    v = q.float()
    assert (v.abs() <= top).all() and not (v * x.sign() < 0).any()
    if D % 128:
        return
    heads = D // (group or D)
    if D // heads > 256:
        return  # wider than a row of the cache
    k = x.reshape(1, rows, heads, -1)
    cache = [torch.zeros(6, 16, heads, k.shape[-1], device="cuda").to(fmt) for _ in range(2)]
    scales = [torch.zeros(6, heads, 16, device="cuda") for _ in range(2)]
    gdr.gdr_cache_write(k, k, *cache, torch.arange(6, dtype=torch.int32, device="cuda")[None],
                        torch.tensor([rows], dtype=torch.int32, device="cuda"), k_scale=scales[0],
                        v_scale=scales[1])
    assert torch.equal(scales[0].transpose(1, 2).reshape(scale.shape), scale)
    assert torch.equal(cache[0].view(torch.uint8).reshape(rows, D), q.view(torch.uint8))


def scan_inputs(lens=(70, 1, 0, 130), C=96, S=16, seed=0):
    T = sum(lens)
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()
    bc = randn(1, T, 2, 1, S, seed=seed)
    return dict(x=randn(1, T, C, seed=seed + 1), dt=randn(1, T, C, seed=seed + 2) - 2.0,
                A=-torch.exp(randn(C, S, seed=seed + 3)), B=bc[:, :, 0], C=bc[:, :, 1],
                D=randn(C, seed=seed + 4), z=randn(1, T, C, seed=seed + 5), dt_bias=randn(C, seed=seed + 6),
                cu_seqlens=cu, h0=randn(len(lens), C, S, seed=seed + 7))


def every_call(s, w, taps, dy, dht, dhc, **kw):
    """Each of the six calls on the same inputs; the outputs by name."""
    x, cu = s["x"], s["cu_seqlens"]
    out = {}
    out["conv y"], out["conv ht"] = gdr.gdr_short_conv_fwd(x, taps, s["D"], cu, output_final_state=True, **kw)
    for name, t in zip(("dx", "dweight", "dbias", "dh0"), gdr.gdr_short_conv_bwd(
            x, taps, dy, s["D"], cu, None, dhc, want_dh0=True, **kw)):
        out["conv " + name] = t
    out["scan y"], out["scan ht"] = gdr.gdr_selective_scan_fwd(**s, **kw)
    for name, t in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"),
                       gdr.gdr_selective_scan_bwd(**s, dy=dy, dht=dht, want_dh0=True, **kw)):
        out["scan " + name] = t
    for name, t in zip("y r".split(), gdr.gdr_rms_norm_fwd(x, w, dy, **kw)):
        out["norm " + name] = t
    q, _, out["norm scale"] = gdr.gdr_rms_norm_fwd(x, w, dtype=torch.float8_e4m3fn, **kw)
    out["norm q"] = q.view(torch.uint8)
    out["norm dx"], out["norm dweight"] = gdr.gdr_rms_norm_bwd(dy, x, w, **kw)
    return out


def call_inputs():
    s = scan_inputs()
    return (s, randn(96, seed=20), randn(96, 4, seed=21), randn(*s["x"].shape, seed=22),
            randn(*s["h0"].shape, seed=23), randn(4, 3, 96, seed=24))


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16, torch.float16], ids=str)
def test_another_default_dtype(default):
    args = call_inputs()
    want = every_call(*args)
    torch.set_default_dtype(default)
    try:
        got = every_call(*args)
    finally:
        torch.set_default_dtype(torch.float32)
    for k in want:
        assert got[k].dtype == want[k].dtype and torch.equal(got[k], want[k]), k


SLEEP = 200_000_000  # cycles that a stream does nothing for: some 100 ms


def warm(args):
    """A side stream that has memory of its own, so that no call on it waits for the device to get
    some; and what the calls give on the current one."""
    side, want = torch.cuda.Stream(), every_call(*args)
    torch.cuda.synchronize()
    every_call(*args, stream=side)
    torch.cuda.synchronize()
    return side, want


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def same(got, want):
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_outputs_on_another_stream_are_not_in_memory_that_this_one_has_let_go():
    """Memory let go on the current stream may still be written there, which a call on another
    stream does not wait for."""
    args = call_inputs()
    side, want = warm(args)
    gone = [torch.empty_like(t) for t in want.values()]
    old = spans(gone)
    torch.cuda._sleep(SLEEP)
    for t in gone:
        t.fill_(77)
    del gone, t
    got = every_call(*args, stream=side)
    for a, b in spans(got.values()):
        assert not any(a < d and c < b for c, d in old)
    same(got, want)


def test_inputs_let_go_while_another_stream_has_yet_to_read_them():
    args = call_inputs()
    side, want = warm(args)
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    shapes = [t.shape for t in list(args[0].values()) + list(args[1:]) if t.is_floating_point()]
    got = every_call(*args, stream=side)
    del args
    for s in shapes:
        torch.full(s, float("nan"), device="cuda")
    junk = [torch.full(s, float("nan"), device="cuda") for s in shapes]
    same(got, want)
    assert len(junk) == len(shapes)


def test_outputs_let_go_while_the_current_stream_has_yet_to_read_them():
    args, other = call_inputs(), list(call_inputs())
    side, want = warm(args)
    other[0] = scan_inputs(seed=40)
    here = torch.cuda.current_stream()
    torch.cuda.synchronize()
    got = every_call(*args, stream=side)
    here.wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = {k: t.clone() for k, t in got.items()}
    del got
    again = every_call(*other, stream=side)
    same(kept, want)
    assert not torch.equal(again["scan y"], want["scan y"])


def test_captured_on_another_stream():
    args = call_inputs()
    side, want = warm(args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = every_call(*args, stream=side)
        here.wait_stream(side)
    for _ in range(2):
        for t in got.values():
            t.zero_()
        graph.replay()
        same(got, want)


def test_status_let_go():
    """A status word that its caller has let go is not handed out again under a call."""
    args = call_inputs()
    s, w, taps, dy = args[:4]
    side, _ = warm(args)
    for call in (lambda **kw: gdr.gdr_short_conv_fwd(s["x"], taps, None, s["cu_seqlens"], **kw),
                 lambda **kw: gdr.gdr_short_conv_bwd(s["x"], taps, dy, None, s["cu_seqlens"], **kw),
                 lambda **kw: gdr.gdr_selective_scan_fwd(**s, **kw),
                 lambda **kw: gdr.gdr_selective_scan_bwd(**s, dy=dy, **kw)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        at, done = status.data_ptr(), torch.cuda.Event()
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        call(status=status, stream=side)
        done.record(side)
        del status
        new = [torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(4)]
        assert not done.query()
        assert all(t.data_ptr() != at for t in new)
        torch.cuda.synchronize()


def test_scan_of_single_tokens_of_more_warps_than_32_bits_count():
    """2^21 sequences of 65536 channels, 2^32 warps of 32 channels and one more sequence's, all but
    the first and the last empty: the last one's tokens are written too."""
    N, C, T = 1 << 21, 65536, 3
    cu = torch.ones(N + 1, dtype=torch.int32, device="cuda")
    cu[0], cu[-1] = 0, T
    x, dt, bc = randn(1, T, C), randn(1, T, C, seed=1) - 1.0, randn(1, T, 2, 1, 1, seed=2)
    A, status = -torch.exp(randn(C, 1, seed=3)), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(x, float("nan"))
    gdr.gdr_selective_scan_fwd(x, dt, A, bc[:, :, 0], bc[:, :, 1], cu_seqlens=cu, max_seqlen=2, y=y,
                               output_final_state=False, status=status)
    want, _ = selective_scan(*(t.cpu().double() for t in (x[0], dt[0], A, bc[0, :, 0], bc[0, :, 1])),
                             None, None, None, [1, 2])
    close("y", y[0], want)
    assert int(status) == 0


def view_of(t, at, pitch):
    """The same values as columns [at, at + C) of rows of ``pitch``."""
    big = randn(*t.shape[:-1], pitch, seed=50 + at).to(t.dtype)
    view = big[..., at:at + t.shape[-1]]
    view.copy_(t)
    assert not view.is_contiguous()
    return view


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("C,at,pitch", [(48, 0, 64), (48, 16, 80), (48, 3, 64), (48, 8, 61), (45, 1, 50)])
def test_gradients_that_come_in_as_views(C, at, pitch, dtype):
    """dy (and x, as the layer has it) as slices of wider rows, on 16 bytes and off them: the bits
    of contiguous tensors, packed and dense."""
    lens = [5, 70, 0, 13, 20]
    T = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    x, dy, z = (randn(1, T, C, seed=i, dtype=dtype) for i in range(3))
    taps, bias = randn(C, 4, seed=3, dtype=dtype), randn(C, seed=4, dtype=dtype)
    dht = randn(5, 3, C, seed=5, dtype=dtype)
    bc = randn(1, T, 2, 1, 16, seed=6, dtype=dtype)
    A, D = -torch.exp(randn(C, 16, seed=7)), randn(C, seed=8)

    def conv(x, dy, cu, dht=None):
        return gdr.gdr_short_conv_bwd(x, taps, dy, bias, cu, None, dht, want_dh0=True)

    def scan(x, dy, z, bc, cu):
        return gdr.gdr_selective_scan_bwd(x, x, A, bc[..., 0, :, :], bc[..., 1, :, :], dy, D, z, D, cu,
                                          want_dh0=True)

    vx, vdy, vz = (view_of(t, at, pitch) for t in (x, dy, z))
    want = conv(x, dy, cu, dht)
    for a, b in ((vx, vdy), (x, vdy), (vx, dy)):
        got = conv(a, b, cu, dht)
        # rows off 16 bytes, or of an odd number of channels, are summed in other runs
        assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
        close("dweight", got[1], want[1])
        close("dbias", got[2], want[2])
    want = scan(x, dy, z, bc, cu)
    for a, b, c in ((vx, vdy, vz), (x, vdy, z), (vx, dy, z)):
        for got, w in zip(scan(a, b, c, bc, cu), want):
            assert torch.equal(got, w)
    # four dense rows of 27 tokens
    rows = [t.reshape(4, 27, *t.shape[2:]) for t in (x, dy, z, bc)]
    wide = [view_of(t, at, pitch) for t in rows[:3]]
    want = scan(*rows, None)
    for got, w in zip(scan(*wide, rows[3], None), want):
        assert torch.equal(got, w)
    want, got = conv(rows[0], rows[1], None), conv(wide[0], wide[1], None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    close("dweight", got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("D,at,pitch", [(96, 0, 128), (96, 8, 104), (96, 2, 100), (96, 1, 97), (1026, 2, 1100),
                                        (2048, 8, 2064), (2048, 3, 2060), (5120, 2, 5200), (10001, 1, 10007)])
def test_norm_gradients_of_views(D, at, pitch, dtype):
    """r, dy and dr as slices of wider rows, one at a time and together: whatever width they are
    loaded in, the gradients of 64 bits."""
    rows = 40
    r, dy, dr = (randn(rows, D, seed=i, dtype=dtype) for i in range(3))
    w = randn(D, seed=3, dtype=dtype)
    lr, lw = (t.cpu().double().requires_grad_() for t in (r, w))
    ((rms_norm(lr, lw, 1e-6) * dy.cpu().double()).sum() + (lr * dr.cpu().double()).sum()).backward()
    vr, vdy, vdr = (view_of(t, at, pitch) for t in (r, dy, dr))
    for a, b, c in ((vr, vdy, vdr), (vr, dy, dr), (r, vdy, dr), (r, dy, vdr)):
        dx, dw = gdr.gdr_rms_norm_bwd(b, a, w, c)
        close("dx", dx, lr.grad)
        close("dweight", dw, lw.grad)
    x = r.clone().requires_grad_()
    y, _ = gdr.rms_norm(x, w)
    y.backward(vdy)
    lr.grad = None
    (rms_norm(lr, lw, 1e-6) * dy.cpu().double()).sum().backward()
    close("dx", x.grad, lr.grad)


def big_randn(*shape):
    """A few GB of BF16, made on the device."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)


def test_channels_at_offsets_of_more_than_32_bits():
    """More than 2^31 values of x: the last sequence's outputs and gradients are those of a call on
    it alone.  (The sums over all tokens, which the other sequence is part of, are left out.)"""
    C, T, tail = 65536, 32900, 77
    x, dy = big_randn(1, T, C), big_randn(1, T, C)
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    taps, bias = randn(C, 4, dtype=torch.bfloat16), randn(C, seed=1, dtype=torch.bfloat16)
    part, part_dy = x[:, -tail:], dy[:, -tail:]
    y, ht = gdr.gdr_short_conv_fwd(x, taps, bias, cu, output_final_state=True)
    y1, ht1 = gdr.gdr_short_conv_fwd(part, taps, bias, output_final_state=True, max_seqlen=tail)
    assert torch.equal(y[:, -tail:], y1) and torch.equal(ht[1:], ht1)
    del y
    dx = gdr.gdr_short_conv_bwd(x, taps, dy, bias, cu)[0]
    assert torch.equal(dx[:, -tail:], gdr.gdr_short_conv_bwd(part, taps, part_dy, bias)[0])
    del dx
    A, bc = -torch.exp(randn(C, 1, seed=2)), randn(1, T, 2, 1, 1, seed=3, dtype=torch.bfloat16)
    B1, C1 = bc[:, :, 0], bc[:, :, 1]
    ends = B1[:, -tail:], C1[:, -tail:]
    for n in (1, 40):
        y, ht = gdr.gdr_selective_scan_fwd(x, x, A, B1, C1, cu_seqlens=cu, n_segments=n, max_seqlen=T)
        y1, ht1 = gdr.gdr_selective_scan_fwd(part, part, A, *ends, n_segments=1)
        close("y", y[:, -tail:], y1)
        close("ht", ht[1:], ht1)
        del y
    got = gdr.gdr_selective_scan_bwd(x, x, A, B1, C1, dy, cu_seqlens=cu, want_dh0=True)
    want = gdr.gdr_selective_scan_bwd(part, part, A, *ends, part_dy, want_dh0=True)
    for i in (0, 1, 3, 4):  # dx, ddt, dB, dC
        assert torch.equal(got[i][:, -tail:], want[i]), i
    assert torch.equal(got[8][1:], want[8])


def test_pools_at_offsets_of_more_than_32_bits():
    C, S, rows = 4096, 64, 8300  # 2^31 values end in row 8192
    scan = torch.zeros(rows, C, S, device="cuda")
    conv = torch.zeros(350000, 3, 2 * C, dtype=torch.bfloat16, device="cuda")  # 8.6e9 values
    idx = torch.tensor([8299, 8191, 8192], dtype=torch.int32, device="cuda")
    far = torch.tensor([349999, 87381, 174763], dtype=torch.int32, device="cuda")
    x = randn(3, 1, C)
    bc = randn(3, 1, 2, 1, S, seed=1)
    A = -torch.exp(randn(C, S, seed=2))
    h = randn(3, C, S, seed=3)
    scan[idx.long()] = h
    y, _ = gdr.gdr_selective_scan_fwd(x, x, A, bc[:, :, 0], bc[:, :, 1], state=scan, state_indices=idx)
    y1, h1 = gdr.gdr_selective_scan_fwd(x, x, A, bc[:, :, 0], bc[:, :, 1], h0=h)
    assert torch.equal(y, y1) and torch.equal(scan[idx.long()], h1)
    scan[idx.long()] = 0
    assert not any(part.any() for part in scan.split(1024))
    x, h = randn(3, 1, 2 * C, dtype=torch.bfloat16), randn(3, 3, 2 * C, seed=4, dtype=torch.bfloat16)
    taps = randn(2 * C, 4, seed=5, dtype=torch.bfloat16)
    conv[far.long()] = h
    y, _ = gdr.gdr_short_conv_fwd(x, taps, state=conv, state_indices=far)
    y1, h1 = gdr.gdr_short_conv_fwd(x, taps, h0=h, output_final_state=True)
    assert torch.equal(y, y1) and torch.equal(conv[far.long()], h1)
    conv[far.long()] = 0
    assert not any(part.any() for part in conv.split(32768))


def test_norm_of_rows_at_offsets_of_more_than_32_bits():
    D, rows, tail = 8192, (1 << 18) + 100, 100
    x, dy, w = big_randn(rows, D), big_randn(rows, D), randn(D, dtype=torch.bfloat16)
    exact = rms_norm(x[-tail:].cpu().double(), w.cpu().double(), 1e-6)
    close("y", gdr.gdr_rms_norm_fwd(x, w)[0][-tail:], exact)
    q, r, scale = gdr.gdr_rms_norm_fwd(x, w, dy, dtype=torch.int8, group=128)
    assert torch.equal(r[-tail:], (x[-tail:].float() + dy[-tail:].float()).bfloat16())
    r1 = r[-tail:].cpu().double()
    del r
    back = q[-tail:].cpu().double().reshape(tail, -1, 128) * scale[-tail:].cpu().double()[..., None]
    err = (back.reshape(tail, D) - rms_norm(r1, w.cpu().double(), 1e-6)).reshape(tail, -1, 128).abs().amax(-1)
    assert (err <= 0.501 * scale[-tail:].cpu().double()).all()  # half a step, and FP32's arithmetic
    del q, scale
    dx, _ = gdr.gdr_rms_norm_bwd(dy, x, w)
    leaf = x[-tail:].cpu().double().requires_grad_()
    (rms_norm(leaf, w.cpu().double(), 1e-6) * dy[-tail:].cpu().double()).sum().backward()
    close("dx", dx[-tail:], leaf.grad)


def test_one_tensor_as_both_inputs():
    """x as its own residual, and as the time step: its gradient is the sum of both."""
    x, w, dy = randn(9, 64), randn(64, seed=1), randn(9, 64, seed=2)
    leaf, ref = x.clone().requires_grad_(), x.cpu().double().requires_grad_()
    gdr.rms_norm(leaf, w, leaf)[0].backward(dy)
    rms_norm(ref + ref, w.cpu().double(), 1e-6).backward(dy.cpu().double())
    close("dx", leaf.grad, ref.grad)
    s = scan_inputs((40,))
    leaf, ref = s["x"].clone().requires_grad_(), s["x"][0].cpu().double().requires_grad_()
    gdr.selective_scan(leaf, leaf, s["A"], s["B"], s["B"], None, leaf)[0].square().sum().backward()
    A, B = s["A"].cpu().double(), s["B"][0].cpu().double()
    selective_scan(ref, ref, A, B, B, None, ref, None, [40])[0].square().sum().backward()
    # a loss of squares: what is left of y in FP32 counts twice
    close("dx", leaf.grad[0], ref.grad, work=2e-5)
