"""The root-mean-square norm on the GPU against 64 bits: with and without the residual, in
the inputs' type and in 8 bits, and its gradients."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import DTYPES, close, rms_norm, wide

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
WIDTHS = [1, 2, 7, 8, 100, 128, 130, 1000, 1024, 1100, 2048, 4104, 5001, 16384]


def inputs(rows, D, dtype="bf16", weight_dtype=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    gain = torch.exp(randn(D))
    return dict(x=(randn(rows, D) * gain).to(dt).cuda(), res=(randn(rows, D) * gain).to(dt).cuda(),
                w=(1.0 + 0.3 * randn(D)).to(DTYPES[weight_dtype or dtype]).cuda(),
                dy=randn(rows, D).to(dt).cuda(), dr=randn(rows, D).to(dt).cuda())


@pytest.mark.parametrize("rows", [1, 5, 700])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(rows, D):
    for dtype, wdt in (("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")):
        s = inputs(rows, D, dtype, wdt)
        y, none, scale = gdr.gdr_rms_norm_fwd(s["x"], s["w"])
        assert none is None and scale is None
        close("y", y, rms_norm(s["x"].cpu().double(), s["w"].cpu().double(), 1e-6))
        y, r, _ = gdr.gdr_rms_norm_fwd(s["x"], s["w"], s["res"], eps=1e-3)
        assert torch.equal(r, (s["x"].float() + s["res"].float()).to(r.dtype))
        close("y", y, rms_norm(r.cpu().double(), s["w"].cpu().double(), 1e-3))
        y, r, _ = gdr.gdr_rms_norm_fwd(s["x"])
        close("y", y, rms_norm(s["x"].cpu().double(), None, 1e-6))


def steps(q, fmt):
    """Distance between neighbouring 8-bit values at q."""
    if fmt is I8:
        return torch.ones_like(q)
    return torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("fmt,group", [(E4M3, 0), (E4M3, 128), (I8, 0), (I8, 128)], ids=str)
def test_eight_bits(rows, D, fmt, group):
    """The scale is max|y| / 448 or / 127 up to FP32's arithmetic (1e-5, as in ``close``), and a
    value is within half a step of y / scale: half of the step at it, and as much again of the
    1e-5."""
    for dtype in ("bf16", "f32", "f16"):
        s = inputs(rows, D, dtype)
        y, r, scale = gdr.gdr_rms_norm_fwd(s["x"], s["w"], s["res"], dtype=fmt, group=group)
        assert y.dtype is fmt and torch.equal(r, (s["x"].float() + s["res"].float()).to(r.dtype))
        ref = rms_norm(r.cpu().double(), s["w"].cpu().double(), 1e-6)
        g = group or D
        parts = -(-D // g)
        assert scale.shape == ((rows, parts) if group else (rows,))
        padded = torch.nn.functional.pad(ref, (0, parts * g - D)).reshape(rows, parts, g)
        top = 448.0 if fmt is E4M3 else 127.0
        one = padded.abs().amax(-1) / top
        got = scale.reshape(rows, parts).cpu().double()
        assert ((got - one).abs() <= 1e-5 * one).all()
        exact = (padded / got[..., None]).reshape(rows, -1)[:, :D]
        q = y.cpu().double() if fmt is I8 else y.cpu().float().double()
        assert (q.abs() <= top).all()
        # the value that rounding gives may lie in the next binade: the larger of both steps
        step = torch.maximum(steps(q, fmt), steps(exact, fmt))
        assert ((q - exact).abs() <= 0.5 * step + 2e-5 * exact.abs() + 1e-9).all()


def test_eight_bits_round_as_the_cache_does():
    """The scale and values are those of gdr_cache_write for the same rows: the norm's own FP32
    output quantised by the cache."""
    s = inputs(64, 128, "f32")
    y, _, _ = gdr.gdr_rms_norm_fwd(s["x"], s["w"])
    for fmt in (E4M3, I8):
        q, _, scale = gdr.gdr_rms_norm_fwd(s["x"], s["w"], dtype=fmt)
        k = y.reshape(1, 64, 1, 128)
        cache = [torch.zeros(4, 16, 1, 128, device="cuda").to(fmt) for _ in range(2)]
        scales = [torch.zeros(4, 1, 16, device="cuda") for _ in range(2)]
        table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        gdr.gdr_cache_write(k, k, *cache, table, torch.tensor([64], dtype=torch.int32, device="cuda"),
                            k_scale=scales[0], v_scale=scales[1])
        assert torch.equal(scales[0].reshape(64), scale)
        assert torch.equal(cache[0].view(torch.uint8).reshape(64, 128), q.view(torch.uint8))


@pytest.mark.parametrize("fmt", [E4M3, I8])
def test_rows_of_zeros_tiny_ones_and_those_that_are_not_finite(fmt):
    x = torch.randn(6, 512, device="cuda")
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e-30  # 1e-6 under the root outweighs the squares: y is about 1e-27
    w = torch.ones(512, device="cuda")
    y, _, scale = gdr.gdr_rms_norm_fwd(x, w, dtype=fmt)
    q = y.view(torch.uint8)
    assert not q[1:4].any() and scale[1] == 0 and torch.isnan(scale[2:4]).all()
    one = (x[4].double() * 1e3).abs().max() / (448.0 if fmt is E4M3 else 127.0)
    assert abs(float(scale[4]) / float(one) - 1) <= 1e-5 and q[4].any()
    # alone in their rows: the others are as without them
    clean, _, s2 = gdr.gdr_rms_norm_fwd(x[[0, 5]], w, dtype=fmt)
    assert torch.equal(clean.view(torch.uint8), q[[0, 5]]) and torch.equal(s2, scale[[0, 5]])
    # 128 columns with a NaN: every column of its row is NaN, as in the norm itself
    y, _, scale = gdr.gdr_rms_norm_fwd(x, w, dtype=fmt, group=128)
    assert torch.isnan(scale[2]).all() and not y.view(torch.uint8)[2].any()


def test_views_and_in_place():
    s = inputs(50, 96, "bf16")
    ref, r, _ = gdr.gdr_rms_norm_fwd(s["x"], s["w"], s["res"])
    big = torch.randn(5, 10, 200, device="cuda").bfloat16()
    for at in (0, 8, 1):
        big[..., at:at + 96] = s["x"].reshape(5, 10, 96)
        y, r2, _ = gdr.gdr_rms_norm_fwd(big[..., at:at + 96], s["w"], s["res"].reshape(5, 10, 96))
        # rows off 16 bytes are summed in another order
        exact = rms_norm(r.cpu().double(), s["w"].cpu().double(), 1e-6)
        close("y", y.reshape(50, 96), exact)
        assert torch.equal(r2.reshape(50, 96), r)
        out = torch.zeros_like(big)
        gdr.gdr_rms_norm_fwd(s["x"].reshape(5, 10, 96), s["w"], s["res"].reshape(5, 10, 96),
                             y=out[..., at:at + 96])
        close("y", out[..., at:at + 96].reshape(50, 96), exact)
        assert not out[..., :at].any() and not out[..., at + 96:].any()
    # x and the residual are replaced by y and r
    x, res = s["x"].clone(), s["res"].clone()
    gdr.gdr_rms_norm_fwd(x, s["w"], res, y=x, residual_out=res)
    assert torch.equal(x, ref) and torch.equal(res, r)
    x = s["x"].clone()
    y, _, _ = gdr.gdr_rms_norm_fwd(x, s["w"], s["res"], residual_out=x)
    assert torch.equal(x, r) and torch.equal(y, ref)
    with pytest.raises(ValueError):
        gdr.gdr_rms_norm_fwd(big[:, :7, :96], s["w"])  # two strides


@pytest.mark.parametrize("rows", [1, 5, 700])
@pytest.mark.parametrize("D", WIDTHS)
def test_gradients(rows, D):
    for dtype, wdt in (("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")):
        s = inputs(rows, D, dtype, wdt)
        for both in (True, False):
            r, w = wide(s["x"]), wide(s["w"])
            loss = (rms_norm(r, w, 1e-6) * s["dy"].cpu().double()).sum()
            if both:
                loss = loss + (r * s["dr"].cpu().double()).sum()
            loss.backward()
            dx, dw = gdr.gdr_rms_norm_bwd(s["dy"], s["x"], s["w"], s["dr"] if both else None)
            # one value a row: its norm is a sign, and dx all but cancels; of each row's terms
            # rstd |w dy| an FP32 part of 2^-22 is left
            big = float((s["dy"].float() * s["w"].float()).norm() /
                        s["x"].float().square().mean(-1).sqrt().min())
            ref = r.grad
            if D == 1 and not both:
                assert float((dx.cpu().double() - ref).norm()) <= 2.0 ** -20 * big
            else:
                close("dx", dx, ref)
            close("dweight", dw, w.grad)
        dx, none = gdr.gdr_rms_norm_bwd(s["dy"], s["x"])
        assert none is None


def test_gradient_is_the_difference_quotient():
    s = inputs(6, 40, "f32")
    dx, dw = gdr.gdr_rms_norm_bwd(s["dy"], s["x"], s["w"])
    for name, grad in (("x", dx), ("w", dw)):
        v, e = torch.randn_like(s[name]), 2.0 ** -9
        def loss(sign):
            t = dict(s, **{name: s[name] + sign * e * v})
            return (gdr.gdr_rms_norm_fwd(t["x"], t["w"])[0].double() * s["dy"].double()).sum()
        quotient = float(loss(1) - loss(-1)) / (2 * e)
        exact = float((grad.double() * v.double()).sum())
        assert abs(quotient - exact) <= 1e-2 * float(grad.double().norm() * v.double().norm()), name


def test_no_rows():
    x, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, r, scale = gdr.gdr_rms_norm_fwd(x, w, x, dtype=E4M3)
    assert y.shape == (0, 64) and r.shape == (0, 64) and scale.shape == (0,)
    dx, dw = gdr.gdr_rms_norm_bwd(x, x, w)
    assert dx.shape == (0, 64) and not dw.any()


def test_captured_calls():
    s = inputs(300, 256)
    def both():
        y, r, _ = gdr.gdr_rms_norm_fwd(s["x"], s["w"], s["res"])
        return (y, r) + gdr.gdr_rms_norm_bwd(s["dy"], r, s["w"], s["dr"])
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    other = inputs(300, 256, seed=5)
    for k in s:
        s[k].copy_(other[k])
    graph.replay()
    for a, b in zip(out, both()):
        assert torch.equal(a, b)


def test_autograd():
    s = inputs(30, 64, "f32")
    leaf = {k: s[k].clone().requires_grad_() for k in ("x", "w", "res")}
    y, r = gdr.rms_norm(leaf["x"], leaf["w"], leaf["res"])
    ((y * s["dy"]).sum() + (r * s["dr"]).sum()).backward()
    ref = {k: wide(s[k]) for k in leaf}
    total = ref["x"] + ref["res"]
    ((rms_norm(total, ref["w"], 1e-6) * s["dy"].cpu().double()).sum()
     + (total * s["dr"].cpu().double()).sum()).backward()
    for k in leaf:
        close("d" + k, leaf[k].grad, ref[k].grad)
    assert leaf["x"].grad.data_ptr() != leaf["res"].grad.data_ptr()


@pytest.mark.parametrize("rows,D", [(1500, 1288), (1300, 2568), (1100, 5120), (500, 12296)])
def test_rows_of_odd_numbers_of_warps(rows, D):
    """Rows enough that a row has as few warps as hold it, not a power of two."""
    test_forward(rows, D)
    for fmt, group in ((E4M3, 0), (E4M3, 128), (I8, 0)):
        test_eight_bits(rows, D, fmt, group)
    test_gradients(rows, D)
