"""The short causal convolution on the GPU against 64 bits: prompts, single tokens, states in
pools, gradients; and what its entry points refuse or leave alone."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import DTYPES, close, offsets, short_conv, wide

pytestmark = pytest.mark.gpu
LENS = {"one": [1], "short": [2, 1, 3], "holes": [0, 5, 0, 0, 64, 65, 1, 0], "runs": [129, 3, 300],
        "long": [1000]}


def inputs(lens, C, W, dtype="bf16", bias=True, weight_dtype=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]

    def randn(*shape):
        return torch.randn(*shape, generator=gen).to(dt).cuda()

    wd = DTYPES[weight_dtype or dtype]
    return dict(x=randn(1, sum(lens), C), w=(randn(C, W) * 0.5).to(wd),
                b=(0.3 * randn(C)).to(wd) if bias else None, h0=randn(len(lens), W - 1, C),
                dy=randn(1, sum(lens), C), dht=randn(len(lens), W - 1, C), cu=offsets(lens).cuda())


def want(s, lens, silu, h0=True):
    x, w, b, h = (wide(s[k]) for k in ("x", "w", "b", "h0"))
    y, ht = short_conv(x[0], w, b, lens, h if h0 else None, silu)
    return dict(x=x, w=w, b=b, h0=h, y=y[None], ht=ht)


@pytest.mark.parametrize("hint", [1, 1000], ids=["step", "runs"])
@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("C,W,dtype,silu,bias", [
    (64, 4, "bf16", True, True), (1001, 4, "f16", True, True), (24, 3, "f32", False, True),
    (8, 2, "bf16", True, False), (7, 2, "f32", True, True), (512, 3, "f16", False, False)])
def test_forward(lens, hint, C, W, dtype, silu, bias):
    s = inputs(lens, C, W, dtype, bias)
    r = want(s, lens, silu)
    act = "silu" if silu else None
    y, ht = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"], s["h0"], activation=act,
                                   output_final_state=True, max_seqlen=hint)
    close("y", y, r["y"])
    assert torch.equal(ht.cpu().double(), r["ht"].detach())  # inputs, as they were
    y0, none = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"], activation=act,
                                      max_seqlen=hint)
    assert none is None
    close("y from zeros", y0, want(s, lens, silu, h0=False)["y"])


@pytest.mark.parametrize("hint", [1, 1000], ids=["step", "runs"])
def test_pool(hint):
    """Rows of a pool move on in place; a sequence with a row outside it is left alone, gives
    zeros and is reported."""
    lens = [3, 0, 1, 70, 2]
    s = inputs(lens, 40, 4, "f16")
    rows = [5, 2, 9, 0, 11]  # of 8: 9 and 11 do not exist
    pool = torch.randn(8, 3, 40, generator=torch.Generator().manual_seed(3)).half().cuda()
    before, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor(rows, dtype=torch.int32).cuda()
    y, st = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"], state=pool, state_indices=idx,
                                   status=status, max_seqlen=hint)
    assert st is pool and int(status) == -7
    s["h0"] = before[[5, 2, 0, 0, 0]]
    r = want(s, lens, True)
    at = 0
    for n, L in enumerate(lens):
        got = y[0, at:at + L]
        if rows[n] < 8:
            close(f"y of {n}", got, r["y"][0, at:at + L])
            assert torch.equal(pool[rows[n]].cpu().double(), r["ht"][n].detach())
        else:
            assert not got.any()
        at += L
    others = [i for i in range(8) if i not in rows]
    assert torch.equal(pool[others], before[others])


def test_tokens_one_by_one_are_the_whole():
    s = inputs([37], 96, 4, "bf16")
    whole, ht = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], h0=s["h0"], output_final_state=True)
    pool = s["h0"].clone()
    got = [gdr.gdr_short_conv_fwd(s["x"][:, t:t + 1], s["w"], s["b"], state=pool)[0] for t in range(37)]
    assert torch.equal(torch.cat(got, 1), whole) and torch.equal(pool, ht)


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("C,W,dtype,silu,bias,wdt", [
    (64, 4, "bf16", True, True, "bf16"), (1001, 4, "f16", True, True, "f32"),
    (24, 3, "f32", False, True, "f32"), (8, 2, "bf16", True, False, "f32"),
    (512, 3, "f32", True, True, "f32"), (12, 4, "bf16", True, True, "bf16")])
def test_gradients(lens, C, W, dtype, silu, bias, wdt):
    s = inputs(lens, C, W, dtype, bias, wdt)
    act = "silu" if silu else None
    for states in (False, True):
        r = want(s, lens, silu, h0=states)
        loss = (r["y"][0] * s["dy"][0].cpu().double()).sum()
        if states:
            loss = loss + (r["ht"] * s["dht"].cpu().double()).sum()
        loss.backward()
        dx, dw, db, dh0 = gdr.gdr_short_conv_bwd(
            s["x"], s["w"], s["dy"], s["b"], s["cu"], s["h0"] if states else None,
            s["dht"] if states else None, activation=act, want_dh0=states)
        close("dx", dx, r["x"].grad)
        close("dweight", dw, r["w"].grad)
        assert dw.dtype == torch.float32 and (db is None) == (not bias)
        if bias:
            close("dbias", db, r["b"].grad)
        if states:
            close("dh0", dh0, r["h0"].grad)


def test_gradient_is_the_difference_quotient():
    """Along a random direction, in FP32: L(x + e v) - L(x - e v) over 2 e, L in 64 bits of the
    library's own forward.  With |y| about 1 and 2^-22 of FP32 error a value, the quotient is
    off by about 2^-22 sqrt(values) / e + e^2, far below 1e-2 of its size."""
    lens = [9, 30]
    s = inputs(lens, 16, 4, "f32", weight_dtype="f32")
    dx, dw, db, _ = gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["cu"])
    for name, grad in (("x", dx), ("w", dw), ("b", db)):
        v, e = torch.randn_like(s[name]), 2.0 ** -7
        def loss(sign):
            t = dict(s, **{name: s[name] + sign * e * v})
            y, _ = gdr.gdr_short_conv_fwd(t["x"], t["w"], t["b"], s["cu"])
            return (y.double() * s["dy"].double()).sum()
        quotient = float(loss(1) - loss(-1)) / (2 * e)
        exact = float((grad.double() * v.double()).sum())
        assert abs(quotient - exact) <= 1e-2 * float(grad.double().norm() * v.double().norm()), name


def test_views_and_offsets_of_64_bits():
    """x and dy as slices of a wider projection, dense batches, int64 offsets: the bits of
    contiguous tensors."""
    lens = [5, 70, 0, 13]
    s = inputs(lens, 48, 4, "bf16")
    ref, _ = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"])
    big = torch.randn(1, sum(lens), 100, device="cuda").bfloat16()
    for at in (0, 16, 3):  # 3: off 16 bytes
        big[..., at:at + 48] = s["x"]
        view = big[..., at:at + 48]
        y, _ = gdr.gdr_short_conv_fwd(view, s["w"], s["b"], s["cu"].long())
        assert torch.equal(y, ref)
        a = gdr.gdr_short_conv_bwd(view, s["w"], s["dy"], s["b"], s["cu"].long())
        b = gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["cu"])
        assert torch.equal(a[0], b[0])
        close("dweight", a[1], b[1])
        out = torch.zeros_like(big)
        gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"], y=out[..., at:at + 48])
        assert torch.equal(out[..., at:at + 48], ref) and not out[..., :at].any() and not out[..., at + 48:].any()
    dense = s["x"][:, :84].reshape(4, 21, 48)
    got, ht = gdr.gdr_short_conv_fwd(dense, s["w"], s["b"], output_final_state=True)
    cu = offsets([21] * 4).cuda()
    same, ht2 = gdr.gdr_short_conv_fwd(s["x"][:, :84], s["w"], s["b"], cu, output_final_state=True)
    assert torch.equal(got.reshape(1, 84, 48), same) and torch.equal(ht, ht2)


@pytest.mark.parametrize("hint", [1, 1000], ids=["step", "runs"])
def test_tokens_of_no_sequence(hint):
    """Tokens behind the last sequence get zeros, and the table is reported."""
    lens = [4, 9]
    s = inputs(lens + [11], 32, 4, "f32", weight_dtype="f32")
    cu = offsets(lens).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(s["x"], 7.0)
    gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], cu, y=y, status=status, max_seqlen=hint)
    assert int(status) == -5 and not y[:, 13:].any()
    part = s["x"][:, :13].contiguous()
    assert torch.equal(y[:, :13], gdr.gdr_short_conv_fwd(part, s["w"], s["b"], cu)[0])
    a = gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], cu)
    b = gdr.gdr_short_conv_bwd(part, s["w"], s["dy"][:, :13].contiguous(), s["b"], cu)
    assert torch.equal(a[0][:, :13], b[0]) and not a[0][:, 13:].any()
    close("dweight", a[1], b[1])
    # offsets that leave the tensors: reported, nothing outside is touched
    for table in ([0, 30, 24], [-3, 5, 24], [0, 20, 10], [0, 1 << 30, 24]):
        status.zero_()
        guard = torch.full((3, 24, 32), 5.0, device="cuda")
        gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], torch.tensor(table, dtype=torch.int32).cuda(),
                               y=guard[1:2], status=status, max_seqlen=hint)
        assert int(status) == -5 and (guard[0] == 5).all() and (guard[2] == 5).all()


def test_no_tokens():
    s = inputs([0, 0], 32, 4)
    y, ht = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"], s["h0"], output_final_state=True)
    assert y.shape == (1, 0, 32) and torch.equal(ht, s["h0"])
    dx, dw, db, dh0 = gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["cu"], s["h0"],
                                             s["dht"], want_dh0=True)
    assert not dw.any() and not db.any() and torch.equal(dh0, s["dht"])


def test_captured_calls():
    """A captured forward and backward replayed on other values give what eager calls give."""
    lens = [40, 3, 100]
    s = inputs(lens, 64, 4)
    def both():
        y, _ = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu"])
        return (y,) + gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["cu"])[:3]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    other = inputs(lens, 64, 4, seed=5)
    for k in ("x", "w", "b", "dy"):
        s[k].copy_(other[k])
    graph.replay()
    for a, b in zip(out, both()):
        assert torch.equal(a, b)


def test_autograd():
    lens = [6, 20]
    s = inputs(lens, 32, 4, "f32", weight_dtype="f32")
    leaf = {k: s[k].clone().requires_grad_() for k in ("x", "w", "b", "h0")}
    y, ht = gdr.short_conv(leaf["x"], leaf["w"], leaf["b"], initial_state=leaf["h0"],
                           output_final_state=True, cu_seqlens=s["cu"])
    ((y * s["dy"]).sum() + (ht * s["dht"]).sum()).backward()
    r = want(s, lens, True)
    ((r["y"] * s["dy"].cpu().double()).sum() + (r["ht"] * s["dht"].cpu().double()).sum()).backward()
    for k in leaf:
        close("d" + k, leaf[k].grad, r[k].grad)
