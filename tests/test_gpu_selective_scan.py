"""The selective scan on the GPU against 64 bits: whole sequences and pieces, single tokens on
a state pool, gradients; and what its entry points refuse or leave alone."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import DTYPES, close, offsets, selective_scan, wide

pytestmark = pytest.mark.gpu
LENS = {"one": [1], "short": [2, 1, 3], "holes": [0, 5, 0, 0, 64, 33, 1, 0], "pieces": [129, 3, 300]}


def inputs(lens, C, S, G=1, dtype="bf16", skip=True, gate=True, bias=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dt, T, n = DTYPES[dtype], sum(lens), len(lens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    s = dict(x=randn(1, T, C).to(dt), dt=(randn(1, T, C) - 2.0).to(dt),
             A=-torch.exp(randn(C, S)), B=randn(1, T, G, S).to(dt), C=randn(1, T, G, S).to(dt),
             D=randn(C) if skip else None, z=randn(1, T, C).to(dt) if gate else None,
             bias=0.5 * randn(C) if bias else None, h0=randn(n, C, S), dy=randn(1, T, C).to(dt),
             dht=randn(n, C, S), cu=offsets(lens))
    return {k: v if v is None else v.cuda() for k, v in s.items()}


NAMES = ("x", "dt", "A", "B", "C", "D", "z", "bias")


def want(s, lens, h0=True, softplus=True):
    r = {k: wide(s[k]) for k in NAMES + ("h0",)}
    flat = {k: r[k][0] if k in ("x", "dt", "B", "C", "z") and r[k] is not None else r[k] for k in NAMES}
    y, ht = selective_scan(flat["x"], flat["dt"], flat["A"], flat["B"], flat["C"], flat["D"], flat["z"],
                           flat["bias"], lens, r["h0"] if h0 else None, softplus)
    return dict(r, y=y[None], ht=ht)


def forward(s, **kw):
    return gdr.gdr_selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"],
                                      kw.pop("cu", s["cu"]), **kw)


def backward(s, **kw):
    return gdr.gdr_selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], s["D"], s["z"],
                                      s["bias"], kw.pop("cu", s["cu"]), **kw)


SHAPES = [(64, 16, 1, "bf16", True, True, True), (40, 16, 2, "f16", True, True, False),
          (33, 5, 1, "f32", False, True, True), (300, 4, 1, "bf16", True, False, True),
          (24, 32, 3, "f32", True, True, True), (20, 64, 1, "bf16", False, False, True),
          (130, 8, 1, "f32", True, False, False), (17, 19, 1, "f16", True, True, True),
          (8, 50, 2, "f32", True, True, True), (257, 1, 1, "f32", True, True, True)]


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(lens, shape):
    s = inputs(lens, *shape)
    r = want(s, lens)
    runs = {"step": dict(max_seqlen=1), "whole": dict(n_segments=1), "planned": dict(max_seqlen=max(lens)),
            "pieces": dict(n_segments=9, max_seqlen=max(lens)), "many": dict(n_segments=2, max_seqlen=33)}
    for name, kw in runs.items():
        y, ht = forward(s, h0=s["h0"], **kw)
        close("y " + name, y, r["y"])
        close("ht " + name, ht, r["ht"])
    y, none = forward(s, output_final_state=False)
    assert none is None
    close("y from zeros", y, want(s, lens, h0=False)["y"])


def test_time_steps_as_they_are_and_far_ones():
    """Without softplus; and with time steps from e^-30 to 40, where softplus is one of its
    asymptotes.  A state that decays by e^-40 and more is gone; FP32 holds e^-30 to its last bit."""
    lens = [50]
    s = inputs(lens, 32, 16, dtype="f32")
    s["dt"] = s["dt"].abs()
    y, ht = forward(s, softplus=False, h0=s["h0"])
    r = want(s, lens, softplus=False)
    close("y", y, r["y"])
    close("ht", ht, r["ht"])
    (r["y"] * s["dy"].cpu().double()).sum().backward()
    got = backward(s, softplus=False, h0=s["h0"])
    for k, g in zip(NAMES, got):
        close("d" + k, g, r[k].grad)
    s["dt"] = torch.linspace(-30.0, 40.0, 50 * 32).reshape(1, 50, 32).cuda()
    y, ht = forward(s, h0=s["h0"])
    r = want(s, lens)
    close("y", y, r["y"])
    close("ht", ht, r["ht"])


@pytest.mark.parametrize("kw", [dict(max_seqlen=1), dict(n_segments=1), dict(n_segments=3, max_seqlen=70)],
                         ids=["step", "whole", "pieces"])
def test_pool(kw):
    lens, rows = [3, 0, 1, 70, 2], [5, 2, 9, 0, -1]  # of 8: 9 and -1 do not exist
    s = inputs(lens, 40, 16, dtype="f32")
    pool = torch.randn(8, 40, 16, generator=torch.Generator().manual_seed(3)).cuda()
    before, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    y, st = forward(s, state=pool, state_indices=torch.tensor(rows, dtype=torch.int32).cuda(),
                    status=status, **kw)
    assert st is pool and int(status) == -7
    s["h0"] = before[[5, 2, 0, 0, 0]]
    r = want(s, lens)
    at = 0
    for n, L in enumerate(lens):
        if 0 <= rows[n] < 8:
            close(f"y of {n}", y[0, at:at + L], r["y"][0, at:at + L])
            close(f"state of {n}", pool[rows[n]], r["ht"][n])
        else:
            assert not y[0, at:at + L].any()
        at += L
    others = [i for i in range(8) if i not in rows]
    assert torch.equal(pool[others], before[others])


def test_tokens_one_by_one_are_the_whole():
    """FP32 sums over the states are taken in another order by the two kernels."""
    s = inputs([37], 96, 16, dtype="f32")
    whole, ht = forward(s, h0=s["h0"], n_segments=1)
    pool, got = s["h0"].clone(), []
    for t in range(37):
        one = {k: v[:, t:t + 1] if k in ("x", "dt", "z", "B", "C") else v for k, v in s.items()}
        got.append(forward(one, cu=None, state=pool)[0])
    close("y", torch.cat(got, 1), whole)
    close("states", pool, ht)


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(lens, shape):
    s = inputs(lens, *shape)
    for states in (False, True):
        r = want(s, lens, h0=states)
        loss = (r["y"] * s["dy"].cpu().double()).sum()
        if states:
            loss = loss + (r["ht"] * s["dht"].cpu().double()).sum()
        loss.backward()
        kw = dict(h0=s["h0"], dht=s["dht"], want_dh0=True) if states else {}
        got = backward(s, **kw)
        for k, g in zip(NAMES, got):
            assert (g is None) == (s[k] is None), k
            if g is not None:
                assert g.dtype == s[k].dtype
                # a loss that does not reach an input leaves no gradient there
                close("d" + k, g, torch.zeros_like(r[k]) if r[k].grad is None else r[k].grad)
        if states:
            close("dh0", got[8], r["h0"].grad)
        else:
            assert got[8] is None


def test_gradient_is_the_difference_quotient():
    """As for the short convolution: 64-bit sums of the library's FP32 outputs."""
    lens = [9, 140]
    s = inputs(lens, 16, 16, dtype="f32")
    got = backward(s)
    for k, grad in zip(NAMES, got):
        v, e = torch.randn_like(s[k]), 2.0 ** -7
        def loss(sign):
            y, _ = forward(dict(s, **{k: s[k] + sign * e * v}))
            return (y.double() * s["dy"].double()).sum()
        quotient = float(loss(1) - loss(-1)) / (2 * e)
        exact = float((grad.double() * v.double()).sum())
        assert abs(quotient - exact) <= 1e-2 * float(grad.double().norm() * v.double().norm()), k


def test_views_and_offsets_of_64_bits():
    lens = [5, 70, 0, 13]
    s = inputs(lens, 48, 16, 2)
    ref, ht = forward(s)
    grads = backward(s)
    for at in (0, 16, 3):  # 3: off 16 bytes
        big = torch.randn(1, 88, 250, device="cuda").bfloat16()
        v = dict(s)
        for i, k in enumerate(("x", "dt", "z")):
            big[..., at + 50 * i:at + 50 * i + 48] = s[k]
            v[k] = big[..., at + 50 * i:at + 50 * i + 48]
        bc = torch.randn(1, 88, 2, 2, 20, device="cuda").bfloat16()
        bc[:, :, 0, :, at % 4:at % 4 + 16], bc[:, :, 1, :, :16] = s["B"], s["C"]
        v["B"], v["C"] = bc[:, :, 0, :, at % 4:at % 4 + 16], bc[:, :, 1, :, :16]
        y, ht2 = forward(v, cu=s["cu"].long())
        assert torch.equal(y, ref) and torch.equal(ht, ht2)
        for a, b in zip(backward(v, cu=s["cu"].long()), grads):
            assert (a is None and b is None) or torch.equal(a, b)
        out = torch.zeros(1, 88, 90, device="cuda").bfloat16()
        forward(s, y=out[..., at:at + 48])
        assert torch.equal(out[..., at:at + 48], ref) and not out[..., :at].any()
    dense = {k: v[:, :84].reshape(4, 21, *v.shape[2:]) if k in ("x", "dt", "z", "B", "C", "dy") else v
             for k, v in s.items()}
    cu = offsets([21] * 4).cuda()
    part = {k: v[:, :84] if k in ("x", "dt", "z", "B", "C", "dy") else v for k, v in s.items()}
    (a, ah), (b, bh) = forward(dense, cu=None), forward(part, cu=cu)
    assert torch.equal(a.reshape(1, 84, 48), b) and torch.equal(ah, bh)
    for p, q in zip(backward(dense, cu=None), backward(part, cu=cu)):
        assert (p is None and q is None) or torch.equal(p.reshape(q.shape), q)


@pytest.mark.parametrize("kw", [dict(max_seqlen=1), dict(n_segments=1), dict(n_segments=3, max_seqlen=90)],
                         ids=["step", "whole", "pieces"])
def test_tokens_of_no_sequence(kw):
    lens = [4, 90]
    s = inputs(lens + [150], 32, 16, dtype="f32")
    cu, status = offsets(lens).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full_like(s["x"], 7.0)
    forward(s, cu=cu, y=y, status=status, **kw)
    assert int(status) == -5 and not y[:, 94:].any()
    rows = ("x", "dt", "z", "B", "C", "dy")
    part = {k: v[:, :94].contiguous() if k in rows else v for k, v in s.items()}
    close("y", y[:, :94], forward(part, cu=cu, n_segments=1)[0])
    a, b = backward(s, cu=cu), backward(part, cu=cu)
    for k, p, q in zip(NAMES, a, b):
        if k in rows:
            assert torch.equal(p[:, :94], q) and not p[:, 94:].any(), k
        else:
            close("d" + k, p, q)
    for table in ([0, 300, 244], [-3, 5, 244], [0, 200, 100], [0, 1 << 30, 244]):
        status.zero_()
        guard = torch.full((3, 244, 32), 5.0, device="cuda")
        bad = torch.tensor(table, dtype=torch.int32).cuda()
        forward(s, cu=bad, y=guard[1:2], status=status, **kw)
        assert int(status) == -5 and (guard[0] == 5).all() and (guard[2] == 5).all()
        status.zero_()
        backward(s, cu=bad, status=status)
        assert int(status) == -5


def test_no_tokens():
    s = inputs([0, 0], 32, 16)
    for kw in (dict(), dict(n_segments=1), dict(n_segments=4, max_seqlen=100)):
        y, ht = forward(s, h0=s["h0"], **kw)
        assert y.shape == (1, 0, 32) and torch.equal(ht, s["h0"])
    got = backward(s, h0=s["h0"], dht=s["dht"], want_dh0=True)
    assert torch.equal(got[8], s["dht"])
    assert not any(t.any() for t in got[:8])


def test_values_that_are_not_finite_stay_in_their_channel_and_sequence():
    lens = [20, 20, 20]
    s = inputs(lens, 32, 16, dtype="f32")
    ref, ht = forward(s, n_segments=1)
    s["x"][0, 25, 3], s["dt"][0, 30, 7] = float("inf"), float("nan")
    y, ht2 = forward(s, n_segments=1)
    ok = torch.ones_like(ref, dtype=torch.bool)
    ok[0, 25:40, 3] = ok[0, 30:40, 7] = False
    assert torch.equal(y[ok], ref[ok]) and not torch.isfinite(y[0, 25, 3])
    assert torch.isnan(y[0, 30:40, 7]).all() and torch.isnan(ht2[1, 7]).all()
    assert torch.equal(ht2[[0, 2]], ht[[0, 2]])


def test_states_that_forget_at_once():
    """A = -inf: a decay of zero for every token, and none for the places past a sequence's end that
    tiles and pieces are filled up with."""
    lens = [20, 33, 100]
    s = inputs(lens, 32, 16, dtype="f32")
    s["A"][3, 5] = -float("inf")
    r = want(dict(s, A=s["A"].clamp(min=-1e30)), lens)
    for kw in (dict(max_seqlen=1), dict(n_segments=1), dict(n_segments=3, max_seqlen=100)):
        y, ht = forward(s, h0=s["h0"], **kw)
        close("y", y, r["y"])
        close("ht", ht, r["ht"])
    got = backward(s, h0=s["h0"])
    (r["y"] * s["dy"].cpu().double()).sum().backward()
    for k, g in zip(NAMES, got):
        close("d" + k, g, r[k].grad)


def test_captured_calls_and_own_scratch():
    """A captured forward (in pieces) and backward replayed on other values, the caller's
    scratch, and a second run give the same bits; too little scratch is refused."""
    lens = [200, 3, 100]
    s = inputs(lens, 64, 16)
    def both(**kw):
        return forward(s, n_segments=4, max_seqlen=200) + backward(s, **kw)[:8]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    other = inputs(lens, 64, 16, seed=5)
    for k in s:
        s[k].copy_(other[k])
    graph.replay()
    from chunked_gated_delta_rule_gb300 import layer
    size = layer.gdr_selective_scan_workspace_size(1, 303, 64, 16, N=3, backward=True)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for a, b, c in zip(out, both(), both(workspace=ws)):
        assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(gdr.GdrError) as e:
        backward(s, workspace=ws[:-256])
    assert e.value.code == -6


def test_autograd():
    lens = [6, 40]
    s = inputs(lens, 32, 16, dtype="f32")
    leaf = {k: s[k].clone().requires_grad_() for k in NAMES + ("h0",)}
    y, ht = gdr.selective_scan(*(leaf[k] for k in NAMES), initial_state=leaf["h0"],
                               output_final_state=True, cu_seqlens=s["cu"])
    ((y * s["dy"]).sum() + (ht * s["dht"]).sum()).backward()
    r = want(s, lens)
    ((r["y"] * s["dy"].cpu().double()).sum() + (r["ht"] * s["dht"].cpu().double()).sum()).backward()
    for k in leaf:
        close("d" + k, leaf[k].grad, r[k].grad)
