"""Measured cases of the operators of a state-space layer: the root-mean-square
norm in front of it (with the residual's addition, and 8-bit outputs), the short
causal convolution, and the selective scan; forward, for training with their
gradients, and for single tokens on rows of a state pool.

``run`` computes them in elementary torch operations, or, where ``own`` is true,
through the library.  Common to all cases: tokens lie in rows, the sequences of a
packed batch one behind the other (``cu``), or as a dense batch; inputs are views
of wider projections, as a layer has them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(op, name, **kw):
    c = dict(name=name, op=op, dtype="bf16")
    if op == "norm":
        c.update(rows=1, width=2048, residual=True, out="same", group=0, train=False)
    else:
        c.update(n=1, lo=1, hi=1, channels=2048, packed=True, pool=False, train=False)
        c.update(dict(taps=4, act=True, bias=True) if op == "conv" else
                 dict(states=16, groups=1, gate=True, skip=True))
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 256 sequences: each takes its last inputs from a pool and puts them back
        _case("conv", "conv step 256", n=256, channels=6144, packed=False, pool=True),
        # prompts of 128 to 512 tokens, FP16, going on from what the pool holds
        _case("conv", "conv prompts 32 f16", n=32, lo=128, hi=512, dtype="f16", pool=True),
        # a training step on 64K tokens in packed sequences of up to 16K
        _case("conv", "conv train 64k", n=8, lo=129, hi=16255, train=True),
        # decode, one sequence: latency
        _case("scan", "scan step 1", channels=1024, packed=False, pool=True),
        # decode, 256 sequences, wide
        _case("scan", "scan step 256", n=256, channels=4096, packed=False, pool=True),
        # prompts of 128 to 512 tokens
        _case("scan", "scan prompts 32", n=32, lo=128, hi=512, pool=True),
        # one long prompt: few sequences, all parallel work lies along the tokens
        _case("scan", "scan one 16k", lo=16384, hi=16384),
        # a training step on a dense batch
        _case("scan", "scan train 8 x 2k", n=8, lo=2048, hi=2048, packed=False, train=True),
        # the same in FP32, odd lengths and channels, two groups, 32 states
        _case("scan", "scan train ragged f32", n=7, lo=1, hi=1023, channels=1000, dtype="f32",
              states=32, groups=2, gate=False, train=True),
        # 64 tokens of a decode step, the norm's output in 8 bits for the next projection
        _case("norm", "norm step 64 e4m3", rows=64, out="e4m3"),
        # 64K tokens of prompts in 8 bits, a scale for each 128 columns
        _case("norm", "norm 64k e4m3", rows=65536, out="e4m3", group=128),
        # a training step, 16K tokens
        _case("norm", "norm train 16k", rows=16384, width=4096, train=True),
    ]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("conv", "scan", "scan", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "norm":
        width = rng.choice((64, 128, 1000, 1024, 1100, 2048, 4096, 8192))
        train = rng.choice((False, True))
        c = _case(op, "", dtype=dtype, width=width, rows=log(1, (1 << 26) // width), train=train,
                  residual=rng.choice((False, True)),
                  out="same" if train else rng.choice(("same", "e4m3", "e4m3")))
        if c["out"] != "same":
            c["group"] = rng.choice((0, 128))
        del c["name"]
        return c
    kind = rng.choice(("step", "prompts", "train"))
    channels = rng.choice((256, 384, 1000, 1024, 2048, 4096))
    top = 134_000_000 if op == "conv" else 33_000_000  # channels x tokens of the largest
    n = log(1, 256 if kind == "step" else 32)
    if kind == "step":
        hi = rng.choice((1, 1, 1, 2, 4))
        c = _case(op, "", n=n, lo=hi, hi=hi, packed=rng.choice((False, True)), pool=True)
    else:
        hi = log(2, min(16384, top // (n * channels)))
        c = _case(op, "", n=n, lo=rng.randint(1, hi), hi=hi, pool=kind == "prompts",
                  train=kind == "train")
    c.update(dtype=dtype, channels=channels)
    if op == "conv":
        c.update(taps=rng.choice((2, 3, 4, 4)), act=rng.choice((True, True, False)),
                 bias=rng.choice((True, False)))
    else:
        c.update(states=rng.choice((8, 16, 16, 16, 24)), groups=rng.choice((1, 1, 2)),
                 gate=rng.choice((True, False)), skip=rng.choice((True, True, False)))
    del c["name"]
    return c


def _lengths(case):
    """Tokens of every sequence, spread over the case's range."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    out = [lo + int(round(((0.5 + 0.6180339887 * i) % 1.0) * (hi - lo))) for i in range(n)]
    if n == 1:
        out[0] = hi
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = dict(case=case)
    if case["op"] == "norm":
        D, R = case["width"], case["rows"]
        # a few channels of a residual stream are much larger than the others
        gain = torch.exp(0.5 * randn(D)) * torch.where(rand(D) < 0.01, 20.0, 1.0)
        x = randn(R, D).to(dt)
        s["w"] = (1.0 + 0.2 * randn(D)).to(dt)
        s["x"] = x if case["residual"] else (x * gain.to(dt))
        s["res"] = (randn(R, D).mul_(gain)).to(dt) if case["residual"] else None
        if case["train"]:
            s["dy"] = randn(R, D).to(dt)
            s["dres"] = randn(R, D).to(dt) if case["residual"] else None
        return s
    lens, C = _lengths(case), case["channels"]
    T, n = sum(lens), case["n"]
    B, L = (1, T) if case["packed"] else (n, lens[0])
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    s.update(T=T, cu=cu.cuda(), longest=max(lens))
    s["cu_arg"] = s["cu"] if case["packed"] else None
    rows = n + n // 8 + 1 if case["pool"] else 0  # some rows of the pool belong to others
    s["idx"] = torch.randperm(rows, generator=gen, device="cuda")[:n].to(torch.int32)
    s["state"] = None
    xz = randn(B, L, 2 * C).to(dt)  # one projection's output
    s["x"], s["z"] = xz[..., :C], None
    if case["op"] == "conv":
        W = case["taps"]
        s["w"] = (randn(C, W) * W ** -0.5).to(dt)
        s["b"] = (0.1 * randn(C)).to(dt) if case["bias"] else None
        if case["pool"]:
            s["state"] = randn(rows, W - 1, C).to(dt)
    else:
        S, G = case["states"], case["groups"]
        if case["gate"]:
            s["z"] = xz[..., C:]
        bc = randn(B, L, 2, G, S).to(dt)
        s["Bm"], s["Cm"] = bc[:, :, 0], bc[:, :, 1]
        s["A"] = -(1.0 + torch.arange(S, device="cuda")) * torch.exp(0.3 * randn(C, S))
        s["D"] = 1.0 + 0.1 * randn(C) if case["skip"] else None
        # time steps of 0.001 to 0.1, a channel's own, moved by its input
        step = torch.exp(math.log(1e-3) + rand(C) * math.log(1e2))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["dt"] = (0.7 * randn(B, L, C)).to(dt)
        if case["pool"]:
            s["state"] = 0.3 * randn(rows, C, S)
    if case["train"]:
        s["dy"] = randn(B, L, C).to(dt)
    return s


# ---- plain forms ----------------------------------------------------------
def _places(s):
    """Sequence of every token, and its place in it."""
    cu, t = s["cu"].long(), torch.arange(s["T"], device=s["cu"].device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, t - cu[seq]


def _rows(x, T):
    return x.reshape(T, *x.shape[2:]).float()


def _plain_conv(s):
    c, T = s["case"], s["T"]
    W, C = c["taps"], c["channels"]
    x, w = _rows(s["x"], T), s["w"].float()
    seq, at = _places(s)
    t = torch.arange(T, device=x.device)
    old = s["state"][s["idx"].long()].float() if s["state"] is not None else None

    def back(j):  # inputs j places before each token's
        y = x[(t - j).clamp(min=0)]
        if old is None:
            return torch.where((at >= j)[:, None], y, torch.zeros_like(y))
        return torch.where((at >= j)[:, None], y, old[seq, (W - 1 + at - j).clamp(max=W - 2)])

    u = s["b"].float().expand(T, C) if s["b"] is not None else torch.zeros(T, C, device=x.device)
    taps = [back(W - 1 - k) for k in range(W)]
    for k in range(W):
        u = u + taps[k] * w[:, k]
    g = torch.sigmoid(u)
    y = (u * g if c["act"] else u).to(s["x"].dtype).reshape(s["x"].shape)
    if c["train"]:
        du = _rows(s["dy"], T)
        if c["act"]:
            du = du * g * (1.0 + u * (1.0 - g))
        left = (s["cu"].long()[1:] - s["cu"].long()[:-1])[seq] - at  # tokens from here on
        dx = torch.zeros_like(x)
        for j in range(W):
            y_j = du[(t + j).clamp(max=T - 1)] * w[:, W - 1 - j]
            dx = dx + torch.where((left > j)[:, None], y_j, torch.zeros_like(y_j))
        dw = torch.stack([(du * taps[k]).sum(0) for k in range(W)], 1)
        out = [y, dx.to(s["x"].dtype).reshape(s["x"].shape), dw]
        return out + ([du.sum(0)] if s["b"] is not None else [])
    if old is None:
        return [y]
    cu = s["cu"].long()
    p = (cu[1:] - cu[:-1])[:, None] + torch.arange(-(W - 1), 0, device=x.device)  # [n, W - 1]
    new = x[(cu[:-1, None] + p).clamp(min=0, max=max(0, T - 1))]
    keep = old[torch.arange(c["n"], device=x.device)[:, None], (W - 1 + p).clamp(max=W - 2)]
    s["state"][s["idx"].long()] = torch.where((p >= 0)[..., None], new, keep).to(s["x"].dtype)
    return [y, s["state"]]


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, h_{-1} = 0, in log2(T) rounds."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _plain_scan(s):
    c, T = s["case"], s["T"]
    C, S, G = c["channels"], c["states"], c["groups"]
    x, dt = _rows(s["x"], T), _rows(s["dt"], T) + s["dt_bias"]
    # log(1 + e^dt), without loss for either sign
    delta = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
    Bm = _rows(s["Bm"], T).repeat_interleave(C // G, 1) if G > 1 else _rows(s["Bm"], T)
    Cm = _rows(s["Cm"], T).repeat_interleave(C // G, 1) if G > 1 else _rows(s["Cm"], T)
    a = torch.exp(delta[..., None] * s["A"])  # [T, C, S]
    b = (delta * x)[..., None] * Bm
    seq, at = _places(s)
    first = (at == 0)[:, None, None]
    idx = s["idx"].long()
    if s["state"] is not None:
        b = b + torch.where(first, a * s["state"][idx][seq], torch.zeros_like(b))
    h = _linear_scan(torch.where(first, torch.zeros_like(a), a), b)
    v = (h * Cm).sum(-1)
    if s["D"] is not None:
        v = v + x * s["D"]
    z = _rows(s["z"], T) if s["z"] is not None else None
    y = v * z * torch.sigmoid(z) if z is not None else v
    y = y.to(s["x"].dtype).reshape(s["x"].shape)
    last = s["cu"].long()[1:] - 1
    if not c["train"]:
        if s["state"] is None:
            return [y, h[last]]
        s["state"][idx] = h[last]
        return [y, s["state"]]
    dv = _rows(s["dy"], T)
    out = {}
    if z is not None:
        g = torch.sigmoid(z)
        out["dz"] = (dv * v * g * (1.0 + z * (1.0 - g))).to(s["x"].dtype).reshape(s["x"].shape)
        dv = dv * z * g
    before = torch.where(first, torch.zeros_like(h), torch.cat([h[:1], h[:-1]]))
    # the gradient of h_t: dh_t = dv_t C_t + a_{t+1} dh_{t+1}, from the last token to the first
    after = torch.cat([a[1:], a[:1]])
    after = torch.where(((s["cu"].long()[1:] - s["cu"].long()[:-1])[seq] - 1 == at)[:, None, None],
                        torch.zeros_like(after), after)
    dh = _linear_scan(after.flip(0), (dv[..., None] * Cm).flip(0)).flip(0)
    del after
    e = dh * a * before
    dhb = (dh * Bm).sum(-1)
    ddelta = (e * s["A"]).sum(-1) + dhb * x
    out["dA"] = (e * delta[..., None]).sum(0)
    dx = dhb * delta
    if s["D"] is not None:
        dx = dx + dv * s["D"]
        out["dD"] = (dv * x).sum(0)
    ddt = ddelta * torch.sigmoid(dt)
    out["ddt_bias"] = ddt.sum(0)
    dB = (dh * (delta * x)[..., None]).reshape(T, G, C // G, S).sum(2)
    dC = (h * dv[..., None]).reshape(T, G, C // G, S).sum(2)
    for name, v_, like in (("dx", dx, s["x"]), ("ddt", ddt, s["dt"]), ("dB", dB, s["Bm"]),
                           ("dC", dC, s["Cm"])):
        out[name] = v_.to(like.dtype).reshape(like.shape)
    out["y"], out["ht"] = y, h[last]
    return out


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(dt)
    v, w = r.float(), s["w"].float()
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
    n = v * rstd
    out = {} if s["res"] is None else {"r": r}
    if c["out"] == "same":
        out["y"] = (n * w).to(dt)
    else:
        R, D = v.shape
        g = c["group"] or D
        y = torch.nn.functional.pad(n * w, (0, -D % g)).reshape(R, -1, g)
        scale = y.abs().amax(-1, keepdim=True) * (1.0 / 448.0)
        q = torch.where(scale > 0, y / scale, torch.zeros_like(y)).reshape(R, -1)[:, :D]
        out["q"], out["scale"] = q.to(torch.float8_e4m3fn), scale[..., 0]
        if not c["group"]:
            out["scale"] = out["scale"][:, 0]
    if c["train"]:
        dy = s["dy"].float()
        wd = w * dy
        dx = rstd * (wd - n * (wd * n).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        out["dx"], out["dw"] = dx.to(dt), (dy * n).sum(0)
    return out


# ---- the library's --------------------------------------------------------
def _own_conv(gdr, s):
    c, act = s["case"], "silu" if s["case"]["act"] else None
    if c["train"]:
        y, _ = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu_arg"], activation=act,
                                      max_seqlen=s["longest"])
        dx, dw, db, _ = gdr.gdr_short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["cu_arg"],
                                               activation=act, max_seqlen=s["longest"])
        return [y, dx, dw] + ([db] if s["b"] is not None else [])
    y, _ = gdr.gdr_short_conv_fwd(s["x"], s["w"], s["b"], s["cu_arg"], activation=act,
                                  state=s["state"], state_indices=s["idx"],
                                  max_seqlen=s["longest"])
    return [y, s["state"]]


def _own_scan(gdr, s):
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    more = (s["D"], s["z"], s["dt_bias"], s["cu_arg"])
    if s["state"] is not None:
        y, _ = gdr.gdr_selective_scan_fwd(*args, *more, state=s["state"], state_indices=s["idx"],
                                          max_seqlen=s["longest"])
        return [y, s["state"]]
    y, ht = gdr.gdr_selective_scan_fwd(*args, *more, max_seqlen=s["longest"])
    if not s["case"]["train"]:
        return [y, ht]
    got = gdr.gdr_selective_scan_bwd(*args, s["dy"], *more, max_seqlen=s["longest"])
    out = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got), y=y, ht=ht)
    return {k: v for k, v in out.items() if v is not None}


def _own_norm(gdr, s):
    c = s["case"]
    y, r, scale = gdr.gdr_rms_norm_fwd(
        s["x"], s["w"], s["res"], dtype=None if c["out"] == "same" else torch.float8_e4m3fn,
        group=c["group"])
    out = {"y": y} if scale is None else {"q": y, "scale": scale}
    if s["res"] is not None:
        out["r"] = r
    if c["train"]:
        out["dx"], out["dw"] = gdr.gdr_rms_norm_bwd(s["dy"], s["x"] if r is None else r, s["w"],
                                                    s["dres"])
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        import chunked_gated_delta_rule_gb300 as gdr
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](gdr, s)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](s)


def work(case):
    es, train = DTYPES[case["dtype"]].itemsize, case["train"]
    if case["op"] == "norm":
        D, R = case["width"], case["rows"]
        res = 1 if case["residual"] else 0
        groups = -(-D // case["group"]) if case["group"] else 1
        y = D * es if case["out"] == "same" else D + 4 * groups
        b = R * (D * es * (1 + 2 * res) + y)
        if train:  # dy, the residual's gradient, dx
            b += R * D * es * (2 + res) + 4 * D
        return {"bytes": float(b + D * es), "flops": float(R * D * (14 if train else 5))}
    T, C, n = sum(_lengths(case)), case["channels"], case["n"]
    pool = 2 if case["pool"] else 0  # rows read and written
    if case["op"] == "conv":
        W = case["taps"]
        b = T * C * es * (4 if train else 2) + pool * n * (W - 1) * C * es + C * W * es
        return {"bytes": float(b), "flops": float(T * C * (2 * W + 4) * (3 if train else 1))}
    S, G = case["states"], case["groups"]
    wide = 3 + case["gate"]
    b = T * C * es * wide + T * 2 * G * S * es + C * S * 4
    b += pool * n * C * S * 4 if case["pool"] else n * C * S * 4
    if train:
        b += T * C * es * (3 + case["gate"]) + T * 2 * G * S * es + C * S * 4
    return {"bytes": float(b), "flops": float(T * C * S * (26 if train else 7))}


# ---- the definitions in 64 bits, token by token and sequence by sequence ----
def _spans(s):
    cu = s["cu"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_conv(s):
    c, T = s["case"], s["T"]
    W, C = c["taps"], c["channels"]
    x, w = s["x"].reshape(T, C), s["w"].double()
    y = torch.zeros(T, C, dtype=torch.float64, device=x.device)
    dx = torch.zeros_like(y) if c["train"] else None
    dw, db = torch.zeros_like(w), torch.zeros(C, dtype=torch.float64, device=x.device)
    state = s["state"].double() if s["state"] is not None else None
    rows = s["idx"].tolist()
    for i, (a, b) in enumerate(_spans(s)):
        head = state[rows[i]] if state is not None else x.new_zeros(W - 1, C, dtype=torch.float64)
        ext, L = torch.cat([head, x[a:b].double()]), b - a
        u = s["b"].double().repeat(L, 1) if s["b"] is not None else torch.zeros_like(y[a:b])
        for k in range(W):
            u = u + ext[k:k + L] * w[:, k]
        y[a:b] = u / (1.0 + torch.exp(-u)) if c["act"] else u
        if state is not None:
            state[rows[i]] = ext[L:]
        if c["train"]:
            du = s["dy"].reshape(T, C)[a:b].double()
            if c["act"]:
                e = torch.exp(-u)
                du = du * (1.0 + e + u * e) / (1.0 + e) ** 2
            dext = torch.zeros_like(ext)
            for k in range(W):
                dext[k:k + L] += du * w[:, k]
                dw[:, k] += (du * ext[k:k + L]).sum(0)
            db += du.sum(0)
            dx[a:b] = dext[W - 1:]
    y = y.reshape(s["x"].shape)
    if c["train"]:
        return [y, dx.reshape(s["x"].shape), dw] + ([db] if s["b"] is not None else [])
    return [y] + ([state] if state is not None else [])


def _exact_scan(s):
    c, T = s["case"], s["T"]
    C, S, G, n = c["channels"], c["states"], c["groups"], c["n"]
    spans = _spans(s)
    L = max(b - a for a, b in spans)
    if c["train"] and n * L * C * S > 1.2e9 or L > 20000:
        return None

    def pad(x):  # [L, n, ...] in 64 bits, zero past each end
        x = x.reshape(T, *x.shape[2:])
        out = x.new_zeros(L, n, *x.shape[1:], dtype=torch.float64)
        for i, (a, b) in enumerate(spans):
            out[:b - a, i] = x[a:b].double()
        return out

    def packed(x):
        return torch.cat([x[:b - a, i] for i, (a, b) in enumerate(spans)])

    A = s["A"].double()
    live = torch.zeros(L, n, 1, dtype=torch.float64, device=A.device)
    for i, (a, b) in enumerate(spans):
        live[:b - a, i] = 1.0
    x, raw = pad(s["x"]), pad(s["dt"]) + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw)) * live  # past the end the state stands still
    Bm, Cm = pad(s["Bm"]), pad(s["Cm"])

    def wide(v):  # [n, G, S] -> [n, C, S]
        return v[:, :, None].expand(n, G, C // G, S).reshape(n, C, S)

    state = s["state"].double() if s["state"] is not None else None
    h = state[s["idx"].long()] if state is not None else A.new_zeros(n, C, S)
    hs = A.new_zeros(L + 1, n, C, S) if c["train"] else None
    v = torch.zeros_like(x)
    for t in range(L):
        h = torch.exp(delta[t][..., None] * A) * h + (delta[t] * x[t])[..., None] * wide(Bm[t])
        v[t] = torch.einsum("ncs,ncs->nc", h, wide(Cm[t]))
        if hs is not None:
            hs[t + 1] = h
    if s["D"] is not None:
        v = v + x * s["D"].double()
    z = pad(s["z"]) if s["z"] is not None else None
    y = v * z / (1.0 + torch.exp(-z)) if z is not None else v
    shape = s["x"].shape
    if state is not None:
        state[s["idx"].long()] = h
        return [packed(y).reshape(shape), state]
    if not c["train"]:
        return [packed(y).reshape(shape), h]
    out = {"y": packed(y).reshape(shape), "ht": h}
    dv = pad(s["dy"])
    if z is not None:
        e = torch.exp(-z)
        out["dz"] = packed(dv * v * (1.0 + e + z * e) / (1.0 + e) ** 2).reshape(shape)
        dv = dv * z / (1.0 + e)
    dA, dh = torch.zeros_like(A), A.new_zeros(n, C, S)
    dx, dd, dB, dC = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(Bm), torch.zeros_like(Cm)
    for t in reversed(range(L)):
        dh = dh + dv[t][..., None] * wide(Cm[t])
        dC[t] = (hs[t + 1] * dv[t][..., None]).reshape(n, G, -1, S).sum(2)
        dB[t] = (dh * (delta[t] * x[t])[..., None]).reshape(n, G, -1, S).sum(2)
        dhb = torch.einsum("ncs,ncs->nc", dh, wide(Bm[t]))
        dx[t] = dhb * delta[t]
        dh = dh * torch.exp(delta[t][..., None] * A)
        e = dh * hs[t]
        dd[t] = torch.einsum("ncs,cs->nc", e, A) + dhb * x[t]
        dA += torch.einsum("ncs,nc->cs", e, delta[t])
    if s["D"] is not None:
        dx = dx + dv * s["D"].double()
        out["dD"] = (dv * x).sum((0, 1))
    ddt = dd * live / (1.0 + torch.exp(-raw))
    out["ddt_bias"], out["dA"] = ddt.sum((0, 1)), dA
    out["dx"], out["ddt"] = packed(dx).reshape(shape), packed(ddt).reshape(shape)
    out["dB"], out["dC"] = packed(dB).reshape(s["Bm"].shape), packed(dC).reshape(s["Cm"].shape)
    return out


def _exact_norm(s):
    c, dt = s["case"], s["x"].dtype
    # the residual's sum is rounded to the inputs' type before the norm sees it
    full = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    r = full if s["res"] is None else full.to(dt).double()
    w = s["w"].double()
    R, D = r.shape
    inv = 1.0 / torch.sqrt((r * r).sum(-1, keepdim=True) / D + 1e-6)
    y = r * inv * w
    out = {} if s["res"] is None else {"r": full}
    if c["out"] == "same":
        out["y"] = y
    else:
        g = c["group"] or D
        q, scale = torch.zeros_like(y), []
        for at in range(0, D, g):
            part = y[:, at:at + g]
            one = part.abs().amax(-1, keepdim=True) / 448.0
            part = part / torch.where(one > 0, one, torch.ones_like(one))
            # E4M3: steps of 2^(e - 3), and of 2^-9 below 2^-6
            unit = torch.exp2(torch.floor(torch.log2(part.abs().clamp(min=2.0 ** -6))) - 3)
            q[:, at:at + g] = torch.round(part / unit) * unit
            scale.append(one)
        out["q"] = q
        out["scale"] = torch.cat(scale, 1) if c["group"] else scale[0][:, 0]
    if c["train"]:
        dn = s["dy"].double() * w
        dx = inv * dn - r * inv ** 3 * (dn * r).sum(-1, keepdim=True) / D
        out["dx"] = dx if s["dres"] is None else dx + s["dres"].double()
        out["dw"] = (s["dy"].double() * r * inv).sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
