"""Measured cases of the paged cache and the attention that reads it.

Three operators: writing new keys and values into a paged cache (quantising
them on the way), reading them back, and softmax attention of new tokens over
the cache (chunks of a prompt, and single tokens).  ``run`` computes them in
elementary torch operations, or, where ``own`` is true, through the library.

Common to all cases: ``kv_lens[n]`` counts sequence n's tokens including this
pass's, token i of its L new ones sits at position ``kv_lens[n] - L + i``, and
position p is slot ``p % page`` of page ``page_table[n, p // page]``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
QMAX = {"e4m3": 448.0, "int8": 127.0}


def _attn(name, **kw):
    c = dict(name=name, op="attn", n=1, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, idle=0, heads=16,
             kv_heads=4, dim=128, page=64, dtype="bf16", fmt="same", window=0, packed=True)
    c.update(kw)
    return c


def _cache(name, **kw):
    c = dict(name=name, op="cache", n=1, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, idle=0, heads=16,
             kv_heads=4, dim=128, page=64, dtype="bf16", fmt="e4m3", window=0, packed=True)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 256 sequences: a token each into the cache
        _cache("cache step 256 e4m3", n=256, kv_lo=1, kv_hi=2048, packed=False),
        # a batch of 32 packed prompts of 128 to 512 tokens, FP16, 8-bit integers
        _cache("cache prompts int8 f16", n=32, q_lo=128, q_hi=512, kv_lo=128, kv_hi=512,
               dtype="f16", fmt="int8", page=16),
        # one 64K-token context at 8 heads, written and read back whole
        _cache("cache 64k x 8 e4m3", q_lo=65536, q_hi=65536, kv_lo=65536, kv_hi=65536, heads=8,
               kv_heads=8),
        # first pass over 32 packed prompts of 128 to 512 tokens, nothing cached before
        _attn("prompts 32", n=32, q_lo=128, q_hi=512, kv_lo=128, kv_hi=512),
        # the last chunk of a 32K context: 4096 new tokens over 28K cached
        _attn("chunk 4096 of 32k", q_lo=4096, q_hi=4096, kv_lo=32768, kv_hi=32768),
        # the same chunk over a quantised cache, half as long
        _attn("chunk 4096 of 16k e4m3", q_lo=4096, q_hi=4096, kv_lo=16384, kv_hi=16384,
              fmt="e4m3"),
        # mixed chunks of odd lengths, FP16, window of 1000, 64-wide heads in groups of three,
        # a page size that ends inside tiles, two sequences idle
        _attn("ragged window f16 d64", n=9, q_lo=1, q_hi=601, kv_lo=601, kv_hi=7001, idle=2,
              heads=12, kv_heads=4, dim=64, page=48, dtype="f16", window=1000),
        # four drafted tokens a sequence, checked in one pass over an 8-bit integer cache
        _attn("draft 4 x 64 int8", n=64, q_lo=4, q_hi=4, kv_lo=100, kv_hi=4096, fmt="int8"),
        # decode, one sequence with a short context: latency
        _attn("decode 1 x 300", kv_lo=300, kv_hi=300, packed=False),
        # decode, 256 sequences of up to 2048 tokens, 8 slots of the batch idle
        _attn("decode 256 x 2k", n=256, kv_lo=1, kv_hi=2048, idle=8, packed=False),
        # decode, 32 sequences of up to 16K tokens over a quantised cache
        _attn("decode 32 x 16k e4m3", n=32, kv_lo=1024, kv_hi=16384, fmt="e4m3", packed=False),
        # decode, one 64K context, every key head its own query head, FP16
        _attn("decode 1 x 64k f16", kv_lo=65536, kv_hi=65536, heads=8, kv_heads=8, dtype="f16",
              page=16, packed=False),
    ]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 8) if kv_heads < 4 else (1, 2, 3, 4))
    heads = min(heads, 16) // kv_heads * kv_heads
    base = dict(heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 48, 64, 128)),
                dtype=rng.choice(("bf16", "f16")))
    kind = rng.choice(("cache", "chunk", "decode"))
    if kind == "cache":
        n = log(1, 256)
        hi = log(1, max(1, min(65536, 380_000 // (n * kv_heads))))
        c = _cache("", n=n, q_lo=rng.randint(1, hi), q_hi=hi, fmt=rng.choice(("e4m3", "int8", "same")),
                   packed=True, **base)
        c["kv_lo"], c["kv_hi"] = hi, hi + log(1, 2048)
    elif kind == "chunk":
        n = log(1, 32)
        hi = log(2, max(2, min(4096, 16384 // n)))
        kv_hi = hi + log(1, max(2, min(28672, 60_000_000 // (n * hi), 900_000 // (n * kv_heads))))
        c = _attn("", n=n, q_lo=rng.randint(1, hi), q_hi=hi, kv_lo=rng.randint(hi, kv_hi), kv_hi=kv_hi,
                  idle=rng.choice((0, 0, 1)) if n > 1 else 0, window=rng.choice((0, 0, log(16, 4096))),
                  fmt=rng.choice(("same", "same", "e4m3", "int8")), **base)
    else:
        n = log(1, 256)
        kv_hi = log(16, max(16, min(65536, 900_000 // (n * kv_heads))))
        t = rng.choice((1, 1, 2, 4)) if kv_hi >= 4 else 1
        c = _attn("", n=n, q_lo=t, q_hi=t, kv_lo=rng.randint(t, kv_hi), kv_hi=kv_hi,
                  idle=rng.choice((0, n // 8)), window=rng.choice((0, 0, 0, log(16, 4096))),
                  fmt=rng.choice(("same", "same", "e4m3", "int8")), packed=t > 1, **base)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, cached tokens including them) of every sequence, spread
    over the case's ranges; the last ``idle`` sequences have none."""
    n, idle = case["n"], case["idle"]
    q, kv = [], []
    for i in range(n):
        u, w = (0.5 + 0.6180339887 * i) % 1.0, (0.9999 + 0.7548776662 * i) % 1.0
        a = case["q_lo"] + int(round(u * (case["q_hi"] - case["q_lo"])))
        b = case["kv_lo"] + int(round(w * (case["kv_hi"] - case["kv_lo"])))
        if i == 0:
            a, b = case["q_hi"], case["kv_hi"]
        if i >= n - idle:  # a slot of the batch without a sequence; dense batches keep its row
            a, b = (0 if case["packed"] else case["q_hi"]), 0
        else:
            b = max(a, b)
        q.append(a)
        kv.append(b)
    return q, kv


def _quantise(x, fmt):
    """Row-wise 8-bit values and FP32 scales, in 32 bits."""
    x = x.float()
    scale = x.abs().amax(-1) * (1.0 / QMAX[fmt])
    y = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    if fmt == "e4m3":
        return y.to(torch.float8_e4m3fn), scale
    return y.round().to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt, fmt, page = DTYPES[case["dtype"]], case["fmt"], case["page"]
    H, Hk, D, n = case["heads"], case["kv_heads"], case["dim"], case["n"]
    q_len, kv_len = _lengths(case)
    T = sum(q_len)
    max_pages = max(1, -(-max(kv_len) // page))
    used = sum(-(-b // page) for b in kv_len)
    n_pages = used + used // 8 + 1  # some pages belong to nobody
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    lens = torch.tensor(kv_len, dtype=torch.int32)
    counts = (lens + page - 1) // page
    first = torch.cumsum(counts, 0) - counts
    at = first[:, None] + torch.arange(max_pages)
    table = perm[at.clamp(max=n_pages - 1).cuda()].contiguous()
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(q_len), 0)
    # keys have channels of different size, tokens values of different size
    gain = torch.exp(0.3 * randn(Hk, D))
    s = dict(case=case, T=T, max_q=max(q_len), max_kv=max(1, max(kv_len)), table=table,
             lens=lens.cuda(), cu=cu.cuda(), scale=1.0 / math.sqrt(D), ks=None, vs=None)
    B, L = (1, T) if case["packed"] else (n, case["q_hi"])
    s["cu_arg"] = s["cu"] if case["packed"] else None
    kc = (randn(n_pages, page, Hk, D) * gain).to(dt)
    vc = (randn(n_pages, page, Hk, D) * torch.exp(0.3 * randn(n_pages, page, Hk, 1))).to(dt)
    if fmt != "same":
        kc, ks = _quantise(kc, fmt)
        vc, vs = _quantise(vc, fmt)
        s["ks"], s["vs"] = (x.transpose(1, 2).contiguous() for x in (ks, vs))
    s["kc"], s["vc"] = kc, vc
    if case["op"] == "cache":
        s["k"] = (randn(B, L, Hk, D) * gain).to(dt)
        s["v"] = (randn(B, L, Hk, D) * torch.exp(0.3 * randn(B, L, Hk, 1))).to(dt)
    else:
        s["q"] = randn(B, L, H, D).to(dt)
    return s


def _slots(s):
    """Page and slot of every new token."""
    lens, cu, page = s["lens"].long(), s["cu"].long(), s["case"]["page"]
    t = torch.arange(s["T"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[seq] - (cu[seq + 1] - t)
    return s["table"][seq, pos // page].long(), pos % page


def _bits(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _plain_write(s, x, cache, scales):
    page, slot = _slots(s)
    x = x.reshape(s["T"], *x.shape[2:])
    if scales is not None:
        x, scale = _quantise(x, s["case"]["fmt"])
        scales[page, :, slot] = scale
    _bits(cache)[page, slot] = _bits(x)


def _plain_read(s, like, cache, scales):
    page, slot = _slots(s)
    x = _bits(cache)[page, slot].view(cache.dtype).float()
    if scales is not None:
        x = x * scales[page, :, slot][..., None]
    return x.to(like.dtype).reshape(like.shape)


def _padded(s, cache, scales):
    """[n, heads, longest, D] in 32 bits, zero past each sequence's end."""
    pos = torch.arange(s["max_kv"], device=cache.device)
    page, slot = s["table"][:, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    x = _bits(cache)[page, slot].view(cache.dtype).float()
    if scales is not None:
        x = x * scales[page, :, slot][..., None]
    live = pos < s["lens"][:, None]
    return torch.where(live[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)


def _plain_attn(s):
    c, q, cu, lens = s["case"], s["q"], s["cu"].long(), s["lens"].long()
    H, Hk, D, n, M = c["heads"], c["kv_heads"], c["dim"], c["n"], s["max_q"]
    k, v = _padded(s, s["kc"], s["ks"]), _padded(s, s["vc"], s["vs"])
    i = torch.arange(M, device=q.device)
    at = (cu[:-1, None] + i).clamp(max=max(0, s["T"] - 1))
    qp = q.reshape(-1, H, D)[at].float()  # [n, M, H, D]
    qp = qp.reshape(n, M, Hk, H // Hk, D).permute(0, 2, 1, 3, 4).reshape(n, Hk, -1, D)
    x = (qp @ k.transpose(2, 3)).mul_(s["scale"]).reshape(n, Hk, M, H // Hk, -1)
    pos = torch.arange(s["max_kv"], device=q.device)
    own_pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i  # [n, M]
    see = (pos <= own_pos[..., None]) & (pos < lens[:, None, None])
    if c["window"]:
        see &= pos > own_pos[..., None] - c["window"]
    x.masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(n, Hk, -1, s["max_kv"]) @ v).reshape(n, Hk, M, -1, D)
    o = o / torch.where(l > 0, l, torch.ones_like(l))
    lse = (torch.log(l) + m).squeeze(-1)
    t = torch.arange(s["T"], device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    row = t - cu[seq]
    o = o.permute(0, 2, 1, 3, 4).reshape(n, M, H, D)[seq, row]
    lse = lse.permute(0, 2, 1, 3).reshape(n, M, H)[seq, row]
    return o.to(q.dtype).reshape(q.shape), lse.reshape(q.shape[:-1])


def run(s):
    if own:
        import chunked_gated_delta_rule_gb300 as gdr
        if s["case"]["op"] == "cache":
            gdr.gdr_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                                s["cu_arg"], k_scale=s["ks"], v_scale=s["vs"])
            k, v = gdr.gdr_cache_read(s["kc"], s["vc"], s["table"], s["lens"], s["k"].shape[1],
                                      s["cu_arg"], k_scale=s["ks"], v_scale=s["vs"],
                                      dtype=s["k"].dtype)
            return [k, v] + ([s["ks"], s["vs"]] if s["ks"] is not None else [])
        return gdr.gdr_paged_attn(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["cu_arg"],
                                  k_scale=s["ks"], v_scale=s["vs"], window=s["case"]["window"],
                                  max_seqlen=s["max_q"])
    if s["case"]["op"] == "cache":
        _plain_write(s, s["k"], s["kc"], s["ks"])
        _plain_write(s, s["v"], s["vc"], s["vs"])
        k = _plain_read(s, s["k"], s["kc"], s["ks"])
        v = _plain_read(s, s["v"], s["vc"], s["vs"])
        return [k, v] + ([s["ks"], s["vs"]] if s["ks"] is not None else [])
    return _plain_attn(s)


def work(case):
    q_len, kv_len = _lengths(case)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    es = DTYPES[case["dtype"]].itemsize
    eb, sb = (es, 0) if case["fmt"] == "same" else (1, 4)
    T = sum(q_len)
    if case["op"] == "cache":
        # rows in, rows written, rows read back, rows out; keys and values
        return {"bytes": 2.0 * T * Hk * 2 * (D * es + D * eb + sb), "flops": 4.0 * T * Hk * D}
    pairs = keys = 0
    w = case["window"]
    for a, b in zip(q_len, kv_len):
        if not a or not b:
            continue
        first = b - a  # the first new token's position
        if w:
            for_p = lambda p: p * (p + 1) // 2 if p < w else w * (w + 1) // 2 + (p - w) * w  # noqa: E731
            keys += b - max(0, first - w + 1)
            pairs += for_p(b) - for_p(first)
        else:
            keys += b
            pairs += a * first + a * (a + 1) // 2
    return {"bytes": float(T * H * (2 * D * es + 4) + keys * Hk * 2 * (D * eb + sb)),
            "flops": 4.0 * D * H * pairs}


# ---- the definition in 64 bits, sequence by sequence ----------------------
def _round64(y, fmt):
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    q_len, kv_len = _lengths(case)
    page, table = case["page"], s["table"].cpu().long()
    H, Hk, D, fmt = case["heads"], case["kv_heads"], case["dim"], case["fmt"]
    if case["op"] == "cache":
        if fmt == "same":
            return [s["k"].double(), s["v"].double()]
        outs, scales = [], []
        for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = x.double()
            amax = x.abs().amax(-1, keepdim=True)
            one = torch.where(amax > 0, amax / QMAX[fmt], torch.ones_like(amax))
            outs.append(_round64(x / one, fmt) * amax / QMAX[fmt])
            sc, flat, at = sc.double(), (amax / QMAX[fmt]).reshape(-1, Hk), 0
            for i, (a, b) in enumerate(zip(q_len, kv_len)):
                if a and b:
                    p = torch.arange(b - a, b)
                    sc[table[i, p // page].cuda(), :, (p % page).cuda()] = flat[at:at + a]
                at += a
            scales.append(sc)
        return outs + scales
    q = s["q"].reshape(-1, H, D).double()
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for i, (a, b) in enumerate(zip(q_len, kv_len)):
        if a and b:
            p = torch.arange(b)
            pg, sl = table[i, p // page].cuda(), (p % page).cuda()

            def rows(cache, sc):
                x = cache[pg, sl] if cache.element_size() > 1 else (
                    cache.view(torch.uint8)[pg, sl].view(cache.dtype))
                x = x.double()
                return x if sc is None else x * sc.double()[pg, :, sl][..., None]

            k, v = rows(s["kc"], s["ks"]), rows(s["vc"], s["vs"])
            qpos = torch.arange(b - a, b, device=q.device)[:, None]
            kpos = torch.arange(b, device=q.device)[None, :]
            hide = kpos > qpos
            if case["window"]:
                hide = hide | (kpos <= qpos - case["window"])
            for h in range(H):
                x = q[at:at + a, h] @ k[:, h // (H // Hk)].T / math.sqrt(D)
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, -1)
                o[at:at + a, h] = torch.exp(x - z[:, None]) @ v[:, h // (H // Hk)]
                lse[at:at + a, h] = z
        at += a
    return o.reshape(s["q"].shape), lse.reshape(s["q"].shape[:-1])
