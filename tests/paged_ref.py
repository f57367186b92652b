"""Plain 64-bit forms of the paged cache and of the attention over it, and
inputs for their tests (CPU, torch float64; no code of the library)."""
import math

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
IO = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CACHE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}

# Relative L2 bounds of o.  16-bit types: the weights and the output are each
# rounded once to nearest, by at most half a unit in the last place (2^-9 of
# the value in BF16, 2^-12 in FP16 beside 2^-11 for its smaller ones), and the
# roundings of different keys are independent, so their sum stays below the
# bound of one: 2^-8 and 2^-10.  FP32: the framework's 1e-5.
TOL_O = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 1e-5}
# lse: FP32 scores of up to 256 products and an exponential good to 2^-21
TOL_LSE = 2e-5


def e4m3_round(y):
    """The nearest E4M3 value (ties to even) of float64 ``y``, |y| <= 448."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def quantise(x, fmt):
    """Stored values (as float64) and FP32 scales of the rows of ``x``: the
    scale is one FP32 product, the quotient is rounded to FP32 first."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = amax * torch.tensor(1.0 / QMAX[fmt], dtype=torch.float32)
    scale = torch.where(torch.isfinite(x).all(-1), scale, torch.tensor(math.nan))
    y = torch.where((scale > 0)[..., None], x / scale[..., None], torch.zeros_like(x)).double()
    q = e4m3_round(y) if fmt == "e4m3" else torch.round(y).clamp(-127, 127)
    return q, scale


class Batch:
    """Lengths, page table and caches of a batch.  ``q_lens`` new tokens and
    ``kv_lens`` cached ones (the new included) of every sequence; every slot
    that no sequence owns holds NaN (16-bit and FP32 caches) or a NaN scale."""

    def __init__(self, q_lens, kv_lens, *, heads=4, kv_heads=2, K=128, V=None, page=16,
                 dtype="bf16", fmt="same", seed=0, dense=False, spare=2):
        g = torch.Generator().manual_seed(seed)
        V = K if V is None else V
        self.q_lens, self.kv_lens, self.page, self.fmt, self.dtype = q_lens, kv_lens, page, fmt, dtype
        self.H, self.Hk, self.K, self.V, self.dense = heads, kv_heads, K, V, dense
        n = len(q_lens)
        counts = [-(-max(0, b) // page) for b in kv_lens]
        self.max_pages = max(1, max(counts, default=1))
        self.n_pages = sum(counts) + spare
        perm = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((n, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = perm[at:at + c]
            at += c
        self.lens = torch.tensor(kv_lens, dtype=torch.int32)
        self.cu = torch.tensor([0] + q_lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        self.T = sum(q_lens)
        lead = (n, q_lens[0] if q_lens else 0) if dense else (1, self.T)
        io = IO[dtype]

        def rows(*shape):
            x = torch.randn(*shape, generator=g)
            return (x * torch.exp(0.5 * torch.randn(*shape[:-1], 1, generator=g))).to(io)

        self.q = torch.randn(*lead, heads, K, generator=g).to(io)
        self.k, self.v = rows(*lead, kv_heads, K), rows(*lead, kv_heads, V)
        self.kc, self.vc = rows(self.n_pages, page, kv_heads, K), rows(self.n_pages, page, kv_heads, V)
        self.ks = self.vs = None
        if fmt != "same":
            (kq, ks), (vq, vs) = quantise(self.kc, fmt), quantise(self.vc, fmt)
            self.kc, self.vc = (x.float().to(CACHE[fmt]) for x in (kq, vq))
            self.ks, self.vs = ks.transpose(1, 2).contiguous(), vs.transpose(1, 2).contiguous()
        owned = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for i, b in enumerate(kv_lens):
            for p in range(max(0, b)):
                owned[self.table[i, p // page], p % page] = True
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            if s is None:
                c[~owned] = math.nan
            else:
                s.transpose(1, 2)[~owned] = math.nan

    def rows64(self, i):
        """Keys and values of sequence i's positions, float64."""
        p = torch.arange(max(0, self.kv_lens[i]))
        pg, sl = self.table[i, p // self.page].long(), p % self.page
        out = []
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            x = c.float()[pg, sl].double()
            out.append(x if s is None else x * s.double()[pg, :, sl][..., None])
        return out

    def attention(self, causal=True, window=0, scale=None):
        """(o, lse), float64, [tokens, H, V] and [tokens, H].  Each row is
        formed from the positions it sees and nothing else."""
        scale = 1 / math.sqrt(self.K) if scale is None else scale
        q = self.q.reshape(-1, self.H, self.K).double()
        o = torch.zeros(q.shape[0], self.H, self.V, dtype=torch.float64)
        lse = torch.full((q.shape[0], self.H), -math.inf, dtype=torch.float64)
        t = 0
        for i, (a, b) in enumerate(zip(self.q_lens, self.kv_lens)):
            k, v = self.rows64(i)
            k, v = (x.repeat_interleave(self.H // self.Hk, 1) for x in (k, v))
            for j in range(a):
                pos = b - a + j
                hi = min(b, pos + 1) if causal else b
                lo = max(0, pos - window + 1) if window else 0
                if hi > lo:
                    s = torch.einsum("hd,jhd->hj", q[t + j], k[lo:hi]) * scale
                    lse[t + j] = torch.logsumexp(s, -1)
                    w = torch.exp(s - lse[t + j][:, None])
                    o[t + j] = torch.einsum("hj,jhd->hd", w, v[lo:hi])
            t += a
        return o, lse

    def on(self, name):
        x = getattr(self, name)
        return None if x is None else x.cuda()

    def run(self, **kw):
        import chunked_gated_delta_rule_gb300 as pkg
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q = kw.pop("q", None)
        o, lse = pkg.gdr_paged_attn(
            self.on("q") if q is None else q, kw.pop("kc", self.on("kc")),
            kw.pop("vc", self.on("vc")), self.on("table"), self.on("lens"),
            None if self.dense else self.on("cu"), k_scale=self.on("ks"), v_scale=self.on("vs"),
            status=status, **kw)
        torch.cuda.synchronize()
        assert int(status) == 0
        return o.reshape(-1, self.H, self.V), lse.reshape(-1, self.H)


def check(batch, o, lse, ref_o, ref_lse, label="", rows=True):
    """o within the bound over the whole tensor and, for every row of 64
    elements and more, within 4 times it; lse by its own bound; rows that see
    nothing exact."""
    o, lse = o.cpu().double(), lse.cpu().double()
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), label
    assert (o[empty] == 0).all(), label
    tol = TOL_O[batch.dtype]
    norm = ref_o.norm()
    err = float((o - ref_o).norm() / norm) if norm > 0 else float((o - ref_o).norm())
    live = ~empty
    dl = ((lse - ref_lse).abs() / (1 + ref_lse.abs()))[live]
    worst = float(dl.max()) if dl.numel() else 0.0
    row = ((o - ref_o).norm(dim=-1) / ref_o.norm(dim=-1).clamp_min(1e-30))[live]
    wrow = float(row.max()) if row.numel() else 0.0
    print(f"{label}: o {err:.2e} (bound {tol:.2e}), worst row {wrow:.2e}, lse {worst:.2e}")
    assert err <= tol, (label, err)
    assert wrow <= 4 * tol, (label, wrow)
    assert worst <= TOL_LSE, (label, worst)
