"""The short convolution, the selective scan and the norm in 64 bits on the CPU, token by
token and sequence by sequence, differentiable; what the GPU tests compare with."""
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def wide(t):
    """A 64-bit leaf on the CPU with the tensor's values."""
    return None if t is None else t.detach().cpu().double().requires_grad_()


def short_conv(x, w, b, lens, h0=None, silu=True):
    """x [tokens, C], h0 [sequences, W - 1, C]; (y, ht)."""
    W, at, ys, hts = w.shape[1], 0, [], []
    for n, L in enumerate(lens):
        head = h0[n] if h0 is not None else x.new_zeros(W - 1, x.shape[1])
        ext = torch.cat([head, x[at:at + L]])
        u = sum(ext[k:k + L] * w[:, k] for k in range(W))
        u = u if b is None else u + b
        ys.append(u * torch.sigmoid(u) if silu else u)
        hts.append(ext[L:])
        at += L
    return torch.cat(ys), torch.stack(hts)


def selective_scan(x, dt, A, B, C, D, z, bias, lens, h0=None, softplus=True):
    """x, dt, z [tokens, C], B and C [tokens, G, S], h0 [sequences, C, S]; (y, ht)."""
    ch, S = A.shape
    rep = ch // B.shape[1]
    d = dt if bias is None else dt + bias
    if softplus:
        d = torch.logaddexp(d, torch.zeros_like(d))
    at, vs, hts = 0, [], []
    for n, L in enumerate(lens):
        h = h0[n] if h0 is not None else x.new_zeros(ch, S)
        for t in range(at, at + L):
            h = torch.exp(d[t][:, None] * A) * h + (d[t] * x[t])[:, None] * B[t].repeat_interleave(rep, 0)
            vs.append((h * C[t].repeat_interleave(rep, 0)).sum(1))
        hts.append(h)
        at += L
    v = torch.stack(vs) if vs else x.new_zeros(0, ch)
    if D is not None:
        v = v + D * x
    if z is not None:
        v = v * z * torch.sigmoid(z)
    return v, torch.stack(hts)


def rms_norm(r, w, eps):
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + eps)
    return n if w is None else n * w


def half_step(dtype):
    """Largest relative error of rounding to dtype (for values in its normal range)."""
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0


def close(name, got, want, dtype=None, work=1e-5):
    """``got`` is ``want`` up to one rounding to its dtype and ``work`` of FP32 arithmetic: relative
    to the whole, and for every value ten times that relative to the root mean square (a sum's
    error follows its terms, not itself).  FP32 products and sums of a few hundred terms, and
    decays of a chain of a few hundred steps, each within 2^-22 of its own, stay within 1e-5."""
    dtype = dtype or got.dtype
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if not want.numel():
        return
    assert torch.isfinite(got).all(), name
    step, err = half_step(dtype), (got - want).abs()
    norm = float(want.norm())
    assert float(err.norm()) <= (step + work) * norm + 1e-30, (name, float(err.norm()) / max(norm, 1e-30))
    rms = norm / want.numel() ** 0.5
    least = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half of FP16's smallest value
    worst = err - (step * want.abs() * 1.001 + 10 * work * rms + least)
    assert float(worst.max()) <= 0, (name, float(worst.max()), rms)
