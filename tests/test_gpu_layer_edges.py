"""The operators of a state-space layer on the GPU where they can go wrong beside their values:
rows in one place, values of FP32's least units, other streams, strided gradients."""
import pytest
import torch

import chunked_gated_delta_rule_gb300 as gdr
from layer_ref import close, rms_norm

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
