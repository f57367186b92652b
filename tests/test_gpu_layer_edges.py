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
