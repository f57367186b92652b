"""The operators of a state-space layer on the CPU: what the binding and the C entry points
refuse before any work.  No compute call is made."""
import pytest
import torch

from chunked_gated_delta_rule_gb300 import layer

D = 16


@pytest.mark.parametrize("rows", [
    torch.zeros(D).expand(8, D), torch.zeros(1, 1, D).expand(1, 8, D), torch.zeros(4, 1, D).expand(4, 8, D),
    torch.zeros(1, 8, D).expand(4, 8, D), torch.zeros(1).expand(8, 1), torch.zeros(1, D).expand(8, 1, D)],
    ids=lambda t: f"{list(t.shape)} at {t.stride()}")
def test_broadcast_rows_are_refused(rows):
    """Their stride is 0, which the C interface takes for rows that lie side by side: as many
    values would be read, or written, far past the one row that there is."""
    with pytest.raises(ValueError, match="rows"):
        layer._row_stride("x", rows)


def test_row_strides():
    wide = torch.zeros(4, 8, 40)
    for t, step in ((wide, 0), (wide[..., :D], 40), (wide[:, 2:3, 3:3 + D], 320), (wide[1:2, :, :D], 40),
                    (wide[:1, :1, 1:1 + D], 0), (wide[0, 0, :D], 0), (wide[:, :, :1], 40),
                    (torch.zeros(0, D), 0), (torch.zeros(1, D).expand(1, D), 0),
                    (torch.zeros(1, 1, D).expand(1, 1, D), 0)):
        assert layer._row_stride("x", t) == step, (t.shape, t.stride())
