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


def test_outputs_in_32_bits_whatever_the_default():
    """What the library writes in FP32 is made as FP32 (with another default dtype it would be
    written past its end): every torch.empty of the binding names its type."""
    import ast
    import inspect
    calls = [n for n in ast.walk(ast.parse(inspect.getsource(layer))) if isinstance(n, ast.Call)
             and isinstance(n.func, ast.Attribute) and n.func.attr in ("empty", "zeros", "ones", "full")]
    assert calls
    for n in calls:
        assert any(k.arg == "dtype" for k in n.keywords), f"line {n.lineno}"
