"""The paged cache and the attention over it at their edges: what a row must not
see, scales and queries of very different size, tables that do not fit, empty
calls, load paths of odd pages.  Bounds are those of paged_ref.py."""
import math

import pytest
import torch

import chunked_gated_delta_rule_gb300 as pkg
from paged_ref import Batch, check

pytestmark = pytest.mark.gpu

ROUTES = [1, 2, 3]


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype,fmt", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"),
                                       ("f16", "int8")])
@pytest.mark.parametrize("q_len,heads", [(1, 4), (1, 32), (2, 32), (4, 4)])
def test_positions_that_left_the_window(route, dtype, fmt, q_len, heads):
    """NaN and infinities in the first page below the window, which is loaded
    with it: a tile whose rows all see the same positions too."""
    b = Batch([q_len], [150], heads=heads, kv_heads=2, dtype=dtype, fmt=fmt, page=64)
    first = 150 - q_len - 36  # what the first token sees
    for at, bad in ((first - 1, math.nan), (first - 3, math.inf), (first - 40, math.nan)):
        page, slot = int(b.table[0, at // 64]), at % 64
        if fmt == "same":
            b.vc[page, slot, :, 5:90] = bad
            b.kc[page, slot, :, 5:90] = bad
        else:
            b.vs[page, :, slot] = math.nan
            b.ks[page, :, slot] = math.nan
    check(b, *b.run(force_path=route, window=37), *b.attention(window=37),
          label=f"{route} {dtype} {fmt} {q_len} {heads}")
