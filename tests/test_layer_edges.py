"""The operators of a state-space layer on the CPU: what the binding and the C entry points
refuse before any work.  No compute call is made."""
import pytest
import torch

from chunked_gated_delta_rule_gb300 import api, layer

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


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_delta_rule_gb300 import build
    build.build()
    import chunked_gated_delta_rule_gb300 as pkg
    return pkg.load_library()


def at(i):
    return 0x100000 * i


SCAN_IN = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
SCAN_OUT = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def scan_bwd(lib, h0=20, dy=21, dht=22, **place):
    """The code of a backward scan whose outputs lie at 30, 31, ..., but for those in ``place``."""
    ins = api.gdr_scan_tensors(*(at(1 + i) for i in range(8)))
    out = api.gdr_scan_grads(*(at(place.get(n, 30 + i)) for i, n in enumerate(SCAN_OUT)))
    dims = api.gdr_scan_dims(1, 64, 128, 16, 1, 0, api.GDR_F32, 0, 1)
    return lib.gdr_selective_scan_bwd(dims, ins, None, at(h0), at(dy), at(dht), out, None, None)


def test_gradients_of_the_scan_in_one_place(lib):
    """dh0 in the place of h0: the launch that turns ends into starts reads the one and writes the
    other, in blocks of which neither waits for the other."""
    for i, name in enumerate(SCAN_OUT):
        for place in list(range(1, 9)) + [20, 21, 22]:
            assert scan_bwd(lib, **{name: place}) == -1, (name, place)
        for j, other in enumerate(SCAN_OUT):
            if other != name:
                assert scan_bwd(lib, **{name: 30 + j}) == -1, (name, other)


def conv_bwd(lib, **place):
    dims = api.gdr_conv_dims(1, 64, 128, 4, 0, api.GDR_F32, 0, api.GDR_F32, 1)
    out = [at(place.get(n, 30 + i)) for i, n in enumerate(("dx", "dw", "db", "dh0"))]
    return lib.gdr_short_conv_bwd(dims, at(1), at(2), at(3), None, at(4), at(5), at(6), *out, None, None)


def test_gradients_of_the_convolution_in_one_place(lib):
    names = ("dx", "dw", "db", "dh0")
    for name in names:
        for place in range(1, 7):
            assert conv_bwd(lib, **{name: place}) == -1, (name, place)
        for j, other in enumerate(names):
            if other != name:
                assert conv_bwd(lib, **{name: 30 + j}) == -1, (name, other)


def test_outputs_in_the_place_of_states_and_parameters(lib):
    """Forward: y anywhere but in a place of its own, states in the place of anything but h0."""
    dims = api.gdr_conv_dims(1, 64, 128, 4, 0, api.GDR_F32, 0, api.GDR_F32, 1)
    for y, ht in ((2, 30), (3, 30), (4, 30), (30, 30), (31, 1), (31, 2), (31, 3)):
        assert lib.gdr_short_conv_fwd(dims, at(1), at(2), at(3), None, at(4), at(ht), 1, None, at(y),
                                      None, None) == -1, (y, ht)
    ins = api.gdr_scan_tensors(*(at(1 + i) for i in range(8)))
    dims = api.gdr_scan_dims(1, 64, 128, 16, 1, 0, api.GDR_F32, 0, 1)
    for y, ht in [(i, 30) for i in list(range(1, 9)) + [20, 30]] + [(31, i) for i in range(1, 9)]:
        assert lib.gdr_selective_scan_fwd(dims, ins, None, at(20), at(ht), 1, None, at(y), 0, None,
                                          None) == -1, (y, ht)


def test_norm_outputs_in_one_place(lib):
    """Backward: dx is written as dense rows, over rows at other strides that other blocks still
    read.  Both ways: the weight is read by every row, a scale is no row."""
    def bwd(dx=30, dw=31, **kw):
        dims = api.gdr_norm_dims(64, 128, api.GDR_F32, api.GDR_F32, api.GDR_F32, 0, 1e-6)
        for k, v in kw.items():
            setattr(dims, k, v)
        return lib.gdr_rms_norm_bwd(dims, at(1), at(2), at(3), at(4), at(dx), at(dw), None, None)

    for place in (1, 2, 3, 4):
        assert bwd(dx=place) == -1 and bwd(dw=place) == -1, place
    for strides in (dict(x_stride=256), dict(y_stride=256), dict(residual_stride=256)):
        for place in (1, 3, 4):
            assert bwd(dx=place, **strides) == -1, (place, strides)
    assert bwd(dx=31) == -1

    def fwd(out=30, y=31, scale=32):
        dims = api.gdr_norm_dims(64, 128, api.GDR_F32, api.GDR_F32, api.GDR_I8, 0, 1e-6)
        return lib.gdr_rms_norm_fwd(dims, at(1), at(2), at(3), at(out), at(y), at(scale), None, None)

    assert fwd(out=3) == -1 and fwd(y=3) == -1
    for place in (1, 2, 3, 30, 31):
        assert fwd(scale=place) == -1, place


def test_outputs_in_the_place_of_offsets_and_indices(lib):
    f32 = api.GDR_F32
    conv = api.gdr_conv_dims(1, 64, 128, 4, 2, f32, 0, f32, 1)
    scan = api.gdr_scan_dims(1, 64, 128, 16, 1, 2, f32, 0, 1)
    ins = api.gdr_scan_tensors(*(at(1 + i) for i in range(8)))
    for y, ht in ((40, 31), (41, 31), (30, 40), (30, 41)):  # offsets at 40, indices at 41
        assert lib.gdr_short_conv_fwd(conv, at(1), at(2), at(3), at(40), at(20), at(ht), 2, at(41), at(y),
                                      None, None) == -1, (y, ht)
        assert lib.gdr_selective_scan_fwd(scan, ins, at(40), at(20), at(ht), 2, at(41), at(y), 0, None,
                                          None) == -1, (y, ht)
    for i in range(4):
        out = [at(40 if k == i else 30 + k) for k in range(4)]
        assert lib.gdr_short_conv_bwd(conv, at(1), at(2), at(3), at(40), at(4), at(5), at(6), *out, None,
                                      None) == -1, i
    for i in range(9):
        out = api.gdr_scan_grads(*(at(40 if k == i else 30 + k) for k in range(9)))
        assert lib.gdr_selective_scan_bwd(scan, ins, at(40), at(20), at(21), at(22), out, None, None) == -1, i
