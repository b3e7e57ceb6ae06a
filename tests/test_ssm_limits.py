"""Sizes of the state space scan near the ends of 32 bits, without a GPU: each call is refused on the host (the
made-up addresses are never used)."""
import pytest

from ssm_form import prefill_form
from test_ssm_abi import ALIGN, BF16, SHAPE, lib, scan  # noqa: F401  (lib is a fixture)

MOST = (1 << 31) - 8  # the most channels that an int32 holds


@pytest.mark.parametrize("fn,T,B", [("ssm_decode", 1, 1), ("ssm_decode", 5, 2), ("ssm_prefill", 1, 1)])
def test_grids_of_most_channels(lib, fn, T, B):  # noqa: F811
    """More workgroups than a launch may have, whatever the form; counted in 32 bits they would be negative."""
    assert scan(lib, fn, B=B, T=T, C=MOST, N=8, G=1, st=BF16 if T > 1 else 0) == SHAPE


@pytest.mark.parametrize("shape", [(300000, 1, 2048, 8, 1), (5592405, 1, 96, 8, 1), (65536, 9, 4800, 16, 200)], ids=str)
def test_a_form_whose_grid_fits(shape):
    """Where the workgroups with 8 or 16 lanes for each channel would be more than a launch may have (in the
    second case once they are rounded up to whole lines), the call runs with four."""
    assert prefill_form(*shape, f32=True) == (4, False, 1, shape[1])
    smaller = (shape[0] // 4, *shape[1:])
    assert prefill_form(*smaller, f32=True)[0] > 4


@pytest.mark.parametrize("shape,f32,one_pass,want", [
    # N = 8: the form that was measured fastest of four lanes, eight (in roles) and segments
    ((16, 1024, 4096, 8, 1), False, False, {(4, False, 1)}),   # 184 us, 197 in eight lanes
    ((64, 300, 1024, 8, 1), False, False, {(4, False, 1)}),    # 56, 71
    ((16, 1024, 4096, 8, 1), True, False, {(8, False, 1)}),    # fp32: 248, 274 in four
    ((8, 1024, 4096, 8, 1), False, False, {(8, False, 1)}),    # 93, 105
    ((4, 1024, 4096, 8, 1), False, True, {(8, False, 1)}),     # 57, 78
    ((1, 8192, 4096, 8, 1), False, True, {(8, True, 1)}),      # 263, 585
    ((1, 8192, 4096, 8, 1), False, False, {(4, False, 16), (4, False, 32)}),  # segments 158 and 161
    ((1, 8192, 4096, 8, 1), True, False, {(4, False, 16), (4, False, 32)}),   # 213 and 218, 352 in eight lanes
    ((1, 8192, 512, 8, 1), False, False, {(4, False, 64)}),    # 43
    ((2, 300, 4096, 8, 1), False, False, {(8, True, 1)}),      # 14, 27
    # N = 16 and 32
    ((16, 1024, 4096, 16, 1), False, False, {(4, False, 1)}),  # 240, 338 in sixteen
    ((4, 1024, 4096, 16, 1), False, False, {(16, False, 1)}),  # 80, 100
    ((1, 8192, 4096, 16, 1), False, False, {(16, True, 1)}),   # 203, segments 220
    ((1, 8192, 512, 16, 1), False, False, {(4, False, 64)}),   # 52, 194
    ((16, 1024, 4096, 32, 1), False, False, {(4, False, 1)}),  # 427, 565
    ((1, 8192, 4096, 32, 1), False, False, {(16, True, 1)}),   # 323, segments 378
], ids=str)
def test_the_form_that_was_measured_fastest(shape, f32, one_pass, want):
    assert prefill_form(*shape, one_pass=one_pass, f32=f32)[:3] in want


def test_the_workspace_does_not_go_by_the_type():
    """Segments, or one pass, whatever the rows' type: ssm_prefill_workspace_size does not know it."""
    for B in (1, 2, 8, 40):
        for T in (100, 1000, 9000):
            for C in (64, 520, 4096):
                for N in (8, 16, 32):
                    a, b = (prefill_form(B, T, C, N, 1, f32=f) for f in (False, True))
                    assert a[2:] == b[2:]


@pytest.mark.parametrize("fn", ["ssm_decode", "ssm_prefill"])
@pytest.mark.parametrize("strides", [(-1, 0, 64), (256, 0, 68), (1 << 61, 0, 64)], ids=str)
def test_strides_of_no_gate_say_nothing(lib, fn, strides):  # noqa: F811
    """Without z its strides are not looked at: the call is refused for what follows in the checks."""
    assert scan(lib, fn, z=None, zs=strides, lens=0x100002) == ALIGN
    assert scan(lib, fn, zs=strides, lens=0x100002) in (SHAPE, ALIGN)
