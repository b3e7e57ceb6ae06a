"""Sizes of the state space scan near the ends of 32 bits, without a GPU: each call is refused on the host (the
made-up addresses are never used)."""
import pytest

from ssm_form import prefill_form
from test_ssm_abi import BF16, SHAPE, lib, scan  # noqa: F401  (lib is a fixture)

MOST = (1 << 31) - 8  # the most channels that an int32 holds


@pytest.mark.parametrize("fn,T,B", [("ssm_decode", 1, 1), ("ssm_decode", 5, 2), ("ssm_prefill", 1, 1)])
def test_grids_of_most_channels(lib, fn, T, B):  # noqa: F811
    """More workgroups than a launch may have, whatever the form; counted in 32 bits they would be negative."""
    assert scan(lib, fn, B=B, T=T, C=MOST, N=8, G=1, st=BF16 if T > 1 else 0) == SHAPE


@pytest.mark.parametrize("shape", [(300000, 1, 2048, 8, 1), (5592405, 1, 96, 8, 1), (65536, 9, 4800, 16, 200)], ids=str)
def test_a_form_whose_grid_fits(shape):
    """Where the workgroups with 8 or 16 lanes for each channel would be more than a launch may have (in the
    second case once they are rounded up to whole lines), the call runs with four."""
    assert prefill_form(*shape) == (4, False, 1, shape[1])
    smaller = (shape[0] // 4, *shape[1:])
    assert prefill_form(*smaller)[0] > 4
