"""Sizes of the state space scan near the ends of 32 bits, without a GPU: each call is refused on the host (the
made-up addresses are never used)."""
import pytest

from test_ssm_abi import BF16, SHAPE, lib, scan  # noqa: F401  (lib is a fixture)

MOST = (1 << 31) - 8  # the most channels that an int32 holds


@pytest.mark.parametrize("fn,T,B", [("ssm_decode", 1, 1), ("ssm_decode", 5, 2), ("ssm_prefill", 1, 1)])
def test_grids_of_most_channels(lib, fn, T, B):  # noqa: F811
    """More workgroups than a launch may have, whatever the form; counted in 32 bits they would be negative."""
    assert scan(lib, fn, B=B, T=T, C=MOST, N=8, G=1, st=BF16 if T > 1 else 0) == SHAPE
