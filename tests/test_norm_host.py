"""Arguments of the block norm on the host (fake, never dereferenced device addresses; no GPU)."""

import pytest

import gated_delta_rule_98_amd as pkg
from test_linear_host import _norm, needs_no_gpu

LARGEST = 3.4028234663852886e38  # of fp32


@needs_no_gpu
@pytest.mark.parametrize("x", [LARGEST, 3.1e38, 1e-45, 0.0])
def test_every_finite_scale_and_eps_is_taken(x):
    """Passes every host check: only the launch itself fails without a device."""
    assert _norm(scale=x) == pkg.KDA_ERR_HIP
    assert _norm(scale=-x) == pkg.KDA_ERR_HIP
    assert _norm(eps=x) == pkg.KDA_ERR_HIP


@needs_no_gpu
@pytest.mark.parametrize("x", [float("inf"), float("nan")])
def test_others_are_refused(x):
    assert _norm(scale=x) == _norm(scale=-x) == _norm(eps=x) == pkg.KDA_ERR_INVALID
