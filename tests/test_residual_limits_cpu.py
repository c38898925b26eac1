"""The largest finite scales of the gated residual and its backward (no GPU: no tokens)."""
import pytest

from depth_wise_attention_attnres_gb300 import binding, build
from tests.test_residual_cpu import INVALID, _bwd, _fwd

MAX = (2 - 2.0 ** -23) * 2.0 ** 127  # fp32's largest


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("scale", [MAX, -MAX, 3.4e38, 0.0, 2.0 ** -149])
def test_every_finite_scale_is_taken(lib, scale):
    assert lib.attnres_gated_residual(*_fwd(T=0, scale=scale)) == 0
    assert lib.attnres_gated_residual_bwd(*_bwd(T=0, scale=scale)) == 0


@pytest.mark.parametrize("scale", [2.0 ** 128, -2.0 ** 128, float("inf"), float("nan")])
def test_others_are_refused(lib, scale):
    assert lib.attnres_gated_residual(*_fwd(T=0, scale=scale)) == INVALID
    assert lib.attnres_gated_residual_bwd(*_bwd(T=0, scale=scale)) == INVALID
