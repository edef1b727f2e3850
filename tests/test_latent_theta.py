"""The latent cache write takes RoPE bases from 1 on: below, frequencies exceed 1 and the angles
leave the range that their reduction is exact over."""
import pytest

from paged_sliding_window_gb300 import binding
from test_latent_host import WRITES, _norm, call, lib  # noqa: F401


@pytest.mark.parametrize("name", WRITES)
def test_bases_below_one_are_refused(lib, name):  # noqa: F811
    for theta in (0.999, 0.5, 1e-30, 0.0, -1.0, float("inf"), float("nan")):
        assert binding.ERRORS.get(call(lib, name, norm=_norm(theta=theta))) == "PSW_EINVAL_ROPE", theta
    for theta in (1.0, 500.0, 1e7):
        assert call(lib, name, norm=_norm(theta=theta)) == 0
