"""Limits of the paged-cache calls' numbers (host arithmetic, no GPU: fake
addresses that never reach a device)."""
import ctypes

import pytest

pytest.importorskip("torch")
from test_paged_host import _attend, api  # noqa: E402,F401


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38])
def test_a_scale_without_a_number_in_base_2_is_refused(api, scale):  # noqa: F811
    assert _attend(api, scale=scale) == api.VQ_ERR_INVALID_ARG
    assert ctypes.c_float(scale).value not in (float("inf"), float("-inf"))
