"""The largest scale of the attention over the 4-bit cache: above it the kernel's factor would overflow, so the call is
refused before anything else happens (CPU; only refused calls: the pointers are not real)."""
import pytest

from test_cache_ops_args import _decode, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.0 ** 94, 1e30, 3.4e38])
def test_a_scale_that_overflows_is_refused(lib, scale):  # noqa: F811
    assert _decode(lib, scale=scale) == 1
