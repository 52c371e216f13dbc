"""Rows of the norm and the appends beyond what one launch's grid holds are refused before anything else happens (CPU).
Only refused calls are made here: the pointers are not real."""
import pytest

from test_cache_ops_args import _append, _norm, lib  # noqa: F401

MOST = 2**31 - 1


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (512, 1), (65536, 1)])   # at least 9 blocks to eight tokens
def test_append_refuses_a_grid_that_does_not_fit(lib, q4, Hq, Hkv):  # noqa: F811
    assert _append(lib, q4, total=MOST, Hq=Hq, Hkv=Hkv, qs=Hq * 128, ks=Hkv * 128, vs=Hkv * 128) == 1


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (512, 1), (65536, 1)])
def test_norm_rope_refuses_a_grid_that_does_not_fit(lib, Hq, Hkv):  # noqa: F811
    assert _norm(lib, B=1, S=MOST, Hq=Hq, Hkv=Hkv) == 1
