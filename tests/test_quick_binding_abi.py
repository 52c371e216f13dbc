"""_quick.so is bound to one torch and one Python (CPU): another one's is rebuilt by build() and never imported, and
the library, which needs neither, loads without it."""
import sys

import pytest

import exact_attention_forward_06_gb300 as A
from exact_attention_forward_06_gb300 import _binding
from exact_attention_forward_06_gb300 import build as B


@pytest.fixture()
def fresh(monkeypatch):
    """load() as in a new process, after which the process's own libraries are back."""
    B.build()                                            # (does nothing when it is up to date)
    A.load()
    monkeypatch.setattr(_binding, "_lib", None)
    monkeypatch.setattr(_binding, "_quick", None)
    return monkeypatch


def _other_abi(tmp_path):
    path = tmp_path / "_quick.abi"
    path.write_text("torch 1.0, C++11 ABI 0, cpython-30")
    return str(path)


def test_build_is_up_to_date_and_another_torch_makes_it_stale(fresh, tmp_path):
    assert B.built_abi() == B.abi_tag() and not B._stale()
    fresh.setattr(B, "QUICK_ABI", _other_abi(tmp_path))
    assert B._stale()
    fresh.setattr(B, "QUICK_ABI", str(tmp_path / "none"))
    assert B.built_abi() is None and B._stale()


@pytest.mark.parametrize("how,why", [("other", "torch 1.0"), ("none", "is missing"), ("no library", "is missing"),
                                     ("broken", "cannot be imported")])
def test_the_library_loads_without_a_usable_quick_way(fresh, tmp_path, how, why):
    if how == "other":
        fresh.setattr(B, "QUICK_ABI", _other_abi(tmp_path))
    elif how == "none":
        fresh.setattr(B, "QUICK_ABI", str(tmp_path / "none"))
    elif how == "no library":
        fresh.setattr(B, "QUICK", str(tmp_path / "_quick.so"))
    else:
        fresh.setitem(sys.modules, _binding.__package__ + "._quick", None)   # importing it raises ImportError
    with pytest.warns(RuntimeWarning, match=why):
        lib = A.load()
    assert lib.attn_version() == A.version()
    for name in ("qk_norm_rope", "append", "gather", "decode", "fwd"):
        assert getattr(_binding._quick, name)(*[None] * 15) is None
    with pytest.raises(TypeError):                       # the long way's own checks
        A.decode_paged_q4(None, None, None, None)
    A.load()                                             # (once: no second warning is needed)
