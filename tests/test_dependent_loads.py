"""Kernels that are launched as programmatic dependents start while the work before them may still be writing: their
sources hold no non-coherent load (CPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_forward_06_gb300", "csrc")


def test_no_non_coherent_loads_in_dependent_kernels():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        if "wait_for_prior_work" in code or "griddepcontrol.wait" in code or path.endswith(".cuh"):
            seen += 1
            assert "__ldg" not in code and "ld.global.nc" not in code, path
            # (a const pointer that nothing else may alias is loaded from so as well)
            assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", code), path
    assert seen >= 6
