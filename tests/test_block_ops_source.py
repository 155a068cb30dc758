"""What the sources of the operators around the routed experts must not contain (no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4afp8_mixture_experts_gb300", "csrc")
FILES = [f for pattern in ("linear*.cu*", "block_norm*", "route_grouped*", "block_ops.cuh")
         for f in glob.glob(os.path.join(CSRC, pattern))]


def test_no_load_that_takes_its_memory_for_constant():
    # These kernels are launched while their predecessor may still write their inputs (programmatic launch).  A
    # non-coherent load's memory must not change during the kernel's whole life, and the compiler may move such a load
    # above the wait for the predecessor.
    assert len(FILES) >= 10
    for f in FILES:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        found = re.findall(r"__ldg|\.nc\b|__restrict__|__builtin_nontemporal_load", code)
        assert not found, (os.path.basename(f), found)
