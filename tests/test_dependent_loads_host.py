"""Kernels that are launched while the one before still runs (programmatic dependent launch) read
only true constants as constant data: an input that the kernel before writes would be undefined
through a non-coherent load, and no run on a GPU shows that reliably.  Read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "phase_disaggregated_quantized_b200", "csrc")

# Weights are constants by the header's rule; t_h is read by an ordinary launch only.
CONSTANT_POINTERS = {"w4a16_gemm.cuh": {"pcodes", "pscales"}, "moe.cuh": {"wr"}, "w4a16_tmem.cuh": set(), "nvfp4_gemm.cuh": set()}
CONSTANT_LOADS = {"w4a16_gemm.cuh": set(), "moe.cuh": {"lo", "hi"}, "w4a16_tmem.cuh": set(), "nvfp4_gemm.cuh": {"p.t_h"}}


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", CONSTANT_LOADS)
def test_only_constants_are_read_as_constant_data(name):
    code = _code(name)
    assert "grid_dependency_wait()" in code
    assert set(re.findall(r"__ldg\(\s*([\w.]+)", code)) <= CONSTANT_LOADS[name]
    assert set(re.findall(r"const\s+[\w:]+\s*\*\s*__restrict__\s+(\w+)", code)) <= CONSTANT_POINTERS[name]


def test_constant_loads_of_the_router_are_of_its_weights():
    code = _code("moe.cuh")
    for row in ("lo", "hi"):
        assert re.search(rf"const uint4\* {row} = reinterpret_cast<const uint4\*>\(wr \+", code)
