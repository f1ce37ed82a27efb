"""The CUDA sources that a recorded kernel's digest is taken over: its own family's."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "shape_driven_tile_gb300", "csrc")


def test_the_16_bit_product_does_not_depend_on_the_8_bit_one():
    fp8 = [n for n in os.listdir(CSRC) if n.startswith("gemm_fp8")]
    assert len(fp8) > 3 and not any(belongs(n) for n in fp8 for belongs in bench.SOURCES.values())
    for name in ("gemm_pair.cuh", "gemm_host.cu", "ptx.cuh", "launch.cuh"):
        assert bench.SOURCES["gemm"](name)
    assert bench.SOURCES["gemv"]("gemv.cu") and not bench.SOURCES["gemm"]("gemv.cu")


def test_what_the_family_includes_belongs_to_it():
    """No source of the 16-bit product includes one that its digest leaves out, but the host's common checks."""
    names = [n for n in os.listdir(CSRC) if bench.SOURCES["gemm"](n)]
    assert names
    for name in names:
        with open(os.path.join(CSRC, name)) as f:
            for other in re.findall(r'#include "(\w+\.cuh)"', f.read()):
                assert bench.SOURCES["gemm"](other) or other == "host_common.cuh", (name, other)
