"""The packed calls of the binding are as long as the C structs that the entry points copy (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from shape_driven_tile_gb300 import fp8, paged, rope

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
CALLS = {"sdt_gemm_fp8": fp8._GEMM, "sdt_quant_fp8": fp8._QUANT, "sdt_rms_norm_fp8": fp8._NORM, "sdt_rope_qk": rope._ROPE,
         "sdt_paged_step": paged._STEP, "sdt_paged_attn": paged._ATTN}


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    compiler = next((c for c in ("cc", "gcc") if shutil.which(c)), None)
    if compiler is None:
        pytest.skip("no C compiler")
    at = tmp_path_factory.mktemp("sizes")
    lines = "".join(f'printf("{name} %zu\\n", sizeof({name}));' for name in CALLS)
    (at / "sizes.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sdt.h"\nint main(void) {' + lines + "return 0;}\n")
    subprocess.run([compiler, "-I", INCLUDE, str(at / "sizes.c"), "-o", str(at / "sizes")], check=True, capture_output=True)
    out = subprocess.run([str(at / "sizes")], check=True, capture_output=True, text=True).stdout
    return {name: int(size) for name, size in (line.split() for line in out.splitlines())}


@pytest.mark.parametrize("name", CALLS)
def test_a_packed_call_has_the_size_of_its_struct(sizes, name):
    assert CALLS[name].size == sizes[name]
