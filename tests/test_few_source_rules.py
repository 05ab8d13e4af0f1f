"""Kernels that start under the end of the one before read nothing as a constant of their lifetime."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_gemm_05_gb300", "csrc")


@pytest.mark.parametrize("name", ["few_kernel.cuh", "ffn.cu"])
def test_no_constant_loads_of_global_memory(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "pdl_wait();" in code and "ProgrammaticStreamSerialization" in code
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__|\.nc\.", code)
