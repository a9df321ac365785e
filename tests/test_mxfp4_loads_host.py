"""The MXFP4 kernels start while the kernel ahead in the stream still runs (programmatic dependent launch), and what
they read may be what that kernel writes.  A non-coherent load (__ldg, or a load through a const __restrict__ pointer
that the compiler may turn into one) asks for memory that nobody writes while the kernel is resident, and is not bound
to stay behind the wait for the kernel ahead: none may stand in these sources (CPU only)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "megatron_tensor_mlp_gb300", "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "mxfp4*.cu*")))


def code(name):
    """The file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)


@pytest.mark.parametrize("name", SOURCES)
def test_no_non_coherent_load_behind_the_wait(name):
    found = re.findall(r"__ldg|__restrict__|ld\.global(?:\.\w+)*\.nc", code(name))
    assert not found, found


def test_the_kernels_are_launched_programmatically():
    """(what makes the rule above necessary)"""
    assert {"mxfp4_quant.cu", "mxfp4_gemm.cu", "mxfp4_gemm.cuh"} <= set(SOURCES)
    for name in ("mxfp4_quant.cu", "mxfp4_gemm.cu"):
        assert "cudaLaunchAttributeProgrammaticStreamSerialization" in code(name)
