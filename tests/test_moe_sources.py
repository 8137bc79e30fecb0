"""How the mixture-of-experts kernels load what an earlier kernel may have
written, checked in their sources.

Every kernel of the chain lets its successor start before its own wait for its
predecessor, so a grid is resident while the data it will read is still being
written. A non-coherent load (__ldg, or a const __restrict__ pointer, which lets
the compiler choose one) asserts data that nothing writes during the grid's
life, and may be moved in front of the wait; so may the cache-hinted load
intrinsics, whose asm does not mention memory."""
import glob
import os
import re

import pytest

import gguf_quant_dequant_q4k_b200 as q4k

CSRC = os.path.join(os.path.dirname(q4k.__file__), "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "q4k_moe_*.cu")))


def code(name):
    """The source without comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_the_kernels_are_there():
    assert FILES == ["q4k_moe_combine.cu", "q4k_moe_gemm.cu", "q4k_moe_gemv.cu", "q4k_moe_route.cu"]


@pytest.mark.parametrize("name", FILES)
def test_launched_early_and_waiting(name):
    """The premise: programmatic launches, and a wait in every kernel."""
    text = code(name)
    kernels = len(re.findall(r"__global__", text))
    assert "cudaLaunchAttributeProgrammaticStreamSerialization" in text
    assert kernels and len(re.findall(r"\bpdl_wait\(\)", text)) == kernels


@pytest.mark.parametrize("name", FILES)
def test_no_noncoherent_loads(name):
    text = code(name)
    assert re.findall(r"\b__ld(?:g|cg|ca|cs|lu|cv)\b|ld\.global\.nc|\bconst\s+[\w:]+\s*\*\s*__restrict__", text) == []
