"""Kernels of the block with experts start beside the kernel before them and wait for
it (programmatic launches), so what that one writes is not read-only while they run:
a const __restrict__ pointer would let the compiler read it by the non-coherent path,
or ahead of the wait."""
import os
import re

import pytest

LM = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "newton_schulz_07_gb300", "csrc", "lm")


@pytest.mark.parametrize("name", ["block8.cuh", "combine.cu", "experts.cu", "experts_gemm.cuh", "quantize8.cu", "rms_norm.cu",
                                  "rms_norm_grad.cu", "route.cu"])
def test_no_read_only_pointers(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(LM, name)).read())
    assert not re.search(r"__restrict__|__ldg|\.nc\b", text)
    # Every kernel of these files waits for the one before it.
    for kernel in re.split(r"__global__", text)[1:]:
        assert "griddep_wait()" in kernel
