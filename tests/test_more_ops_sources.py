"""The rules of test_ops_sources.py for layer norm's and the linear layer's sources, and what they share
with the other operators (CPU)."""
import os
import re

from tests.test_ops_sources import CSRC, _code


def test_only_weights_are_read_through_the_non_coherent_path():
    """Kernels in front of these may still write what they read (x, its scales, the residual, and in a training
    step's graph the parameters): only the few-token kernel's weights bypass L1's coherence, behind the wait."""
    for name in ("layernorm.cu", "linear.cu", "linear_few.cu", "linear_shares.cu", "rowops.cuh", "tile_gemm.cuh"):
        code = _code(os.path.join(CSRC, name))
        assert "__ldg" not in code, name
        assert len(re.findall(r"\.nc\b", code)) == (name == "linear_few.cu"), name  # load_once
        for at in re.finditer(r"load_once\((?!const)(\w+)", code):
            assert at.group(1) == "w", (name, at.group(1))


def test_every_kernel_waits_for_the_kernels_in_front_of_it():
    """Each kernel of these files is launched so that it may start early: it has to wait before it reads."""
    for name in ("layernorm.cu", "linear.cu", "linear_few.cu", "linear_shares.cu", "rowops.cuh", "tile_gemm.cuh"):
        code = _code(os.path.join(CSRC, name))
        kernels = re.findall(r"__global__ void", code)
        assert len(re.findall(r"grid_wait_prior\(\);", code)) == len(kernels), name
        assert "<<<" not in code, name
