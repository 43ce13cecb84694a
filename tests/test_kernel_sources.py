"""CPU checks of rules that the kernels' sources keep and that no run would show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_core_gemm_tcgen05_gb300", "csrc")


def code(path):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


FILES = {os.path.basename(f): code(f) for f in sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.cu")))}


@pytest.mark.parametrize("name", [f for f in FILES if f != "softmax_kernel.cuh"])
def test_no_read_only_loads_beside_the_kernel_before(name):
    """Kernels that start while the one before them still writes read with ordinary loads what an operator may have written: __ldg
    (ld.global.nc), and pointers that let the compiler choose it, are for data that no one writes in the kernel's lifetime, which
    of a batch is q_start (load_start)."""
    loads = re.findall(r"__ldg\s*\(|ld\.global\.nc|ld\.nc|__restrict__", FILES[name])
    assert loads == (["__ldg("] if name == "serving_common.cuh" else [])
    assert all("q_start" in x for x in re.findall(r"\bload_start\(([^)]*)\)", FILES[name]) if x != "const int *at")


def test_the_other_kernels_start_when_all_is_written():
    """row_softmax's kernels are launched in the ordinary way."""
    assert "grid_dependency_wait" not in FILES["softmax_kernel.cuh"]
    launches = re.findall(r"row_softmax\w*kernel[^;]*;", FILES["gemm_api.cu"])
    assert launches and not any("launch_serving" in x or "cudaLaunchKernelEx" in x for x in launches)


@pytest.mark.parametrize("name", [f for f, text in FILES.items() if "extern __shared__" in text])
def test_dynamic_shared_memory_is_aligned_for_vectors(name):
    """It is read in vectors of 16 bytes (or written by TMA): declared as such, or aligned by the kernel itself."""
    for kind, what in re.findall(r"extern __shared__ (\w+) (\w+)\[\]", FILES[name]):
        assert kind == "uint4" or re.search(r"smem_u32\(" + what + r"\).*\+ 1023u\) & ~1023u", FILES[name], re.S), (kind, what)
