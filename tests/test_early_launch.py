"""Kernels that may start while the kernel before them on the stream still runs read global memory by coherent loads that stay behind
their wait: neither __ldg (ld.global.nc, for data that nothing writes during the whole kernel) nor const __restrict__, which
lets the compiler choose it. Read in the sources; what the loads see is tested on the GPU."""
import os
import re

import pytest

from int8_quantized_gemm_gb300 import build

EARLY = ["q8_fp4_quant.cu", "q8_fp4_gemm.cu", "q8_gemv_mma.cu"]


def code(name):
    """A source without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_the_list_is_complete():
    """Every source that launches a kernel with the attribute, itself or by the 4-bit operators' helper."""
    found = [s for s in build.SOURCES if re.search(r"launch_dependent\(|ProgrammaticStreamSerialization", code(s))]
    assert sorted(found) == sorted(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_no_load_that_may_miss_the_kernel_before(name):
    text = code(name)
    assert not re.search(r"\b__ldg\b|ld\.global\.[a-z0-9_:.]*nc\b|__restrict__", text)
    assert not re.search(r"\bGroups\b|GroupsOf<false>|\bepi_bias\(|\bepi_bias<false>", text)   # shared helpers: their form for it


def test_shared_helpers_have_a_form_for_them():
    text = code("q8_tiles.cuh")
    body = text[text.index("struct GroupsOf"):text.index("using Groups")]
    assert re.search(r"if constexpr \(kEarly\)\s+return load_int", body) and body.count("__ldg") == 1
    assert re.search(r"using EarlyGroups = GroupsOf<true>;", text)
    text = code("q8_internal.h")
    assert re.search(r"if constexpr \(kEarly\)\s+return ep\.bias \? __fadd_rn\(v, load_float", text) and text.count("__ldg") == 1
    loads = code("q8_loads.cuh")
    assert loads.count("asm volatile") == loads.count("ld.global.") == loads.count('"memory"') and ".nc" not in loads
