"""Float8 and routed-expert entry points at the ends of their ranges: batches of nothing and the largest sizes. Validation
runs before any CUDA call, so these need no GPU (the pointers are never read)."""
import os
import shutil
import subprocess

import pytest

from .test_fp8_abi import FAKE, GEMM, GROUPED, INVALID, OK, QUANT, UNSUPPORTED, call, lib  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("change,status", [
    (dict(top_k=8, rows_out=0), OK),                          # the empty tensors of a batch of no token
    (dict(top_k=8, rows_out=5), OK),
    (dict(top_k=8, rows_out=0, slots=FAKE), OK),
    (dict(top_k=0, rows_out=0), OK),
    (dict(top_k=-1, rows_out=0), INVALID),
    (dict(top_k=8, rows_out=-1), INVALID),
    (dict(top_k=0, rows_out=0, slots=FAKE), INVALID),
    (dict(top_k=33, rows_out=0), UNSUPPORTED),
])
def test_no_rows_to_quantize_into_slots(lib, change, status):  # noqa: F811
    before = lib.q8_launch_count()
    assert call(lib, "q8_quantize_fp8", QUANT, M=0, x=None, q=None, s=None, **change) == status
    assert lib.q8_launch_count() == before


@pytest.mark.parametrize("name,defaults,change", [
    ("q8_gemm_fp8", GEMM, dict(K=(1 << 31) - 16)),            # the block after the last would end past 2^31
    ("q8_gemm_fp8", GEMM, dict(K=(1 << 31) - 112)),
    ("q8_gemm_fp8", GEMM, dict(M=(1 << 31) - 1)),             # and so would the rows of a tile
    ("q8_gemm_fp8", GEMM, dict(M=(1 << 31) - 200)),
    ("q8_gemm_fp8", GEMM, dict(N=(1 << 31) - 1)),
    ("q8_gemm_fp8_grouped", GROUPED, dict(K=(1 << 31) - 112)),
    ("q8_gemm_fp8_grouped", GROUPED, dict(rows=(1 << 31) - 16)),
    ("q8_gemm_fp8_grouped", GROUPED, dict(E=2, N=(1 << 30) - 8)),
])
def test_products_next_to_32_bits_are_refused(lib, name, defaults, change):  # noqa: F811
    before = lib.q8_launch_count()
    assert call(lib, name, defaults, **change) == UNSUPPORTED
    assert lib.q8_launch_count() == before


def test_error_code_tells_the_float8_products_apart(tmp_path):
    """The code that q8_device_error makes of the kernels' error words: a byte for each family, and the highest bit where a
    float8 product gave up, which shares its byte with the int8 CTA-pair kernel."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_quantized_gemm_gb300", "csrc")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src, exe = tmp_path / "code.cu", tmp_path / "code"
    src.write_text('#include <stdio.h>\n#include "q8_internal.h"\nint main() {\n'
                   'const unsigned w[][6] = {{0, 0, 0, 0, 0, 0}, {2, 0, 0, 0, 0, 0}, {0, 128, 0, 0, 0, 0}, {0, 0, 8, 0, 0, 0},\n'
                   '{0, 0, 0, 2, 0, 0}, {0, 0, 0, 0, 33, 0}, {0, 0, 0, 0, 0, 33}, {1, 128, 2, 4, 8, 64}};\n'
                   'for (auto& v : w) printf("%u ", q8::device_error_code(v[0], v[1], v[2], v[3], v[4], v[5]));\n}\n')
    subprocess.run([nvcc, "-std=c++17", "-I", csrc, "-o", str(exe), str(src)], check=True, capture_output=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [0, 2, 128, 8 << 8, 2 << 16, 33 << 24, 33 << 24 | 1 << 31,
                                     1 | 128 | 2 << 8 | 4 << 16 | 72 << 24 | 1 << 31]
