"""Float8 and routed-expert entry points at the ends of their ranges: batches of nothing and the largest sizes. Validation
runs before any CUDA call, so these need no GPU (the pointers are never read)."""
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
