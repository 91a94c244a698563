"""What the binding of the FP8 operators refuses before any call into the library."""
import pytest

from helpers import ensure_built


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


def test_fp32_sums_do_not_go_into_a_bf16_output(chord):
    """CHORD_FLAG_OUTPUT_FP32 with a bf16 `out` would be written with rows twice as long as they are."""
    import torch
    rows, N, K, E = 4, 128, 128, 2
    xq, w = torch.zeros((E * rows, K), dtype=torch.uint8), torch.zeros((E, N, K), dtype=torch.uint8)
    xs, ws = torch.zeros((1, E * rows)), torch.zeros((E, 1, 1))
    out = torch.zeros((E * rows, N), dtype=torch.bfloat16)
    work, m = torch.zeros(1 << 17, dtype=torch.uint8), torch.zeros(E * rows, dtype=torch.int32)
    flag = chord.CHORD_FLAG_OUTPUT_FP32
    with pytest.raises(AssertionError, match="OUTPUT_FP32"):
        chord.chord_fp8_gemm(xq, xs, w[0], ws[0], out, work, flag)
    with pytest.raises(AssertionError, match="OUTPUT_FP32"):
        chord.chord_fp8_grouped_contiguous(xq, xs, m, w, ws, out, work, flag)
    with pytest.raises(AssertionError, match="OUTPUT_FP32"):
        chord._fp8_out(out, E * rows, N, flag)
