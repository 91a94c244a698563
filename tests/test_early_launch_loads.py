"""Kernels that start while the kernel before them still writes do not read its output as read-only
data (ld.global.nc): the scored router and the grouped routing pass let the W4A16 gate_up kernel
start while they write the routing tensors, gate_up the down kernel while it writes the
intermediate, and an FP8 product its successor while it writes rows that this may read."""
import os
import re

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "w4a16_int4_mixture_align_b200", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


@pytest.mark.parametrize("name", ["stream_gemm.cu", "stream_gemm_short.cu", "stream_common.cuh"])
def test_routing_and_activations(name):
    assert not re.search(r"__ldg\(|ld\.global\.nc|__restrict__", source(name))


@pytest.mark.parametrize("name", ["router.cu", "grouped.cu", "fp8_quant.cu", "fp8_stream.cu", "fp8_tile.cu"])
def test_kernels_that_are_always_launched_early(name):
    text = source(name)
    assert "grid_dep_wait" in text and "__ldg(" not in text and "ld.global.nc" not in text


@pytest.mark.parametrize("name", ["stream_gemm.cu", "stream_gemm_short.cu"])
def test_no_block_ends_before_the_kernel_before_it(name):
    """A grid that ends at once (another weight's blob) must not let its successor overtake its
    predecessor."""
    text = source(name)
    before_roles = text[text.index("abort_flag = 2;"):text.index("// ---", text.index("abort_flag = 2;"))]
    left = before_roles[before_roles.index("if (abort_flag)"):]
    assert "grid_dep_wait();" in left[:left.index("return;")]
