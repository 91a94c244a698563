"""GPU FP8 products by the tile kernel with operands that come from HBM, where copies land out of
order: the bits stay the same call after call and are the product's."""
import numpy as np
import pytest

import ref64
from test_gpu_fp8 import check_rows, chord, codes, cuda, scales, workspace  # noqa: F401

pytestmark = pytest.mark.gpu
B = ref64.BLOCK


# Up to 128 rows the estimates always give 128 x 128 tiles to the tensor cores (one wave of them
# takes 2.6 + 0.265 KB + 1.4 us against 3.0 + 0.485 KB + 0.9 of the pairs). The last two go to pairs
# with 256 x 256 tiles (estimates of 22 us against 31, and 38 against 43).
@pytest.mark.parametrize("M,N,K", [(128, 4096, 7168), (100, 18944, 1040), (1, 4096, 8192), (2048, 9216, 1024),
                                   (4096, 4096, 2048)])
def test_cold_operands(chord, M, N, K):  # noqa: F811
    import torch
    xq, wq = codes((M, K), M + 1), codes((N, K), N)
    xs, ws = scales((-(-K // B), M), 3), scales((-(-N // B), -(-K // B)), 4)
    args, work = [cuda(v) for v in (xq, xs, wq, ws)], workspace(chord, M)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")   # twice the L2
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 24)])
    want = torch.full((M, N), float("nan"), device="cuda")
    chord.chord_fp8_gemm(*args, want, work, chord.CHORD_FLAG_FORCE_TENSOR)
    check_rows(want[torch.from_numpy(rows).cuda()], *ref64.product(xq[rows], xs[:, rows], wq, ws), K)
    out = torch.empty_like(want)
    for i in range(30):
        flush.fill_(i)
        chord.chord_fp8_gemm(*args, out, work, chord.CHORD_FLAG_FORCE_TENSOR)
        assert torch.equal(out, want), i
    assert chord.chord_moe_check_status(work) == 0
