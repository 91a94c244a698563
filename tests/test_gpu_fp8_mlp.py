"""GPU ChordFP8MLP: outputs, buffers and weights over the life of a layer."""
import pytest

from test_gpu_fp8 import chord, codes, cuda, scales  # noqa: F401

pytestmark = pytest.mark.gpu
H, I = 256, 128


def weights(seed):
    return [cuda(v) for v in (codes((2 * I, H), seed), scales((2, 2), seed + 2), codes((H, I), seed + 1),
                              scales((2, 1), seed + 3))]


def rows(T, seed):
    import torch
    return torch.randn((T, H), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(torch.bfloat16)


def test_fp32_sums_by_flag(chord):  # noqa: F811
    """CHORD_FLAG_OUTPUT_FP32 goes with an fp32 `out`, and is refused for any other."""
    import torch
    mlp, x = chord.ChordFP8MLP(*weights(5), max_tokens=9), rows(9, 1)
    want = mlp(x, out=torch.empty((9, H), device="cuda"))
    got = mlp(x, out=torch.empty((9, H), device="cuda"), flags=chord.CHORD_FLAG_OUTPUT_FP32)
    assert torch.equal(want, got) and mlp.check_status() == 0
    for out in (None, torch.empty((9, H), dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(AssertionError, match="OUTPUT_FP32"):
            mlp(x, out=out, flags=chord.CHORD_FLAG_OUTPUT_FP32)
