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


def test_weights_that_are_replaced(chord):  # noqa: F811
    """A call multiplies by the weights that the layer holds then, and checks them."""
    import torch
    a, b, x = weights(5), weights(40), rows(6, 2)
    other = chord.ChordFP8MLP(*b, max_tokens=6)
    want_a, want_b = chord.ChordFP8MLP(*a, max_tokens=6)(x), other(x)
    mlp = chord.ChordFP8MLP(*[v.clone() for v in a], max_tokens=6)
    assert torch.equal(mlp(x), want_a)
    mlp.w13, mlp.s13, mlp.w2, mlp.s2 = [v.clone() for v in b]
    junk = [torch.full((2 * I * H,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]  # where the old ones were
    assert torch.equal(mlp(x), want_b)
    mlp.w13.data, mlp.s13.data, mlp.w2.data, mlp.s2.data = [v.clone() for v in a]
    assert torch.equal(mlp(x), want_a) and mlp.check_status() == 0
    for name, bad in (("w13", a[0][:I].clone()), ("s13", a[1].double()), ("w2", a[2].T), ("s2", a[3].cpu())):
        setattr(mlp, name, bad)
        with pytest.raises(AssertionError):
            mlp(x)
        setattr(mlp, name, getattr(other, name))
    assert torch.equal(mlp(x), want_b)
    del junk
