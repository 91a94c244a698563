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


def test_buffers_of_a_creeping_batch_stay_bounded(chord):  # noqa: F811
    """Outgrown buffers are kept for graphs, so they must not add up to more than a few times the
    largest; a smaller reservation keeps what is there."""
    import torch
    mlp = chord.ChordFP8MLP(*weights(5))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in range(1, 400):
        mlp.reserve(T)
        assert mlp.max_tokens >= T
    for T in (1, 399, 7, 2):
        mlp.reserve(T)
    held = torch.cuda.memory_allocated() - before
    # what one layer of this many tokens allocates (512-byte granules and 64 KiB headers included)
    one = chord.ChordFP8MLP(*weights(5), max_tokens=mlp.max_tokens)
    own = sum(t.numel() * t.element_size() for t in (one.xq, one.xs, one.aq, one.as_, one.workspace))
    growths = 16                                          # of a factor of 1.5 and one row at least: 1, 2, 3, 4, 6, 9, .. 474
    assert held <= 3 * own + growths * (65536 + 32768)
    x = rows(399, 3)
    assert torch.equal(mlp(x), one(x)) and mlp.max_tokens < 2 * 399


def test_status_outlives_growth(chord):  # noqa: F811
    """An error raised by a call, or by the replay of a graph, on buffers that the layer has outgrown
    is still reported, once."""
    import torch
    mlp = chord.ChordFP8MLP(*weights(5), max_tokens=2)
    word = mlp.workspace[:4].view(torch.int32)
    mlp(rows(50, 1))
    word.fill_(chord.CHORD_DEV_TIMEOUT)
    later = mlp.workspace[:4].view(torch.int32)
    assert later.data_ptr() != word.data_ptr()
    assert mlp.check_status() == chord.CHORD_DEV_TIMEOUT and mlp.check_status() == 0
    word.fill_(chord.CHORD_DEV_TIMEOUT)
    later.fill_(chord.CHORD_DEV_ROUTING_INVALID)
    assert mlp.check_status() == chord.CHORD_DEV_TIMEOUT | chord.CHORD_DEV_ROUTING_INVALID
    assert mlp.check_status() == 0


@pytest.mark.parametrize("T,h,i", [(1, 7168, 2048), (16, 7168, 2048), (300, 1024, 512), (2500, 1024, 512)])
def test_repeats_bit_for_bit(chord, T, h, i):  # noqa: F811
    """The same call on the same rows gives the same bits, whether its operands come from L2 or HBM."""
    import torch
    g = torch.Generator("cuda").manual_seed(T)

    def code(*shape):  # finite codes of both signs
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8).bitwise_and(0xBF)

    mlp = chord.ChordFP8MLP(code(2 * i, h), torch.full((2 * i // 128, h // 128), 0.01, device="cuda"), code(h, i),
                            torch.full((h // 128, i // 128), 0.01, device="cuda"), max_tokens=T)
    x = torch.randn((T, h), generator=g, device="cuda").to(torch.bfloat16)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    want = mlp(x)
    assert torch.isfinite(want.float()).all()
    for n in range(12):
        if n % 2:
            flush.fill_(n)
        assert torch.equal(mlp(x), want), n
    assert mlp.check_status() == 0
