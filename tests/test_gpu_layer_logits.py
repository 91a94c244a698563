"""GPU layer from gate logits: steps of changing routing that follow one another without a wait give
what each gives alone."""
import numpy as np
import pytest

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


@pytest.mark.parametrize("T,block_m,config", [(1, 8, "tiny"), (16, 8, "tiny"), (17, 16, "tiny"), (200, 32, "tiny"), (300, 64, "tiny")])
def test_steps_in_a_row(chord, T, block_m, config):
    import torch
    from w4a16_int4_mixture_align_b200 import inputs
    d = inputs.make_inputs(inputs.CONFIGS[config])
    E, k = d["qw13"].shape[0], 2
    layer = chord.ChordMoE(d["qw13"], d["s13"].view(np.int16), d["qw2"], d["s2"].view(np.int16), topk=k, max_tokens=T,
                           block_m=block_m)
    g = torch.Generator("cuda").manual_seed(T)
    steps = [(torch.randn((T, layer.H), generator=g, device="cuda").to(torch.bfloat16),
              torch.randn((T, E), generator=g, device="cuda")) for _ in range(24)]
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    want = []
    for x, logits in steps:
        ids, w = layer.route(logits, bias=bias, scale=2.0)
        torch.cuda.synchronize()
        want.append((layer.forward(x, ids, w), ids, w))
        torch.cuda.synchronize()

    def run():
        return [layer.forward_logits(x, logits, bias=bias, scale=2.0) for x, logits in steps]
    for _ in range(3):
        for a, b in zip(run(), want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert layer.check_status() == 0


@pytest.mark.parametrize("T", [4, 16])
def test_hidden_rows_straight_from_an_fp8_product(chord, T):
    """The layer's input written by the kernel right before its first one, on changing inputs."""
    import torch
    from w4a16_int4_mixture_align_b200 import inputs
    d = inputs.make_inputs(inputs.CONFIGS["tiny"])
    E, H, I = d["qw13"].shape[0], d["qw13"].shape[2] * 8, 256
    layer = chord.ChordMoE(d["qw13"], d["s13"].view(np.int16), d["qw2"], d["s2"].view(np.int16), topk=2, max_tokens=T,
                           block_m=8)
    g = torch.Generator("cuda").manual_seed(T)

    def code(*shape):  # finite codes of both signs
        return torch.randint(0, 120, shape, generator=g, device="cuda").add(128 * torch.randint(
            0, 2, shape, generator=g, device="cuda")).to(torch.uint8)

    mlp = chord.ChordFP8MLP(code(2 * I, H), torch.full((2 * I // 128, H // 128), 2.0 ** -10, device="cuda"), code(H, I),
                            torch.full((H // 128, I // 128), 2.0 ** -10, device="cuda"), max_tokens=T)
    xs = [torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(16)]
    ids, w = layer.route(torch.randn((T, E), generator=g, device="cuda"))
    h = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")

    def step(x, wait):
        layer.align(ids)
        mlp(x, out=h)
        if wait:
            torch.cuda.synchronize()
        out = layer._forward_sorted(h, ids, w, None, 0)
        if wait:
            torch.cuda.synchronize()
        return out
    want = [step(x, True) for x in xs]
    assert all(torch.isfinite(y.float()).all() for y in want)
    for _ in range(3):
        for got, y in zip([step(x, False) for x in xs], want):
            assert torch.equal(got, y)


def test_mismatched_blob_behind_the_router(chord):
    """A gate_up kernel that refuses its weights ends at once; the down kernel, whose weights are right,
    and the next step still find the routing complete."""
    import torch
    from w4a16_int4_mixture_align_b200 import inputs
    d = inputs.make_inputs(inputs.CONFIGS["tiny"])
    E, T = d["qw13"].shape[0], 16
    layer = chord.ChordMoE(d["qw13"], d["s13"].view(np.int16), d["qw2"], d["s2"].view(np.int16), topk=2, max_tokens=T,
                           block_m=8)
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((T, layer.H), generator=g, device="cuda").to(torch.bfloat16)
    steps = [torch.randn((T, E), generator=g, device="cuda") for _ in range(8)]
    want = [layer.forward_logits(x, logits)[0] for logits in steps]
    right, wrong = layer.w13, layer.w2.clone()
    got = []
    for logits in steps:
        layer.w13 = wrong
        layer.forward_logits(x, logits.flip(0))
        layer.w13 = right
        got.append(layer.forward_logits(x, logits)[0])
    assert layer.check_status() == chord.CHORD_DEV_BLOB_MISMATCH
    for a, b in zip(got, want):
        assert torch.equal(a, b)
