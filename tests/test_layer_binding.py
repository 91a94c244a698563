"""What ChordMoE.forward_logits refuses before any call into the library."""
import pytest

from helpers import ensure_built


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


def bare_layer(chord, route):
    """A layer of the sizes alone, whose routing is `route`."""
    layer = object.__new__(chord.ChordMoE)
    layer.H, layer.topk, layer.E, layer.max_tokens = 256, 2, 8, 16
    layer.route = route
    return layer


def reached(*args, **kw):
    raise RuntimeError("routed")


@pytest.mark.parametrize("shape", [(5, 256), (3, 256), (4, 128), (4, 512)])
def test_rows_of_another_number_or_width(chord, shape):
    """The forward takes its number of tokens from `hidden`: more rows than logits would read ids
    and weights that are not there."""
    import torch
    with pytest.raises(AssertionError, match="hidden has shape"):
        bare_layer(chord, reached).forward_logits(torch.zeros(shape), torch.zeros((4, 8)))


def test_ids_of_another_width(chord):
    """Ids in a buffer with other than topk columns would be read with its width."""
    import torch
    ids, w = torch.zeros((4, 4), dtype=torch.int32), torch.zeros((4, 4))
    layer = bare_layer(chord, lambda logits, topk_ids=None, topk_weights=None: (topk_ids, topk_weights))
    layer._forward_sorted = reached
    with pytest.raises(AssertionError, match="topk_ids"):
        layer.forward_logits(torch.zeros((4, 256)), torch.zeros((4, 8)), topk_ids=ids, topk_weights=w)


def sums(chord, out, flags):
    """forward_logits with a forward that only notes its output."""
    import torch
    layer = bare_layer(chord, lambda logits: (torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))))
    layer.device, layer.block_m, layer.I = torch.device("cpu"), 8, 128
    layer.sorted_ids = layer.expert_ids = layer.ntp = layer.w13 = layer.w2 = layer.workspace = None
    return layer.forward_logits(torch.zeros((4, 256)), torch.zeros((4, 8)), out=out, flags=flags)[0]


def test_output_is_as_large_as_the_flag_makes_it(chord, monkeypatch):
    """CHORD_FLAG_OUTPUT_FP32 writes four bytes an element: into an fp32 tensor of its own, or into an
    `out` that holds them."""
    import torch
    monkeypatch.setattr(chord, "chord_moe_forward", lambda *args, **kw: None)
    flag = chord.CHORD_FLAG_OUTPUT_FP32
    assert sums(chord, None, 0).dtype == torch.bfloat16 and sums(chord, None, flag).dtype == torch.float32
    for dtype, flags in ((torch.bfloat16, 0), (torch.float32, flag)):
        out = torch.zeros((4, 256), dtype=dtype)
        assert sums(chord, out, flags) is out
    with pytest.raises(AssertionError, match="out holds"):
        sums(chord, torch.zeros((4, 256), dtype=torch.bfloat16), flag)
    with pytest.raises(AssertionError, match="out holds"):
        sums(chord, torch.zeros((3, 256), dtype=torch.bfloat16), 0)


def test_one_stream_for_routing_and_forward(chord):
    """`stream` is an argument of the router alone: the forward would not wait for it."""
    import torch
    with pytest.raises(TypeError, match="stream"):
        bare_layer(chord, reached).forward_logits(torch.zeros((4, 256)), torch.zeros((4, 8)), stream=object())
