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
