"""GPU scored router (chord_router_scored_align) vs a 64-bit reference: ids and routing
tensors exact, weights within FP32 rounding."""
import numpy as np
import pytest

import oracle
import ref64
from helpers import ensure_built

pytestmark = pytest.mark.gpu

LOWEST = {"float32": float(np.finfo(np.float32).min), "bfloat16": -3.3895313892515355e38, "float16": -65504.0}


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


def run(chord, logits, topk, E, bm, **kw):
    import torch
    T, _ = logits.shape
    dev = "cuda"
    cap = chord.chord_moe_align_capacity(T, topk, E, bm)
    nb = chord.chord_moe_align_num_blocks(T, topk, E, bm)

    def full(*shape, value=-7, dtype=torch.int32):
        return torch.full(shape, value, dtype=dtype, device=dev)
    ids, w = full(T, topk), full(T, topk, dtype=torch.float32)
    s, e, n, o = full(max(cap, 1)), full(max(nb, 1)), full(2), full(E + 1)
    wsb = chord.chord_moe_align_workspace_bytes(T, topk, E)
    ws = full(wsb, value=0x5A, dtype=torch.uint8) if wsb else None
    chord.chord_router_scored_align(logits, topk, E, bm, ids, w, s, e, n, o, ws, **kw)
    torch.cuda.synchronize()
    return [v.cpu().numpy() for v in (ids, w, s[:cap], e[:nb], n, o)]


def check(chord, logits, bias, topk, E, bm, score="sigmoid", n_group=1, topk_group=1, group_top=1, renormalize=True,
          scale=1.0):
    """`logits`: a torch CUDA tensor [T, G]."""
    import torch
    name = str(logits.dtype).replace("torch.", "")
    got = run(chord, logits, topk, E, bm, bias=None if bias is None else torch.from_numpy(bias).cuda(), score=score,
              n_group=n_group, topk_group=topk_group, group_top=group_top, renormalize=renormalize, scale=scale)
    ids, w = ref64.route(logits.double().cpu().numpy(), LOWEST[name],
                         None if bias is None else bias.astype(np.float64), topk, score, n_group, topk_group,
                         group_top, renormalize, scale)
    np.testing.assert_array_equal(got[0], ids)
    # the scores are FP64, rounded once to FP32 (2^-24, with room for the two exps' own last
    # bits 2^-23); an un-normalised softmax divides by an FP32 sum of at most 1024
    # exponentials (2 ulp each, 32 + 5 additions): (2 * 2 + 37 + 2) * 2^-24
    rtol = 43 * 2.0 ** -24 if score == "softmax" and not renormalize else 2.0 ** -23
    np.testing.assert_allclose(got[1], w, rtol=rtol, atol=1e-38)
    rs, re_, rn, ro = oracle.moe_align(ids, E, bm)
    np.testing.assert_array_equal(got[2], rs)
    np.testing.assert_array_equal(got[3], re_)
    assert int(got[4][0]) == rn and int(got[4][1]) == chord.routing_tag(bm)
    np.testing.assert_array_equal(got[5], ro)
    return got


def normal(T, G, seed, dtype="float32", spread=1.0):
    import torch
    rng = np.random.default_rng(seed)
    return torch.from_numpy((spread * rng.standard_normal((T, G))).astype(np.float32)).cuda().to(getattr(torch, dtype))


CASES = [
    # T, G, topk, E, bm, dtype, score, bias, n_group, topk_group, group_top, renormalize
    (1, 384, 8, 48, 8, "float32", "sigmoid", True, 1, 1, 1, True),     # one launch
    (8, 384, 8, 48, 8, "bfloat16", "softmax", True, 8, 4, 2, True),    # one launch, largest batch
    (9, 384, 8, 48, 8, "float16", "sigmoid", True, 8, 4, 2, True),
    (128, 384, 8, 48, 8, "bfloat16", "sigmoid", True, 8, 4, 2, True),
    (700, 384, 8, 384, 64, "float32", "sigmoid", False, 1, 1, 1, True),  # multi-CTA sort
    (300, 256, 8, 32, 16, "float32", "softmax", False, 8, 3, 1, False),
    (300, 160, 6, 160, 8, "bfloat16", "softmax", False, 8, 3, 1, False),  # many equal logits
    (300, 160, 6, 160, 8, "bfloat16", "sigmoid", False, 4, 2, 2, True),
    (65, 100, 3, 10, 4, "float32", "softmax", True, 5, 2, 2, True),    # G not a multiple of 32, five groups
    (33, 96, 4, 96, 1, "float32", "sigmoid", True, 32, 5, 2, True),    # groups of three
    (20, 64, 64, 64, 8, "float32", "sigmoid", True, 1, 1, 1, True),    # every expert, more than 32
    (20, 64, 32, 64, 8, "float32", "softmax", True, 2, 1, 1, True),    # a whole group
    (50, 1024, 1, 16, 1, "float32", "sigmoid", True, 1, 1, 1, True),
    (40, 1024, 40, 1024, 1, "bfloat16", "softmax", True, 16, 3, 2, False),
    (7, 1, 1, 1, 8, "float32", "softmax", False, 1, 1, 1, True),       # one expert
    (12, 32, 2, 32, 8, "float32", "sigmoid", True, 32, 2, 1, True),    # groups of one
    (200, 500, 16, 125, 32, "float32", "sigmoid", True, 1, 1, 1, False),
]


@pytest.mark.parametrize("T,G,k,E,bm,dtype,score,bias,ng,tg,gt,renorm", CASES)
def test_matches_reference(chord, T, G, k, E, bm, dtype, score, bias, ng, tg, gt, renorm):
    b = (0.1 * np.random.default_rng(G + k).standard_normal(G)).astype(np.float32) if bias else None
    check(chord, normal(T, G, T + G + k, dtype), b, k, E, bm, score, ng, tg, gt, renorm, scale=2.5)


def test_empty_batch(chord):
    import torch
    check(chord, torch.empty((0, 384), device="cuda"), None, 8, 48, 8)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [5, 40])
def test_masked_logits(chord, score, T):
    """-inf, the type's lowest value and NaN mask; rows with fewer than topk experts left, and
    with none, get id -1 and weight 0."""
    import torch
    for dtype in ("float32", "bfloat16", "float16"):
        x = normal(T, 64, 3, dtype)
        x[0] = float("-inf")                        # nothing left
        x[1] = torch.finfo(x.dtype).min
        x[2, 3:] = float("nan")                     # three left
        x[3, ::2] = torch.finfo(x.dtype).min
        x[4, 5] = float("inf")
        b = (np.arange(64) / 64).astype(np.float32)  # a masked expert's bias must not count
        for bias in (None, b):
            for ng, tg, gt in ((1, 1, 1), (8, 2, 2), (8, 2, 1)):
                got = check(chord, x, bias, 6, 64, 8, score, ng, tg, gt)
                assert (got[0][0] == -1).all() and (got[1][0] == 0).all()


def test_near_ties_go_by_exact_scores(chord):
    """Choice scores that FP32 cannot tell apart: sigmoids next to 1 with tiny biases, and sums
    of groups that differ in the last bits."""
    import torch
    rng = np.random.default_rng(5)
    l = (12 + 1e-3 * rng.standard_normal((64, 128))).astype(np.float32)   # 1 - s ~ 6e-6, differences ~ 6e-9
    b = (1e-9 * rng.standard_normal(128)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        for ng, tg, gt in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
            check(chord, torch.from_numpy(l).cuda(), b, 8, 128, 8, score, ng, tg, gt)


def test_ties_go_to_the_lower_id(chord):
    import torch
    x = torch.zeros((70, 96), device="cuda")
    x[1::2] = normal(35, 96, 9, "bfloat16").float().round()
    zero = np.zeros(96, np.float32)
    for bias in (None, zero):
        for score in ("sigmoid", "softmax"):
            for ng, tg, gt in ((1, 1, 1), (6, 2, 2)):
                check(chord, x, bias, 8, 24, 8, score, ng, tg, gt)


def test_large_logits_and_biases(chord):
    x = normal(60, 128, 4, spread=60.0)
    rng = np.random.default_rng(1)
    for b in ((1000 * rng.standard_normal(128)).astype(np.float32), (0.5 * rng.standard_normal(128)).astype(np.float32)):
        for score in ("sigmoid", "softmax"):
            check(chord, x, b, 8, 128, 8, score, 4, 2, 2)
            check(chord, x, b, 8, 128, 8, score, renormalize=False)


def test_small_sigmoids_keep_their_ratio(chord):
    """Scores far below the FP32 range still renormalise to weights."""
    x = normal(30, 64, 8) - 300.0
    got = check(chord, x, None, 4, 64, 8)
    np.testing.assert_allclose(got[1].sum(1), 1.0, rtol=1e-6)


def test_rows_that_lie_apart(chord):
    import torch
    wide = normal(50, 200, 6)
    a = check(chord, wide[:, 40:136], None, 4, 96, 8)
    b = check(chord, wide[:, 40:136].contiguous(), None, 4, 96, 8)
    for u, v in zip(a, b):
        np.testing.assert_array_equal(u, v)
    del torch


def test_graph_replay_and_other_stream(chord):
    import torch
    x = normal(300, 384, 2)
    bias = torch.zeros(384, device="cuda")
    cap = chord.chord_moe_align_capacity(300, 8, 48, 8)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.zeros((300, 8), **i32), torch.zeros((300, 8), device="cuda")
    s, e, n = torch.zeros(cap, **i32), torch.zeros((cap + 7) // 8, **i32), torch.zeros(2, **i32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        chord.chord_router_scored_align(x, 8, 48, 8, ids, w, s, e, n, bias=bias)
    x.copy_(normal(300, 384, 77))
    g.replay()
    torch.cuda.synchronize()
    ref, _ = ref64.route(x.double().cpu().numpy(), LOWEST["float32"], None, 8, "sigmoid", 1, 1, 1, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)


# The sort behind the router: one CTA up to 16 tokens, one cluster up to 256, a cluster kernel up to
# 65536 and up to 262144 slots, then the kernels of the plain sort; both sides of each border.
@pytest.mark.parametrize("T,G,k,E,bm", [(16, 128, 64, 128, 8), (17, 128, 64, 128, 8), (256, 128, 64, 100, 16),
                                        (257, 128, 64, 100, 16), (8192, 64, 8, 64, 128), (8193, 64, 8, 64, 128),
                                        (8193, 1024, 8, 1024, 4), (32768, 64, 8, 9, 64), (32769, 64, 8, 9, 64)])
def test_sorts(chord, T, G, k, E, bm):
    b = (0.1 * np.random.default_rng(G).standard_normal(G)).astype(np.float32)
    check(chord, normal(T, G, T), b, k, E, bm)


def test_every_token_masked(chord):
    """A batch of padding alone routes nothing."""
    import torch
    for T in (3, 200, 3000):
        got = check(chord, torch.full((T, 96), float("-inf"), device="cuda"), np.ones(96, np.float32), 4, 96, 16)
        assert (got[0] == -1).all() and int(got[4][0]) == 0


def test_all_tokens_to_the_same_experts(chord):
    """The longest run of one expert, with ties everywhere."""
    import torch
    for T in (16, 256, 5000):
        check(chord, torch.zeros((T, 256), device="cuda"), None, 8, 4, 64)
