"""GPU FP8 block-128 operators vs 64-bit references: quantised codes and scales bit for bit,
products within the rounding of FP32 sums."""
import numpy as np
import pytest

import ref64
from helpers import ensure_built

pytestmark = pytest.mark.gpu
B = ref64.BLOCK


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(a):
    """fp32 array -> bf16 CUDA tensor and its exact fp32 values."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def codes(shape, seed, spread=1.0):
    """Finite E4M3 codes of normal values (subnormals, zeros and +-448 among them)."""
    rng = np.random.default_rng(seed)
    v = ref64.e4m3_round(spread * rng.standard_normal(shape) * 2.0 ** rng.integers(-6, 4, shape))
    order = np.argsort(ref64.CODES[:127])
    c = order[np.searchsorted(ref64.CODES[:127], np.abs(v))].astype(np.uint8)
    return np.where(np.signbit(v), c | 0x80, c).astype(np.uint8)


def scales(shape, seed):
    rng = np.random.default_rng(seed)
    return (2.0 ** rng.uniform(-9, 1, shape)).astype(np.float32)


# ------------------------------------------------------------------ quantise

def check_quantised(q, s, x32):
    v, ref_s = ref64.quantise(x32)
    np.testing.assert_array_equal(s, ref_s)
    np.testing.assert_array_equal(ref64.CODES[q], ref64.e4m3_round(v.astype(np.float64)))


@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (8, 1024), (9, 1040), (77, 7168), (300, 272)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_quantise(chord, rows, K, dtype):
    import torch
    rng = np.random.default_rng(rows + K)
    x = rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((rows, 1)))
    x[rng.random((rows, K)) < 0.01] *= 100
    x[0, :min(K, 64)] = 0
    t, x32 = bf16(x)
    if dtype == "float32":
        x32 = x.astype(np.float32)
        t = cuda(x32)
    q = torch.full((rows, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-K // B), rows), -1.0, device="cuda")
    chord.chord_fp8_quantize(t, q, s)
    check_quantised(q.cpu().numpy(), s.cpu().numpy(), x32)


def test_quantise_extremes(chord):
    """Zeros, the smallest and largest finite values, and blocks with infinities or NaN, which
    spoil themselves and nothing else."""
    import torch
    x = np.ones((6, 256), np.float32)
    x[0] = 0
    x[1, :128] = 1e-39
    x[2, :128] = 3.38e38
    x[3, 5] = np.inf
    x[4, 200] = np.nan
    x[5, 7] = -np.inf
    q = torch.zeros((6, 256), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2, 6), device="cuda")
    for t, x32 in (bf16(x), (cuda(x), x)):
        chord.chord_fp8_quantize(t, q, s)
        qn, sn = q.cpu().numpy(), s.cpu().numpy()
        good = np.ones((2, 6), bool)
        good[0, 3] = good[1, 4] = good[0, 5] = False
        assert np.isnan(sn[~good]).all()
        clean = np.where(np.repeat(good.T, B, 1), x32, 0)
        v, ref_s = ref64.quantise(clean)
        np.testing.assert_array_equal(sn[good], ref_s[good])
        at = np.repeat(good.T, B, 1)
        np.testing.assert_array_equal(ref64.CODES[qn][at], ref64.e4m3_round(v.astype(np.float64))[at])


@pytest.mark.parametrize("rows,I", [(1, 16), (5, 128), (33, 400), (64, 2048)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_silu_quantise(chord, rows, I, dtype):
    import torch
    rng = np.random.default_rng(rows + I)
    h = 3 * rng.standard_normal((rows, 2 * I))
    h[0, :4] = [-100, -50, 90, 0]
    t, h32 = bf16(h)
    if dtype == "float32":
        h32 = h.astype(np.float32)
        t = cuda(h32)
    q = torch.zeros((rows, I), dtype=torch.uint8, device="cuda")
    s = torch.zeros((-(-I // B), rows), device="cuda")
    chord.chord_fp8_silu_quantize(t, q, s)
    a = ref64.silu_mul(h32.astype(np.float64))
    # silu * up in FP32: exp within 2 ulp, one addition, one division, one product, then the
    # quotient and the product of the quantisation: at most 8 roundings of 2^-24
    p = np.zeros((rows, s.shape[0] * B))
    p[:, :I] = np.abs(a)
    amax = np.maximum(p.reshape(rows, -1, B).max(2), 2.0 ** -100)
    np.testing.assert_allclose(s.cpu().numpy().T, amax / 448, rtol=8 * 2.0 ** -24)
    v = a * np.repeat(448 / amax, B, 1)[:, :I]
    clear = ref64.border_distance(v) > 24 * 2.0 ** -24   # codes are certain away from a border
    assert clear.mean() > 0.99
    np.testing.assert_array_equal(ref64.CODES[q.cpu().numpy()][clear], ref64.e4m3_round(v)[clear])


@pytest.mark.parametrize("silu", [False, True])
def test_quantise_masked_rows_and_strides(chord, silu):
    """Rows behind the counts are neither read nor written; rows may lie apart; counts out of
    range are clamped."""
    import torch
    E, max_m, K = 5, 7, 272
    counts = np.array([0, 7, 3, -2, 100], np.int32)
    width = 2 * K if silu else K
    rng = np.random.default_rng(1)
    t, x32 = bf16(rng.standard_normal((E * max_m, width)))
    wide = torch.full((E * max_m, width + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + width] = t
    live = (np.arange(max_m)[None, :] < counts[:, None]).ravel()
    wide[torch.from_numpy(~live).cuda()] = float("nan")
    q = torch.full((E * max_m, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((3, E * max_m), -1.0, device="cuda")
    (chord.chord_fp8_silu_quantize if silu else chord.chord_fp8_quantize)(wide[:, 8:8 + width], q, s, masked_m=cuda(counts))
    q2 = torch.empty((int(live.sum()), K), dtype=torch.uint8, device="cuda")
    s2 = torch.empty((3, int(live.sum())), device="cuda")
    (chord.chord_fp8_silu_quantize if silu else chord.chord_fp8_quantize)(t[torch.from_numpy(live).cuda()], q2, s2)
    np.testing.assert_array_equal(q.cpu().numpy()[live], q2.cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy()[:, live], s2.cpu().numpy())
    assert (q.cpu().numpy()[~live] == 0x55).all() and (s.cpu().numpy()[:, ~live] == -1).all()


# ------------------------------------------------------------------ products

def flag(chord, schedule):
    return {"auto": 0, "stream": chord.CHORD_FLAG_FORCE_STREAM, "tensor": chord.CHORD_FLAG_FORCE_TENSOR}[schedule]


def workspace(chord, rows, E=1):
    import torch
    return torch.zeros(chord.chord_fp8_workspace_bytes(rows, E), dtype=torch.uint8, device="cuda")


def check_rows(out, y, a, K, rows=slice(None)):
    import torch
    got = out.double().cpu().numpy()[rows]
    bound = ref64.product_bound(y, a, K, out.dtype == torch.bfloat16)
    worst = (np.abs(got - y) / bound).max() if y.size else 0.0
    assert np.isfinite(got).all() and worst <= 1.0, worst


DENSE = [
    # M, N, K
    (1, 8, 16), (1, 128, 128), (1, 4096, 7168), (3, 72, 144), (8, 136, 256), (9, 264, 400), (17, 24, 1024),
    (32, 512, 272), (33, 576, 1520), (64, 136, 2048), (100, 256, 128), (128, 264, 384), (129, 256, 640),
    (255, 520, 272), (300, 1032, 512), (513, 264, 896),
    (40, 128, 7168), (65, 384, 1040), (120, 136, 4096), (2, 24, 144),
]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("schedule", ["stream", "tensor", "auto"])
def test_dense(chord, M, N, K, schedule):
    import torch
    xq, wq = codes((M, K), M + N + K), codes((N, K), M + N + K + 1)
    xs, ws = scales((-(-K // B), M), 3), scales((-(-N // B), -(-K // B)), 4)
    y, a = ref64.product(xq, xs, wq, ws)
    work = workspace(chord, M)
    args = [cuda(v) for v in (xq, xs, wq, ws)]
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        chord.chord_fp8_gemm(*args, out, work, flag(chord, schedule))
        check_rows(out, y, a, K)
    again = torch.empty_like(out)
    chord.chord_fp8_gemm(*args, again, work, flag(chord, schedule))
    assert torch.equal(out, again)                       # the same bits call after call
    assert chord.chord_moe_check_status(work) == 0


def test_dense_nan_stays_in_its_row(chord):
    import torch
    xq, wq = codes((70, 256), 1), codes((136, 256), 2)
    xs, ws = scales((2, 70), 3), scales((2, 2), 4)
    y, a = ref64.product(xq, xs, wq, ws)
    xq[5, 3] = 0x7F
    xs[1, 66] = np.nan
    for schedule in ("stream", "tensor"):
        out = torch.zeros((70, 136), device="cuda")
        chord.chord_fp8_gemm(*[cuda(v) for v in (xq, xs, wq, ws)], out, workspace(chord, 70), flag(chord, schedule))
        ok = np.ones(70, bool)
        ok[[5, 66]] = False
        assert torch.isnan(out[5]).all() and torch.isnan(out[66]).all()
        check_rows(out, y[ok], a[ok], 256, ok)


def test_no_rows(chord):
    import torch
    out = torch.empty((0, 128), device="cuda")
    w, ws = cuda(codes((128, 128), 1)), cuda(scales((1, 1), 1))
    xq, xs = torch.empty((0, 128), dtype=torch.uint8, device="cuda"), torch.empty((1, 0), device="cuda")
    chord.chord_fp8_gemm(xq, xs, w, ws, out, workspace(chord, 0))


MASKED = [
    # E, max_m, N, K, counts
    (3, 1, 136, 272, [1, 0, 1]),
    (4, 5, 128, 256, [0, 5, 2, 1]),
    (6, 33, 72, 400, [33, 0, 7, 32, 9, 0]),
    (3, 130, 264, 640, [130, 128, 1]),
    (2, 300, 520, 272, [257, 300]),
    (5, 16, 512, 1024, [0, 0, 0, 0, 0]),
    (4, 16, 136, 272, [-3, 99, 4, 16]),      # clamped
]


@pytest.mark.parametrize("E,max_m,N,K,counts", MASKED)
@pytest.mark.parametrize("schedule", ["stream", "tensor", "auto"])
def test_masked(chord, E, max_m, N, K, counts, schedule):
    import torch
    rows = E * max_m
    xq, wq = codes((rows, K), rows), codes((E * N, K), 2).reshape(E, N, K)
    xs, ws = scales((-(-K // B), rows), 3), scales((E, -(-N // B), -(-K // B)), 4)
    live = (np.arange(max_m)[None, :] < np.array(counts)[:, None]).ravel()
    xq[~live], xs[:, ~live] = 0x7F, np.nan               # what stands in dead rows must not matter
    work = workspace(chord, rows, E)
    out = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    chord.chord_fp8_grouped_masked(cuda(xq), cuda(xs), cuda(np.array(counts, np.int32)), max(1, max(counts)), cuda(wq),
                                   cuda(ws), out, work, flag(chord, schedule))
    assert (out[torch.from_numpy(~live).cuda()] == -7).all()
    for e in range(E):
        at = np.flatnonzero(live & (np.arange(rows) // max_m == e))
        if at.size:
            check_rows(out, *ref64.product(xq[at], xs[:, at], wq[e], ws[e]), K, at)
    bad = any(c < 0 or c > max_m for c in counts)
    assert chord.chord_moe_check_status(work) == (chord.CHORD_DEV_ROUTING_INVALID if bad else 0)


CONTIGUOUS = [
    # E, N, K, blocks: (expert, valid rows at the start of the 128-row block) ; tail rows of the last block
    (3, 136, 272, [(1, 128), (1, 5), (2, 128), (0, 1)], 128),
    (2, 264, 640, [(0, 128), (0, 128), (1, 77)], 128),
    (4, 512, 256, [(3, 128), (-1, 0), (0, 64), (0, 128), (2, 3)], 40),
    (1, 72, 144, [(0, 9)], 9),
    (2, 128, 128, [(-1, 0), (-1, 0)], 128),
]


@pytest.mark.parametrize("E,N,K,blocks,tail", CONTIGUOUS)
@pytest.mark.parametrize("schedule", ["stream", "tensor", "auto"])
def test_contiguous(chord, E, N, K, blocks, tail, schedule):
    import torch
    rows = 128 * (len(blocks) - 1) + tail
    m = np.full(rows, -1, np.int32)
    rng = np.random.default_rng(rows)
    for b, (e, n) in enumerate(blocks):
        m[128 * b:128 * b + n] = e
        if e >= 0 and n == 64:                           # holes inside a block are padding too
            m[128 * b + rng.integers(0, 64, 20)] = -1
    m = m[:rows]
    live = m >= 0
    xq, wq = codes((rows, K), rows), codes((E * N, K), 2).reshape(E, N, K)
    xs, ws = scales((-(-K // B), rows), 3), scales((E, -(-N // B), -(-K // B)), 4)
    xq[~live], xs[:, ~live] = 0x7F, np.nan
    work = workspace(chord, rows, E)
    out = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    chord.chord_fp8_grouped_contiguous(cuda(xq), cuda(xs), cuda(m), cuda(wq), cuda(ws), out, work, flag(chord, schedule))
    assert (out[torch.from_numpy(~live).cuda()] == -7).all()
    for e in range(E):
        at = np.flatnonzero(m == e)
        if at.size:
            check_rows(out, *ref64.product(xq[at], xs[:, at], wq[e], ws[e]), K, at)
    assert chord.chord_moe_check_status(work) == 0


def test_contiguous_refuses_mixed_blocks(chord):
    """A block of two experts, or of an unknown one, is not computed and is reported."""
    import torch
    m = np.zeros(384, np.int32)
    m[130] = 1
    m[256:] = 9
    xq, wq = codes((384, 128), 1), codes((2 * 128, 128), 2).reshape(2, 128, 128)
    xs, ws = scales((1, 384), 3), scales((2, 1, 1), 4)
    y, a = ref64.product(xq, xs, wq[0], ws[0])
    for schedule in ("stream", "tensor"):
        work = workspace(chord, 384, 2)
        out = torch.full((384, 128), -7.0, dtype=torch.bfloat16, device="cuda")
        chord.chord_fp8_grouped_contiguous(*[cuda(v) for v in (xq, xs, m, wq, ws)], out, work, flag(chord, schedule))
        check_rows(out, y[:128], a[:128], 128, slice(0, 128))
        assert (out[128:] == -7).all()
        assert chord.chord_moe_check_status(work) == chord.CHORD_DEV_ROUTING_INVALID


# ------------------------------------------------------------------ gate_up and the MLP

def mlp_reference(xq, xs, w13, s13, w2, s2):
    """The MLP behind given codes, in 64 bits, and the intermediate before its quantisation."""
    h, _ = ref64.product(xq, xs, w13, s13)
    return ref64.silu_mul(h)


@pytest.mark.parametrize("M,H,I", [(1, 128, 128), (5, 400, 256), (16, 1024, 384), (130, 272, 128), (300, 512, 256),
                                   (1, 7168, 128), (33, 4096, 256), (70, 2048, 640), (2500, 272, 256)])
@pytest.mark.parametrize("schedule", ["stream", "tensor", "auto"])
def test_gate_up(chord, M, H, I, schedule):
    import torch
    xq, w13 = codes((M, H), M), codes((2 * I, H), 5)
    xs, s13 = scales((-(-H // B), M), 3), scales((2 * I // B, -(-H // B)), 4) * np.float32(2.0 ** -6)
    q = torch.zeros((M, I), dtype=torch.uint8, device="cuda")
    s = torch.zeros((I // B, M), device="cuda")
    work = torch.zeros(chord.chord_fp8_gate_up_workspace_bytes(M, I), dtype=torch.uint8, device="cuda")
    chord.chord_fp8_gate_up(*[cuda(v) for v in (xq, xs, w13, s13)], q, s, work, flag(chord, schedule))
    h, ha = ref64.product(xq, xs, w13, s13)
    off = ref64.product_bound(h, ha, H, False)               # of the FP32 sums
    a = ref64.silu_mul(h)
    g, u = h[:, :I], h[:, I:]
    # |silu'| <= 1.1 and |silu(g)| <= |g|; 8 FP32 roundings follow
    aoff = 1.1 * off[:, :I] * np.abs(u) + np.abs(g) * off[:, I:] + 1.1 * off[:, :I] * off[:, I:] + np.abs(a) * 8 * 2.0 ** -24
    amax = np.abs(a).reshape(M, -1, B).max(2)
    amax_off = aoff.reshape(M, -1, B).max(2)
    got_s = s.cpu().numpy().T.astype(np.float64)
    assert (np.abs(got_s - amax / 448) <= (amax_off + amax * 2.0 ** -23) / 448).all()
    # a code stands for the value within half a step: 2^-4 of it, 2^-10 near zero
    v = ref64.CODES[q.cpu().numpy()] * np.repeat(got_s, B, 1)
    step = np.maximum(np.abs(a) * 2.0 ** -4, np.repeat(got_s, B, 1) * 2.0 ** -10)
    assert (np.abs(v - a) <= step * (1 + 2.0 ** -3) + aoff * (1 + 2.0 ** -3) + 1e-37).all()
    assert chord.chord_moe_check_status(work) == 0


@pytest.mark.parametrize("T", [1, 3, 40, 200])
def test_mlp_beside_routed_experts(chord, T):
    """The block a user runs: scored routing, the W4A16 experts and the FP8 shared expert, whose
    outputs are added; the shared expert against its own codes in 64 bits."""
    import torch
    import oracle
    from w4a16_int4_mixture_align_b200 import inputs
    H, I, E, k = 256, 128, 8, 2
    rng = np.random.default_rng(T)
    d = inputs.make_inputs(inputs.CONFIGS["tiny"])
    layer = chord.ChordMoE(d["qw13"], d["s13"].view(np.int16), d["qw2"], d["s2"].view(np.int16), topk=k, max_tokens=T)
    x, x32 = bf16(rng.standard_normal((T, H)))
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    routed, ids, w = layer.forward_logits(x, logits, bias=cuda(bias), score="sigmoid", scale=2.0)
    ref_ids, ref_w = ref64.route(logits.double().cpu().numpy(), float(np.finfo(np.float32).min),
                                 bias.astype(np.float64), k, "sigmoid", 1, 1, 1, True, 2.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    want = oracle.moe_forward((x.view(torch.int16).cpu().numpy().view(np.uint16)), ref_ids,
                              ref_w.astype(np.float32), d["qw13"], d["s13"], d["qw2"], d["s2"])
    from helpers import assert_layer_close
    assert_layer_close(routed.view(torch.int16).cpu().numpy().view(np.uint16), want)

    w13, w2 = codes((2 * I, H), 5), codes((H, I), 6)
    s13, s2 = scales((2 * I // B, H // B), 7) * np.float32(0.01), scales((H // B, I // B), 8) * np.float32(0.01)
    mlp = chord.ChordFP8MLP(*[cuda(v) for v in (w13, s13, w2, s2)], max_tokens=max(1, T // 2))
    shared = mlp(x, out=torch.empty((T, H), device="cuda"))
    v, xs = ref64.quantise(x32)
    h = ref64.product(_code(ref64.e4m3_round(v.astype(np.float64))), xs, w13, s13)[0]
    a = ref64.silu_mul(h)
    # the codes of `a` differ from a by half a step each: 2^-4 of it (2^-10 of the block's
    # scale near zero), which the down product carries on; FP32 rounding is far below
    w = ref64.CODES[w2] * np.repeat(np.repeat(s2.astype(np.float64), B, 0), B, 1)[:H, :I]
    amax = np.repeat(np.abs(a).reshape(T, -1, B).max(2) / 448, B, 1)
    half = np.maximum(np.abs(a) * 2.0 ** -4, amax * 2.0 ** -10) * 1.01
    assert (np.abs(shared.double().cpu().numpy() - a @ w.T) <= half @ np.abs(w).T + 1e-30).all()
    assert mlp.check_status() == 0 and layer.check_status() == 0
    assert torch.isfinite(routed.float() + shared).all()


def _code(v):
    c = np.searchsorted(ref64.CODES[:127], np.abs(v)).astype(np.uint8)
    return np.where(np.signbit(v), c | 0x80, c).astype(np.uint8)


def test_graph_replay_on_another_stream(chord):
    """The MLP captured on a side stream, replayed on new inputs, gives the eager bits."""
    import torch
    H, I, T = 512, 256, 70
    args = [cuda(v) for v in (codes((2 * I, H), 5), scales((4, 4), 7) * np.float32(0.01), codes((H, I), 6), scales((4, 2), 8))]
    mlp = chord.ChordFP8MLP(*args, max_tokens=T)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mlp(x, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        mlp(x, out=out)
    for seed in (1, 2):
        x.copy_(torch.randn((T, H), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, mlp(x, out=out))


def test_masked_quantise_takes_expert_batches(chord):
    """[E, max_m, K] tensors as they are; a transposed code tensor is refused, not lost."""
    import torch
    x = torch.randn((3, 4, 256), device="cuda", dtype=torch.float32)
    q = torch.zeros((3, 4, 256), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2, 12), device="cuda")
    m = torch.tensor([4, 4, 4], dtype=torch.int32, device="cuda")
    chord.chord_fp8_quantize(x, q, s, masked_m=m)
    check_quantised(q.view(12, 256).cpu().numpy(), s.cpu().numpy(), x.view(12, 256).cpu().numpy())
    with pytest.raises(AssertionError):
        chord.chord_fp8_quantize(x, q.transpose(0, 1), s, masked_m=m)
    with pytest.raises(RuntimeError):
        chord.chord_fp8_quantize(x.transpose(0, 1), q, s, masked_m=m)


def test_graph_outlives_a_larger_call(chord):
    """A graph captured before the MLP's buffers grew replays on the ones it was captured with."""
    import torch
    H, I = 256, 128
    mlp = chord.ChordFP8MLP(*[cuda(v) for v in (codes((2 * I, H), 5), scales((2, 2), 7), codes((H, I), 6),
                                                scales((2, 1), 8))], max_tokens=4)
    x = torch.randn((4, H), device="cuda").to(torch.bfloat16)
    want = mlp(x).clone()
    out = torch.empty((4, H), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp(x, out=out)
    mlp(torch.randn((300, H), device="cuda").to(torch.bfloat16))
    junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del junk


def test_two_streams_at_once(chord):
    """Products with workspaces of their own on two streams give what they give alone."""
    import torch
    jobs = []
    for M, N, K, schedule in ((5, 512, 2048, "stream"), (300, 520, 1024, "tensor"), (64, 256, 4096, "auto")):
        a = [cuda(v) for v in (codes((M, K), M), scales((-(-K // B), M), 1), codes((N, K), N), scales((-(-N // B), -(-K // B)), 2))]
        w = workspace(chord, M)
        ref = torch.empty((M, N), device="cuda")
        chord.chord_fp8_gemm(*a, ref, w, flag(chord, schedule))
        jobs.append((a, ref, torch.empty_like(ref), w, flag(chord, schedule), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, _, out, w, f, s in jobs:
            with torch.cuda.stream(s):
                chord.chord_fp8_gemm(*a, out, w, f)
    torch.cuda.synchronize()
    for _, ref, out, w, _, _ in jobs:
        assert torch.equal(ref, out) and chord.chord_moe_check_status(w) == 0


def test_far_rows(chord):
    """Offsets beyond 2^31 bytes: the last rows of an activation matrix of 2.3 GB."""
    import torch
    rows, K, N = 150016, 16000, 8
    xq = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
    xs = torch.ones((-(-K // B), rows), device="cuda")
    tail = codes((16, K), 3)
    xq[-16:] = cuda(tail)
    wq, ws = codes((N, K), 4), scales((1, -(-K // B)), 5)
    y, a = ref64.product(tail, np.ones((-(-K // B), 16), np.float32), wq, ws)
    for schedule in ("stream", "tensor"):
        out = torch.full((rows, N), -7.0, device="cuda")
        chord.chord_fp8_gemm(xq, xs, cuda(wq), cuda(ws), out, workspace(chord, rows), flag(chord, schedule))
        check_rows(out, y, a, K, slice(rows - 16, rows))
        assert (out[:-16] == 0).all()


# More items than the kernels have CTAs, so that each takes several in turn: rings, buffers and
# output staging carry over from one item to the next.
@pytest.mark.parametrize("M,N,K,schedule", [(200, 13000, 400, "stream"), (16, 40008, 272, "stream"),
                                            (1100, 4104, 272, "tensor"), (6000, 4104, 400, "tensor"),
                                            (3001, 40008, 144, "tensor"), (6000, 4104, 400, "auto")])
def test_several_items_a_cta(chord, M, N, K, schedule):
    import torch
    xq, wq = codes((M, K), M), codes((N, K), N)
    xs, ws = scales((-(-K // B), M), 3), scales((-(-N // B), -(-K // B)), 4)
    args, work = [cuda(v) for v in (xq, xs, wq, ws)], workspace(chord, M)
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 60)])
    y, a = ref64.product(xq[rows], xs[:, rows], wq, ws)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        chord.chord_fp8_gemm(*args, out, work, flag(chord, schedule))
        assert torch.isfinite(out).all()
        check_rows(out[torch.from_numpy(rows).cuda()], y, a, K)
    assert chord.chord_moe_check_status(work) == 0


@pytest.mark.parametrize("layout", ["masked", "contiguous"])
@pytest.mark.parametrize("schedule", ["stream", "tensor", "auto"])
def test_many_experts(chord, layout, schedule):
    """Experts with no row, one, a few tiles and parts of them; several units a CTA."""
    import torch
    E, N, K, max_m = 40, 1032, 272, 384
    rng = np.random.default_rng(11)
    counts = rng.choice([0, 1, 77, 128, 129, 300, 384], E)
    if layout == "masked":
        m = np.where(np.arange(max_m)[None, :] < counts[:, None], np.arange(E)[:, None], -1).ravel()
    else:  # experts out of order, each padded to whole 128-row blocks
        m = np.concatenate([np.r_[np.full(counts[e], e), np.full(-counts[e] % 128, -1)] for e in rng.permutation(E)])
    m = m.astype(np.int32)
    rows = m.size
    xq, wq = codes((rows, K), rows), codes((E * N, K), 2).reshape(E, N, K)
    xs, ws = scales((-(-K // B), rows), 3), scales((E, -(-N // B), -(-K // B)), 4)
    xq[m < 0], xs[:, m < 0] = 0x7F, np.nan
    work = workspace(chord, rows, E)
    out = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    x = [cuda(xq), cuda(xs)]
    tail = [cuda(wq), cuda(ws), out, work, flag(chord, schedule)]
    if layout == "masked":
        chord.chord_fp8_grouped_masked(*x, cuda(counts.astype(np.int32)), 200, *tail)
    else:
        chord.chord_fp8_grouped_contiguous(*x, cuda(m), *tail)
    assert (out[torch.from_numpy(m < 0).cuda()] == -7).all()
    assert torch.isfinite(out).all() and chord.chord_moe_check_status(work) == 0
    for e in range(E):
        at = np.flatnonzero(m == e)
        if at.size:
            at = np.unique(np.r_[at[0], at[-1], rng.choice(at, 6)])
            check_rows(out, *ref64.product(xq[at], xs[:, at], wq[e], ws[e]), K, at)


@pytest.mark.parametrize("M,H,I,schedule", [(500, 400, 2560, "stream"), (6000, 272, 1280, "tensor")])
def test_gate_up_several_items_a_cta(chord, M, H, I, schedule):
    import torch
    xq, w13 = codes((M, H), M), codes((2 * I, H), 5)
    xs, s13 = scales((-(-H // B), M), 3), scales((2 * I // B, -(-H // B)), 4) * np.float32(2.0 ** -6)
    args = [cuda(v) for v in (xq, xs, w13, s13)]
    q = torch.zeros((M, I), dtype=torch.uint8, device="cuda")
    s = torch.zeros((I // B, M), device="cuda")
    work = torch.zeros(chord.chord_fp8_gate_up_workspace_bytes(M, I), dtype=torch.uint8, device="cuda")
    chord.chord_fp8_gate_up(*args, q, s, work, flag(chord, schedule))
    assert chord.chord_moe_check_status(work) == 0
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 60)])
    h, ha = ref64.product(xq[rows], xs[:, rows], w13, s13)
    off = ref64.product_bound(h, ha, H, False)
    a, g, u = ref64.silu_mul(h), h[:, :I], h[:, I:]
    aoff = 1.1 * off[:, :I] * np.abs(u) + np.abs(g) * off[:, I:] + 1.1 * off[:, :I] * off[:, I:] + np.abs(a) * 8 * 2.0 ** -24
    amax, amax_off = (v.reshape(rows.size, -1, B).max(2) for v in (np.abs(a), aoff))
    got_s = s.cpu().numpy().T.astype(np.float64)[rows]
    assert (np.abs(got_s - amax / 448) <= (amax_off + amax * 2.0 ** -23) / 448).all()
    v = ref64.CODES[q.cpu().numpy()[rows]] * np.repeat(got_s, B, 1)
    step = np.maximum(np.abs(a) * 2.0 ** -4, np.repeat(got_s, B, 1) * 2.0 ** -10)
    assert (np.abs(v - a) <= step * (1 + 2.0 ** -3) + aoff * (1 + 2.0 ** -3) + 1e-37).all()
    # every row was written: no block of real sums is all zero
    assert (s > 0).all() and (q != 0).any(1).all()


def test_mlps_in_a_row(chord):
    """Two layers that feed each other, twenty times without a wait between them, give the bits of
    calls made one at a time."""
    import torch
    H, I, T = 512, 256, 40
    a, b = (chord.ChordFP8MLP(*[cuda(v) for v in (codes((2 * I, H), k), scales((4, 4), k) * np.float32(0.004),
                                                  codes((H, I), k + 1), scales((4, 2), k) * np.float32(0.004))], max_tokens=T)
            for k in (5, 9))
    x0 = torch.randn((T, H), device="cuda").to(torch.bfloat16)

    def run(wait):
        x = x0
        for _ in range(10):
            for layer in (a, b):
                y = layer(x)
                # back to rows of size 1, so that the values stay in range
                x = (y.float() / y.float().abs().amax(1, keepdim=True).clamp_min(1e-30)).to(torch.bfloat16)
                if wait:
                    torch.cuda.synchronize()
        return x
    want = run(True)
    assert torch.isfinite(want).all()
    for _ in range(3):
        assert torch.equal(run(False), want)
