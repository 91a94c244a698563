"""Host-side checks of the scored router's and the FP8 operators' arguments: each refusal is
returned before any device access."""
import ctypes

import pytest

from helpers import ensure_built


@pytest.fixture(scope="module")
def chord():
    ensure_built()
    from w4a16_int4_mixture_align_b200 import chord as c
    return c


P = ctypes.c_void_p(0x100000)       # an aligned address that nothing reads
ODD = ctypes.c_void_p(0x100004)
BIG = 1 << 30


def router(chord, **kw):
    a = dict(logits=P, dtype=0, ld=64, bias=None, T=16, G=64, topk=4, E=8, bm=8, score=1, ng=1, tg=1, gt=1, renorm=1,
             scale=1.0, ids=P, w=P, s=P, e=P, n=P, o=None, ws=None, wsb=0)
    a.update(kw)
    return chord.lib().chord_router_scored_align(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), "INVALID_ARG"), (dict(topk=0), "INVALID_ARG"), (dict(topk=65), "INVALID_ARG"),
    (dict(G=1025, ld=1025), "UNSUPPORTED"), (dict(G=3, ld=3), "UNSUPPORTED"), (dict(E=0), "UNSUPPORTED"),
    (dict(bm=0), "UNSUPPORTED"), (dict(bm=257), "UNSUPPORTED"), (dict(dtype=3), "UNSUPPORTED"),
    (dict(dtype=-1), "UNSUPPORTED"), (dict(score=2), "UNSUPPORTED"), (dict(ng=0), "UNSUPPORTED"),
    (dict(ng=33), "UNSUPPORTED"), (dict(ng=5), "UNSUPPORTED"), (dict(ng=8, tg=0), "INVALID_ARG"),
    (dict(ng=8, tg=9), "INVALID_ARG"), (dict(ng=8, tg=4, gt=0), "INVALID_ARG"),
    (dict(ng=8, tg=4, gt=3), "INVALID_ARG"), (dict(ng=32, tg=1), "INVALID_ARG"),  # 4 of 2 experts
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(ld=63), "INVALID_ARG"), (dict(logits=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"),
    (dict(w=None), "INVALID_ARG"), (dict(s=None), "INVALID_ARG"), (dict(n=None), "INVALID_ARG"),
    (dict(T=4096), "WORKSPACE_TOO_SMALL"), (dict(T=4096, ws=ODD, wsb=BIG), "INVALID_ARG"),
    (dict(T=1 << 40), "UNSUPPORTED"),
])
def test_router_refusals(chord, bad, status):
    assert router(chord, **bad) == getattr(chord, "CHORD_ERR_" + status), chord.chord_last_error_detail()
    assert chord.chord_last_error_detail()


def quantise(chord, name="chord_fp8_quantize", **kw):
    a = dict(x=P, dtype=1, ld=256, rows=16, K=256, m=None, E=0, q=P, s=P)
    if "silu" in name:
        a["ld"] = 512
    a.update(kw)
    return getattr(chord.lib(), name)(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(K=0), "UNSUPPORTED"), (dict(K=24), "UNSUPPORTED"), (dict(K=-16), "UNSUPPORTED"),
    (dict(rows=-1), "INVALID_ARG"), (dict(rows=1 << 31), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"),
    (dict(ld=240), "INVALID_ARG"), (dict(ld=1001), "INVALID_ARG"), (dict(x=ODD), "INVALID_ARG"),
    (dict(q=ODD), "INVALID_ARG"), (dict(s=ctypes.c_void_p(0x100002)), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(s=None), "INVALID_ARG"), (dict(E=4), "INVALID_ARG"),
    (dict(m=P, E=0), "INVALID_ARG"), (dict(m=P, E=3), "INVALID_ARG"), (dict(m=P, E=2000), "INVALID_ARG"),
])
@pytest.mark.parametrize("name", ["chord_fp8_quantize", "chord_fp8_silu_quantize"])
def test_quantise_refusals(chord, name, bad, status):
    assert quantise(chord, name, **bad) == getattr(chord, "CHORD_ERR_" + status), chord.chord_last_error_detail()


def dense(chord, **kw):
    a = dict(xq=P, xs=P, M=16, K=256, w=P, ws=P, N=128, out=P, work=P, have=BIG, flags=0)
    a.update(kw)
    return chord.lib().chord_fp8_gemm(*a.values(), None)


def contiguous(chord, **kw):
    a = dict(xq=P, xs=P, M=256, K=256, m=P, w=P, ws=P, E=4, N=128, out=P, work=P, have=BIG, flags=0)
    a.update(kw)
    return chord.lib().chord_fp8_grouped_contiguous(*a.values(), None)


def masked(chord, **kw):
    a = dict(xq=P, xs=P, E=4, max_m=16, K=256, m=P, expected=4, w=P, ws=P, N=128, out=P, work=P, have=BIG, flags=0)
    a.update(kw)
    return chord.lib().chord_fp8_grouped_masked(*a.values(), None)


def gate_up(chord, **kw):
    a = dict(xq=P, xs=P, M=16, K=256, w=P, ws=P, I=128, out=P, s=P, work=P, have=BIG, flags=0)
    a.update(kw)
    return chord.lib().chord_fp8_gate_up(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(K=0), "UNSUPPORTED"), (dict(K=24), "UNSUPPORTED"), (dict(xq=ODD), "INVALID_ARG"),
    (dict(w=ODD), "INVALID_ARG"), (dict(out=ODD), "INVALID_ARG"), (dict(xs=ctypes.c_void_p(0x100002)), "INVALID_ARG"),
    (dict(xq=None), "INVALID_ARG"), (dict(xs=None), "INVALID_ARG"), (dict(w=None), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(work=None), "INVALID_ARG"),
    (dict(work=ODD), "INVALID_ARG"), (dict(have=1024), "WORKSPACE_TOO_SMALL"), (dict(flags=6), "INVALID_ARG"),
    (dict(flags=1), "INVALID_ARG"), (dict(flags=16), "INVALID_ARG"),
])
@pytest.mark.parametrize("call", [dense, contiguous, masked, gate_up])
def test_product_refusals(chord, call, bad, status):
    assert call(chord, **bad) == getattr(chord, "CHORD_ERR_" + status), chord.chord_last_error_detail()


def test_refusals_of_single_products(chord):
    inv, uns = chord.CHORD_ERR_INVALID_ARG, chord.CHORD_ERR_UNSUPPORTED
    assert dense(chord, M=-1) == inv and dense(chord, M=1 << 31) == uns and dense(chord, N=12) == uns
    assert contiguous(chord, M=-1) == inv and contiguous(chord, E=0) == uns and contiguous(chord, E=1025) == uns
    assert contiguous(chord, m=None) == inv and contiguous(chord, m=ODD) == inv
    assert masked(chord, m=None) == inv and masked(chord, max_m=0) == inv and masked(chord, expected=0) == inv
    assert masked(chord, max_m=1 << 62) == uns and masked(chord, E=0) == uns
    assert gate_up(chord, I=64) == uns and gate_up(chord, I=192) == uns and gate_up(chord, s=None) == inv
    assert gate_up(chord, flags=8) == inv and gate_up(chord, M=-1) == inv
    assert gate_up(chord, s=ctypes.c_void_p(0x100002)) == inv


def test_workspace_sizes(chord):
    assert chord.chord_fp8_workspace_bytes(-1, 1) == 0 and chord.chord_fp8_workspace_bytes(1, 0) == 0
    assert chord.chord_fp8_workspace_bytes(0, 1) >= 65536
    assert chord.chord_fp8_gate_up_workspace_bytes(-1, 128) == 0 and chord.chord_fp8_gate_up_workspace_bytes(1, 0) == 0
    assert chord.chord_fp8_gate_up_workspace_bytes(16, 128) >= chord.chord_fp8_workspace_bytes(16, 1)


def test_binding_checks(chord):
    """The binding refuses wrong types and shapes before the library is called."""
    import torch
    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        chord.chord_router_scored_align(cpu, 4, 8, 8, cpu, cpu, cpu, cpu, cpu, score="max")
    with pytest.raises(AssertionError):
        chord.chord_router_scored_align(cpu.double(), 4, 8, 8, cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(AssertionError):
        chord.chord_fp8_quantize(cpu, cpu, cpu)
    with pytest.raises(AssertionError):
        chord.chord_fp8_gemm(cpu, cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError):
        chord.ChordFP8MLP(torch.zeros((256, 128)), cpu, torch.zeros((256, 128)), cpu)
