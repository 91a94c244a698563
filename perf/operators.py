"""Measured cases of the scored router, the FP8 block quantisation, the FP8 block-128 products and the FP8 gated MLP.

`run` computes each operator in plain torch operations (`own` false) or through the framework's entry points (`own`
true); `exact` gives the same results in 64 bits. Sizes are those of this repository's workloads (hidden 7168,
intermediate 2048, 384 experts of which 48 are local, top-8) or generic ragged ones."""
import torch

own = False

DEV = "cuda"
B = 128  # scale block


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token: sigmoid scores with a balance bias, sorted for the weight-streaming schedule
        dict(name="route one token", op="route", T=1, G=384, topk=8, E=48, block_m=8, dtype="float32", score="sigmoid",
             bias=True, n_group=1, topk_group=1, group_top=1, renorm=True, scale=2.5, pad=0),
        # a decode batch of an expert-parallel shard, experts limited to 4 of 8 groups, bf16 gate output
        dict(name="route decode groups", op="route", T=128, G=384, topk=8, E=48, block_m=8, dtype="bfloat16",
             score="sigmoid", bias=True, n_group=8, topk_group=4, group_top=2, renorm=True, scale=2.5, pad=0),
        # a prefill batch of the same shard without groups
        dict(name="route prefill", op="route", T=8192, G=384, topk=8, E=48, block_m=256, dtype="float32",
             score="sigmoid", bias=True, n_group=1, topk_group=1, group_top=1, renorm=True, scale=2.5, pad=0),
        # a ragged batch with padded rows (all logits masked): softmax scores kept as they are, 3 of 8 groups of 20
        dict(name="route padded softmax", op="route", T=2741, G=160, topk=6, E=160, block_m=64, dtype="float32",
             score="softmax", bias=False, n_group=8, topk_group=3, group_top=1, renorm=False, scale=16.0, pad=300),
        # hidden rows of a prefill batch, one row short of a round number
        dict(name="quantise prefill", op="quant", rows=8191, K=7168),
        # SiLU(gate)*up of 48 experts' decode rows in the masked layout, between the two grouped products
        dict(name="silu quantise masked", op="silu", E=48, max_m=256, I=2048, tokens=6144),
        # the smallest product: one token through a shared expert's gate and up matrix
        dict(name="product one row", op="dense", M=1, N=4096, K=7168, out="bfloat16"),
        # a small ragged projection whose last blocks are partial, kept in fp32 for a tensor-parallel sum
        dict(name="product ragged", op="dense", M=333, N=576, K=1520, out="float32"),
        # decode through 48 local experts held in FP8 (gate and up), a handful of rows each, some none
        dict(name="grouped masked decode", op="masked", E=48, max_m=64, N=4096, K=7168, tokens=384),
        # prefill through the down matrices of 48 local experts, runs padded to 128 rows
        dict(name="grouped contiguous", op="contiguous", E=48, N=7168, K=2048, tokens=8192),
        # the shared expert of a decode batch
        dict(name="mlp decode", op="mlp", T=16, H=7168, I=2048),
        # the shared expert of a prefill batch
        dict(name="mlp prefill", op="mlp", T=8192, H=7168, I=2048),
    ]


def _spread(rng, lo, hi, step=1):
    """A size from lo to hi, spread over its logarithm, a multiple of step."""
    v = lo * (hi / lo) ** rng.random()
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["route", "route", "quant", "silu", "dense", "dense", "masked", "contiguous", "mlp"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8])
        G = n_group * rng.randint(max(2, 40 // n_group), 512 // n_group)
        E = G if rng.random() < 0.4 else max(1, G // rng.choice([2, 4, 8]))
        topk_group = rng.randint((n_group + 1) // 2, n_group)
        topk = rng.randint(1, min(16, G // n_group * topk_group))
        T = _spread(rng, 1, 8192)
        score = rng.choice(["sigmoid", "softmax"])
        return dict(op="route", T=T, G=G, topk=topk, E=E, block_m=rng.choice([8, 16, 32, 64, 128, 256]),
                    dtype=rng.choice(["float32", "bfloat16", "float16"]), score=score, bias=rng.random() < 0.6,
                    n_group=n_group, topk_group=topk_group, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, T // 10]))
    if op == "quant":
        return dict(op="quant", rows=_spread(rng, 1, 8192), K=_spread(rng, 256, 7168, 16))
    if op == "silu":
        E, max_m = rng.randint(1, 48), _spread(rng, 1, 256)
        return dict(op="silu", E=E, max_m=max_m, I=_spread(rng, 256, 2048, 16), tokens=max(1, E * max_m // 2))
    if op == "dense":
        return dict(op="dense", M=_spread(rng, 1, 4096), N=_spread(rng, 128, 7168, 8), K=_spread(rng, 256, 7168, 16),
                    out=rng.choice(["bfloat16", "bfloat16", "float32"]))
    if op == "masked":
        E, max_m = rng.randint(2, 48), _spread(rng, 4, 128)
        return dict(op="masked", E=E, max_m=max_m, N=_spread(rng, 512, 4096, 8), K=_spread(rng, 256, 7168, 16),
                    tokens=max(1, E * max_m // rng.choice([2, 4])))
    if op == "contiguous":
        return dict(op="contiguous", E=rng.randint(2, 48), N=_spread(rng, 512, 7168, 8), K=_spread(rng, 256, 2048, 16),
                    tokens=_spread(rng, 64, 8192))
    return dict(op="mlp", T=_spread(rng, 1, 8192), H=_spread(rng, 512, 7168, 128), I=_spread(rng, 256, 2048, 128))


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _blocks(n):
    return (n + B - 1) // B


def _weights(E, N, K, g):
    """E4M3 codes [E, N, K] and scales [E, N/128, K/128] of N(0, 0.02) matrices, as a checkpoint holds them."""
    q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device=DEV)
    for e in range(E):
        w = torch.randn((N, K), generator=g, device=DEV) * 0.02
        p = torch.zeros((_blocks(N) * B, _blocks(K) * B), device=DEV)
        p[:N, :K] = w
        p = p.view(_blocks(N), B, _blocks(K), B)
        s[e] = p.abs().amax((1, 3)) / 448.0
        q[e] = (p / s[e][:, None, :, None]).view(_blocks(N) * B, _blocks(K) * B)[:N, :K].to(torch.float8_e4m3fn)
    return q, s


def _hidden(rows, K, g):
    """bf16 rows N(0, 1) with a size of their own each, a few large channels among them."""
    x = torch.randn((rows, K), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    x *= 1 + 9 * (torch.rand((1, K), generator=g, device=DEV) < 0.01)
    return x.to(torch.bfloat16)


def _activations(rows, K, g):
    """E4M3 codes [rows, K] and scales [K/128, rows] of such rows."""
    return _plain_quantise(_hidden(rows, K, g).float())


def _counts(case, g):
    """Rows of each expert: `tokens` drawn over the experts, none for two of them where there are many."""
    E = case["E"]
    lo = 2 if E > 4 else 0
    c = torch.bincount(torch.randint(lo, E, (case["tokens"],), generator=g, device=DEV), minlength=E)
    return c if "max_m" not in case else c.clamp(max=case["max_m"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    i32 = dict(dtype=torch.int32, device=DEV)
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    if op == "route":
        T, G, k, E, bm = (case[n] for n in ("T", "G", "topk", "E", "block_m"))
        x = torch.randn((T, G), generator=g, device=DEV).to(getattr(torch, case["dtype"]))
        if case["pad"]:
            x[T - case["pad"]:] = float("-inf")
        s["logits"] = x
        s["b"] = 0.1 * torch.randn(G, generator=g, device=DEV) if case["bias"] else None
        cap = T * k + E * (bm - 1)
        s["ids"], s["w"] = torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["sorted"], s["experts"] = torch.empty(cap, **i32), torch.empty((cap + bm - 1) // bm, **i32)
        s["ntp"], s["offsets"] = torch.empty(2, **i32), torch.empty(E + 1, **i32)
        if own:
            from w4a16_int4_mixture_align_b200 import chord
            n = chord.chord_moe_align_workspace_bytes(T, k, E)
            s["work"] = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        return s
    if op in ("quant", "silu"):
        rows, K = (case["rows"], case["K"]) if op == "quant" else (case["E"] * case["max_m"], case["I"])
        s["x"] = _hidden(rows, K if op == "quant" else 2 * K, g)
        s["counts"] = _counts(case, g).to(torch.int32) if op == "silu" else None
        s["q"] = torch.zeros((rows, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        s["scales"] = torch.zeros((_blocks(K), rows), dtype=torch.float32, device=DEV)
        return s
    if op == "mlp":
        T, H, I = (case[n] for n in ("T", "H", "I"))
        s["x"] = _hidden(T, H, g)
        s["w13"], s["s13"] = (v[0] for v in _weights(1, 2 * I, H, g))
        s["w2"], s["s2"] = (v[0] for v in _weights(1, H, I, g))
        s["y"] = torch.empty((T, H), **bf16)
        if own:
            from w4a16_int4_mixture_align_b200 import chord
            s["layer"] = chord.ChordFP8MLP(s["w13"], s["s13"], s["w2"], s["s2"], max_tokens=T)
        return s
    if op == "dense":
        rows, E = case["M"], 1
    elif op == "masked":
        rows, E = case["E"] * case["max_m"], case["E"]
        s["counts"] = _counts(case, g).to(torch.int32)
    else:
        E = case["E"]
        rows = (case["tokens"] // B + E) * B
        c = _counts(case, g)
        padded = (c + B - 1) // B * B
        start = padded.cumsum(0) - padded
        r = torch.arange(rows, device=DEV)
        e = (r[:, None] >= start[None, :]).sum(1) - 1
        s["m_indices"] = torch.where(r < start[e] + c[e], e, -1).to(torch.int32)
    s["xq"], s["xs"] = _activations(rows, case["K"], g)
    s["wq"], s["ws"] = _weights(E, case["N"], case["K"], g)
    if op == "dense":
        s["wq"], s["ws"] = s["wq"][0], s["ws"][0]
    s["y"] = torch.zeros((rows, case["N"]), dtype=getattr(torch, case.get("out", "bfloat16")), device=DEV)
    if own:
        from w4a16_int4_mixture_align_b200 import chord
        s["work"] = torch.zeros(chord.chord_fp8_workspace_bytes(rows, E), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from w4a16_int4_mixture_align_b200 import chord
    op = s["op"]
    if op == "route":
        chord.chord_router_scored_align(
            s["logits"], s["topk"], s["E"], s["block_m"], s["ids"], s["w"], s["sorted"], s["experts"], s["ntp"],
            s["offsets"], s["work"], bias=s["b"], score=s["score"], n_group=s["n_group"], topk_group=s["topk_group"],
            group_top=s["group_top"], renormalize=s["renorm"], scale=s["scale"])
        return {n: s[n] for n in ("ids", "w", "sorted", "experts", "ntp", "offsets")}
    if op == "quant":
        chord.chord_fp8_quantize(s["x"], s["q"], s["scales"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "silu":
        chord.chord_fp8_silu_quantize(s["x"], s["q"], s["scales"], masked_m=s["counts"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "mlp":
        return s["layer"](s["x"], out=s["y"])
    if op == "dense":
        chord.chord_fp8_gemm(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], s["work"])
    elif op == "masked":
        chord.chord_fp8_grouped_masked(s["xq"], s["xs"], s["counts"], max(1, s["tokens"] // s["E"]), s["wq"], s["ws"],
                                       s["y"], s["work"])
    else:
        chord.chord_fp8_grouped_contiguous(s["xq"], s["xs"], s["m_indices"], s["wq"], s["ws"], s["y"], s["work"])
    return s["y"]


def _run_plain(s):
    op = s["op"]
    if op == "route":
        return _plain_route(s)
    if op in ("quant", "silu"):
        x = s["x"].float()
        if op == "silu":
            gate, up = x.chunk(2, 1)
            x = gate / (1 + torch.exp(-gate)) * up
        q, scales = _plain_quantise(x)
        if s["counts"] is None:
            return {"q": q, "scales": scales}
        live = _live_rows(s)
        bits = torch.where(live[:, None], q.view(torch.uint8), s["q"].view(torch.uint8))
        return {"q": bits.view(torch.float8_e4m3fn), "scales": torch.where(live[None, :], scales, s["scales"])}
    if op == "mlp":
        q, scales = _plain_quantise(s["x"].float())
        gate, up = (_rows(q, scales) @ _matrix(s["w13"], s["s13"]).T).chunk(2, 1)
        q, scales = _plain_quantise(gate / (1 + torch.exp(-gate)) * up)
        return (_rows(q, scales) @ _matrix(s["w2"], s["s2"]).T).to(torch.bfloat16)
    x = _rows(s["xq"], s["xs"])
    if op == "dense":
        return (x @ _matrix(s["wq"], s["ws"]).T).to(s["y"].dtype)
    if op == "masked":
        y = torch.bmm(x.view(s["E"], s["max_m"], -1), _matrix(s["wq"], s["ws"]).transpose(1, 2)).view(s["y"].shape)
        return torch.where(_live_rows(s)[:, None], y.to(s["y"].dtype), s["y"])
    block = s["m_indices"].view(-1, B).amax(1).long().clamp(min=0)  # the expert of each 128-row block
    y = torch.bmm(x.view(block.numel(), B, -1), _matrix(s["wq"].view(torch.uint8)[block].view(torch.float8_e4m3fn), s["ws"][block]).transpose(1, 2))
    return torch.where(s["m_indices"][:, None] >= 0, y.view(s["y"].shape).to(s["y"].dtype), s["y"])


def _live_rows(s):
    return (torch.arange(s["max_m"], device=DEV)[None, :] < s["counts"][:, None]).view(-1)


def _plain_quantise(x):
    rows, K = x.shape
    p = torch.zeros((rows, _blocks(K) * B), dtype=torch.float32, device=x.device)
    p[:, :K] = x
    p = p.view(rows, _blocks(K), B)
    amax = p.abs().amax(2).clamp(min=2.0 ** -100)
    most = torch.full_like(amax, 448.0)  # a tensor: torch turns a division by or of a number into a product
    q = (p * (most / amax)[:, :, None]).view(rows, -1)[:, :K].to(torch.float8_e4m3fn).contiguous()
    return q, (amax / most).T.contiguous()


def _rows(q, scales):
    K = q.shape[1]
    return q.float() * scales.T.repeat_interleave(B, 1)[:, :K]


def _matrix(q, scales):
    N, K = q.shape[-2:]
    return q.float() * scales.repeat_interleave(B, -2)[..., :N, :].repeat_interleave(B, -1)[..., :K]


def _plain_route(s):
    T, G, k, n_group = s["T"], s["G"], s["topk"], s["n_group"]
    lowest = torch.finfo(s["logits"].dtype).min
    l = s["logits"].double()  # choices next to a border need 64 bits
    masked = ~(l > lowest)
    l = l.clamp(min=lowest, max=-lowest)
    top = torch.where(masked, -torch.inf, l).amax(1, keepdim=True).clamp(min=lowest)
    if s["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.where(masked, 0.0, torch.exp(l - top))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    c = torch.where(masked, -torch.inf, p if s["b"] is None else p + s["b"].double())
    key = torch.where(masked, -torch.inf, l) if s["b"] is None else c
    if n_group > 1:
        best = c.view(T, n_group, -1).sort(dim=2, descending=True).values[:, :, :s["group_top"]]
        score = torch.where(best > -torch.inf, best, 0.0).sum(2)
        if s["b"] is None and s["group_top"] == 1:
            score = key.view(T, n_group, -1).amax(2)
        score = torch.where(best[:, :, 0] > -torch.inf, score, -torch.inf)
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
        kept = torch.zeros((T, n_group), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(G // n_group, 1), key, -torch.inf)
    value, order = key.sort(dim=1, descending=True, stable=True)
    value, order = value[:, :k], order[:, :k]
    none = value == -torch.inf
    w = torch.where(none, 0.0, p.gather(1, order))
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    ids = torch.where(none, -1, order).to(torch.int32)
    return {"ids": ids, "w": (w * s["scale"]).float(), **_plain_sort(s, ids)}


def _plain_sort(s, ids):
    E, bm, n = s["E"], s["block_m"], ids.numel()
    cap = n + E * (bm - 1)
    flat = ids.view(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = flat.sort(stable=True).indices
    count = (flat[None, :] == torch.arange(E, device=flat.device)[:, None]).sum(1)
    padded = (count + bm - 1) // bm * bm
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    e = flat[order]
    rank = torch.arange(n, device=flat.device) - (count.cumsum(0) - count)[e.clamp(max=E - 1)]
    at = torch.where(e < E, offsets[e.clamp(max=E - 1)] + rank, cap)
    out = torch.full((cap + 1,), n, dtype=torch.int32, device=flat.device)
    out[at] = torch.where(e < E, order, n).to(torch.int32)
    row = torch.arange((cap + bm - 1) // bm, device=flat.device) * bm
    expert = (offsets[None, 1:] <= row[:, None]).sum(1)
    tag = torch.tensor([0x52540000 + bm], device=flat.device)
    return {"sorted": out[:cap], "experts": torch.where(row < offsets[E], expert, -1).to(torch.int32),
            "ntp": torch.cat([offsets[E:], tag]).to(torch.int32), "offsets": offsets.to(torch.int32)}


# ------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        T, G, k, E, bm = (case[n] for n in ("T", "G", "topk", "E", "block_m"))
        size = 4 if case["dtype"] == "float32" else 2
        cap = T * k + E * (bm - 1)
        return {"bytes": T * G * size + (4 * G if case["bias"] else 0) + T * k * 8 + 4 * (cap + cap // bm + E + 3),
                "flops": 8 * T * G}
    if op == "quant":
        rows, K = case["rows"], case["K"]
        return {"bytes": rows * (3 * K + 4 * _blocks(K)), "flops": 3 * rows * K}
    if op == "silu":
        rows, K = min(case["tokens"], case["E"] * case["max_m"]), case["I"]
        return {"bytes": rows * (5 * K + 4 * _blocks(K)) + 4 * case["E"], "flops": 8 * rows * K}

    def product(rows, E, N, K, size):
        return (E * (N * K + 4 * _blocks(N) * _blocks(K)) + rows * (K + 4 * _blocks(K)) + rows * N * size,
                2 * rows * N * K)
    if op == "mlp":
        T, H, I = (case[n] for n in ("T", "H", "I"))
        weights = 3 * H * I + 4 * 3 * _blocks(H) * _blocks(I)
        return {"bytes": weights + 4 * T * H, "flops": 6 * T * H * I}
    if op == "dense":
        n, f = product(case["M"], 1, case["N"], case["K"], 2 if case["out"] == "bfloat16" else 4)
        return {"bytes": n, "flops": f}
    E = case["E"]
    live = E - 2 if E > 4 else E
    n, f = product(case["tokens"], min(live, case["tokens"]), case["N"], case["K"], 2)
    return {"bytes": n, "flops": f}


# ------------------------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return {"w": _exact_route_weights(s)}
    if op == "quant":
        q, scales = _exact_quantise(s["x"].double())
        return {"q": q, "scales": scales}
    if op == "silu":
        I = case["I"]
        h = s["x"].double()
        q, scales = _exact_quantise(torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:])
        row = torch.arange(h.shape[0], device=DEV)
        dead = row % case["max_m"] >= s["counts"].long()[row // case["max_m"]]
        q[dead], scales[:, dead] = 0, 0
        return {"q": q, "scales": scales}
    if op == "mlp":
        I = case["I"]
        h = _exact_product(*_exact_quantise(s["x"].double()), s["w13"], s["s13"])
        a = torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:]
        return _exact_product(*_exact_quantise(a), s["w2"], s["s2"])
    if op == "dense":
        return _exact_product(s["xq"], s["xs"], s["wq"], s["ws"])
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    row = torch.arange(y.shape[0], device=DEV)
    if op == "masked":
        owner = torch.where(row % case["max_m"] < s["counts"][row // case["max_m"]], row // case["max_m"], -1)
    else:
        owner = s["m_indices"]
    for e in range(case["E"]):
        at = (owner == e).nonzero().view(-1)
        if at.numel():
            y[at] = _exact_product(s["xq"].view(torch.uint8)[at].view(torch.float8_e4m3fn), s["xs"][:, at],
                                   s["wq"][e], s["ws"][e])
    return y


def _exact_quantise(x):
    """Codes (as their values) and scales. The definition rounds x, 448 / amax and their product to fp32 before the
    code is chosen: bf16 rows often fall on the very border between two codes, and that product decides."""
    def fp32(v):
        return v.float().double()
    x = fp32(x)
    rows, K = x.shape
    q, scales = torch.empty_like(x), x.new_empty((_blocks(K), rows))
    for kb in range(_blocks(K)):
        v = x[:, kb * B:(kb + 1) * B]
        m = torch.maximum(v.abs().max(1).values, v.new_tensor(2.0 ** -100))
        scales[kb] = m / 448
        v = fp32(v * fp32(448 / m)[:, None])
        # nearest of the values with 3 mantissa bits, ties to even; below 2^-6 the step stays 2^-9
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, kb * B:(kb + 1) * B] = torch.round(v / step) * step
    return q, scales


def _exact_product(q, scales, wq, ws):
    y = torch.zeros((q.shape[0], wq.shape[0]), dtype=torch.float64, device=DEV)
    col = torch.arange(wq.shape[0], device=DEV) // B
    for kb in range(scales.shape[0]):
        part = q[:, kb * B:(kb + 1) * B].double() @ wq[:, kb * B:(kb + 1) * B].double().T
        y += part * scales[kb].double()[:, None] * ws[:, kb].double()[col][None, :]
    return y


def _exact_route_weights(s):
    """The chosen experts' weights, token by token over ranks: the best expert left at each step."""
    T, G, n_group = s["T"], s["G"], s["n_group"]
    x = s["logits"].double()
    dead = torch.isnan(x) | (x <= torch.finfo(s["logits"].dtype).min)
    x = torch.where(dead, 0.0, x)
    if s["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(torch.where(dead, -1e300, x), 1)
    choice = p + (s["b"].double() if s["b"] is not None else 0.0)
    choice = choice.masked_fill(dead, -torch.inf)
    if n_group > 1:
        group = torch.arange(G, device=DEV) // (G // n_group)
        score = []
        for i in range(n_group):
            v = choice[:, group == i].clone()
            total = torch.full((T,), -torch.inf, dtype=torch.float64, device=DEV)
            for _ in range(min(s["group_top"], v.shape[1])):
                best, at = v.max(1)
                total = torch.where(best > -torch.inf, best + total.clamp(min=-1e290) * (total > -torch.inf), total)
                v.scatter_(1, at[:, None], -torch.inf)
            score.append(total)
        score = torch.stack(score, 1)
        beaten = ((score[:, None, :] > score[:, :, None]).sum(2)
                  + ((score[:, None, :] == score[:, :, None]).tril(-1)).sum(2))
        choice = choice.masked_fill((beaten >= s["topk_group"])[:, group], -torch.inf)
    w = []
    for _ in range(s["topk"]):
        best, at = choice.max(1)
        w.append(torch.where(best > -torch.inf, p.gather(1, at[:, None])[:, 0], 0.0))
        choice = choice.scatter(1, at[:, None], -torch.inf)
    w = torch.stack(w, 1)
    if s["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return w * s["scale"]
