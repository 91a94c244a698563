"""64-bit references of the scored router and the FP8 block-128 operators, in numpy, from
their definitions (no code shared with the library)."""
import numpy as np

BLOCK = 128


# ------------------------------------------------------------------ router

def route(logits, lowest, bias, topk, score, n_group, topk_group, group_top, renormalize, scale):
    """ids int32 [T, topk], weights float64 [T, topk]. `logits` float64 values of a type whose
    lowest finite value is `lowest`."""
    T, G = logits.shape
    ids = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    size = G // n_group
    for t in range(T):
        l = logits[t]
        alive = l > lowest                       # NaN compares false
        l = np.where(alive, np.minimum(l, -lowest), 0.0)
        with np.errstate(over="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                m = l[alive].max() if alive.any() else 0.0
                s = np.where(alive, np.exp(np.where(alive, l - m, 0.0)), 0.0)
                s = s / (s.sum() if s.sum() > 0 else 1.0)
        c = s + (bias if bias is not None else 0.0)
        key = c if bias is not None else l       # the same order, without rounding
        experts = [e for e in range(G) if alive[e]]
        if n_group > 1:
            value = []
            for g in range(n_group):
                of = sorted((e for e in experts if e // size == g), key=lambda e: (-key[e], e))[:group_top]
                if bias is None and group_top == 1:
                    value.append(key[of[0]] if of else -np.inf)
                else:
                    value.append(sum(c[e] for e in of) if of else -np.inf)
            keep = sorted((g for g in range(n_group) if value[g] > -np.inf), key=lambda g: (-value[g], g))[:topk_group]
            experts = [e for e in experts if e // size in keep]
        chosen = sorted(experts, key=lambda e: (-key[e], e))[:topk]
        w = np.array([s[e] for e in chosen])
        if renormalize and len(chosen):
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    return ids, weights


# ------------------------------------------------------------------ E4M3

def e4m3_values():
    """The 256 code values (NaN for 0x7f and 0xff)."""
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (e == 15 and m == 7) else (-x if s else x)
    return v


CODES = e4m3_values()


def e4m3_round(x):
    """Nearest E4M3 value (as float64), ties to the even code, saturating at 448."""
    pos = CODES[:127]                             # 0 .. 448, increasing
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(np.where(take_hi, pos[hi], pos[lo]), x)


def border_distance(x):
    """Relative distance of |x| (<= 448) to the nearest border between two E4M3 values."""
    pos = CODES[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    a = np.abs(x)
    i = np.clip(np.searchsorted(mid, a), 1, len(mid) - 1)
    return np.minimum(np.abs(a - mid[i]), np.abs(a - mid[i - 1])) / np.maximum(a, 1e-300)


def quantise(x):
    """(values before rounding, scales [blocks, rows]) of fp32 rows x, every operation rounded
    to fp32."""
    rows, K = x.shape
    kb = -(-K // BLOCK)
    p = np.zeros((rows, kb * BLOCK), np.float32)
    p[:, :K] = x
    p = p.reshape(rows, kb, BLOCK)
    amax = np.maximum(np.abs(p).max(2), np.float32(2.0 ** -100))
    r = (np.float32(448) / amax).astype(np.float32)
    v = (p * r[:, :, None]).astype(np.float32).reshape(rows, -1)[:, :K]
    return v, np.ascontiguousarray((amax / np.float32(448)).astype(np.float32).T)


def silu_mul(h):
    I = h.shape[1] // 2
    g = h[:, :I].astype(np.float64)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * h[:, I:]


# ------------------------------------------------------------------ products

def product(xq, xs, wq, ws):
    """(result, sum of absolute terms), float64 [rows, N], from codes (uint8) and scales."""
    x, w = CODES[xq], CODES[wq]
    rows, K = x.shape
    y = np.zeros((rows, w.shape[0]))
    a = np.zeros_like(y)
    col = np.arange(w.shape[0]) // BLOCK
    for kb in range(-(-K // BLOCK)):
        k = slice(kb * BLOCK, (kb + 1) * BLOCK)
        f = xs[kb].astype(np.float64)[:, None] * ws[:, kb].astype(np.float64)[col][None, :]
        y += (x[:, k] @ w[:, k].T) * f
        a += (np.abs(x[:, k]) @ np.abs(w[:, k]).T) * np.abs(f)
    return y, a


def product_bound(y, a, K, bf16):
    """How far FP32 sums may be off: a block's products are added in at most 4 steps of the
    tensor core (each rounding the running sum by at most 2^-23 of the terms' size), the
    ceil(K/128) blocks in as many FP32 operations of two roundings (the scale, the fused
    multiply-add), and the parts of a split K in at most 8 more; then bf16 rounds by half a step, 2^-8."""
    steps = 4 + 2 * (-(-K // BLOCK)) + 8
    return a * steps * 2.0 ** -23 + (np.abs(y) * 2.0 ** -8 if bf16 else 0.0) + 1e-37
