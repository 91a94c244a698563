"""GPU scored router where the FP32 softmax denominator is furthest off: one large logit in a lane
whose 31 others are each lost in the addition."""
import numpy as np
import pytest

from test_gpu_router_scored import check, chord  # noqa: F401

pytestmark = pytest.mark.gpu


def off_by(logits):
    """The kernel's FP32 sum of exponentials (lane l: experts l, l + 32, ...) against the exact one."""
    e = np.exp((logits - logits.max()).astype(np.float64)).astype(np.float32)
    z = np.zeros(32, np.float32)
    for i in range(0, logits.size, 32):
        z = z + e[i:i + 32]
    for o in (16, 8, 4, 2, 1):
        z = z + z[np.arange(32) ^ o]
    return abs(float(z[0]) / e.astype(np.float64).sum() - 1)


@pytest.mark.parametrize("topk", [1, 4, 8])
def test_denominator_far_off(chord, topk):  # noqa: F811
    """Sixteen experts whose choice scores lie 2e-7 apart around the one that the denominator's error
    moves by 1.7e-6; every other lane's best is far below."""
    import torch
    G, T = 1024, 40
    rng = np.random.default_rng(topk)
    logits = np.full((T, G), -16.7, np.float32)
    bias = np.full(G, -1.0, np.float32)
    top = 5
    near = np.array([l + 32 * rng.integers(1, 32) for l in rng.permutation(32)[:16]])
    near = near[near % 32 != top % 32][:15]
    logits[:, top] = 0.0
    p = np.exp(np.float64(logits[0]))
    p /= p.sum()
    assert off_by(logits[0]) > 1.5e-6
    # biases are FP32: near experts at 0.01 + steps, the top one at the middle of them
    bias[near] = (0.01 + 2e-7 * rng.permutation(near.size)).astype(np.float32)
    bias[top] = np.float32(0.01 + 2e-7 * near.size / 2 - p[top])
    for t in range(T):   # each token's large logit a little different, so that the order changes
        logits[t, top] = rng.integers(-2, 3) * np.float32(2.0 ** -9)
    check(chord, torch.from_numpy(logits).cuda(), bias, topk, G, 8, "softmax")
    check(chord, torch.from_numpy(logits).cuda(), bias, topk, G, 8, "softmax", 8, 4, 2)
