"""The barrier protocol of the FP8 tile kernel, by exhaustive search on the CPU: whatever the order
in which copies land, no block is multiplied before it is in shared memory.

A ring of S stages is filled in order, copies land in any order, two issuers multiply the even and
the odd blocks into B buffers, the adding warps empty the buffers in order. A wait on an mbarrier
for the end of phase n looks at the phase's parity only, so it also passes while phase n - 1 is
still open."""
import os
import re

import pytest

from helpers import ROOT

TILE = os.path.join(ROOT, "w4a16_int4_mixture_align_b200", "csrc", "fp8_tile.cu")


def first_fault(S, B, blocks, buffer_first):
    """A reachable state (blocks loaded, landed, multiplied, added) in which an issuer multiplies a
    block that has not landed or into a buffer not yet read; None if there is none."""
    def passed(completed, n):
        return completed % 2 != n % 2

    def phases(done, s):  # completions of stage s's barrier after the blocks in `done`
        return sum(1 for i in range(s, blocks, S) if done >> i & 1)

    start = (0, 0, 0, 0, (0, 0), (1, 0))  # loads issued, landed, multiplied, added, issuers (block, waits behind it)
    seen, todo = {start}, [start]
    while todo:
        loaded, landed, mul, added, *issuers = state = todo.pop()
        nxt = []
        if loaded < blocks and (loaded < S or passed(phases(mul, loaded % S), loaded // S - 1)):
            nxt.append((loaded + 1, landed, mul, added, *issuers))
        for i in range(loaded):
            if not landed >> i & 1:
                nxt.append((loaded, landed | 1 << i, mul, added, *issuers))
        if added < blocks and passed(phases(mul, added % S), added // S):
            if not mul >> added & 1:
                return state
            nxt.append((loaded, landed, mul, added + 1, *issuers))
        for w in (0, 1):
            it, waits = issuers[w]
            if it >= blocks:
                continue
            full = passed(phases(landed, it % S), it // S)
            emptied = sum(1 for i in range(it % B, added, B))
            free = it < B or passed(emptied, it // B - 1)
            if (free, full)[waits if buffer_first else 1 - waits]:
                after = list(issuers)
                if waits == 0:
                    after[w] = (it, 1)
                    nxt.append((loaded, landed, mul, added, *after))
                else:
                    if not landed >> it & 1 or (it >= B and added <= it - B):
                        return state
                    after[w] = (it + 2, 0)
                    nxt.append((loaded, landed, mul | 1 << it, added, *after))
        for n in nxt:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return None


@pytest.mark.parametrize("S,B", [(2, 2), (3, 2), (5, 2), (6, 2), (4, 4), (5, 4), (6, 4), (7, 4)])
def test_buffer_first_is_safe(S, B):
    assert first_fault(S, B, S + 4, True) is None


def test_stage_first_is_not():
    """The search sees the fault of the other order in a ring of five stages and four buffers."""
    assert first_fault(5, 4, 9, False) is not None


def test_the_kernel_waits_for_its_buffer_first():
    text = open(TILE).read()
    loop = re.search(r"for \(; it < blocks; it \+= 2\) \{(.*?)commit<CG>", text, re.S).group(1)
    assert loop.index("acc_empty[b]") < loop.index("full[s]")
