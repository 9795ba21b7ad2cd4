"""The load ring of the paged decode kernel, restated and run on the CPU.

Blocks of keys stream through S shared-memory stages. Block u goes to stage u % S, is loaded by
warp u % L and multiplied by the warps of group u % G. It has the barriers u % B: "full" (the
loading warp arrives, and the copies complete their bytes) and "empty" (the group's warps
arrive). Copies land in any order. mbarrier waits test a phase's parity only, so a wait that is
two phases behind passes at once. With B a multiple of S, G and L every barrier belongs to one
group and one loading warp, which see each of its phases. With a barrier per stage and S no
multiple of G, a copy that lands late lets another group read a stage before its own copy is
there.
"""
import math
import random
import re

import pytest

from sink_aware_sliding_head_b200.build import CSRC

MATH_WARPS, LOAD_WARPS = 8, 2


class Barrier:
    """An mbarrier: phases complete when the expected arrivals and bytes are in."""

    def __init__(self, count):
        self.count = self.pending = count
        self.phase, self.tx = 0, 0

    def _step(self):
        assert self.pending >= 0, "more arrivals than the phase expects"
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        self._step()

    def complete(self, tx):
        self.tx -= tx
        self._step()

    def passed(self, parity):
        """What a parity wait sees: the running phase has the other parity."""
        return (self.phase & 1) != parity


def run(stages, bars, group_warps, units, seed):
    """True if every block is read after its own copy landed, no stage is overwritten while it
    is read, and every role ends."""
    rng = random.Random(seed)
    groups = MATH_WARPS // group_warps
    full = [Barrier(1) for _ in range(bars)]
    empty = [Barrier(group_warps) for _ in range(bars)]
    holds = [None] * stages                       # the block whose bytes are in the stage
    flying = []
    load_at = list(range(LOAD_WARPS))
    warps = [(g, w) for g in range(groups) for w in range(group_warps)]
    at = {x: x[0] for x in warps}
    slow = rng.random()
    for _ in range(600 * units + 6000):
        if not flying and min(load_at) >= units and all(u >= units for u in at.values()):
            return True
        role = rng.randrange(4)
        if role == 0:
            w = rng.randrange(LOAD_WARPS)
            u, d = load_at[w], load_at[w] - stages
            if u < units and (d < 0 or empty[d % bars].passed((d // bars) & 1)):
                if d >= 0 and any(n <= d for x, n in at.items() if x[0] == d % groups):
                    return False                  # block d is still being read
                full[u % bars].arrive(tx=1)
                flying.append(u)
                load_at[w] = u + LOAD_WARPS
        elif role == 1 and flying and rng.random() > slow:
            u = flying.pop(rng.randrange(len(flying)))
            holds[u % stages] = u
            full[u % bars].complete(1)
        elif role >= 2:
            x = rng.choice(warps)
            u = at[x]
            if u < units and full[u % bars].passed((u // bars) & 1):
                if holds[u % stages] != u:
                    return False
                empty[u % bars].arrive()
                at[x] = u + groups
    return False


def ends_badly(stages, bars, seed):
    try:
        return not run(stages, bars, 2, 60, seed)
    except AssertionError:
        return True


def kernel_rings():
    """(stages, barriers, warps of a group) of the kernel's four variants."""
    src = open(f"{CSRC}/decode_paged.cu").read()
    m = re.search(r"kStages = \(NG == 1 \? (\d+) : (\d+)\) \* \(kF8 \? (\d+) : 1\)", src)
    b = re.search(r"kBars = NG == 1 \? (\d+) : (\d+);", src)
    assert m and b, "the ring sizes moved: adapt this test"
    assert "kGroupWarps = 2 * NG, kGroups = kMathWarps / kGroupWarps" in src
    assert f"constexpr int kMathWarps = {MATH_WARPS};" in src
    assert f"constexpr int kLoadWarps = {LOAD_WARPS};" in src
    one, two, f8 = map(int, m.groups())
    return [(s * f, int(b.group(ng)), 2 * ng) for ng, s in ((1, one), (2, two)) for f in (1, f8)]


def test_the_kernels_rings_keep_their_order():
    for stages, bars, group_warps in kernel_rings():
        groups = MATH_WARPS // group_warps
        assert bars % math.lcm(stages, groups, LOAD_WARPS) == 0
        for seed in range(60):
            assert run(stages, bars, group_warps, 5 * stages + seed % 7, seed), (stages, seed)


@pytest.mark.parametrize("stages", [5, 6, 10])
def test_a_barrier_per_stage_is_caught(stages):
    assert any(ends_badly(stages, stages, seed) for seed in range(80))
