"""The load ring of the paged decode kernel, restated and run on the CPU.

Blocks of keys stream through S shared-memory stages; four groups of two math warps (two of
four over more than 8 heads) take the blocks in turn (block n: stage n % S, group n % 4). A stage has a "full" barrier (the
loading warp arrives, and the copies complete their bytes) and an "empty" one (the group's
warps arrive). Copies land in any order. mbarrier waits test a phase's parity only, so a wait
that is two phases behind passes at once: when S is no multiple of the groups, a stage changes
hands between them, a group does not see every phase of it, and a copy that lands late lets
another group read a stage before its own copy is there. Otherwise each stage belongs to one
group.
"""
import random
import re

import pytest

from sink_aware_sliding_head_b200.build import CSRC

GROUPS, GROUP_WARPS = 4, 2


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


def run(stages, units, seed):
    """True if every block is read after its own copy landed and every role ends."""
    rng = random.Random(seed)
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(GROUP_WARPS) for _ in range(stages)]
    holds = [None] * stages                       # the block whose bytes are in the stage
    flying, issued = [], 0
    warps = [(g, w) for g in range(GROUPS) for w in range(GROUP_WARPS)]
    at = {x: x[0] for x in warps}
    slow = rng.random()
    for _ in range(400 * units + 4000):
        if issued == units and not flying and all(n >= units for n in at.values()):
            return True
        role = rng.randrange(4)
        if role == 0 and issued < units:
            n, s = issued, issued % stages
            if n < stages or empty[s].passed((n // stages - 1) & 1):
                full[s].arrive(tx=1)
                flying.append(n)
                issued += 1
        elif role == 1 and flying and rng.random() > slow:
            n = flying.pop(rng.randrange(len(flying)))
            holds[n % stages] = n
            full[n % stages].complete(1)
        elif role >= 2:
            x = rng.choice(warps)
            n = at[x]
            if n < units and full[n % stages].passed((n // stages) & 1):
                if holds[n % stages] != n:
                    return False
                empty[n % stages].arrive()
                at[x] = n + GROUPS
    return False


def test_rings_of_whole_turns_keep_their_order():
    for stages in (4, 8, 12):
        for seed in range(60):
            assert run(stages, 5 * stages + seed % 7, seed), (stages, seed)


@pytest.mark.parametrize("stages", [5, 6])
def test_other_rings_are_caught(stages):
    def ends_badly(seed):
        try:
            return not run(stages, 40, seed)
        except AssertionError:
            return True
    assert any(ends_badly(seed) for seed in range(60))


def test_the_kernel_uses_such_rings():
    src = open(f"{CSRC}/decode_paged.cu").read()
    m = re.search(r"kStages = kF8 \? (\d+) : (\d+);", src)
    assert m, "the ring sizes moved: adapt this test"
    assert all(int(s) % GROUPS == 0 for s in m.groups())
    assert "static_assert(kStages % kGroups == 0" in src
    assert "kGroupWarps = 2 * NG, kGroups = kMathWarps / kGroupWarps" in src
    assert "constexpr int kMathWarps = 8;" in src and "constexpr int kLoadWarps = 4;" in src
