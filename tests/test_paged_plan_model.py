"""The paged decode kernel's plan, restated and checked on the CPU.

Every SM's block of threads computes its own range of the batch's keys from the lengths alone:
no two ranges may disagree. For random batches the segments of all ranges must cover every
64-position block of every (row, KV head) pair once, a pair's segments must lie in exactly the
ranges c0 .. c1 that its segments name (the counter that finds the last one expects c1 - c0 + 1
of them), and no two partial results may share a slot.
"""
import random
import re

import pytest

from sink_aware_sliding_head_b200.build import CSRC

BLK = 64


def row_range(p, W, cap):
    """(lo, first block, blocks) of a row with p cached tokens; no blocks: nothing to do."""
    lo = max(0, p - W + 1) if W > 0 else 0
    if not 0 <= p < cap:
        return lo, 0, 0
    return lo, lo // BLK, (p - 1) // BLK - lo // BLK + 1 if p > lo else 1


def segments(lens, Hk, W, cap, grid, cost, groups):
    """[(range, row, head, first block, blocks, pair's blocks, c0, c1)] of all ranges."""
    ns = [row_range(p, W, cap)[2] for p in lens]
    if len(lens) == 1:
        n, most = ns[0], grid // Hk
        if n == 0:
            return []
        if most > 0:
            ranges = min(most, -(-n // groups))
            share = -(-n // ranges)
            cost = -(-n // share) * share - n
        else:
            share = (cost + n) * -(-Hk // grid)
        units = (cost + n) * Hk
    else:
        units = sum(cost + n for n in ns if n) * Hk
        share = max(-(-units // grid), cost + groups)
    starts, at = [], 0                            # the first unit of each row
    for n in ns:
        starts.append(at)
        at += (cost + n) * Hk if n else 0
    out = []
    for i in range(grid):
        u, end = share * i, min(units, share * (i + 1))
        while u < end:
            b = max(x for x in range(len(ns)) if ns[x] and starts[x] <= u)
            n = ns[b]
            g, pos = divmod(u - starts[b], cost + n)
            take = min(cost + n - pos, end - u)
            blk = max(0, pos - cost)
            length = max(0, pos + take - cost) - blk
            if length > 0:
                last = u + take - 1 + (n - blk - length)
                out.append((i, b, g, blk, length, n, (last - (n - 1)) // share, last // share))
            u += take
    return out


def check(lens, Hk, W, cap, grid, cost, groups):
    seen, slots, firsts, lasts = {}, set(), set(), set()
    segs = segments(lens, Hk, W, cap, grid, cost, groups)
    for i, b, g, blk, length, n, c0, c1 in segs:
        for x in range(blk, blk + length):
            assert (b, g, x) not in seen
            seen[b, g, x] = i
        if length < n:
            slot = 2 * i + (blk == 0)
            assert slot not in slots and 0 <= slot < 2 * grid
            slots.add(slot)
            kind = lasts if blk == 0 else firsts  # a block of threads keeps one of each
            assert i not in kind
            kind.add(i)
            mine = [s for s in segs if s[1:3] == (b, g)]
            assert [s[0] for s in mine] == list(range(c0, c1 + 1))
            assert all(2 * s[0] + (s[3] == 0) == 2 * s[0] + (s[0] == c0) for s in mine)
    want = {(b, g, x) for b, p in enumerate(lens) for g in range(Hk)
            for x in range(row_range(p, W, cap)[2])}
    assert set(seen) == want


@pytest.mark.parametrize("cost,groups", [(4, 4), (8, 4), (4, 2), (8, 2)])
def test_every_block_once_and_joins_complete(cost, groups):
    rng = random.Random(cost * 10 + groups)
    for _ in range(150):
        B = rng.choice([1, 1, 2, 3, 7, 20, 60])
        top = rng.choice([1, 63, 64, 65, 300, 3000])
        lens = [rng.randint(-1, top) for _ in range(B)]
        check(lens, rng.choice([1, 2, 3, 8, 19]), rng.choice([0, 0, 1, 64, 100, 1000]),
              rng.choice([top, top + 1, 1 << 20]), rng.choice([1, 2, 7, 16, 148]), cost, groups)


def test_edges():
    check([-1, -1], 4, 0, 1000, 148, 4, 4)
    check([0], 4, 0, 1000, 148, 4, 4)
    check([9473], 3, 0, 1 << 20, 148, 4, 4)
    check([500], 40, 0, 1 << 20, 16, 8, 2)        # more heads than SMs


def test_the_kernel_has_these_costs():
    src = open(f"{CSRC}/decode_paged.cu").read()
    assert "kCost = kF8 ? 8 : 4;" in src and "constexpr int kBlk = 64;" in src
    assert re.search(r"kGroupWarps = 2 \* NG, kGroups = kMathWarps / kGroupWarps", src)
    assert "share = max(quotient(units + gridDim.x - 1, gridDim.x), " \
           "(long long)(w.cost + C::kGroups));" in src


def test_page_quotients_are_exact():
    """pos / P as the high half of pos * ceil(2^(31+s) / P), shifted by s - 1, 2^s >= P."""
    rng = random.Random(3)
    src = open(f"{CSRC}/decode_paged.cu").read()
    assert "A.page_mul = (uint32_t)(((1ull << (31 + s)) + a.c.P - 1) / a.c.P);" in src
    assert "A.page_shift = s - 1;" in src
    for P in list(range(16, 2064, 16)) + [4096, 48 * 1111, 1 << 20, (1 << 30) - 16, 1 << 30]:
        s = (P - 1).bit_length()
        mul = ((1 << (31 + s)) + P - 1) // P
        assert mul < 1 << 32
        top = (1 << 30) + 4096                    # past every position of a table
        for pos in [0, 1, P - 1, P, P + 1, top] + [rng.randrange(top) for _ in range(100)] + \
                [k * P + d for k in (1, 2, top // P) for d in (-1, 0, 1)]:
            assert ((pos * mul) >> 32) >> (s - 1) == pos // P, (P, pos)
