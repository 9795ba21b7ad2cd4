"""The bounds of paged_precision.py tell operands in two 16-bit parts from operands in one: the
kernel's roundings, emulated on the CPU, with parts left out on purpose."""
import numpy as np
import pytest
import torch

import paged_precision as pp
from paged_util import Paged, to64

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16
PART = {E4M3: torch.float16, BF16: BF16}          # the products' operand type over each cache


def emulate(dtype, q_parts, p_parts, small=1.0, lift=1.0):
    """(rms of the LSE's error, of the output's) / bound, with that many parts of q and P."""
    lens = np.random.RandomState(5).randint(0, 130, 16).tolist()
    w = Paged(lens, H=16, Hk=2, P=16, dtype=dtype, seed=61)
    got, want = [], []
    for b in range(len(lens)):
        q, K, V = pp.operands(w, b, 0, w.kp, w.vp)
        q, K = q * small, K / small
        a = q, K, V, to64(w.sink), 128 ** -0.5
        want.append(pp.attend(*a))
        got.append(pp.attend(*a, q_parts=pp.in_parts(PART[dtype], q_parts, lift),
                             p_parts=pp.in_parts(PART[dtype], p_parts, 64.0)))
    return [x / y for x, y in zip(pp.off_by(got, want), pp.BOUND[dtype])]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_two_parts_pass_and_one_part_of_either_fails(dtype):
    assert max(emulate(dtype, 2, 2)) < 0.5
    lse, out = emulate(dtype, 1, 2)
    assert lse > 4 and out > 4
    lse, out = emulate(dtype, 2, 1)
    assert lse < 0.5 and out > 4


@pytest.mark.parametrize("small", [2.0 ** -10, 2.0 ** -20])
def test_small_q_in_fp16_fails_unless_lifted(small):
    """fp16 parts of a q that is small (against large key scales): steps of 2^-24 at the least.
    Unlifted, what is rounded is q in log2 units."""
    assert emulate(E4M3, 2, 2, small, 128 ** -0.5 * np.log2(np.e))[0] > 4
    lift = 2.0 ** (11 - np.floor(np.log2(small)))
    assert max(emulate(E4M3, 2, 2, small, lift)) < 0.5
