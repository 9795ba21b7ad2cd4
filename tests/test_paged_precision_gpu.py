"""The precision of flint_attn_decode_paged with a float32 output, by root mean squares over
many rows and heads: the probabilities and q keep two 16-bit parts over both cache types."""
import numpy as np
import pytest
import torch

import paged_precision as pp
from paged_util import Paged, decode

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("H,Hk,W,rope", [(32, 4, 0, True), (18, 2, 40, True), (16, 1, 0, False)])
def test_output_and_lse_keep_two_parts_of_each_operand(cuda_lib, H, Hk, W, rope, dtype):
    lens = np.random.RandomState(H).randint(0, 130, 40).tolist()
    w = Paged(lens, H=H, Hk=Hk, P=16, dtype=dtype, rope=rope, seed=60)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, W, fp32_out=True)
    pp.check(w, out, lse, d["kp"], d["vp"], W)
