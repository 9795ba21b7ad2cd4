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


@pytest.mark.parametrize("softmax_scale", [False, True])
@pytest.mark.parametrize("power", [-20, -10, 8, 20])
def test_q_of_any_size_over_e4m3(cuda_lib, power, softmax_scale):
    """Norm weights (or a softmax scale) and key scales whose powers of two cancel: the scores
    are of the usual size, q is not."""
    lens = np.random.RandomState(7).randint(0, 130, 40).tolist()
    w = Paged(lens, H=16, Hk=2, P=16, dtype=E4M3, seed=62)
    w.k_scale = w.k_scale * 2.0 ** -power
    w.wk = w.wk * 2.0 ** -power
    scale = 128 ** -0.5
    if softmax_scale:
        scale = scale * 2.0 ** power
    else:
        w.wq = w.wq * 2.0 ** power
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True, softmax_scale=scale)
    pp.check(w, out, lse, d["kp"], d["vp"], 0, scale)


def test_weights_of_q_that_differ_by_channel(cuda_lib):
    """q's small channels meet large keys, over e4m3."""
    w = Paged([0, 9, 65, 100] * 10, H=16, Hk=2, P=16, dtype=E4M3, rope=False, seed=63)
    ramp = 2.0 ** -torch.arange(128).remainder(8).float()      # 1 to 2^-7
    w.wq = (w.wq.float() * ramp).to(BF16)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    pp.check(w, out, lse, d["kp"], d["vp"], 0)


def test_zero_weights_of_q(cuda_lib):
    """All scores are zero: nothing to lift, the weights are equal."""
    w = Paged([0, 1, 70], H=8, Hk=2, P=16, dtype=E4M3, seed=64)
    w.wq = torch.zeros_like(w.wq)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    pp.check(w, out, lse, d["kp"], d["vp"], 0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_long_sums_are_not_cut_off(cuda_lib, dtype):
    """Values around one, 30000 keys in one range of keys: the errors of single keys average out,
    what is left is what the long sums do. A matrix product's sums are cut off toward zero, some
    2^-24.5 a step, and a running output would be cut in each of its ~470 steps here (2^-15.7).

    Bound: 2^-17 of each weight (bf16 parts) over 30000 keys of like weights, sqrt(30000) =
    2^7.4: 2^-24. The roundings in 32 bits that all keys share or that have one sign, twenty of
    2^-23 at the most: below 2^-18."""
    Hk, p, P = 148, 30000, 64                     # one row, a range for each of its KV heads
    n = -(-(p + 1) // P)
    gen = torch.Generator(device="cuda").manual_seed(65)
    kp, vp = (torch.empty(n, Hk, P, 128, dtype=dtype, device="cuda") for _ in "kv")
    for at in range(0, n, 64):
        shape = kp[at:at + 64].shape
        kp[at:at + 64] = torch.randn(shape, generator=gen, device="cuda").to(dtype)
        vp[at:at + 64] = (1 + 0.2 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)
    table = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)[None]
    w = Paged([0], H=Hk, Hk=Hk, P=16, rope=False, seed=66)
    d = w.dev()
    lens = torch.tensor([p], dtype=torch.int32, device="cuda")
    d["v"] = torch.ones_like(d["v"])
    out, _ = cuda_lib.decode_paged(d["q"], d["k"], d["v"], d["wq"], d["wk"], d["sink"], lens,
                                   table, kp, vp, 0, False, 1e6, check_status=True, fp32_out=True)
    w.lens = [p]
    q = torch.as_tensor(pp.fo.prologue(w.q.double().numpy(), w.wq.double().numpy(),
                                       np.array([p]), False, 1e6, 1e-6)[0]).cuda()
    errors = []
    for h in range(Hk):
        K, V = (x[table[0].long(), h].reshape(-1, 128)[:p + 1].double() for x in (kp, vp))
        z = torch.cat([K @ q[h] * 128 ** -0.5, d["sink"][h:h + 1].double()])
        e = torch.softmax(z, 0)[:-1]
        errors.append((out[0, h].double() - e @ V) / (e @ V.abs()))
    assert pp.rms(torch.stack(errors).cpu().numpy()) <= 2.0 ** -18


@pytest.mark.parametrize("power", [-112, 112])
def test_key_scales_near_the_ends_of_float32(cuda_lib, power):
    """Neither the cached keys' scores nor the new one's pass through a product that is larger
    or smaller than float32 holds."""
    w = Paged([0, 0, 9, 65, 100] * 6, H=16, Hk=2, P=16, dtype=E4M3, seed=67)
    w.k_scale = w.k_scale * 2.0 ** -power
    w.wk = w.wk * 2.0 ** -power
    w.wq = w.wq * 2.0 ** power
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    pp.check(w, out, lse, d["kp"], d["vp"], 0)
