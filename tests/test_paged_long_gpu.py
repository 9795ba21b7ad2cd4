"""Calls long enough that the paged kernels use everything twice: the decode kernel's ring stages,
barriers and segment slots in all four variants, and further turns of the append kernel's loop.
Also e4m3 pools that one tensor map cannot hold together, and a dense cache as a pool."""
import numpy as np
import pytest
import torch

from paged_util import Paged, append, decode
from test_paged_plan_model import segments

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def used(w, W, G):
    """(blocks, segments) of the SM that has the most, by the plan restated on the CPU."""
    cost, groups = 8 if w.e4m3 else 4, 4 if G <= 8 else 2
    per = {}
    for i, _, _, _, length, *_ in segments(w.lens, w.Hk, W, w.table.shape[1] * w.P, sms(), cost,
                                           groups):
        n = per.setdefault(i, [0, 0])
        n[0] += length
        n[1] += 1
    return max(n[0] for n in per.values()), max(n[1] for n in per.values())


# No variant has more than 10 stages, 20 barriers or 4 segment slots.
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("G", [8, 9, 16])
def test_many_segments_to_a_range(cuda_lib, G, dtype):
    """Short rows, many to an SM."""
    lens = np.random.RandomState(G).randint(-1, 330, 2200).tolist()
    w = Paged(lens, H=G, Hk=1, P=32, dtype=dtype, seed=80)
    blocks, segs = used(w, 0, G)
    assert blocks > 40 and segs > 8
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    rows = [b for b, p in enumerate(lens) if p >= 0]
    w.check_pool(d["kp"], d["vp"], rows)
    w.check_decode(out, lse, 0, rows)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("G,P", [(8, 64), (9, 16), (16, 48)])
def test_long_ranges(cuda_lib, G, P, dtype):
    """A few long rows: an SM streams dozens of blocks of one segment."""
    w = Paged([230001, 5, 177777, 0], H=G, Hk=1, P=P, dtype=dtype, rope=False, seed=81)
    blocks, _ = used(w, 0, G)
    assert blocks > 40
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    w.check_pool(d["kp"], d["vp"])
    w.check_decode(out, lse, 0)


@pytest.mark.parametrize("dtype,Hk,tokens,resident", [
    (BF16, 1, 40007, 8 * 4), (BF16, 2, 40007, 8 * 4), (BF16, 4, 24001, 5 * 4),
    (BF16, 7, 20011, 4 * 4), (E4M3, 1, 11003, 8), (E4M3, 2, 11003, 8), (E4M3, 3, 7001, 5),
    (E4M3, 8, 6007, 4), (E4M3, 24, 5003, 4)])
def test_append_of_more_tokens_than_one_turn(cuda_lib, dtype, Hk, tokens, resident):
    """resident: blocks of eight tokens per SM that the variant's grid has at most."""
    assert tokens > resident * 8 * sms()
    new = [1, 0, 701, 0, 17, 0]
    new.append(tokens - sum(new))
    w = Paged([0, 3, 90, 0, 15, 5, 33], new, H=Hk, Hk=Hk, P=48, dtype=dtype, seed=82)
    d = w.dev()
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])


@pytest.mark.parametrize("P", [16, 32, 64])
def test_keys_and_values_in_one_pool(cuda_lib, P):
    """One e4m3 tensor as keys and as values (no distance to step by, so K and V take a copy
    each). Its new slots are written twice and are not compared."""
    lens = [0, 5, 200, 333]
    w = Paged(lens, H=18, Hk=2, P=P, dtype=E4M3, seed=83)
    w.v_scale = w.k_scale.clone()
    w.vp = w.kp
    d = w.dev()
    d["vp"] = d["kp"]
    out, lse = decode(cuda_lib, w, d, 60, fp32_out=True)
    w.check_decode(out, lse, 60)
    same = torch.ones(w.kp.shape[0], P, dtype=torch.bool)
    for b, p in enumerate(lens):
        pg, sl = w.slots(b, p, p + 1)
        same[int(pg[0]), int(sl[0])] = False
    a, c = (t.cpu().view(torch.uint8).transpose(1, 2)[same] for t in (d["kp"], w.kp))
    assert torch.equal(a, c)


def test_a_dense_cache_is_a_pool_of_one_page_to_a_row(cuda_lib):
    """[B, Hk, C, D] with row b in page b gives the bits that scattered pages of C slots give."""
    lens = [0, 511, 63, 300]
    w = Paged(lens, H=16, Hk=2, P=512, seed=84, extra_cols=0)
    d = w.dev()
    dense = [t[d["table"][:, 0].long()].contiguous() for t in (d["kp"], d["vp"])]
    rows = torch.arange(4, device="cuda", dtype=torch.int32)[:, None]
    out, lse = decode(cuda_lib, w, d, 200, fp32_out=True)
    w.check_decode(out, lse, 200)
    scattered = d["table"][:, 0].long()
    e = dict(d, kp=dense[0], vp=dense[1], table=rows)
    again = decode(cuda_lib, w, e, 200, fp32_out=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert torch.equal(dense[0], d["kp"][scattered]) and torch.equal(dense[1], d["vp"][scattered])
