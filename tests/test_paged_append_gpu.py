"""flint_attn_paged_append against the formulas in 64 bits: new rows in their slots, every
other bit of the pools unchanged, and its device-side refusals."""
import pytest
import torch

from paged_util import Paged, append

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("lens,new,Hk,P,dtype,layout,rope", [
    ([0], [1], 4, 16, BF16, "head", True),
    ([0], [200], 4, 16, BF16, "head", False),
    ([5, 0, 31, 64], [27, 1, 1, 300], 4, 32, BF16, "head", True),
    ([7, 0, 100, 3], [0, 33, 0, 15], 4, 16, BF16, "token", True),     # sequences without a token
    ([1, 17, 250], [130, 1, 64], 1, 48, BF16, "both", True),
    ([131000, 9], [72, 3], 2, 128, BF16, "head", True),               # far positions
    ([0, 12], [65, 18], 3, 16, BF16, "token", True),
    ([0], [40], 24, 64, BF16, "head", True),                          # many heads
    ([3, 0, 90], [62, 1, 7], 4, 16, E4M3, "head", True),
    ([3, 0, 90], [62, 5, 0], 8, 48, E4M3, "token", True),
    ([1000], [129], 1, 256, E4M3, "both", False),
])
def test_append_matches_the_formulas(cuda_lib, lens, new, Hk, P, dtype, layout, rope):
    w = Paged(lens, new, H=Hk, Hk=Hk, P=P, dtype=dtype, layout=layout, rope=rope, seed=3)
    d = w.dev()
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])


def test_append_takes_slices_of_a_fused_projection(cuda_lib):
    w = Paged([9, 40], [21, 16], H=8, Hk=2, P=16, seed=4)
    d = w.dev()
    qkv = torch.cat([d["q"], d["k"], d["v"]], 1).contiguous()          # [T, H + 2 Hk, D]
    d["k"], d["v"] = qkv[:, 8:10], qkv[:, 10:12]
    wide = torch.full((2, d["table"].shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, :d["table"].shape[1]] = d["table"]
    d["table"] = wide[:, :d["table"].shape[1]]                         # a strided table
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])


def test_append_ignores_rows_behind_the_last_sequence(cuda_lib):
    """A fixed-size buffer partly filled, with sequences that are not in use."""
    w = Paged([4, -1, 30], [3, 0, 18], P=16, seed=5)
    d = w.dev()
    tail = torch.full((50, 4, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    d["k"], d["v"] = torch.cat([d["k"], tail]), torch.cat([d["v"], tail])
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"], rows=[0, 2])


def test_append_of_no_tokens_is_a_no_op(cuda_lib):
    w = Paged([4, 7], [0, 0], P=16, seed=6)
    d = w.dev()
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])


def test_append_saturates_and_keeps_extremes(cuda_lib):
    """Values past e4m3's range become +-448 of the scale; a zero row stays zero."""
    w = Paged([0], [4], H=2, Hk=2, P=16, dtype=E4M3, rope=False, seed=7)
    w.v[0] = 1000.0
    w.v[1] = -1000.0
    w.k[2] = 0.0
    w.v[3] = torch.linspace(-7, 7, 128).to(BF16)
    d = w.dev()
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])
    pg, sl = w.slots(0, 0, 4)
    assert torch.all(d["vp"][int(pg[0]), :, 0].float() == 448)
    assert torch.all(d["vp"][int(pg[1]), :, 1].float() == -448)
    assert torch.all(d["kp"][int(pg[2]), :, 2].float() == 0)


def test_append_reports_and_skips_what_has_no_page(cuda_lib):
    w = Paged([10, 20, 5], [4, 40, 2], P=16, seed=8, extra_cols=0)
    d = w.dev()
    d["table"][1, 2] = w.kp.shape[0]                                   # not a page: 32..47
    d["lens"][2] = -3                                                  # not a length
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    append(cuda_lib, w, d, status=status, check=False)
    assert status[0].item() != 0
    with pytest.raises(cuda_lib.FlintError) as e:
        append(cuda_lib, w, d, status=status)
    assert e.value.code == 1
    assert status[0].item() == 0                                       # cleared by the check
    # sequence 1: positions 20..31 and 48..59 written, 32..47 skipped
    bits = torch.int16
    pg, sl = w.slots(1, 32, 48)
    for got, was in ((d["kp"], w.kp), (d["vp"], w.vp)):
        for p in set(pg.tolist()):
            assert torch.equal(got[p].cpu().view(bits), was[p].view(bits))
    kn, _ = w.new_rows(1)
    pg, sl = w.slots(1, 48, 60)
    x = d["kp"][torch.as_tensor(pg, dtype=torch.long), :, torch.as_tensor(sl)].cpu().double()
    assert float((x - torch.as_tensor(kn[28:40])).abs().max()) <= 2.0 ** -7 * 8   # |k_hat| < 8


def test_append_past_the_table_is_skipped(cuda_lib):
    w = Paged([10], [6], P=16, seed=9, extra_cols=0)                   # fills slots 10..15
    d = w.dev()
    d["lens"][0] = 13                                                  # 13..18: three have no page
    with pytest.raises(cuda_lib.FlintError):
        append(cuda_lib, w, d)
    pg, _ = w.slots(0, 13, 14)
    same = torch.arange(16) < 13
    for got, was in ((d["kp"], w.kp), (d["vp"], w.vp)):
        assert torch.equal(got[int(pg[0])][:, same.cuda()].cpu(), was[int(pg[0])][:, same])
        other = torch.arange(got.shape[0]) != int(pg[0])
        assert torch.equal(got[other.cuda()].cpu(), was[other])


def test_append_on_another_stream_and_replayed(cuda_lib):
    w = Paged([5, 0], [20, 33], P=16, seed=10)
    d = w.dev()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    append(cuda_lib, w, d, stream=s)
    s.synchronize()
    w.check_pool(d["kp"], d["vp"])
    d = w.dev()
    status = torch.zeros(64, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(cuda_lib, w, d, status=status, check=False)
    graph.replay()
    torch.cuda.synchronize()
    w.check_pool(d["kp"], d["vp"])
    assert status[0].item() == 0
