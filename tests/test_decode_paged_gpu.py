"""flint_attn_decode_paged against the formulas in 64 bits, by the roundings on the way: cache
types and layouts, group sizes, windows, lengths from none to many splits, masked garbage,
and its device-side refusals."""
import numpy as np
import pytest
import torch

from paged_util import Paged, append, decode, to64

pytestmark = pytest.mark.gpu

E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


def check(fa, w, window, **kw):
    d = w.dev()
    out, lse = decode(fa, w, d, window, **kw)
    rows = [b for b, p in enumerate(w.lens) if p >= 0]
    w.check_decode(out, lse, window, rows)
    w.check_pool(d["kp"], d["vp"], rows)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,H,Hk,P,W,layout,rope", [
    ([0], 32, 4, 16, 0, "head", True),                        # the first token
    ([0, 1, 15, 16, 17, 63, 64, 65], 32, 4, 16, 0, "head", True),
    ([300, 0, 599, 127, 128], 32, 4, 64, 128, "token", True),
    ([5, 0, 599], 32, 4, 16, 1, "head", True),                # only the new token in the window
    ([5, 70, 599], 32, 4, 32, 2, "both", True),
    ([100, 513, 64, 1], 32, 4, 48, 65, "token", False),
    ([299, 5, 150], 32, 2, 16, 64, "head", True),             # G = 16
    ([199, 0, 77], 4, 4, 128, 0, "head", True),               # G = 1
    ([299, 0, 100], 8, 4, 16, 0, "token", True),              # G = 2
    ([249, 3, 130], 6, 2, 32, 0, "head", True),               # G = 3
    ([399, 250, 0], 16, 4, 256, 200, "both", False),          # G = 4
    ([259, 40], 18, 2, 16, 100, "head", True),                # G = 9
    ([1099, 513, 1024], 32, 4, 64, 1000, "token", False),
    ([4000], 16, 1, 16, 0, "head", True),                     # one pair over many splits
    ([70000], 2, 1, 128, 0, "head", True),                    # a far position
    ([9000], 16, 1, 64, 0, "head", True),                     # 36 and more partials, G = 16
])
def test_decode_matches_the_formulas(cuda_lib, lens, H, Hk, P, W, layout, rope, dtype):
    w = Paged(lens, H=H, Hk=Hk, P=P, dtype=dtype, layout=layout, rope=rope, seed=11)
    check(cuda_lib, w, W, fp32_out=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_ragged_batch_bf16_out(cuda_lib, dtype):
    """More rows than threads of a block, lengths mixed, some rows not in use."""
    rng = np.random.RandomState(5)
    lens = rng.randint(-1, 200, 331).tolist()
    w = Paged(lens, H=4, Hk=2, P=16, dtype=dtype, seed=12)
    out, _ = check(cuda_lib, w, 50)
    assert out.dtype == BF16


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,top,W", [(700, 150, 0), (1500, 40, 33)])
def test_more_rows_than_a_block_keeps_lengths_of(cuda_lib, B, top, W, dtype):
    lens = np.random.RandomState(B).randint(-1, top, B).tolist()
    w = Paged(lens, H=2, Hk=1, P=16, dtype=dtype, seed=40)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, W, fp32_out=True)
    rows = [b for b, p in enumerate(lens) if p >= 0]
    w.check_pool(d["kp"], d["vp"], rows)
    w.check_decode(out, lse, W, rows[:5] + rows[B // 2:B // 2 + 40] + rows[-40:])


def test_a_range_of_more_rows_than_kept_lengths(cuda_lib):
    """90000 rows on one KV head: over 512 rows to an SM's range, their lengths read late."""
    B = 90000
    lens = np.random.RandomState(1).randint(0, 3, B).tolist()
    w = Paged(lens, H=1, Hk=1, P=16, seed=41, extra_cols=0)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    w.check_decode(out, lse, 0, list(range(0, B, 997)) + [B - 1])
    assert torch.all(torch.isfinite(out)) and torch.all(torch.isfinite(lse))


@pytest.mark.parametrize("lens", [[70], [333, 64]])
def test_more_kv_heads_than_sms(cuda_lib, lens):
    w = Paged(lens, H=200, Hk=200, P=16, seed=42)
    check(cuda_lib, w, 100, fp32_out=True)


@pytest.mark.parametrize("P", [80, 112, 272, 512])
def test_page_sizes_off_the_block(cuda_lib, P):
    w = Paged([P - 1, P, P + 1, 3 * P + 5], H=8, Hk=2, P=P, seed=43)
    check(cuda_lib, w, 0, fp32_out=True)


@pytest.mark.parametrize("lens", [[1], [64], [255], [256], [257], [2048], [9473]])
def test_one_row_over_its_ranges(cuda_lib, lens):
    """One row alone: its blocks end anywhere in the last range."""
    w = Paged(lens, H=24, Hk=3, P=16, seed=44)
    check(cuda_lib, w, 0, fp32_out=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pools_in_either_order(cuda_lib, dtype):
    """V's pool before K's in memory, as well as behind it."""
    for flip in (False, True):
        w = Paged([200, 31], H=8, Hk=2, P=16, dtype=dtype, seed=48)
        d = w.dev()
        one = torch.empty(2, *w.kp.shape, dtype=dtype, device="cuda")
        one[int(flip)].copy_(d["kp"])
        one[1 - int(flip)].copy_(d["vp"])
        d["kp"], d["vp"] = one[int(flip)], one[1 - int(flip)]
        out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
        w.check_decode(out, lse, 0)
        w.check_pool(d["kp"], d["vp"])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_offsets_past_32_bits(cuda_lib, dtype):
    """Pages that lie more than 2^32 bytes (and 2^31 elements) into their pool."""
    w = Paged([200, 31, 77], new=[1, 1, 1], H=8, Hk=2, P=16, dtype=dtype, seed=49)
    d = w.dev()
    n = w.kp.shape[0]
    pages = (1 << 32) // (2 * 16 * 128) + n + 1                # of 4096 elements
    far = torch.arange(pages - n, pages, device="cuda")
    pools = []
    for x in (d["kp"], d["vp"]):
        big = torch.empty(pages, 2, 16, 128, dtype=dtype, device="cuda")
        big[far] = x
        pools.append(big)
    d["kp"], d["vp"] = pools
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - n), d["table"])
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    w.check_decode(out, lse, 0)
    w.check_pool(pools[0][far], pools[1][far])
    again = Paged([200, 31, 77], new=[5, 0, 20], H=8, Hk=2, P=16, dtype=dtype, seed=49)
    e = again.dev()
    m = again.kp.shape[0]
    assert m < n + 20
    far = torch.arange(pages - m, pages, device="cuda")
    pools[0][far], pools[1][far] = e["kp"], e["vp"]
    e["kp"], e["vp"] = pools
    e["table"] = torch.where(e["table"] >= 0, e["table"] + (pages - m), e["table"])
    append(cuda_lib, again, e)
    again.check_pool(pools[0][far], pools[1][far])


def test_rows_not_in_use_stay_as_they_were(cuda_lib):
    w = Paged([-1, 37, -1, 0, -1], P=16, seed=13)
    d = w.dev()
    out = torch.full((5, 32, 128), 7.0, device="cuda")
    lse = torch.full((5, 32), 7.0, device="cuda")
    decode(cuda_lib, w, d, 0, out=out, lse=lse, fp32_out=True)
    w.check_decode(out, lse, 0, rows=[1, 3])
    w.check_pool(d["kp"], d["vp"], rows=[1, 3])
    for b in (0, 2, 4):
        assert torch.all(out[b] == 7.0) and torch.all(lse[b] == 7.0)


def test_all_rows_unused(cuda_lib):
    w = Paged([-1, -1], P=16, seed=14)
    d = w.dev()
    out = torch.full((2, 32, 128), 7.0, device="cuda")
    decode(cuda_lib, w, d, 0, out=out, fp32_out=True)
    assert torch.all(out == 7.0)
    w.check_pool(d["kp"], d["vp"], rows=[])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,W", [([37, 130], 0), ([200, 333], 77)])
def test_garbage_in_masked_slots_is_not_seen(cuda_lib, dtype, lens, W):
    """NaN and infinities in slots past the new token and before the window."""
    w = Paged(lens, P=64, dtype=dtype, seed=15)
    for b, p in enumerate(lens):
        lo = max(0, p - W + 1) if W else 0
        pos = np.array([t for t in range(-(-(p + 1) // 64) * 64) if t < lo or t > p])
        pg, sl = w.table[b].numpy()[pos // 64], pos % 64
        for pool, bad in ((w.kp, float("inf")), (w.vp, float("nan"))):
            for x, y in zip(pg.tolist(), sl.tolist()):
                pool[x, :, y] = torch.full((4, 128), bad).to(dtype)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, W, fp32_out=True)
    w.check_decode(out, lse, W)


def test_shared_prefix_pages(cuda_lib):
    """Two sequences that read the same pages of a common prefix."""
    w = Paged([80, 90], P=16, seed=16)
    w.table[1, :5] = w.table[0, :5]
    check(cuda_lib, w, 0, fp32_out=True)


def test_sinks_of_minus_infinity_and_large_scores(cuda_lib):
    w = Paged([50, 0, 700], P=16, seed=17)
    w.sink[::2] = float("-inf")
    w.sink[1] = 60.0
    w.kp *= 8.0                                   # scores to about +-80: the running max moves
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 0, fp32_out=True)
    w.check_decode(out, lse, 0)


def test_rising_scores_move_the_maximum(cuda_lib):
    """Keys that line up better and better with the query, along many blocks."""
    w = Paged([1000], H=8, Hk=1, P=16, rope=False, seed=18)
    q = to64(w.q[0, 0]) * to64(w.wq)
    q = q / np.linalg.norm(q)
    pg, sl = w.slots(0, 0, 1000)
    ramp = np.linspace(0, 900, 1000)[:, None, None] * q[None, None, :]
    w.kp[torch.as_tensor(pg, dtype=torch.long), :, torch.as_tensor(sl)] = \
        torch.as_tensor(ramp).to(BF16)
    check(cuda_lib, w, 0, fp32_out=True)


def test_softmax_scale_and_fused_projection_strides(cuda_lib):
    w = Paged([33, 257], H=8, Hk=2, P=32, seed=19)
    d = w.dev()
    qkv = torch.cat([d["q"], d["k"], d["v"]], 1).contiguous()
    d["q"], d["k"], d["v"] = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    out, lse = decode(cuda_lib, w, d, 0, softmax_scale=0.25, fp32_out=True)
    w.check_decode(out, lse, 0, scale=0.25)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_same_bits_every_run_and_ready_workspace(cuda_lib, dtype):
    """One workspace over calls of different sizes; results repeat bit for bit."""
    big = Paged([3000, 17, 900], P=16, dtype=dtype, seed=20)
    small = Paged([40], H=8, Hk=2, P=16, dtype=dtype, seed=21)
    ws = cuda_lib.alloc_decode_paged_workspace(3, 32, 4)
    first = None
    for _ in range(3):
        a = decode(cuda_lib, big, big.dev(), 0, workspace=ws)
        b = decode(cuda_lib, small, small.dev(), 16, workspace=ws)
        if first is None:
            first = a + b
            big.check_decode(a[0], a[1], 0)
            small.check_decode(b[0], b[1], 16)
        for x, y in zip(first, a + b):
            assert torch.equal(x, y)


def test_bad_lengths_are_reported_and_skipped(cuda_lib):
    w = Paged([10, 20, 30], P=16, seed=22, extra_cols=0)
    d = w.dev()
    d["lens"][0], d["lens"][2] = -2, w.table.shape[1] * 16            # no such slot
    out = torch.full((3, 32, 128), 7.0, device="cuda")
    lse = torch.full((3, 32), 7.0, device="cuda")
    ws = cuda_lib.alloc_decode_paged_workspace(3, 32, 4)
    with pytest.raises(cuda_lib.FlintError) as e:
        decode(cuda_lib, w, d, 0, out=out, lse=lse, fp32_out=True, workspace=ws)
    assert e.value.code == 1
    for b in (0, 2):
        assert torch.all(out[b] == 7.0) and torch.all(lse[b] == 7.0)
    w.check_decode(out, lse, 0, rows=[1])
    w.check_pool(d["kp"], d["vp"], rows=[1])
    good = w.dev()                                                     # the workspace still serves
    out, lse = decode(cuda_lib, w, good, 0, fp32_out=True, workspace=ws)
    w.check_decode(out, lse, 0)


def test_pages_before_the_window_are_not_looked_at(cuda_lib):
    w = Paged([300, 100, 200], P=16, seed=23)
    d = w.dev()
    d["table"][0, 4], d["table"][2, 1] = -1, 1 << 30                   # slots 64.. and 16..
    out, lse = decode(cuda_lib, w, d, 150, fp32_out=True)
    w.check_decode(out, lse, 150)
    w.check_pool(d["kp"], d["vp"])


@pytest.mark.parametrize("col", [10, 12, 18])                          # slots 151.. to the new one
def test_bad_pages_give_nan_and_a_status(cuda_lib, col):
    w = Paged([300, 100, 200], P=16, seed=23)
    ws = cuda_lib.alloc_decode_paged_workspace(3, 32, 4)
    for bad in (-1, w.kp.shape[0], 1 << 30, -(1 << 31)):
        d = w.dev()
        d["table"][0, col] = bad
        out, lse = decode(cuda_lib, w, d, 150, fp32_out=True, workspace=ws, check=False)
        assert cuda_lib.load_library().flint_attn_check_status(ws.data_ptr(), None) == 1
        assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
        w.check_decode(out, lse, 150, rows=[1, 2])
        w.check_pool(d["kp"], d["vp"], rows=[1, 2] if col == 18 else [0, 1, 2])


def test_two_streams_two_workspaces(cuda_lib):
    ws = [Paged([900, 31], P=16, seed=24), Paged([450, 1200], P=64, seed=25)]
    devs, streams = [w.dev() for w in ws], [torch.cuda.Stream() for _ in ws]
    got = []
    for w, d, s in zip(ws, devs, streams):
        s.wait_stream(torch.cuda.current_stream())
        got.append(decode(cuda_lib, w, d, 0, check=False, stream=s, fp32_out=True))
    torch.cuda.synchronize()
    for w, (out, lse) in zip(ws, got):
        w.check_decode(out, lse, 0)


def test_two_graphs_share_a_workspace(cuda_lib):
    ws = cuda_lib.alloc_decode_paged_workspace(2, 32, 4)
    cases, graphs, outs = [Paged([2000, 3], P=16, seed=26), Paged([64, 700], P=16, seed=27)], [], []
    devs = [w.dev() for w in cases]
    for w, d in zip(cases, devs):
        out = torch.empty(2, 32, 128, device="cuda")
        lse = torch.empty(2, 32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(cuda_lib, w, d, 0, check=False, fp32_out=True, out=out, lse=lse, workspace=ws)
        graphs.append(g)
        outs.append((out, lse))
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for w, (out, lse) in zip(cases, outs):
        w.check_decode(out, lse, 0)


def test_a_captured_call_follows_its_lengths(cuda_lib):
    """One capture, replayed after the lengths, the table and the new rows changed."""
    runs = [Paged(lens, P=16, seed=45 + i, extra_cols=100 - max(lens) // 16)
            for i, lens in enumerate([[10, 700, -1], [1500, 0, 63], [-1, -1, 64]])]
    cols = min(w.table.shape[1] for w in runs)
    pages = max(w.kp.shape[0] for w in runs)
    d = runs[0].dev()
    d["table"] = torch.zeros(3, cols, dtype=torch.int32, device="cuda")
    d["kp"], d["vp"] = (torch.zeros(pages, 4, 16, 128, dtype=BF16, device="cuda") for _ in "kv")
    ws = cuda_lib.alloc_decode_paged_workspace(3, 32, 4)
    out, lse = torch.empty(3, 32, 128, device="cuda"), torch.empty(3, 32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(cuda_lib, runs[0], d, 0, check=False, fp32_out=True, out=out, lse=lse, workspace=ws)
    for w in runs:
        for name in ("q", "k", "v", "wq", "wk", "sink"):
            d[name].copy_(getattr(w, name))
        d["lens"].copy_(torch.tensor(w.lens, dtype=torch.int32))
        d["table"].copy_(w.table[:, :cols])
        d["kp"][:w.kp.shape[0]] = w.kp.cuda()
        d["vp"][:w.vp.shape[0]] = w.vp.cuda()
        graph.replay()
        torch.cuda.synchronize()
        w.check_decode(out, lse, 0, rows=[b for b, p in enumerate(w.lens) if p >= 0])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_prompt_then_decode_steps(cuda_lib, dtype):
    """As a server uses them: append a prompt in two chunks, then decode three tokens; every
    step's cache is what the formulas give for all tokens so far."""
    w = Paged([0, 0], new=[70, 33], H=8, Hk=2, P=16, dtype=dtype, seed=28, extra_cols=4)
    pages = w.kp.shape[0]
    w.table[:, :] = torch.randperm(2 * w.table.shape[1], generator=torch.Generator().manual_seed(1)).view(2, -1).to(torch.int32)
    grow = 2 * w.table.shape[1] - pages
    w.kp, w.vp = (torch.cat([x.float(), torch.zeros(grow, *x.shape[1:])]).to(dtype)
                  for x in (w.kp, w.vp))
    d = w.dev()
    append(cuda_lib, w, d)
    w.check_pool(d["kp"], d["vp"])
    ws = cuda_lib.alloc_decode_paged_workspace(2, 8, 2)
    lens = [70, 33]
    for step in range(3):
        n = Paged(lens, H=8, Hk=2, P=16, dtype=dtype, seed=29 + step)
        n.table, n.kp, n.vp = w.table, d["kp"].cpu(), d["vp"].cpu()
        n.k_scale, n.v_scale = w.k_scale, w.v_scale
        s = n.dev()
        s["kp"], s["vp"] = d["kp"], d["vp"]
        out, lse = decode(cuda_lib, n, s, 48, fp32_out=True, workspace=ws)
        n.check_decode(out, lse, 48)
        n.check_pool(d["kp"], d["vp"])
        lens = [p + 1 for p in lens]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_append_and_decode_store_the_same_bits(cuda_lib, dtype):
    w = Paged([77, 0, 15], P=16, dtype=dtype, seed=33)
    a, b = w.dev(), w.dev()
    append(cuda_lib, w, a)
    decode(cuda_lib, w, b, 0)
    bits = torch.uint8 if dtype == E4M3 else torch.int16
    assert torch.equal(a["kp"].view(bits), b["kp"].view(bits))
    assert torch.equal(a["vp"].view(bits), b["vp"].view(bits))


def test_matches_the_dense_decode(cuda_lib):
    """The same step through flint_attn_decode's dense cache: each is within its own bound of
    the formulas, so the two are within both bounds of each other."""
    lens = [0, 63, 200, 511]
    w = Paged(lens, P=64, seed=34)
    C = w.table.shape[1] * 64
    dense = [torch.zeros(4, 4, C, 128, dtype=BF16) for _ in range(2)]
    for b, p in enumerate(lens):
        pg, sl = w.slots(b, 0, p)
        for x, pool in zip(dense, (w.kp, w.vp)):
            x[b, :, :p] = pool[torch.as_tensor(pg, dtype=torch.long), :,
                               torch.as_tensor(sl)].transpose(0, 1)
    d = w.dev()
    out, lse = decode(cuda_lib, w, d, 128, fp32_out=True)
    o2, l2 = cuda_lib.decode(d["q"], d["k"], d["v"], d["wq"], d["wk"], d["sink"], d["lens"],
                             dense[0].cuda(), dense[1].cuda(), 128, True, 1e6, fp32_out=True,
                             check_status=True)
    # the dense kernel sums the rounded probabilities: 2^-8 more in its denominator
    for b in range(4):
        ro, rl, mag, dz = w.decode64(b, 128)
        tol = (2 * 2.0 ** -8 + 2.0 ** -8 + 6 * dz[:, None]) * mag
        assert np.all(np.abs(to64(out[b]) - to64(o2[b])) <= tol)
        assert np.all(np.abs(to64(lse[b]) - to64(l2[b])) <= 2.0 ** -8 + 3 * dz)
