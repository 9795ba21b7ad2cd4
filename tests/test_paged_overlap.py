"""The paged kernels may be set up while the kernel before them on the stream is finishing: what
that kernel wrote (lengths, tables, rows, scales) is read after it is done, and by loads that
cannot be taken for invariant and moved before the wait."""
import os
import re

import pytest
import torch

from paged_util import D, Paged, THETA
from sink_aware_sliding_head_b200.build import CSRC

FILES = ("paged.cuh", "paged_append.cu", "decode_paged.cu")


def code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)


def test_no_read_only_loads_under_an_overlapped_start():
    """Memory that an earlier kernel writes is not read-only for the lifetime of this one."""
    for name in FILES:
        for word in ("__ldg", "ld.global.nc", "__restrict__", "doc_of"):
            assert word not in code(name), (name, word)
    shared = code("common.cuh")                   # why doc_of is among them
    assert "__ldg" in shared[shared.index("int doc_of("):][:400]


def test_the_kernels_wait_before_their_first_global_access():
    for name in FILES[1:]:
        src = code(name)
        body = src[src.index("__global__"):]
        before = body[body.index("{"):body.index("previous_done();")]
        for word in ("load(", "load_row(", "a.lens", "a.cu", "a.status", "atomic", "tma_load"):
            assert word not in before, (name, word)
        assert src.count("__global__") == src.count("previous_done();") == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_steps_back_to_back_are_the_steps_one_by_one(cuda_lib, dtype):
    """A serving loop whose every input is made by the kernel right before the call: a product
    (q, k, v), a table row, lengths, scales. Without any wait on the host it gives the bits that
    it gives with one after every kernel."""
    fa, B, H, Hk, P, steps = cuda_lib, 6, 16, 2, 16, 24
    w = Paged([40, 0, 15, 63, 300, 7], H=H, Hk=Hk, P=P, dtype=dtype, seed=70, extra_cols=6)
    gen = torch.Generator().manual_seed(71)
    x = torch.randn(steps, B, 256, generator=gen).to(torch.bfloat16).cuda()
    proj = torch.randn(256, (H + 2 * Hk) * D, generator=gen).to(torch.bfloat16).cuda() / 16
    cols = w.table.shape[1]
    pages = torch.randperm(B * cols, generator=gen).view(B, cols).to(torch.int32).cuda()

    def loop(wait):
        d = w.dev()
        kp, vp = (torch.zeros(B * cols, *t.shape[1:], dtype=dtype, device="cuda")
                  for t in (d["kp"], d["vp"]))
        table = torch.full_like(pages, -1)
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        ks = vs = None
        if dtype is not torch.bfloat16:
            ks, vs = torch.ones(Hk, device="cuda"), torch.ones(Hk, device="cuda")
        status = torch.zeros(64, dtype=torch.int32, device="cuda")
        ws = fa.alloc_decode_paged_workspace(B, H, Hk)
        outs = []
        for i in range(steps):
            def done():
                if wait:
                    torch.cuda.synchronize()
            table.copy_(pages); done()
            if ks is not None:
                ks.fill_(0.01 + 0.001 * i); done()
                vs.fill_(0.02 - 0.0005 * i); done()
            qkv = (x[i] @ proj).view(B, H + 2 * Hk, D); done()
            q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
            torch.arange(B + 1, out=cu); done()
            fa.paged_append(k, v, d["wk"], cu, lens, table, kp, vp, True, THETA, k_scale=ks,
                            v_scale=vs, status=status); done()
            lens.add_(1); done()
            out, lse = fa.decode_paged(q, k, v, d["wq"], d["wk"], d["sink"], lens, table, kp, vp,
                                       0, True, THETA, k_scale=ks, v_scale=vs, workspace=ws); done()
            lens.add_(1); done()
            outs += [out, lse]
        torch.cuda.synchronize()
        assert status[0].item() == 0
        return outs + [kp.view(torch.uint8), vp.view(torch.uint8)]

    for a, b in zip(loop(True), loop(False)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_behind_copies_fills_and_joined_streams(cuda_lib):
    """In a captured step the paged calls follow copies, fills and a second stream, not only
    kernels of their own stream."""
    fa = cuda_lib
    w = Paged([70, 3, 200], H=16, Hk=2, P=16, seed=72)
    d = w.dev()
    kp0, vp0 = d["kp"].clone(), d["vp"].clone()
    host = torch.tensor(w.lens, dtype=torch.int32).pin_memory()
    lens = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    lens2 = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    status = torch.ones(64, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(3, 16, D, device="cuda"), torch.zeros(3, 16, device="cuda")
    ws = fa.alloc_decode_paged_workspace(3, 16, 2)
    side = torch.cuda.Stream()
    args = d["k"], d["v"], d["wk"], d["cu"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lens2.copy_(host, non_blocking=True)                  # a copy node on the other stream
            fa.paged_append(*args, lens2, d["table"], d["kp"], d["vp"], w.rope, THETA,
                            status=torch.zeros(64, dtype=torch.int32, device="cuda"))
        status.zero_()
        lens.copy_(host, non_blocking=True)
        torch.cuda.current_stream().wait_stream(side)
        fa.paged_append(*args, lens, d["table"], d["kp"], d["vp"], w.rope, THETA, status=status)
        lens.copy_(host, non_blocking=True)
        fa.decode_paged(d["q"], d["k"], d["v"], d["wq"], d["wk"], d["sink"], lens, d["table"],
                        d["kp"], d["vp"], 0, w.rope, THETA, out=out, lse=lse, fp32_out=True,
                        workspace=ws)
        lens.fill_(-1)
    for _ in range(3):
        d["kp"].copy_(kp0)
        d["vp"].copy_(vp0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        w.check_decode(out, lse, 0)
        w.check_pool(d["kp"], d["vp"])
        assert status[0].item() == 0
