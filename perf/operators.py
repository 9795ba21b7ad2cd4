"""Cases and plain forms of the paged key-value cache operators.

``paged_append`` writes new tokens' keys (normalised, rotated) and values into the pages of
a cache; ``decode_paged`` attends with one new token per sequence over such a cache and
appends it. Where ``own`` is false, ``run`` computes them with elementary torch operations in
32 bits (angles in 64), rounded once where a value is stored.
"""
import math
import random

import torch

own = False

D = 128
EPS = 1e-6
THETA = 1e6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _decode(name, **kw):
    c = dict(name=name, op="decode", seqs=1, heads=32, kv_heads=4, window=0, rope=True, page=16,
             fp8=False, token_major=False, len_lo=0, len_hi=0)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", seqs=1, kv_heads=4, rope=True, page=16, fp8=False,
             token_major=False, new_lo=1, new_hi=1, len_lo=0, len_hi=0)
    c.update(kw)
    return c


def listed():
    return [
        # the first tokens of one chat turn on a sliding layer: launch latency
        _decode("decode 1 short", window=512, len_lo=230, len_hi=230),
        # the serving shape: 64 sequences on a sliding layer, the window full
        _decode("decode 64 window 4096", seqs=64, window=4096, page=64, len_lo=4096, len_hi=8191),
        # the same batch over an e4m3 cache whose pages keep a token's heads together
        _decode("decode 64 window 4096 e4m3", seqs=64, window=4096, fp8=True, token_major=True,
                len_lo=4096, len_hi=8191),
        # a full layer (no rotation) near the longest context
        _decode("decode 4 full 131072", seqs=4, rope=False, page=128, len_lo=98303, len_hi=131071),
        # one long sequence alone over an e4m3 cache: all the parallelism is along the keys
        _decode("decode 1 full 131072 e4m3", rope=False, fp8=True, page=32, len_lo=131071,
                len_hi=131071),
        # a large ragged batch, new and old sequences mixed, nine query heads to a KV head
        _decode("decode 201 ragged G9", seqs=201, heads=18, kv_heads=2, window=1024, page=48,
                len_lo=0, len_hi=2513),
        # one new token for each sequence of a decode batch
        _append("append 64 tokens", seqs=64, len_lo=100, len_hi=8000),
        # a packed batch of prompts, 128 to 8192 tokens each
        _append("append 65536 prompts", seqs=16, page=64, new_lo=128, new_hi=8064),
        # the prompt of a full layer near the longest context
        _append("append 131072 full", rope=False, page=128, new_lo=131072, new_hi=131072),
        # prompts quantised to e4m3 behind cached prefixes, odd lengths, token-major pages
        _append("append ragged e4m3", seqs=11, kv_heads=8, fp8=True, token_major=True, page=32,
                new_lo=1, new_hi=4097, len_lo=0, len_hi=5001),
        # one chunk of a long prompt at a far position
        _append("append chunk 509", page=16, new_lo=509, new_hi=509, len_lo=100003, len_hi=100003),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 48, 64, 128, 256])
    fp8, token_major, rope = rng.random() < 0.4, rng.random() < 0.4, rng.random() < 0.7
    kv_heads = rng.choice([1, 2, 4, 8])
    if rng.random() < 0.6:
        seqs = _log_int(rng, 1, 256)
        longest = max(2, min(131071, 1_900_000 // (seqs * kv_heads)))
        hi = _log_int(rng, 1, longest)
        return dict(op="decode", seqs=seqs, heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 9, 16]),
                    kv_heads=kv_heads, window=rng.choice([0, 0, 512, _log_int(rng, 1, 8192)]),
                    rope=rope, page=page, fp8=fp8, token_major=token_major,
                    len_lo=rng.randint(0, hi), len_hi=hi)
    seqs = _log_int(rng, 1, 128)
    new = max(1, min(131072, _log_int(rng, 1, 500_000) // kv_heads) // seqs)
    past = _log_int(rng, 1, max(2, min(100_000, 1_500_000 // (seqs * kv_heads))))
    return dict(op="append", seqs=seqs, kv_heads=kv_heads, rope=rope, page=page, fp8=fp8,
                token_major=token_major, new_lo=rng.randint(1, new), new_hi=new,
                len_lo=rng.randint(0, past), len_hi=past)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly apart; their set depends on the case alone."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    past = _spread(case["len_lo"], case["len_hi"], case["seqs"])
    new = _spread(case["new_lo"], case["new_hi"], case["seqs"]) if case["op"] == "append" else \
        [1] * case["seqs"]
    return past, new


def work(case):
    past, new = _lens(case)
    hk, e = case["kv_heads"], 1 if case["fp8"] else 2
    if case["op"] == "append":
        tokens = sum(new)
        return {"bytes": 2 * tokens * hk * D * (2 + e), "flops": 12 * tokens * hk * D}
    w = case["window"]
    keys = sum(min(p, w - 1) if w > 0 else p for p in past)
    rows = case["seqs"]
    moved = 2 * keys * hk * D * e + rows * (2 * case["heads"] * 2 * D + 2 * hk * D * (2 + e)
                                            + 4 * case["heads"])
    return {"bytes": moved, "flops": 4 * case["heads"] * D * (keys + rows)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dev, bf = "cuda", torch.bfloat16
    past, new = _lens(case)
    order = list(range(case["seqs"]))
    rng.shuffle(order)                           # which sequence has which length
    past = [past[i] for i in order]
    rng.shuffle(order)
    new = [new[i] for i in order]
    hk, page = case["kv_heads"], case["page"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    # each sequence's pages, anywhere in the pool; unused entries of the table are -1
    need = [(p + n + page - 1) // page for p, n in zip(past, new)]
    pool = 3 + sum(-(-p // page) - (-n // page) for p, n in zip(past, new))     # at least all
    perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    cols = torch.arange(max(need), device=dev)
    count = torch.tensor(need, device=dev)
    first = torch.cumsum(count, 0) - count
    idx = (first[:, None] + cols[None, :]).clamp(max=pool - 1)
    table = torch.where(cols[None, :] < count[:, None], perm[idx], torch.full_like(perm[idx], -1))
    s = dict(case=case, block_table=table.contiguous(),
             cache_lens=torch.tensor(past, device=dev, dtype=torch.int32))

    k_scale = v_scale = None
    if case["fp8"]:                              # about 6 standard deviations inside e4m3's range
        k_scale = 0.014 + 0.002 * torch.rand(hk, generator=gen, device=dev)
        v_scale = 0.014 + 0.002 * torch.rand(hk, generator=gen, device=dev)
    s.update(k_scale=k_scale, v_scale=v_scale)
    for name, scale in (("k_pages", k_scale), ("v_pages", v_scale)):
        shape = (pool, page, hk, D) if case["token_major"] else (pool, hk, page, D)
        x = torch.empty(shape, device=dev, dtype=torch.float8_e4m3fn if case["fp8"] else bf)
        y = x.transpose(1, 2) if case["token_major"] else x          # [pages, heads, slots, D]
        step = max(1, (1 << 26) // (hk * page * D))
        for at in range(0, pool, step):
            n = min(step, pool - at)
            z = randn(n, hk, page, D)
            if case["fp8"]:
                z = (z / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX)
            y[at:at + n].copy_(z)
        s[name] = y

    rows = sum(new)
    s["k"], s["v"] = randn(rows, hk, D).to(bf), randn(rows, hk, D).to(bf)
    s["w_k"] = (1 + 0.1 * randn(D)).to(bf)
    if case["op"] == "append":
        ends = [0]
        for n in new:
            ends.append(ends[-1] + n)
        s["cu_new_lens"] = torch.tensor(ends, device=dev, dtype=torch.int32)
        s["status"] = torch.zeros(64, device=dev, dtype=torch.int32)
    else:
        s["q"] = randn(rows, case["heads"], D).to(bf)
        s["w_q"] = (1 + 0.1 * randn(D)).to(bf)
        s["sink"] = randn(case["heads"])
        if own:
            from sink_aware_sliding_head_b200 import flint_attn as fa
            s["workspace"] = fa.alloc_decode_paged_workspace(rows, case["heads"], hk)
    return s


# ------------------------------------------------------------------ the operators

def _norm_rotate(x, w, pos, rope):
    """RMSNorm of each head, then the rotation of channel j with channel j + D/2 at pos."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
    if not rope:
        return y
    freq = THETA ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    angle = pos.double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _store(pages, page, slot, x, scale):
    if scale is None:
        pages[page, :, slot] = x.to(pages.dtype)
    else:
        q = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(pages.dtype)
        pages.view(torch.uint8)[page, :, slot] = q.view(torch.uint8)


def _load(pages, page, slot, scale):
    if scale is None:
        return pages[page, :, slot].float()
    x = pages.view(torch.uint8)[page, :, slot].view(pages.dtype).float()
    return x * scale[:, None]


def _plain_append(s):
    case, lens, table, page = s["case"], s["cache_lens"], s["block_table"], s["case"]["page"]
    cu = s["cu_new_lens"]
    t = torch.arange(s["k"].shape[0], device=cu.device, dtype=cu.dtype)
    seq = torch.bucketize(t, cu[1:], right=True)
    pos = (lens[seq] + t - cu[seq]).long()
    at, slot = table[seq, pos // page].long(), pos % page
    k_hat = _norm_rotate(s["k"], s["w_k"], pos, case["rope"])
    _store(s["k_pages"], at, slot, k_hat, s["k_scale"])
    _store(s["v_pages"], at, slot, s["v"].float(), s["v_scale"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_decode(s):
    case, table, page = s["case"], s["block_table"], s["case"]["page"]
    p, w = s["cache_lens"].long(), case["window"]
    b, h, hk = case["seqs"], case["heads"], case["kv_heads"]
    q_hat = _norm_rotate(s["q"], s["w_q"], p, case["rope"])
    k_hat = _norm_rotate(s["k"], s["w_k"], p, case["rope"])
    at = table.gather(1, (p // page)[:, None])[:, 0].long()
    _store(s["k_pages"], at, p % page, k_hat, s["k_scale"])
    _store(s["v_pages"], at, p % page, s["v"].float(), s["v_scale"])
    widest = min(w, case["len_hi"] + 1) if w > 0 else case["len_hi"] + 1
    lo = (p - w + 1).clamp(min=0) if w > 0 else torch.zeros_like(p)
    pos = lo[:, None] + torch.arange(widest, device=p.device)
    seen = pos <= p[:, None]
    at = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1)).clamp(min=0).long()
    keys = _load(s["k_pages"], at, pos % page, s["k_scale"])            # [B, n, Hk, D]
    z = q_hat.view(b, hk, h // hk, D) @ keys.permute(0, 2, 3, 1) / math.sqrt(D)
    del keys
    z = z.masked_fill(~seen[:, None, None, :], -math.inf)
    sink = s["sink"].view(1, hk, h // hk, 1)
    m = torch.maximum(z.max(-1, keepdim=True).values, sink)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True) + torch.exp(sink - m)
    values = _load(s["v_pages"], at, pos % page, s["v_scale"])
    out = (e @ values.permute(0, 2, 1, 3)) / total
    return {"out": out.view(b, h, D).to(torch.bfloat16),
            "lse": (m + total.log()).view(b, h),
            "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(s):
    case = s["case"]
    if not own:
        return _plain_append(s) if case["op"] == "append" else _plain_decode(s)
    from sink_aware_sliding_head_b200 import flint_attn as fa
    if case["op"] == "append":
        fa.paged_append(s["k"], s["v"], s["w_k"], s["cu_new_lens"], s["cache_lens"],
                        s["block_table"], s["k_pages"], s["v_pages"], case["rope"], THETA,
                        rms_eps=EPS, k_scale=s["k_scale"], v_scale=s["v_scale"],
                        status=s["status"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    out, lse = fa.decode_paged(s["q"], s["k"], s["v"], s["w_q"], s["w_k"], s["sink"],
                               s["cache_lens"], s["block_table"], s["k_pages"], s["v_pages"],
                               case["window"], case["rope"], THETA, rms_eps=EPS,
                               k_scale=s["k_scale"], v_scale=s["v_scale"],
                               workspace=s["workspace"])
    return {"out": out, "lse": lse, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ------------------------------------------------------------------ in 64 bits

def _hat64(row, w, t, rope):
    """k_hat or q_hat of the rows [heads, D] of the token at position t."""
    x = row.double()
    x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
    if rope:
        j = torch.arange(D // 2, device=row.device, dtype=torch.float64)
        turn = torch.polar(torch.ones_like(j), t * torch.exp(-j * (2 * math.log(THETA) / D)))
        z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
        x = torch.cat([z.real, z.imag], -1)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    page, past = case["page"], s["cache_lens"].tolist()
    table = s["block_table"].tolist()
    k64, v64 = s["k_pages"].double(), s["v_pages"].double()      # stored values, before scales
    hk = case["kv_heads"]
    ones = torch.ones(hk, device="cuda")
    ks = (s["k_scale"] if case["fp8"] else ones).double()[:, None]
    vs = (s["v_scale"] if case["fp8"] else ones).double()[:, None]

    def kept(x):                                                  # e4m3 saturates
        return x.clamp(-E4M3_MAX, E4M3_MAX) if case["fp8"] else x

    if case["op"] == "append":
        ends = s["cu_new_lens"].tolist()
        for b, p in enumerate(past):
            t = torch.arange(p, p + ends[b + 1] - ends[b], device="cuda")
            rows = slice(ends[b], ends[b + 1])
            at, slot = s["block_table"][b][t // page].long(), t % page
            k64[at, :, slot] = kept(_hat64(s["k"][rows], s["w_k"], t.double()[:, None, None],
                                           case["rope"]) / ks)
            v64[at, :, slot] = kept(s["v"][rows].double() / vs)
        return {"k_pages": k64, "v_pages": v64}

    out = torch.empty(case["seqs"], case["heads"], D, device="cuda", dtype=torch.float64)
    lse = torch.empty(case["seqs"], case["heads"], device="cuda", dtype=torch.float64)
    group, kind = case["heads"] // hk, s["k_pages"].dtype
    for b, p in enumerate(past):
        t = torch.tensor(float(p), device="cuda", dtype=torch.float64)
        q = _hat64(s["q"][b], s["w_q"], t, case["rope"]).view(hk, group, D)
        new_k = kept(_hat64(s["k"][b], s["w_k"], t, case["rope"]) / ks)
        new_v = kept(s["v"][b].double() / vs)
        first = max(0, p + 1 - case["window"]) if case["window"] > 0 else 0
        j = torch.arange(first, p, device="cuda")
        at, slot = s["block_table"][b][j // page].long(), j % page
        # the new row is attended as it is stored: rounded to the cache's type
        keys = torch.cat([k64[at, :, slot], new_k.to(kind).double()[None]]) * ks
        vals = torch.cat([v64[at, :, slot], new_v.to(kind).double()[None]]) * vs
        z = torch.einsum("gid,jgd->gij", q, keys) * D ** -0.5
        z = torch.cat([z, s["sink"].double().view(hk, group, 1)], -1)    # the sink: value zero
        lse[b] = torch.logsumexp(z, -1).view(-1)
        out[b] = torch.einsum("gij,jgd->gid", torch.softmax(z, -1)[..., :-1], vals).reshape(-1, D)
        at, slot = table[b][p // page], p % page
        k64[at, :, slot], v64[at, :, slot] = new_k, new_v
    return {"out": out, "lse": lse, "k_pages": k64, "v_pages": v64}
