"""How exact a paged decode step is: the formulas in 64 bits over what the cache holds, the
roundings of the kernel's operands restated, and bounds on root mean squares.

Bounds on single values must add up all magnitudes (about |q| |K| times a step) and hardly
tell an operand of 22 bits from one of 11. Independent roundings add up in squares, and their
root mean square over thousands of outputs is sharp.
"""
import numpy as np
import torch

from oracle import flint_oracle as fo
from paged_util import THETA, to64

# Root mean squares that a call may be off by: the LSE (absolute), and the output relative to
# the weighted |v|. With channels q_i K_i of a like size, independent relative errors e of the
# channels move a score by e |z|-like amounts: sqrt(128) e |q_i K_i| / sqrt(128) = e.
#   Two parts: the second leaves at most half its step, 2^-22 in fp16 (11 bits each), 2^-17 in
#   bf16 (8 bits each), a root mean square of 1/sqrt(3) of that and less.
#   In 32 bits: the norm, the angle, eight products of 16 channels each, 2^x and the joins, some
#   20 roundings of at most 2^-23 (sums in a product may be cut off, not rounded): sqrt(20) 2^-23
#   = 2^-20.8; twice that for scores above one and for a cut that always has the same sign.
# fp16: 2^-19.8 + 2^-22 < 2^-19. bf16: 2^-17.8 + 2^-19.8 < 2^-17; the output has q's and P's
# parts, 2^-16. A single part leaves 2^-11 / sqrt(3) = 2^-11.8 (fp16) or 2^-8.8 (bf16).
BOUND = {torch.float8_e4m3fn: (2.0 ** -19, 2.0 ** -18), torch.bfloat16: (2.0 ** -17, 2.0 ** -16)}


def operands(w, b, window, kp, vp):
    """q_hat [H, D], K and V [keys, Hk, D] of row b in 64 bits, the new row as kp, vp hold it."""
    p = w.lens[b]
    sk, sv = w.scales()
    q = fo.prologue(to64(w.q[b][None]), to64(w.wq), np.array([p]), w.rope, THETA, 1e-6)[0]
    lo = max(0, p - window + 1) if window > 0 else 0
    pg, sl = w.slots(b, lo, p + 1)
    at = torch.as_tensor(pg, dtype=torch.long), slice(None), torch.as_tensor(sl)
    return q, to64(kp[at].float()) * sk[:, None], to64(vp[at].float()) * sv[:, None]


def attend(q, K, V, sink, scale, q_parts=None, p_parts=None):
    """(out [H, D], lse [H], weighted |v|) of one row; q_parts and p_parts round the operands."""
    H, G = len(q), len(q) // K.shape[1]
    K, V = np.repeat(K, G, 1), np.repeat(V, G, 1)
    if q_parts:
        q = q_parts(q)
    z = scale * np.einsum("hd,nhd->hn", q, K)
    m = np.maximum(z.max(1), sink)
    e = np.exp(z - m[:, None])
    total = e.sum(1) + np.exp(sink - m)
    if p_parts:
        e = p_parts(e)
    e = e / total[:, None]
    return (np.einsum("hn,nhd->hd", e, V), m + np.log(total),
            np.einsum("hn,nhd->hd", e, np.abs(V)))


def in_parts(dtype, parts, lift=1.0):
    """Rounds to the sum of that many 16-bit parts of x * lift."""
    def f(x):
        x = x * lift
        got = np.zeros_like(x)
        for _ in range(parts):
            got = got + torch.as_tensor(x - got).to(dtype).double().numpy()
        return got / lift
    return f


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def off_by(got, want):
    """(rms of the LSE's error, rms of the output's error relative to the weighted |v|)."""
    lse = np.concatenate([g[1] - r[1] for g, r in zip(got, want)])
    out = np.concatenate([((g[0] - r[0]) / np.maximum(r[2], 1e-30)).ravel()
                          for g, r in zip(got, want)])
    return rms(lse), rms(out)


def check(w, out, lse, kp, vp, window, scale=128 ** -0.5):
    """out (float32) and lse of all rows (device tensors) within BOUND of the formulas."""
    kp, vp, sink = kp.cpu(), vp.cpu(), to64(w.sink)
    o, s = to64(out), to64(lse)
    want = [attend(*operands(w, b, window, kp, vp), sink, scale) for b in range(len(w.lens))]
    l, x = off_by([(o[b], s[b]) for b in range(len(w.lens))], want)
    assert l <= BOUND[w.dtype][0], ("lse", l / BOUND[w.dtype][0])
    assert x <= BOUND[w.dtype][1], ("out", x / BOUND[w.dtype][1])
