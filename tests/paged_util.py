"""Helpers of the paged-cache tests: inputs with scattered pages, and the formulas in 64 bits."""
import numpy as np
import torch

from oracle import flint_oracle as fo

D = 128
THETA = 1e6


def to64(t):
    return t.detach().cpu().double().numpy()


def make_pool(pages, Hk, P, dtype, layout="head", gen=None, scale=None):
    """(k_pages, v_pages) [pages, Hk, P, D] filled with N(0,1) values, on the CPU."""
    def fill(shape, axis):
        x = torch.randn(shape, generator=gen)
        if dtype == torch.float8_e4m3fn:
            x = (x / scale.view([-1 if i == axis else 1 for i in range(len(shape))])).clamp(-448, 448)
        return x.to(dtype)
    if layout == "head":
        return fill((pages, Hk, P, D), 1), fill((pages, Hk, P, D), 1)
    if layout == "token":
        return tuple(fill((pages, P, Hk, D), 2).transpose(1, 2) for _ in range(2))
    both = fill((pages, 2, Hk, P, D), 2)                      # K and V of a page side by side
    return both[:, 0], both[:, 1]


class Paged:
    """One batch over a paged cache: CPU inputs, their device copies, the formulas in 64 bits."""

    def __init__(self, lens, new=None, H=32, Hk=4, P=16, dtype=torch.bfloat16, layout="head",
                 rope=True, seed=0, extra_cols=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hk, self.P, self.rope = list(lens), H, Hk, P, rope
        self.new = [1] * len(lens) if new is None else list(new)
        self.dtype, self.layout = dtype, layout
        self.e4m3 = dtype == torch.float8_e4m3fn
        self.k_scale = self.v_scale = None
        if self.e4m3:
            self.k_scale = 0.014 + 0.004 * torch.rand(Hk, generator=g)
            self.v_scale = 0.014 + 0.004 * torch.rand(Hk, generator=g)
        need = [(max(p, 0) + n + P - 1) // P if p >= 0 else 0 for p, n in zip(self.lens, self.new)]
        pool = sum(need) + 2
        perm = torch.randperm(pool, generator=g).to(torch.int32)
        cols = max(need + [1]) + extra_cols
        self.table = torch.full((len(lens), cols), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.kp, self.vp = make_pool(pool, Hk, P, dtype, layout, g, self.k_scale)
        T = sum(self.new)
        bf = torch.bfloat16
        self.q = torch.randn(T, H, D, generator=g).to(bf)
        self.k = torch.randn(T, Hk, D, generator=g).to(bf)
        self.v = torch.randn(T, Hk, D, generator=g).to(bf)
        self.wq = (1 + 0.1 * torch.randn(D, generator=g)).to(bf)
        self.wk = (1 + 0.1 * torch.randn(D, generator=g)).to(bf)
        self.sink = torch.randn(H, generator=g)
        self.cu = torch.tensor([0] + np.cumsum(self.new).tolist(), dtype=torch.int32)

    def dev(self):
        """Device copies in the pool's own layout, as a dict."""
        d = {n: getattr(self, n).cuda() for n in ("q", "k", "v", "wq", "wk", "sink", "cu", "table")}
        d["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        d["ks"] = None if self.k_scale is None else self.k_scale.cuda()
        d["vs"] = None if self.v_scale is None else self.v_scale.cuda()
        if self.layout == "both":
            both = torch.stack([self.kp, self.vp], 1).cuda()
            d["kp"], d["vp"] = both[:, 0], both[:, 1]
        elif self.layout == "token":
            d["kp"], d["vp"] = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                                for x in (self.kp, self.vp))
        else:
            d["kp"], d["vp"] = self.kp.contiguous().cuda(), self.vp.contiguous().cuda()
        return d

    def scales(self):
        one = np.ones(self.Hk)
        return (one, one) if self.k_scale is None else (to64(self.k_scale), to64(self.v_scale))

    def stored(self, x, scale):
        """The values [.., Hk, D] a cache holds for x, in 64 bits (before the scale)."""
        y = torch.as_tensor(x / scale[:, None])
        if self.e4m3:
            y = y.clamp(-448, 448)
        return y.to(self.dtype).double().numpy()

    def new_rows(self, b):
        """k_hat and v of sequence b's new tokens in 64 bits, unrounded, [n, Hk, D]."""
        lo, hi = int(self.cu[b]), int(self.cu[b + 1])
        pos = self.lens[b] + np.arange(hi - lo)
        k = fo.prologue(to64(self.k[lo:hi]), to64(self.wk), pos, self.rope, THETA, 1e-6)
        return k, to64(self.v[lo:hi])

    def slots(self, b, first, last):
        """(pages, slots) of positions first..last-1 of sequence b."""
        pos = np.arange(first, last)
        return self.table[b].numpy()[pos // self.P], pos % self.P

    def decode64(self, b, window, scale=D ** -0.5):
        """(out, lse, weighted |v|, score error bound) of sequence b in 64 bits.

        The score bound: q enters the products as two parts of 16 bits in all (2^-16 of each
        channel) and they are summed in 32 bits (128 terms: 2^-16 of the sum of magnitudes
        covers the sums, the norm and the angle), so |dz| <= 2^-15 * scale * |q| |k|.
        """
        p = self.lens[b]
        sk, sv = self.scales()
        kn, vn = self.new_rows(b)
        q = fo.prologue(to64(self.q[int(self.cu[b])][None]), to64(self.wq), np.array([p]),
                        self.rope, THETA, 1e-6)[0]
        lo = max(0, p - window + 1) if window > 0 else 0
        pg, sl = self.slots(b, lo, p)
        at = torch.as_tensor(pg, dtype=torch.long), slice(None), torch.as_tensor(sl)
        K = np.concatenate([to64(self.kp[at].float()), self.stored(kn[:1], sk)]) * sk[:, None]
        V = np.concatenate([to64(self.vp[at].float()), self.stored(vn[:1], sv)]) * sv[:, None]
        G = self.H // self.Hk
        out, lse = np.zeros((self.H, D)), np.zeros(self.H)
        mag, dz = np.zeros((self.H, D)), np.zeros(self.H)
        for h in range(self.H):
            z = scale * (K[:, h // G] @ q[h])
            s = float(self.sink[h])
            m = max(z.max(), s)
            e = np.exp(z - m)
            tot = e.sum() + np.exp(s - m)
            out[h] = (e / tot) @ V[:, h // G]
            mag[h] = (e / tot) @ np.abs(V[:, h // G])
            lse[h] = m + np.log(tot)
            dz[h] = 2.0 ** -15 * scale * np.linalg.norm(q[h]) * \
                np.linalg.norm(K[:, h // G], axis=1).max()
        return out, lse, mag, dz

    def check_decode(self, out, lse, window, rows=None, scale=D ** -0.5):
        """out and lse (device tensors) against the formulas, by the roundings on the way.

        The probabilities enter the second product as two bf16 parts (2^-16 of each; fp16,
        2^-11, over e4m3 caches) and carry the score error dz twice (in the weight and in the
        sum); sums and 2^x in 32 bits stay below 2^-18 of the sum of magnitudes; a bf16 out
        adds 2^-8 of its value.
        """
        o, s = to64(out.float()), to64(lse)
        p_step = (2.0 ** -11 if self.e4m3 else 2.0 ** -16) + 2.0 ** -18
        for b in (range(len(self.lens)) if rows is None else rows):
            ro, rl, mag, dz = self.decode64(b, window, scale)
            tol = (p_step + 2 * dz[:, None]) * mag + 1e-30
            if out.dtype == torch.bfloat16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ro)
            err = np.abs(o[b] - ro)
            assert np.all(err <= tol), (b, float(np.max(err / tol)))
            lerr = np.abs(s[b] - rl)
            assert np.all(lerr <= dz + 2.0 ** -21 * (1 + np.abs(rl))), (b, float(np.max(lerr)))

    def check_pool(self, kp, vp, rows=None):
        """The pools (device) hold the new rows in their slots, and all other bits as before.

        A stored key is one rounding of a value in 32 bits, so it is off by half a step of the
        cache's type (bf16 2^-8, e4m3 2^-4; 2^-10 absolute below e4m3's normal range) and the
        32-bit arithmetic's 2^-18 of the row's largest channel; a bf16 value is exact.
        """
        half = 2.0 ** -4 if self.e4m3 else 2.0 ** -8
        tiny = 2.0 ** -10 if self.e4m3 else 1e-38
        got_k, got_v = kp.cpu(), vp.cpu()
        was_k, was_v = self.kp, self.vp
        bits = torch.uint8 if self.e4m3 else torch.int16
        same = torch.ones(got_k.shape[0], self.P, dtype=torch.bool)
        sk, sv = self.scales()
        for b in (range(len(self.lens)) if rows is None else rows):
            n, p = self.new[b], self.lens[b]
            if n == 0:
                continue
            pg, sl = self.slots(b, p, p + n)
            same[torch.as_tensor(pg, dtype=torch.long), torch.as_tensor(sl)] = False
            kn, vn = self.new_rows(b)
            for got, want, s, exact in ((got_k, kn, sk, False), (got_v, vn, sv, not self.e4m3)):
                y = want / s[:, None]
                if self.e4m3:
                    y = np.clip(y, -448, 448)
                x = to64(got[torch.as_tensor(pg, dtype=torch.long), :, torch.as_tensor(sl)].float())
                tol = 0 if exact else half * np.abs(y) + tiny + \
                    2.0 ** -18 * np.abs(y).max(-1, keepdims=True)
                assert np.all(np.abs(x - y) <= tol), (b, float(np.max(np.abs(x - y))))
        for got, was in ((got_k, was_k), (got_v, was_v)):
            a = got.contiguous().view(bits).transpose(1, 2)[same]
            c = was.contiguous().view(bits).transpose(1, 2)[same]
            assert torch.equal(a, c), "a slot that belongs to no new token changed"


def append(fa, w, d, status=None, check=True, **kw):
    fa.paged_append(d["k"], d["v"], d["wk"], d["cu"], d["lens"], d["table"], d["kp"], d["vp"],
                    w.rope, THETA, k_scale=d["ks"], v_scale=d["vs"], status=status,
                    check_status=check, **kw)


def decode(fa, w, d, window=0, check=True, **kw):
    return fa.decode_paged(d["q"], d["k"], d["v"], d["wq"], d["wk"], d["sink"], d["lens"],
                           d["table"], d["kp"], d["vp"], window, w.rope, THETA, k_scale=d["ks"],
                           v_scale=d["vs"], check_status=check, **kw)
