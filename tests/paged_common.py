"""Plain 64-bit forms of the paged-cache operators (append with rotation,
shared-prefix attention) and the cases their tests run on."""
import math

import numpy as np
import torch

PAGE = 16


def place(t, d, hd):
    """Offset of (token t, dim d) in one block of 8x8 tiles."""
    return ((t // 8) * (hd // 8) + d // 8) * 64 + (t % 8) * 8 + d % 8


def block_rows(x, hd):
    """[..., T*hd] blocks of 8x8 tiles -> [..., T, hd]."""
    T = x.shape[-1] // hd
    t = torch.arange(T, device=x.device)[:, None]
    d = torch.arange(hd, device=x.device)
    return x[..., place(t, d, hd)]


def rotate(x, t, theta, gain=None, eps=1e-6):
    """float64 per-head RMS norm (optional) and rotate-half rotation of
    x [n][heads][hd] at positions t [n].  Returns (y, |a| + |b|): the values and
    the sum of magnitudes each was made of, for error bounds."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    hd = x.shape[-1]
    h = hd // 2
    w = theta ** (-2.0 * torch.arange(h, dtype=torch.float64, device=x.device) / hd)
    ang = (t.double()[:, None] * w)[:, None]
    a, b = x[..., :h], x[..., h:]
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    mag = a.abs() + b.abs()
    return y, torch.cat([mag, mag], -1)


def rotate_bound(y, mag, dtype):
    """Bound on the error of a rotated value: half a step of the stored type,
    plus the 32-bit arithmetic.  The angle is off by at most 2^-25 turns' worth of
    conversion (2 pi 2^-26 < 2^-23 rad), sine and cosine by 2 steps of 2^-23, the
    norm's factor by under 2^-20, and the two products and the sum by 2^-23: in
    all below 2^-19 of |a| + |b|."""
    return torch.finfo(dtype).eps / 2 * (y.abs() + 2.0 ** -19 * mag) + 2.0 ** -19 * mag


class AttnCase:
    """Inputs of one shared-prefix attention call.  lens: cached length of each
    sequence; those of at least 16*S take part in the shared prefix.  Whatever a
    row must not see (page tails, window pad rows, pages nobody names) is NaN or
    infinite."""

    def __init__(self, lens, W, nq, nkv, hd, S, dtype, seed=0, kscale=None, extra_cols=2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.B, self.W, self.nq, self.nkv, self.hd, self.S = B, W, nq, nkv, hd, S
        self.lens, self.dtype = list(lens), dtype
        cols = max((max(lens) + PAGE - 1) // PAGE, 1) + extra_cols
        need = [(n + PAGE - 1) // PAGE - (S if n >= PAGE * S else 0) for n in lens]
        spare = 3
        total = S + sum(need) + spare
        ids = rng.permutation(total).astype(np.int32)
        table = np.full((B, cols), -7, np.int32)  # never read where no key lies
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        pool = rnd(total, 2, nkv, PAGE * hd)
        at = S
        for b, n in enumerate(lens):
            first = S if n >= PAGE * S else 0
            table[b, first:first + need[b]] = ids[at:at + need[b]]
            at += need[b]
            if n % PAGE and need[b]:  # the last page's tail
                off = place(torch.arange(n % PAGE, PAGE)[:, None], torch.arange(hd), hd)
                pool[int(ids[at - 1]), :, :, off.reshape(-1).cuda()] = float("nan")
        pool[torch.from_numpy(ids[at:].astype(np.int64)).cuda()] = float("inf")
        if kscale is not None:  # keys of page j of every list grow
            for row in [ids[:S]] + [table[b][table[b] >= 0] for b in range(B)]:
                for j, p in enumerate(row):
                    pool[int(p), 0] *= kscale(j)
        wp = (W + PAGE - 1) // PAGE * PAGE
        win = rnd(B, 2, nkv, wp * hd)
        if wp > W:
            off = place(torch.arange(W, wp)[:, None], torch.arange(hd), hd).reshape(-1).cuda()
            win[..., off] = float("nan")
        T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.pool, self.win, self.q = pool, win, rnd(B * W, nq, hd)
        self.shared = T(ids[:S]) if S else None
        self.table, self.seq_len = T(table), T(np.array(lens, np.int32))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def out(self):
        return torch.full((self.B * self.W, self.nq * self.hd), float("nan"), dtype=self.dtype,
                          device="cuda")

    def call(self, o=None, **kw):
        from serving_wedlm_step_gb300 import binding
        o = self.out() if o is None else o
        return binding.shared_prefix_attention(self.q, self.pool, self.shared, self.table,
                                               self.seq_len, self.win, o, error=self.err, **kw)

    def keys(self, b):
        """K and V of sequence b's cached positions and window, float64
        [2][L + W][nkv][hd]."""
        n, W, hd = self.lens[b], self.W, self.hd
        pages = self.table[b].clone()
        if self.S and n >= PAGE * self.S:
            pages[:self.S] = self.shared
        pages = pages[:(n + PAGE - 1) // PAGE].long()
        kv = block_rows(self.pool[pages], hd)                 # [P, 2, nkv, 16, hd]
        kv = kv.permute(1, 0, 3, 2, 4).reshape(2, -1, self.nkv, hd)[:, :n]
        win = block_rows(self.win[b], hd)[:, :, :W].transpose(1, 2)
        return torch.cat([kv, win], 1).double()

    def expect(self):
        """(o, bound): the formula in 64 bits and how far a result may be off.

        Rounding of p and of the output: half a step each, the first weighted by
        sum p |v|.  Scores: hd products summed in 32 bits are off by at most
        hd 2^-23 sum |q k| (a tensor core may truncate), which moves p by twice
        that in relative terms (numerator and sum); 2^-18 covers the
        exponential, the scale and the merge.  32-bit sums over n keys add
        n 2^-23 at most."""
        B, W, nq, nkv, hd = self.B, self.W, self.nq, self.nkv, self.hd
        G, sc = nq // nkv, hd ** -0.5
        half = torch.finfo(self.dtype).eps / 2
        o = torch.empty(B * W, nq, hd, dtype=torch.float64, device="cuda")
        bound = torch.empty_like(o)
        later = torch.ones(W, W, dtype=torch.bool, device="cuda").triu(1)
        for b in range(B):
            k, v = self.keys(b)
            n = k.shape[0]
            for h in range(nkv):
                q = self.q[b * W:(b + 1) * W, h * G:(h + 1) * G].double().transpose(0, 1)
                s = q @ k[:, h].T * sc
                mag = q.abs() @ k[:, h].abs().T * sc
                s[:, :, n - W:][:, later] = -math.inf
                mag[:, :, n - W:][:, later] = 0
                p = torch.softmax(s, -1)
                at = (slice(b * W, (b + 1) * W), slice(h * G, (h + 1) * G))
                r, a = p @ v[:, h], p @ v[:, h].abs()
                rel = half + 2 * hd * 2.0 ** -23 * mag.amax(-1, keepdim=True) + 2.0 ** -18 \
                    + n * 2.0 ** -23
                o[at] = r.transpose(0, 1)
                bound[at] = (a * rel + half * r.abs()).transpose(0, 1)
        return o.view(B * W, nq * hd), bound.view(B * W, nq * hd)

    def check(self, o):
        ref, bound = self.expect()
        bad = ~((o.double() - ref).abs() <= bound)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                               o[bad][:4].tolist(), ref[bad][:4].tolist())
