"""The K/V append and the shared-prefix attention: cases, plain forms and exact values.

`append`: raw q, k, v rows of B sequences (views of one packed projection, as a
user's linear layer leaves them) are normalised per head (optional), rotated at
their positions and written: q to its own tensor, K/V to the window block and
to the pages of the cache.

`attend`: window attention of B sequences of W rows that share their first
16*S positions (one list of S pages), over [shared pages || own pages ||
window rows 0..p].

`own` selects the framework's calls instead of the plain torch forms.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    a = dict(op="append", dtype="bf16", nq=32, nkv=8, hd=128, norm=True, q=True, win=True,
             theta=1000000.0)
    s = dict(op="attend", dtype="bf16", nq=32, nkv=8, hd=128)
    return [
        # one new token of one sequence: what a single decode step appends in each layer
        dict(a, name="append_one_token", batch=1, rows=1, past=500, cut=False),
        # the 32-slot window of 8 sequences at long prefixes; the committed run goes to the pages
        dict(a, name="append_window", batch=8, rows=32, past=32768, cut=True),
        # a small fp32 model (4 query and 2 kv heads of 64), nine rows, no norm
        dict(a, name="append_small_fp32", dtype="fp32", nq=4, nkv=2, hd=64, norm=False,
             theta=10000.0, batch=5, rows=9, past=130, cut=True),
        # K/V of a batch of short prompts, heads of 64, queries handled elsewhere
        dict(a, name="append_prompts_kv_only", nq=10, nkv=4, hd=64, norm=False, q=False,
             win=False, batch=7, rows=333, past=0, cut=True),
        # prompt chunks of 2000 tokens of 16 sequences, each at its own length
        dict(a, name="append_prompt_chunks", win=False, batch=16, rows=2000, past=3000, cut=False),
        # the smallest serving call: two sequences, one token each, a one-page-of-text prompt
        dict(s, name="attend_two_tokens", batch=2, window=1, shared=16, tail=40),
        # plain decoding of 64 requests that share an 8192-token prompt
        dict(s, name="attend_decode_batch", batch=64, window=1, shared=512, tail=1024),
        # the 16-slot window of 8 sequences on a shared prompt of 4096
        dict(s, name="attend_window_16", batch=8, window=16, shared=256, tail=512),
        # the 32-slot window of 8 sequences on a shared prompt of 32768
        dict(s, name="attend_window_32_long", batch=8, window=32, shared=2048, tail=700),
        # the largest: 64 sequences, 32-slot windows, a shared prompt of 16384
        dict(s, name="attend_window_32_wide", batch=64, window=32, shared=1024, tail=2000),
        # heads of 64, five query heads to a kv head, odd batch and window
        dict(s, name="attend_heads_of_64", nq=10, nkv=2, hd=64, batch=13, window=7, shared=77,
             tail=301),
        # a small fp32 model
        dict(s, name="attend_small_fp32", dtype="fp32", nq=4, nkv=2, hd=64, batch=12, window=8,
             shared=128, tail=300),
    ]


_HEADS = [(32, 8, 128), (28, 4, 128), (16, 16, 64), (10, 2, 64), (8, 1, 128), (4, 2, 64),
          (24, 8, 64), (14, 2, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        nq, nkv, hd = rng.choice(_HEADS)
        dtype = "fp32" if rng.random() < 0.25 else "bf16"
        if rng.random() < 0.4:
            c = dict(op="append", dtype=dtype, nq=nq, nkv=nkv, hd=hd, norm=rng.random() < 0.5,
                     theta=rng.choice([10000.0, 500000.0, 1000000.0]), batch=_log(rng, 1, 64),
                     rows=_log(rng, 1, 2000), past=_log(rng, 1, 8000) - 1, cut=rng.random() < 0.5)
            c["q"] = rng.random() < 0.7
            c["win"] = c["rows"] <= 64 and rng.random() < 0.7
            if work(c)["bytes"] <= 4.0e8:
                return c
        else:
            c = dict(op="attend", dtype=dtype, nq=nq, nkv=nkv, hd=hd, batch=_log(rng, 1, 64),
                     window=_log(rng, 1, 64), shared=_log(rng, 1, 1024), tail=_log(rng, 1, 2000))
            if work(c)["flops"] <= (2.0e10 if dtype == "fp32" else 3.0e11):
                return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _torch_dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _lengths(c):
    """Lengths of a case's sequences: a fixed spread over the range the case names, so that
    work() can count them without the inputs."""
    B = c["batch"]
    if c["op"] == "append":
        past = [c["past"] - (c["past"] * 37 * b) // (100 * B) for b in range(B)]
        count = [(c["rows"] * (7 * b + 3)) // (7 * B) if c["cut"] else c["rows"] for b in range(B)]
        return past, [min(n, c["rows"]) for n in count]
    own_len = [(c["tail"] * (B - b)) // B for b in range(B)]
    return own_len, None


def _randn(g, shape, dtype, mul=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat, step = out.view(-1), 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=g, device="cuda") * mul).to(dtype)
    return out


def prepare(case, seed):
    c, dt = case, _torch_dtype(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, nq, nkv, hd = c["batch"], c["nq"], c["nkv"], c["hd"]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    if c["op"] == "append":
        n = c["rows"]
        past, count = _lengths(c)
        # pages that hold the rows written here, and as many others of the same sequences
        cols = max(past) // PAGE + (n + PAGE - 1) // PAGE + 1
        first = [p // PAGE for p in past]
        need = [(p + n + PAGE - 1) // PAGE - f for p, f in zip(past, first)]
        ids = rng.permutation(sum(need)).astype(np.int32)
        table = np.full((B, cols), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, first[b]:first[b] + need[b]] = ids[at:at + need[b]]
            at += need[b]
        qkv = _randn(g, (B, n, nq + 2 * nkv, hd), dt)
        st = dict(case=c, qkv=qkv, q=qkv[:, :, :nq], k=qkv[:, :, nq:nq + nkv],
                  v=qkv[:, :, nq + nkv:], pool=_randn(g, (at, 2, nkv, PAGE * hd), dt),
                  table=dev(table), seq_len=dev(np.array(past, np.int32)),
                  count=dev(np.array(count, np.int32)),
                  new_len=torch.zeros(B, dtype=torch.int32, device="cuda"))
        # the window's rows are reordered: row p of a sequence carries its own position
        pos = np.stack([past[b] + rng.permutation(n) for b in range(B)]).astype(np.int32)
        st["pos"] = dev(pos) if c["win"] else None
        st["k_norm"] = _randn(g, (hd,), dt, 0.1) + 1 if c["norm"] else None
        st["q_norm"] = _randn(g, (hd,), dt, 0.1) + 1 if c["norm"] and c["q"] else None
        st["q_out"] = torch.empty(B * n, nq, hd, dtype=dt, device="cuda") if c["q"] else None
        wp = (n + PAGE - 1) // PAGE * PAGE
        st["win"] = torch.empty(B, 2, nkv, wp * hd, dtype=dt, device="cuda") if c["win"] else None
        return st
    W, S = c["window"], c["shared"]
    tail, _ = _lengths(c)
    cols = S + (max(tail) + PAGE - 1) // PAGE + 1
    need = [(t + PAGE - 1) // PAGE for t in tail]
    ids = rng.permutation(S + sum(need)).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = S
    for b in range(B):
        table[b, :S] = ids[:S]
        table[b, S:S + need[b]] = ids[at:at + need[b]]
        at += need[b]
    wp = (W + PAGE - 1) // PAGE * PAGE
    win = _randn(g, (B, 2, nkv, wp * hd), dt)
    o = torch.empty(B * W, nq * hd, dtype=dt, device="cuda")
    return dict(case=c, q=_randn(g, (B * W, nq, hd), dt), pool=_randn(g, (at, 2, nkv, PAGE * hd), dt),
                shared=dev(ids[:S]), table=dev(table), win=win, o=o,
                seq_len=dev(np.array([PAGE * S + t for t in tail], np.int32)))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if c["op"] == "append":
        return _append_own(state) if own else _append_plain(state)
    return _attend_own(state) if own else _attend_plain(state)


def _append_out(st):
    return {k: st[k] for k in ("pool", "new_len", "q_out", "win") if st[k] is not None}


def _append_own(st):
    from serving_wedlm_step_gb300 import binding
    c = st["case"]
    binding.append_kv(st["k"], st["v"], st["pool"], st["table"], st["seq_len"],
                      counts=st["count"], pos=st["pos"], q=st["q"] if c["q"] else None,
                      q_out=st["q_out"], kv_win=st["win"], k_norm=st["k_norm"],
                      q_norm=st["q_norm"], rms_eps=1e-6, rope_theta=c["theta"],
                      new_seq_len=st["new_len"])
    return _append_out(st)


def _attend_own(st):
    from serving_wedlm_step_gb300 import binding
    return binding.shared_prefix_attention(st["q"], st["pool"], st["shared"], st["table"],
                                           st["seq_len"], st["win"], st["o"])


def _tiles(x):
    """[..., T, hd] rows -> the cache's order of 8x8 tiles: [..., T*hd]."""
    T, hd = x.shape[-2:]
    x = x.reshape(*x.shape[:-2], T // 8, 8, hd // 8, 8)
    return x.transpose(-3, -2).reshape(*x.shape[:-4], T * hd)


def _rows(x, hd):
    """The inverse of _tiles: [..., T*hd] -> [..., T, hd]."""
    T = x.shape[-1] // hd
    x = x.reshape(*x.shape[:-1], T // 8, hd // 8, 8, 8)
    return x.transpose(-3, -2).reshape(*x.shape[:-4], T, hd)


def _norm_rotate(x, gain, cos, sin):
    """Per-head RMS norm (optional) and rotation of [B, n, heads, hd] rows, in 32 bits."""
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.float()
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(st):
    c, dt = st["case"], st["qkv"].dtype
    B, n, hd = c["batch"], c["rows"], c["hd"]
    p = torch.arange(n, device="cuda")
    at = st["seq_len"].long()[:, None] + p  # place in the cache
    t = at if st["pos"] is None else st["pos"].long()
    i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
    ang = t.double()[..., None] * torch.pow(c["theta"], -2.0 * i / hd)
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    k = _norm_rotate(st["k"], st["k_norm"], cos, sin).to(dt)
    v = st["v"]
    if st["q_out"] is not None:
        st["q_out"].copy_(_norm_rotate(st["q"], st["q_norm"], cos, sin).to(dt).view(B * n, -1, hd))
    if st["win"] is not None:
        w = torch.zeros(B, 2, c["nkv"], st["win"].shape[-1] // hd, hd, dtype=dt, device="cuda")
        w[:, 0, :, :n] = k.transpose(1, 2)
        w[:, 1, :, :n] = v.transpose(1, 2)
        st["win"].copy_(_tiles(w))
    b, r = torch.nonzero(p < st["count"][:, None], as_tuple=True)
    s = at[b, r]
    page, s = st["table"][b, s // PAGE].long(), s % PAGE
    pool = st["pool"].view(-1, 2, c["nkv"], 2, hd // 8, 8, 8)  # token group, dim group, token, dim
    pool[page, 0, :, s // 8, :, s % 8] = k[b, r].view(-1, c["nkv"], hd // 8, 8)
    pool[page, 1, :, s // 8, :, s % 8] = v[b, r].view(-1, c["nkv"], hd // 8, 8)
    st["new_len"].copy_(st["seq_len"] + st["count"])
    return _append_out(st)


def _attend_plain(st):
    c = st["case"]
    B, W, nq, nkv, hd, S = (c[k] for k in ("batch", "window", "nq", "nkv", "hd", "shared"))
    G = nq // nkv
    q = st["q"].float().view(B, W, nkv, G, hd) / math.sqrt(hd)
    # the shared pages, one product for all rows
    kv = _rows(st["pool"][st["shared"].long()].float(), hd)  # [S, 2, nkv, 16, hd]
    kv = kv.permute(1, 2, 0, 3, 4).reshape(2, nkv, S * PAGE, hd)
    qs = q.permute(2, 0, 1, 3, 4).reshape(nkv, B * W * G, hd)
    ss = qs @ kv[0].transpose(1, 2)
    ms = ss.amax(-1, keepdim=True)
    ss.sub_(ms).exp_()
    ls, os_ = ss.sum(-1, keepdim=True), ss @ kv[1]
    del ss
    back = lambda x: x.view(nkv, B, W, G, -1).permute(1, 0, 2, 3, 4).reshape(B, nkv, W * G, -1)  # noqa: E731
    ms, ls, os_ = back(ms), back(ls), back(os_)
    # each sequence's own pages and window, padded to the longest
    cols = st["table"][:, S:].long()
    C = cols.shape[1]
    own_len = st["seq_len"].long() - S * PAGE
    kv = _rows(st["pool"][cols.clamp(min=0)].float(), hd)  # [B, C, 2, nkv, 16, hd]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, nkv, C * PAGE, hd)
    win = _rows(st["win"].float(), hd)[..., :W, :].transpose(0, 1)  # [2, B, nkv, W, hd]
    kv = torch.cat([kv, win], 3)
    qp = q.permute(0, 2, 1, 3, 4).reshape(B, nkv, W * G, hd)
    sp = qp @ kv[0].transpose(2, 3)
    r = torch.arange(W, device="cuda")
    see_own = torch.arange(C * PAGE, device="cuda") < own_len[:, None]  # [B, C*16]
    see = torch.cat([see_own[:, None].expand(B, W, -1), (r <= r[:, None]).expand(B, W, W)], 2)
    see = see.repeat_interleave(G, 1)[:, None]
    sp = sp.masked_fill(~see, float("-inf"))
    mp = sp.amax(-1, keepdim=True)
    m = torch.maximum(ms, mp)
    e = (sp - m).exp()
    a = (ms - m).exp()
    o = (os_ * a + e @ kv[1]) / (ls * a + e.sum(-1, keepdim=True))
    o = o.view(B, nkv, W, G, hd).transpose(1, 2).reshape(B * W, nq * hd)
    st["o"].copy_(o.to(st["o"].dtype))
    return st["o"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    B, nq, nkv, hd = c["batch"], c["nq"], c["nkv"], c["hd"]
    if c["op"] == "append":
        n = c["rows"]
        _, count = _lengths(c)
        kv_rows = B * n if c["win"] else sum(count)
        vals = 2 * kv_rows * nkv * hd + 2 * sum(count) * nkv * hd  # read, pages
        flops = 3 * kv_rows * nkv * hd
        if c["win"]:
            vals += 2 * B * ((n + PAGE - 1) // PAGE * PAGE) * nkv * hd
        if c["q"]:
            vals += 2 * B * n * nq * hd
            flops += 3 * B * n * nq * hd
        return {"bytes": vals * es + 4 * (3 * B + sum(count) // PAGE + B + B * n * int(c["win"])),
                "flops": flops}
    W, S = c["window"], c["shared"]
    tail, _ = _lengths(c)
    keys = S * PAGE + sum(tail) + B * W  # read once each
    pairs = sum(W * (S * PAGE + t) + W * (W + 1) // 2 for t in tail) * nq
    return {"bytes": 2 * keys * nkv * hd * es + 2 * B * W * nq * hd * es
            + 4 * (S + B + sum(t // PAGE + 1 for t in tail)), "flops": 4 * hd * pairs}


# ---------------------------------------------------------------------------
# exact values: straight from the definitions, row by row or sequence by sequence, in 64 bits
# ---------------------------------------------------------------------------
def _place(t, d, hd):
    """Place of (token t, dim d) in one page's or window's block of 8x8 tiles."""
    return ((t // 8) * (hd // 8) + d // 8) * 64 + (t % 8) * 8 + d % 8


def exact(case, seed):
    st = prepare(case, seed)
    return _append_exact(st) if case["op"] == "append" else _attend_exact(st)


def _append_exact(st):
    c = st["case"]
    B, n, nq, nkv, hd = (c[k] for k in ("batch", "rows", "nq", "nkv", "hd"))
    h = hd // 2
    lens, counts, table = st["seq_len"].tolist(), st["count"].tolist(), st["table"]
    pool = st["pool"].double()
    win = torch.zeros(st["win"].shape, dtype=torch.float64, device="cuda") if c["win"] else None
    q_out = torch.empty(B * n, nq, hd, dtype=torch.float64, device="cuda") if c["q"] else None
    freq = torch.tensor([c["theta"] ** (-2.0 * i / hd) for i in range(h)], dtype=torch.float64,
                        device="cuda")
    d = torch.arange(hd, device="cuda")
    heads = torch.arange(nkv, device="cuda")

    def turn(x, gain, ang):
        x = x.double()
        if gain is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / hd + 1e-6).sqrt() * gain.double()
        z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(ang), ang)
        return torch.cat([z.real, z.imag], -1)

    for b in range(B):
        t = torch.arange(n, device="cuda") + lens[b] if st["pos"] is None else st["pos"][b]
        ang = (t.double()[:, None] * freq)[:, None]
        kk, vv = turn(st["k"][b], st["k_norm"], ang), st["v"][b].double()
        if c["q"]:
            q_out[b * n:(b + 1) * n] = turn(st["q"][b], st["q_norm"], ang)
        if c["win"]:
            to = _place(torch.arange(n, device="cuda")[:, None], d, hd)  # [n, hd]
            win[b, 0, :, to.reshape(-1)] = kk.permute(1, 0, 2).reshape(nkv, -1)
            win[b, 1, :, to.reshape(-1)] = vv.permute(1, 0, 2).reshape(nkv, -1)
        m = counts[b]
        if m:
            s = torch.arange(m, device="cuda") + lens[b]
            page = table[b][s // PAGE].long()
            to = _place((s % PAGE)[:, None], d, hd)
            pool[page[:, None, None], 0, heads[None, :, None], to[:, None]] = kk[:m]
            pool[page[:, None, None], 1, heads[None, :, None], to[:, None]] = vv[:m]
    out = dict(pool=pool, new_len=None, q_out=q_out, win=win)
    return {k: out[k] for k in _append_out(st)}


def _attend_exact(st):
    c = st["case"]
    B, W, nq, nkv, hd, S = (c[k] for k in ("batch", "window", "nq", "nkv", "hd", "shared"))
    G = nq // nkv
    lens, pool, win = st["seq_len"].tolist(), st["pool"], st["win"]
    out = torch.empty(B * W, nq, hd, dtype=torch.float64, device="cuda")
    to = _place(torch.arange(PAGE, device="cuda")[:, None], torch.arange(hd, device="cuda"), hd)
    to_w = _place(torch.arange(W, device="cuda")[:, None], torch.arange(hd, device="cuda"), hd)
    ahead = torch.ones(W, W, dtype=torch.bool, device="cuda").triu(1)
    for b in range(B):
        L = lens[b]
        page = st["table"][b][:(L + PAGE - 1) // PAGE].long()
        for h in range(nkv):
            k, v = (torch.cat([pool[page, i, h][:, to].reshape(-1, hd)[:L],
                               win[b, i, h][to_w]]).double() for i in (0, 1))
            q = st["q"][b * W:(b + 1) * W, h * G:(h + 1) * G].double().transpose(0, 1)
            s = torch.matmul(q, k.T) * hd ** -0.5  # [G, W, L + W]
            s[:, :, L:][:, ahead] = float("-inf")
            p = torch.softmax(s, -1)
            out[b * W:(b + 1) * W, h * G:(h + 1) * G] = torch.matmul(p, v).transpose(0, 1)
    return out.view(B * W, nq * hd)
