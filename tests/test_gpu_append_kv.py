"""wedlm_append_kv: K/V appended to the paged cache with the rotation on the
way, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from tests.paged_common import PAGE, block_rows, place, rotate, rotate_bound

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, n, nq, nkv, hd, dtype, past, counts, win, norm, pos, seed=0, theta=1e6,
                 spare=2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        T = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        self.B, self.n, self.nq, self.nkv, self.hd = B, n, nq, nkv, hd
        self.theta, self.dtype = theta, dtype
        self.past = [past] * B if isinstance(past, int) else past
        self.counts = counts
        self.cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
        cols = (max(self.past) + n + PAGE - 1) // PAGE + 1
        table = np.full((B, cols), -1, np.int32)
        need = [(p + n + PAGE - 1) // PAGE - p // PAGE for p in self.past]
        ids = rng.permutation(sum(need) + spare)
        at = 0
        for b, p in enumerate(self.past):
            table[b, p // PAGE:p // PAGE + need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.table, self.seq_len = T(table), T(self.past)
        self.pool = rnd(sum(need) + spare, 2, nkv, PAGE * hd)
        # one packed projection row: q heads, k heads, v heads, and a pad that is never read
        self.qkv = rnd(B, n, nq + 2 * nkv + 1, hd)
        self.qkv[:, :, -1] = float("nan")
        self.q = self.qkv[:, :, :nq] if nq else None
        self.k, self.v = self.qkv[:, :, nq:nq + nkv], self.qkv[:, :, nq + nkv:nq + 2 * nkv]
        self.kn = (rnd(hd).float() * 0.1 + 1).to(dtype) if norm else None
        self.qn = (rnd(hd).float() * 0.1 + 1).to(dtype) if norm and nq else None
        self.pos = T(np.stack([p + rng.permutation(n) for p in self.past])) if pos else None
        nan = lambda *s: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        self.wp = (n + PAGE - 1) // PAGE * PAGE
        self.win = nan(B, 2, nkv, self.wp * hd) if win else None
        self.q_out = nan(B * n, nq, hd) if nq else None
        self.new_len = torch.full((B,), -5, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        from serving_wedlm_step_gb300 import binding
        args = dict(counts=self.cnt, pos=self.pos, q=self.q, q_out=self.q_out, kv_win=self.win,
                    k_norm=self.kn, q_norm=self.qn, rope_theta=self.theta,
                    new_seq_len=self.new_len, error=self.err)
        args.update(kw)
        binding.append_kv(self.k, self.v, self.pool, self.table, self.seq_len, **args)

    def check(self, before):
        """Every written value against the formula, everything else untouched."""
        B, n, hd = self.B, self.n, self.hd
        counts = [n] * B if self.counts is None else self.counts
        want, touched = before.clone(), torch.zeros_like(before, dtype=torch.bool)
        bound = torch.zeros(before.shape, dtype=torch.float64, device="cuda")
        want = want.double()
        for b in range(B):
            t = self.pos[b] if self.pos is not None else \
                torch.arange(n, device="cuda") + self.past[b]
            y, mag = rotate(self.k[b], t, self.theta, self.kn)
            tol = rotate_bound(y, mag, self.dtype)
            if self.q_out is not None:
                yq, mq = rotate(self.q[b], t, self.theta, self.qn)
                got = self.q_out[b * n:(b + 1) * n].double()
                assert ((got - yq).abs() <= rotate_bound(yq, mq, self.dtype)).all(), "q_out"
            if self.win is not None:
                got = block_rows(self.win[b], hd)              # [2, nkv, Wp, hd]
                assert ((got[0, :, :n].double() - y.transpose(0, 1)).abs()
                        <= tol.transpose(0, 1)).all(), "window K"
                assert torch.equal(got[1, :, :n], self.v[b].transpose(0, 1)), "window V"
                assert (got[:, :, n:] == 0).all(), "window pad rows"
            for p in range(counts[b]):
                s = self.past[b] + p
                page = int(self.table[b, s // PAGE])
                off = place(s % PAGE, torch.arange(hd, device="cuda"), hd)
                want[page, 0][:, off] = y[p]
                bound[page, 0][:, off] = tol[p]
                want[page, 1][:, off] = self.v[b, p].double()
                touched[page][:, :, off] = True
        got = self.pool.double()
        assert ((got - want).abs() <= bound).all(), "pool"
        assert torch.equal(self.pool[~touched], before[~touched])
        assert self.new_len.tolist() == [p + c for p, c in zip(self.past, counts)]
        assert int(self.err) == 0


BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("B,n,nq,nkv,hd,dtype,past,counts,win,norm,pos", [
    (1, 1, 32, 8, 128, BF, 500, None, True, True, False),     # one token
    (1, 1, 0, 1, 64, FP, 0, None, False, False, False),       # K/V alone, empty cache
    (3, 16, 4, 2, 128, BF, [15, 16, 31], [0, 16, 7], True, True, True),
    (5, 9, 4, 2, 64, FP, [0, 1, 7, 8, 130], [9, 0, 1, 5, 9], True, False, True),
    (2, 64, 5, 5, 64, BF, [3, 1000], [64, 33], True, True, True),   # largest window
    (4, 77, 14, 2, 128, FP, [0, 5, 16, 77], [77, 76, 1, 0], False, True, False),
    (3, 333, 10, 2, 64, BF, 11, None, False, False, False),   # more rows than a window
    (70, 1, 28, 4, 128, BF, list(range(70)), None, True, False, False),
    (2, 2, 3, 1, 128, FP, 131071, None, False, True, False),  # far positions
    (2, 5, 2, 2, 64, FP, [1000003, 1 << 22], None, True, False, True),
])
def test_append_matches_formula(B, n, nq, nkv, hd, dtype, past, counts, win, norm, pos):
    theta = 1e4 if hd == 64 else 1e6
    c = Case(B, n, nq, nkv, hd, dtype, past, counts, win, norm, pos, seed=B * n, theta=theta)
    before = c.pool.clone()
    c.call()
    c.check(before)


def test_head_major_and_offset_rows():
    """k as [B][heads][n][hd] memory, v and q as every second row of larger tensors."""
    c = Case(2, 6, 4, 2, 128, BF, [9, 30], [6, 3], True, True, True, seed=3)
    before = c.pool.clone()
    c.k = c.k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    big = torch.full((2, 12, 4, 136), float("nan"), dtype=BF, device="cuda")
    big[:, 1::2, :2, 8:] = c.v
    c.v = big[:, 1::2, :2, 8:]
    bq = torch.full((2, 12, 5, 128), float("nan"), dtype=BF, device="cuda")
    bq[:, ::2, 1:] = c.q
    c.q = bq[:, ::2, 1:]
    c.call()
    c.check(before)


def test_same_rotation_as_the_step():
    """The far end of a long cache: the K of the step's own QKV epilogue (float64
    angles) and of the append agree to rounding."""
    from serving_wedlm_step_gb300.binding import WedlmContext
    from synth import TINY, make_weights_torch
    s = TINY.replace(qk_norm=True)
    w = make_weights_torch(s, seed=5, norm_jitter=0.2)
    B, W = 2, 8
    ctx = WedlmContext(s, w, window=W, max_batch=B, max_pages_per_seq=4)
    x = torch.randn(B * W, s.hidden, device="cuda")
    pos = (torch.arange(B * W, dtype=torch.int32, device="cuda") + 32000).view(B, W)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = torch.zeros(4, 2, s.n_kv_heads, PAGE * s.head_dim, device="cuda")
    pt = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    win = torch.empty(B, 2, s.n_kv_heads, PAGE * s.head_dim, device="cuda")
    q = torch.empty(B * W, s.n_q_heads * s.head_dim, device="cuda")
    lw = w["layers"][0]
    xn = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s.rms_eps) * lw["attn_norm"]
    rows = torch.cat([xn @ lw[k].T for k in ("w_q", "w_k", "w_v")], 1)
    ctx.layer(0, x, pos, zero, pt, 4, pool, kv_win_out=win, q_out=q)
    torch.cuda.synchronize()
    c = Case(B, W, s.n_q_heads, s.n_kv_heads, s.head_dim, FP, 0, [0] * B, True, False, True)
    h = s.n_q_heads + s.n_kv_heads
    rows = rows.view(B, W, -1, s.head_dim)
    c.q, c.k, c.v = rows[:, :, :s.n_q_heads], rows[:, :, s.n_q_heads:h], rows[:, :, h:]
    c.pos, c.theta, c.kn, c.qn = pos, s.rope_theta, lw["k_norm"], lw["q_norm"]
    c.call()
    torch.testing.assert_close(c.q_out.view(B * W, -1), q, atol=2e-5, rtol=0)
    got, ref = block_rows(c.win, s.head_dim)[..., :W, :], block_rows(win, s.head_dim)[..., :W, :]
    torch.testing.assert_close(got, ref, atol=2e-5, rtol=0)
    ctx.close()


def test_errors_are_reported_and_nothing_else_is_written():
    from serving_wedlm_step_gb300 import binding as Bd
    c = Case(4, 20, 0, 2, 64, FP, [0, 10, 20, 30], [20, 20, 20, 20], False, False, False)
    c.table[1, 0] = c.pool.shape[0]              # sequence 1: rows 0..5 on a bad page
    c.seq_len[2] = -3                            # sequence 2: appends nothing
    c.table = c.table[:, :3].contiguous()        # sequence 3: rows 18, 19 beyond 48 positions
    before = c.pool.clone()
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == Bd.DEV_BAD_PAGE | Bd.DEV_BAD_SEQLEN | Bd.DEV_CAPACITY
    assert c.new_len.tolist() == [20, 30, -3, 48]
    assert torch.isfinite(c.pool).all()
    changed = (c.pool != before).flatten(1).any(1).nonzero().flatten().tolist()
    named = {int(c.table[0, j]) for j in (0, 1)} | {int(c.table[1, 1])} | \
        {int(c.table[3, j]) for j in (1, 2)}
    assert set(changed) == named
    # a count beyond the rows is cut and told
    c = Case(2, 4, 0, 1, 64, FP, 0, [9, -1], False, False, False)
    c.call()
    assert int(c.err) == Bd.DEV_BAD_SEQLEN and c.new_len.tolist() == [4, 0]


def test_captured_and_replayed_on_new_rows():
    c = Case(3, 8, 4, 2, 128, BF, [4, 40, 100], [8, 3, 0], True, True, True, seed=11)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        c.call()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        c.call()
    c.qkv[:, :, :-1].normal_()
    before = c.pool.clone()
    g.replay()
    torch.cuda.synchronize()
    c.check(before)


def test_on_another_stream():
    """The call's stream is the one given: it waits there for what fills its rows."""
    c = Case(4, 40, 8, 2, 128, BF, [0, 3, 16, 100], [40, 1, 0, 33], True, True, False, seed=12)
    before = c.pool.clone()
    rows = c.qkv.clone()
    c.qkv.zero_()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        c.qkv.copy_(rows)
    c.call(stream=st)
    st.synchronize()
    c.check(before)


def test_rows_expanded_over_the_batch():
    """One prompt for all sequences: rows with a batch stride of zero."""
    c = Case(3, 5, 4, 2, 64, FP, [2, 17, 30], [5, 2, 4], True, True, False, seed=13)
    before = c.pool.clone()
    c.k, c.v, c.q = (t[:1].expand(3, -1, -1, -1) for t in (c.k, c.v, c.q))
    c.call()
    c.check(before)


def test_binding_refuses_before_anything_is_enqueued():
    from serving_wedlm_step_gb300 import binding as Bd
    c = Case(2, 4, 4, 2, 64, FP, 0, [4, 4], True, True, False, seed=14)
    before = c.pool.clone()
    bad = [dict(counts=c.cnt.long()), dict(counts=c.cnt[:1]), dict(q=None), dict(q_out=None),
           dict(q=c.q.to(BF)), dict(q_out=c.q_out[:, :, :32]), dict(kv_win=c.win[:1]),
           dict(k_norm=c.kn.cpu()), dict(pos=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
           dict(new_seq_len=c.seq_len), dict(error=torch.zeros(2, dtype=torch.int32).cuda()),
           dict(rope_theta=0.0), dict(rms_eps=float("inf")), dict(q=c.qkv[:, :, :4, 1:])]
    for kw in bad:
        with pytest.raises(Bd.WedlmError) as e:
            c.call(**kw)
        assert e.value.code == Bd.ERR_INVALID_ARG, kw
    k = c.k
    for c.k in (k[:, :, :1], k[..., :48], k[:, :, :, 2:], k.half()):
        with pytest.raises(Bd.WedlmError):
            c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.pool, before)


def test_pages_are_there_for_the_window_attention_behind_it():
    """wedlm_attention reads cached pages before it waits for the kernel in front
    of it: straight behind an append it must still see the appended rows."""
    from serving_wedlm_step_gb300 import binding as Bd
    from synth import make_weights_torch, qwen3_layers
    s = qwen3_layers(1).replace(vocab=256, ffn=128)
    B, n, W = 4, 48, 16
    c = Case(B, n, 0, 8, 128, BF, [0, 5, 16, 40], None, False, False, False, seed=15)
    c.pool.zero_()
    ctx = Bd.WedlmContext(s, make_weights_torch(s, seed=0), window=W, max_batch=B,
                          max_pages_per_seq=c.table.shape[1])
    table = c.table.clamp(min=0)
    q = torch.randn(B * W, 32, 128, device="cuda").to(BF)
    win = torch.randn(B, 2, 8, W * 128, device="cuda").to(BF)
    outs = []
    for i in range(8):
        c.qkv[:, :, :-1].normal_()
        o, ref = (torch.empty(B * W, 32 * 128, dtype=BF, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        c.call()
        ctx.attention(q, c.pool, table, c.new_len, c.pool.shape[0], win, o)
        torch.cuda.synchronize()
        ctx.attention(q, c.pool, table, c.new_len, c.pool.shape[0], win, ref)
        torch.cuda.synchronize()
        assert ctx.status() == 0 and torch.equal(o, ref)
        Bd.shared_prefix_attention(q, c.pool, None, table, c.new_len, win, ref)
        # two bf16 results of one sum, each within 2^-8 of it for P and for the output
        torch.testing.assert_close(o.float(), ref.float(), rtol=0, atol=4 * 2.0 ** -8)
        outs.append(o)
    assert not torch.equal(outs[0], outs[1])
    ctx.close()


def test_pool_beyond_32_bit_offsets():
    """Pages whose first value lies past 2^31 values and 2^32 bytes."""
    c = Case(2, 40, 0, 8, 128, BF, [0, 7], None, False, False, False, seed=2)
    pages = (1 << 31) // (2 * 8 * PAGE * 128) + 64
    small, c.pool = c.pool, torch.empty(pages, 2, 8, PAGE * 128, dtype=BF, device="cuda")
    base = pages - small.shape[0]
    c.pool[base:] = small
    c.table = torch.where(c.table >= 0, c.table + base, c.table)
    whole = c.pool
    c.call()
    c.pool, c.table = whole[base:], torch.where(c.table >= 0, c.table - base, c.table)
    c.check(small)
