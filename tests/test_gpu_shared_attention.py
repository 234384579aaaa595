"""wedlm_shared_attention: window attention over a shared prefix, each
sequence's own pages and the window, against the formula in 64 bits."""
import pytest
import torch

from tests.paged_common import PAGE, AttnCase, block_rows, rotate

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("S,own,W,nq,nkv,hd", [
    (0, [0], 1, 1, 1, 64),                      # nothing cached at all
    (0, [0, 1, 15, 16, 17, 200], 5, 4, 2, 128),  # nothing shared
    (1, [0, 0], 1, 32, 8, 128),                 # shared only, single tokens
    (3, [0, 1, 16, 40], 16, 8, 2, 128),
    (8, [0, 128, 127, 129], 1, 8, 1, 64),       # whole tiles and their neighbours
    (9, [5] * 13, 7, 10, 2, 64),                # five q heads to a kv head
    (17, [0, 300, 33], 33, 14, 2, 128),         # seven; windows of three pages
    (30, [100, 0], 64, 8, 2, 128),              # two row blocks in a window
    (12, [64, 3, 250], 64, 16, 16, 64),         # one q head to a kv head
    (5, [20] * 40, 1, 8, 8, 64),                # more units than blocks
    (64, [900, 0, 10], 2, 128, 1, 128),         # 128 q heads to a kv head
    (40, [700, 77], 40, 36, 4, 128),            # 360 rows a window
])
def test_matches_formula(dtype, S, own, W, nq, nkv, hd):
    lens = [PAGE * S + n for n in own]
    c = AttnCase(lens, W, nq, nkv, hd, S, dtype, seed=S + W)
    o = c.call()
    c.check(o)
    assert int(c.err) == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("S,own,W", [(3, [0, 0], 1), (40, [0, 300], 1), (9, [0, 20], 40)])
def test_a_visible_nan_is_not_lost_with_its_range(dtype, S, own, W):
    """The one key of its own that a row sees is NaN, the shared ones are finite: the
    row is NaN, the other sequences are what they were."""
    c = AttnCase([PAGE * S + n for n in own], W, 8, 2, 128, S, dtype, seed=S)
    before = c.call()
    c.win[0, 0, 1, :8] = float("nan")  # 8 dims of K of the first window row, kv head 1
    o = c.call().view(len(own), W, 8, 128)
    assert o[0, :, 4:].isnan().all()
    old = before.view(len(own), W, 8, 128)
    assert torch.equal(o[0, :, :4], old[0, :, :4]) and torch.equal(o[1:], old[1:])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("W,lens", [
    (1, [0, 160, 159, 1, 500, 0]),    # padded slots and sequences shorter than the prefix
    (16, [0, 0, 0]),                  # nobody takes part
    (33, [161, 2, 170, 100]),
])
def test_sequences_shorter_than_the_prefix(dtype, W, lens):
    c = AttnCase(lens, W, 8, 2, 128, 10, dtype, seed=W)
    c.check(c.call())
    assert int(c.err) == 0


@pytest.mark.parametrize("dtype", [BF, FP])
def test_growing_scores(dtype):
    """Keys grow page by page: row maxima keep rising along every range."""
    c = AttnCase([16 * 60 + 700, 16 * 60 + 90, 300], 9, 8, 2, 128, 60, dtype, seed=4,
                 kscale=lambda j: 1.0 + 0.25 * (j % 32))
    c.check(c.call())


def test_shrinking_scores_keep_the_first_maximum():
    c = AttnCase([16 * 70 + 40, 16 * 70], 4, 8, 2, 128, 70, BF, seed=5,
                 kscale=lambda j: 8.0 / (1 + j))
    c.check(c.call())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_row_blocks_and_long_ranges(dtype):
    """Several shared row blocks per kv head, each cut over many blocks of the grid."""
    B, W = (24, 16) if dtype == BF else (6, 16)
    c = AttnCase([16 * 130 + 37 * b for b in range(B)], W, 8, 2, 128, 130, dtype, seed=6)
    c.check(c.call())


@pytest.mark.parametrize("B,own", [(300, 5), (500, 0), (200, 130)])
def test_many_short_private_units_behind_shared_ones(B, own):
    """Blocks that go from long shared segments to a run of one- and two-tile
    private ones."""
    c = AttnCase([16 * 40 + own] * B, 1, 8, 2, 128, 40, BF, seed=B)
    c.check(c.call())


def test_batch_of_1024_single_tokens():
    c = AttnCase([16 * 4 + (b % 40) for b in range(1024)], 1, 4, 1, 64, 4, BF, seed=7)
    c.check(c.call())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_repeated_calls_are_bit_identical_whatever_the_workspace_held(dtype):
    from serving_wedlm_step_gb300 import binding as Bd
    c = AttnCase([16 * 33 + 20 * b for b in range(9)], 12, 8, 2, 128, 33, dtype, seed=8)
    need = Bd.shared_prefix_workspace(9, 12, 8, 2, 128, Bd.BF16 if dtype == BF else Bd.FP32,
                                      c.table.shape[1], 33)
    a = c.call()
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(a, c.call(workspace=ws))


def test_agrees_with_the_window_attention():
    """The same call through wedlm_attention, every sequence on its own pages."""
    from serving_wedlm_step_gb300.binding import WedlmContext
    from synth import make_weights_torch, qwen3_layers
    s = qwen3_layers(1).replace(vocab=256, ffn=128)
    B, W, S = 4, 16, 20
    c = AttnCase([16 * S + n for n in (0, 33, 64, 100)], W, 32, 8, 128, S, BF, seed=9)
    c.pool.nan_to_num_(0, 0, 0)
    c.win.nan_to_num_(0, 0, 0)
    table = c.table.clone()
    table[:, :S] = c.shared
    table.clamp_(min=0)
    ctx = WedlmContext(s, make_weights_torch(s, seed=0), window=W, max_batch=B,
                       max_pages_per_seq=table.shape[1])
    ref = c.out()
    ctx.attention(c.q, c.pool, table, c.seq_len, c.pool.shape[0], c.win, ref)
    o = c.call()
    torch.cuda.synchronize()
    assert ctx.status() == 0
    _, bound = c.expect()
    assert ((o.double() - ref.double()).abs() <= 2 * bound).all()
    ctx.close()


def test_bad_pages_and_lengths_are_reported():
    from serving_wedlm_step_gb300 import binding as Bd
    S = 6
    c = AttnCase([16 * S + 50, 16 * S + 50, 16 * S], 8, 8, 2, 128, S, BF, seed=10)
    good = c.call().clone()
    c.table[1, S + 1] = c.pool.shape[0] + 9   # sequence 1's own page
    o = c.call()
    assert int(c.err) == Bd.DEV_BAD_PAGE
    assert torch.isfinite(o).all()
    per = 8
    assert torch.equal(o[:per], good[:per]) and torch.equal(o[2 * per:], good[2 * per:])
    c.err.zero_()
    c.seq_len[1] = -1                         # counts as 0
    o = c.call()
    assert int(c.err) == Bd.DEV_BAD_SEQLEN and torch.isfinite(o).all()
    c.err.zero_()
    c.seq_len[1] = 16 * c.table.shape[1] + 1  # beyond the table: cut to it
    c.table[1, S:] = 0
    c.pool.nan_to_num_(0, 0, 0)
    o = c.call()
    assert int(c.err) == Bd.DEV_CAPACITY and torch.isfinite(o).all()
    c.err.zero_()
    c.shared[2] = -1                          # a shared page
    o = c.call()
    assert int(c.err) & Bd.DEV_BAD_PAGE and torch.isfinite(o).all()


def test_binding_refuses_before_anything_is_enqueued():
    from serving_wedlm_step_gb300 import binding as Bd
    c = AttnCase([16 * 3 + 5, 16 * 3], 4, 4, 2, 64, 3, BF, seed=17)
    o = c.out()

    def refused(code=Bd.ERR_INVALID_ARG, **kw):
        args = dict(q=c.q, pool=c.pool, shared_pages=c.shared, page_table=c.table,
                    seq_len=c.seq_len, kv_win=c.win, o=o)
        args.update(kw)
        with pytest.raises(Bd.WedlmError) as e:
            Bd.shared_prefix_attention(**args)
        assert e.value.code == code, kw

    refused(q=c.q.float())
    refused(q=c.q[:, :3].contiguous())
    refused(q=c.q[1:])
    refused(q=c.q.transpose(0, 1).contiguous().transpose(0, 1))
    refused(pool=c.pool[:, :, :, 1:])
    refused(pool=c.pool.view(-1)[8:])
    refused(shared_pages=c.shared.long())
    refused(shared_pages=c.shared.cpu())
    refused(page_table=c.table[:1])
    refused(page_table=c.table[:, ::2])
    refused(seq_len=c.seq_len.long())
    refused(kv_win=c.win[:, :, :, 16:])
    refused(o=o[:, :64])
    refused(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), code=Bd.ERR_CAPACITY)
    refused(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    torch.cuda.synchronize()
    assert torch.isnan(o).all()


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    a = AttnCase([16 * 80 + 100] * 8, 8, 8, 2, 128, 80, BF, seed=12)
    b = AttnCase([16 * 40 + 300] * 12, 4, 16, 4, 64, 40, BF, seed=13)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [a.out() for _ in range(6)], [b.out() for _ in range(6)]
    torch.cuda.synchronize()
    for x, y in zip(oa, ob):
        a.call(x, stream=s1)
        b.call(y, stream=s2)
    torch.cuda.synchronize()
    a.check(oa[0])
    b.check(ob[0])
    assert all(torch.equal(oa[0], x) for x in oa) and all(torch.equal(ob[0], y) for y in ob)


def test_captured_and_replayed_on_new_contents():
    c = AttnCase([16 * 20 + 30 * b for b in range(6)], 8, 8, 2, 128, 20, BF, seed=14)
    o = c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(o)
    d = AttnCase([16 * 20 + 30 * b for b in (5, 4, 3, 2, 1, 0)], 8, 8, 2, 128, 20, BF, seed=15)
    for name in ("q", "win", "seq_len", "shared"):
        getattr(c, name).copy_(getattr(d, name))
    c.pool[:d.pool.shape[0]] = d.pool[:c.pool.shape[0]]
    c.table.fill_(-1)
    c.table[:, :d.table.shape[1]] = d.table[:, :c.table.shape[1]]
    c.lens = d.lens
    g.replay()
    torch.cuda.synchronize()
    c.check(o)


def test_pool_beyond_32_bit_offsets():
    c = AttnCase([16 * 4 + 100, 16 * 4 + 3], 16, 32, 8, 128, 4, BF, seed=16)
    pages = (1 << 31) // (2 * 8 * PAGE * 128) + 64
    small, c.pool = c.pool, torch.empty(pages, 2, 8, PAGE * 128, dtype=BF, device="cuda")
    base = pages - small.shape[0]
    c.pool[base:] = small
    c.shared += base
    c.table = torch.where(c.table >= 0, c.table + base, c.table)
    c.check(c.call())


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (FP, 64)])
def test_append_then_attend(dtype, hd):
    """The two together over three steps, as a decode loop uses them: the window's
    projections are rotated into the window block, the observed run is appended
    to the pages, the attention reads [shared || own pages || window], and the
    next step starts from the new lengths."""
    from serving_wedlm_step_gb300 import binding as Bd
    S, W, nq, nkv, theta = 5, 6, 8, 2, 1e6
    lens = [16 * S, 16 * S + 9, 16 * S + 31]
    B = len(lens)
    c = AttnCase(lens, W, nq, nkv, hd, S, dtype, seed=20, extra_cols=3)
    table = c.table.clone()
    first = [(n + 15) // 16 for n in lens]   # a fresh page at the end of every row
    c.pool = torch.cat([c.pool, torch.full((3 * B, *c.pool.shape[1:]), float("nan"), dtype=dtype,
                                           device="cuda")])
    n0 = c.pool.shape[0] - 3 * B
    for b in range(B):
        for j in range(2):
            table[b, first[b] + j] = n0 + 3 * b + j
    c.table = table
    lens_dev, new_len = c.seq_len, torch.empty_like(c.seq_len)
    q_out = torch.empty(B * W, nq, hd, dtype=dtype, device="cuda")
    gain = torch.rand(hd, device="cuda").to(dtype) + 0.5
    err = c.err
    for step, counts in enumerate([[2, 0, 6], [1, 3, 0], [6, 6, 6]]):
        qkv = torch.randn(B, W, nq + 2 * nkv, hd, device="cuda").to(dtype)
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        Bd.append_kv(qkv[:, :, nq:nq + nkv], qkv[:, :, nq + nkv:], c.pool, c.table, lens_dev,
                     counts=cnt, q=qkv[:, :, :nq], q_out=q_out, kv_win=c.win, k_norm=gain,
                     q_norm=gain, rope_theta=theta, new_seq_len=new_len, error=err)
        c.q, c.seq_len = q_out, lens_dev
        o = c.call()
        c.check(o)
        # what the window block and q hold is what the formula says
        for b in range(B):
            t = torch.arange(W, device="cuda") + c.lens[b]
            y, _ = rotate(qkv[b, :, nq:nq + nkv], t, theta, gain)
            got = block_rows(c.win[b], hd)[0, :, :W].transpose(0, 1)
            torch.testing.assert_close(got.double(), y, rtol=torch.finfo(dtype).eps, atol=1e-4)
        c.lens = [n + k for n, k in zip(c.lens, counts)]
        lens_dev, new_len = new_len, lens_dev
        assert lens_dev.tolist() == c.lens
    assert int(err) == 0
