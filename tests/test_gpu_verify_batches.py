"""wedlm_verify_drafts in the forms that decoding batches run in, against its definition in
64 bits: spans of several rounds, clusters of every size, the largest sums of a block, logits
straight from the LM head; and how often tokens come."""
import pytest
import torch

from tests.verify_common import Case, p_bound, rows, weights

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
TEMPS = (1.0, 0.7, 0.0, 1.6)


# On 152 SMs: rounds of a span = rows x ceil(V / 1024 or 512) / 4864, 1 to 5; blocks of a sequence
# 16 for up to 9 sequences, 8 for up to 38, 4 for up to 76, 2 for up to 152, 1 beyond, fewer
# where the vocabulary is small and more where a block's sums would not fit.
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("dtype,B,K,V,pad", [
    (BF, 12, 5, 151936, 0),    # 2 rounds, 8 blocks
    (BF, 12, 8, 151936, 3),    # 3 rounds
    (BF, 11, 13, 151935, 1),   # 4 rounds, rows off any boundary
    (BF, 38, 4, 151936, 0),    # 5 rounds
    (BF, 10, 2, 40001, 7),     # 1 round, 8 blocks
    (BF, 64, 3, 100003, 1),    # 5 rounds, 4 blocks
    (BF, 90, 3, 50257, 2),     # 3 rounds, 2 blocks
    (BF, 160, 3, 20000, 5),    # 2 rounds, 1 block
    (FP, 12, 3, 151936, 0),    # 2 rounds, 8 blocks
    (FP, 12, 5, 151935, 1),    # 4 rounds
    (FP, 38, 2, 100003, 3),    # 4 rounds
    (FP, 64, 2, 50257, 1),     # 3 rounds, 4 blocks
    (FP, 90, 3, 32003, 2),     # 4 rounds, 2 blocks
])
def test_wide_calls(dtype, B, K, V, pad, probs):
    c = Case(B, K, V, dtype, probs, seed=B + K, pad=pad, temps=TEMPS, n_drafts=rows(B, V, K))
    for b in range(B):  # not read
        c.logits[b, int(c.n[b]) + 1:] = float("nan")
    c.call()
    assert len(set(c.check().tolist())) > 1


@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 1])
@pytest.mark.parametrize("dtype,pad", [(BF, 0), (BF, 1), (BF, 9), (FP, 0), (FP, 3)])
def test_the_largest_sums_of_a_block(dtype, V, pad):
    """12 sequences: eight blocks each, with sums of up to 16385 groups."""
    c = Case(12, 0, V, dtype, False, seed=V % 97 + pad, pad=pad, temps=TEMPS, mask_id=-1)
    c.call()
    c.check()


@pytest.mark.parametrize("V,pad", [(98289, 0), (98290, 0), (98297, 1), (98304, 3), (98305, 7), (131071, 1),
                                   (196608, 0), (196609, 1)])
def test_more_sequences_than_places(V, pad):
    """170 sequences: one block each, until its sums would not fit."""
    c = Case(170, 1, V, BF, V % 2 == 1, seed=V % 89, pad=pad, temps=TEMPS)
    c.call()
    c.check()


def test_logits_of_the_lm_head():
    """The framework's own logits, as the LM head leaves them."""
    from serving_wedlm_step_gb300.binding import WedlmContext
    from synth import make_weights_torch, qwen3_layers
    s, B, W = qwen3_layers(1), 12, 8
    ctx = WedlmContext(s, make_weights_torch(s, seed=5, norm_jitter=0.2), window=W, max_batch=B,
                       max_pages_per_seq=4)
    x = torch.randn(B * W, s.hidden, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    recs = torch.empty(B * W, 4, dtype=torch.int32, device="cuda")
    logits = torch.empty(B * W, s.vocab, dtype=FP, device="cuda")
    ctx.lm_head(B, x.to(BF), recs, logits=logits)
    c = Case(B, W - 1, s.vocab, FP, False, seed=7, temps=(0.3, 0.0, 1.0), mask_id=s.mask_id)
    c.logits = logits.view(B, W, s.vocab)
    c.x = recs[:, 0].view(B, W)[:, :W - 1].contiguous()  # the records' tokens as drafts
    c.x[::4, 3] = 17
    c.call()
    acc = c.check()
    assert ctx.status() == 0 and acc[1] == W - 1 and len(set(acc.tolist())) > 1
    ctx.close()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [2, 31, 256])
def test_p_to_a_few_roundings(dtype, V):
    """Rows of one span and one round: eight additions, one rescaling and the quotient, 10 x
    2^-24; the exponentials of the sum, of the rescaling and of the logit, 3 x 2^-22; the
    exponents' roundings as in p_bound."""
    c = Case(30, 4, V, dtype, False, seed=V, spread=0.3, temps=(1.0, 0.8), mask_id=-1)
    c.call()
    c.check()
    for b in range(c.B):
        for i in range(c.K):
            z = c.logits[b, i].float()
            p = weights(z, float(c.temp[b]))
            x = int(c.x[b, i])
            rel = float(p_bound(z, float(c.temp[b]), p)[x]) - 2.0 ** -20 - 100 * 2.0 ** -24
            rel += 10 * 2.0 ** -24 + 3 * 2.0 ** -22
            assert abs(float(c.dp[b, i]) - float(p[x])) <= rel * float(p[x])


@pytest.mark.parametrize("V", [2, 1024, 1 << 17, 1 << 20])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_p_of_equal_logits(dtype, V):
    """Logits of 0: every exponential is 1 and every sum exact."""
    c = Case(3, 1, V, dtype, False, seed=1, temps=(1.0, 0.7, 3.0), mask_id=-1)
    c.logits[:] = 0
    c.call()
    assert (c.dp == 1.0 / V).all() and (c.sp == 1.0 / V).all()


@pytest.mark.parametrize("probs", [False, True])
def test_rare_tokens_come_as_often_as_the_target_has_them(probs):
    """Accepted or replaced: 200000 sequences with one draft, what is rare under the target
    mostly frequent under the drafter.  A count with mean m is off by 6 of its standard deviations
    + 2 with a probability below 10^-6 (by Bernstein's bound, for m >= 30)."""
    n = 200000
    p = torch.tensor([0.3, 0.25, 0.2, 0.1, 0.08, 0.05, 0.0155, 0.003, 0.001, 0.0003, 0.0002], dtype=torch.float64)
    q = torch.tensor([0.05, 0.3, 0.0, 0.02, 0.08, 0.1, 0.2, 0.1, 0.1, 0.05, 0.0], dtype=torch.float64)
    p, q = p / p.sum(), q / q.sum()
    c = Case(n, 1, 12, FP, True, seed=35, temps=(1.0,))
    c.logits[..., :11] = p.log().float().cuda()
    c.logits[..., 11] = 3.0  # the mask token
    c.au = torch.rand(n, 1, generator=torch.Generator(device="cuda").manual_seed(36), device="cuda")
    if probs:
        c.probs = torch.cat([q, q.new_zeros(1)]).float().cuda().expand(n, 1, 12).contiguous()
        c.x = torch.multinomial(q, n, replacement=True,
                                generator=torch.Generator().manual_seed(37)).int().view(n, 1).cuda()
    else:  # certain drafts, whatever they are
        c.probs = None
        c.x = (torch.arange(n, device="cuda") % 11).int().view(n, 1)
    c.call()
    got = torch.bincount(c.tok[:, 0].long(), minlength=12).double().cpu()
    assert int(got[11]) == 0 and int(c.err) == 0
    assert ((got[:11] - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt() + 2).all(), (got[:11], n * p)
