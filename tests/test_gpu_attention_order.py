"""wedlm_attention straight behind a kernel that writes what it reads."""
import pytest
import torch

from tests.paged_common import AttnCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_pages_of_the_kernel_in_front(captured):
    """The merge of wedlm_shared_attention lets the next kernel start before it has
    written its output.  That output taken as the pages (120 of them), the lengths
    copied by a kernel of torch's: wedlm_attention sees both whole."""
    from serving_wedlm_step_gb300 import binding as Bd
    from synth import make_weights_torch, qwen3_layers
    bf = torch.bfloat16
    s = qwen3_layers(1).replace(vocab=256, ffn=128)
    B, W, per = 4, 16, 30
    ctx = Bd.WedlmContext(s, make_weights_torch(s, seed=0), window=W, max_batch=B,
                          max_pages_per_seq=per)
    c = AttnCase([16] * 60, 16, 32, 8, 128, 1, bf, seed=41)  # 960 rows of 32 heads
    pages = torch.empty(960, 32 * 128, dtype=bf, device="cuda")
    pool = pages.view(B * per, 2, 8, 16 * 128)
    table = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    lens = torch.tensor([16 * per, 16 * per - 5, 100, 0], dtype=torch.int32, device="cuda")
    now = torch.zeros_like(lens)
    q = torch.randn(B * W, 32, 128, device="cuda").to(bf)
    win = torch.randn(B, 2, 8, W * 128, device="cuda").to(bf)
    o, ref = (torch.empty(B * W, 32 * 128, dtype=bf, device="cuda") for _ in range(2))
    ws = torch.empty(Bd.shared_prefix_workspace(60, 16, 32, 8, 128, Bd.BF16, c.table.shape[1], 1),
                     dtype=torch.uint8, device="cuda")

    def run():
        now.copy_(lens)
        c.call(pages, workspace=ws)
        ctx.attention(q, pool, table, now, B * per, win, o)

    replay = run
    if captured:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        replay = g.replay
    outs = []
    for i in range(12):
        c.q.normal_()
        c.pool[c.shared.long()] = torch.randn_like(c.pool[c.shared.long()])
        pages.zero_()
        now.zero_()
        torch.cuda.synchronize()
        replay()
        torch.cuda.synchronize()
        ctx.attention(q, pool, table, now, B * per, win, ref)
        torch.cuda.synchronize()
        assert ctx.status() == 0 and int(c.err) == 0 and torch.equal(o, ref), i
        outs.append(o.clone())
    assert not torch.equal(outs[0], outs[1])
    ctx.close()
