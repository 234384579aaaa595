"""wedlm_verify_drafts behind kernels that rewrite its inputs, over the same memory again and
again: the call takes what the kernel directly in front of it has written."""
import pytest
import torch

from tests.verify_common import Case

pytestmark = pytest.mark.gpu
NAMES = ("logits", "x", "n", "temp", "su", "probs", "au")  # accept_u last, directly in front


def outputs(c):
    return [t.clone() for t in (c.acc, c.tok, c.dp, c.sp)]


@pytest.mark.parametrize("last", ["au", "su", "n", "logits", "temp"])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,K,V,dtype", [(6, 5, 32003, torch.bfloat16), (40, 3, 33000, torch.float32),
                                         (3, 4, 700, torch.bfloat16)])
def test_inputs_rewritten_in_front(B, K, V, dtype, captured, last):
    from serving_wedlm_step_gb300 import binding as Bd
    cases = [Case(B, K, V, dtype, True, seed=40 + s, n_drafts=[(b + s) % (K + 1) for b in range(B)],
                  temps=[(1.0, 0.7, 0.0), (0.5, 1.0), (0.0, 1.3, 0.8, 1.0)][s]) for s in range(3)]
    want = []
    for c in cases:
        c.call()
        c.check()
        want.append(outputs(c))
    live = Case(B, K, V, dtype, True, seed=40, n_drafts=[0] * B)
    live.outputs()
    order = [n for n in NAMES if n != last] + [last]
    turns = [t % 3 for t in (0, 1, 2, 1, 0, 2, 2, 0, 1)] * 4
    results = [[torch.empty_like(w) for w in want[0]] for _ in turns]
    ws = torch.empty(Bd.verify_drafts_workspace(B, K, V, Bd.BF16 if dtype == torch.bfloat16 else Bd.FP32),
                     dtype=torch.uint8, device="cuda")

    def enqueue():
        for i, out in zip(turns, results):
            for n in order:  # kernels, not copies
                torch.mul(getattr(cases[i], n), 1, out=getattr(live, n))
            live.enqueue(workspace=ws)
            for t, r in zip((live.acc, live.tok, live.dp, live.sp), out):
                torch.mul(t, 1, out=r)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            enqueue()
        for _ in range(3):
            graph.replay()
    else:
        enqueue()
    torch.cuda.synchronize()
    for i, out in zip(turns, results):
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
