"""Page calls where some arrays of the state are updated in place and others written anew."""
import numpy as np
import pytest
import torch

from tests import pages_common as P
from tests.test_gpu_pages import dev, many, pools, word

pytestmark = pytest.mark.gpu
MIXED = [(a, b, c) for a in (0, 1) for b in (0, 1) for c in (0, 1)]


class Mixed:
    """Table, lengths and counts; fresh[i]: array i has a successor of its own."""

    def __init__(self, state, fresh):
        self.old = [dev(x) for x in state]
        self.keep = [x.clone() for x in self.old]
        self.new = [torch.full_like(x, 12345) if f else x for x, f in zip(self.old, fresh)]
        self.fresh, self.err = fresh, word()

    def kw(self, lens=True):
        names = ("new_page_table", "new_seq_len", "new_page_refs")
        return dict(error=self.err, **{k: v for k, v, f, use in zip(
            names, self.new, self.fresh, (True, lens, True)) if f and use})

    def check(self, table, lens, refs, err):
        torch.cuda.synchronize()
        for x, want in zip(self.new, (table, lens, refs)):
            assert want is None or np.array_equal(x.cpu().numpy(), want)
        for x, k, f in zip(self.old, self.keep, self.fresh):
            assert not f or torch.equal(x, k)
        assert int(self.err) == err


def state(B, cols, spare=0):
    lens, shared, rng = many(B, B + cols, 16 * cols - 40)
    ahead = rng.integers(0, 2, B)
    used = sum(P.up(n) + x for n, x in zip(lens, ahead))
    return P.State(lens, cols, used + spare + 1, shared, ahead, seed=B), rng


# few and many values of a state: copied by the kernel that changes it, or ahead of it
SIZES = [(6, 14), (200, 60), (700, 130)]


@pytest.mark.parametrize("fresh", MIXED)
@pytest.mark.parametrize("B,cols", SIZES)
def test_fork(B, cols, fresh):
    from serving_wedlm_step_gb300 import binding as Bd
    st, rng = state(B, cols)
    n = max(1, B // 2)
    src, dst = rng.integers(-1, B, n).astype(np.int32), rng.permutation(B)[:n].astype(np.int32)
    cut = np.where(src < 0, 0, rng.integers(0, st.lens[src] + 1)).astype(np.int32)
    a = Mixed(st.arrays(), fresh)
    Bd.fork_pages(dev(src), dev(dst), *a.old, lens=dev(cut), **a.kw())
    a.check(*P.fork(*st.arrays(), src, dst, cut))


@pytest.mark.parametrize("fresh", MIXED)
@pytest.mark.parametrize("B,cols", SIZES + [(3, 2500)])
def test_free(B, cols, fresh):
    from serving_wedlm_step_gb300 import binding as Bd
    st, rng = state(B, cols)
    keep = rng.integers(0, 16 * cols + 20, B).astype(np.int32)
    a = Mixed(st.arrays(), fresh)
    Bd.free_pages(dev(keep), *a.old, **a.kw())
    a.check(*P.free(*st.arrays(), keep))
    a = Mixed(st.arrays(), fresh)
    Bd.free_pages(a.old[1], *a.old, **a.kw())  # the lengths themselves
    a.check(*P.free(*st.arrays(), st.lens))


@pytest.mark.parametrize("fresh", [(a, 0, c) for a in (0, 1) for c in (0, 1)])
@pytest.mark.parametrize("B,cols", SIZES)
def test_reserve(B, cols, fresh):
    from serving_wedlm_step_gb300 import binding as Bd
    st, rng = state(B, cols, 2 * B)
    counts = rng.integers(0, 38, B).astype(np.int32)
    a, pool = Mixed(st.arrays(), fresh), pools(2, len(st.refs), 16, 1)
    before = pool.clone()
    Bd.reserve_pages(37, *a.old, pool, counts=dev(counts), **a.kw(lens=False))
    want = P.reserve(*st.arrays(), 37, counts)
    a.check(want[0], st.lens, want[1], want[5])
    for s, d in want[4]:
        before[:, d] = before[:, s]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("fresh", [(a, 0, c) for a in (0, 1) for c in (0, 1)])
@pytest.mark.parametrize("B,cols", SIZES)
def test_compact(B, cols, fresh):
    from serving_wedlm_step_gb300 import binding as Bd
    st, rng = state(B, cols, 500)
    a, pool = Mixed(st.arrays(), fresh), pools(2, len(st.refs), 16, 1)
    before = pool.clone()
    Bd.compact_pages(a.old[0], a.old[2], pool, **a.kw(lens=False))
    want = P.compact(st.table, st.refs)
    a.check(want[0], st.lens, want[1], want[5])
    for s, d in want[4]:
        before[:, d] = before[:, s]
    assert torch.equal(pool, before)
