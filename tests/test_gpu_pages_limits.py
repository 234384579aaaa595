"""Calls on a cache's pages at the sizes where their arithmetic could go wrong."""
import pytest
import torch

from tests.test_gpu_pages import word

pytestmark = pytest.mark.gpu


def test_reserve_needs_past_32_bits():
    """32 rows that each need all of 2^26 columns: with the two pages of the row in front the
    needs add up to 2^31 + 2, above any number of pages.  None of the 32 is served, nor the row
    behind them that needs one page; the first row and the one that needs nothing are."""
    from serving_wedlm_step_gb300 import binding as Bd
    cols, B, N, tail = 1 << 26, 35, 64, 4096
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, cols), -1, **i32)
    lens, refs, granted, left, err = torch.zeros(B, **i32), torch.zeros(N, **i32), torch.full((B,), -9, **i32), word(), word()
    refs[3] = 1  # pinned
    counts = torch.full((B,), 16 * cols, **i32)
    counts[0], counts[33], counts[34] = 20, 1, 0
    pool = torch.randn(2, N, 8, device="cuda")
    before = pool.clone()
    n = Bd.reserve_pages_workspace(B, cols, N, 2, 32, 16 * cols)
    ws = torch.full((n + tail,), 77, dtype=torch.uint8, device="cuda")
    Bd.reserve_pages(16 * cols, table, lens, refs, pool, counts=counts, granted=granted, n_free=left,
                     error=err, workspace=ws)
    torch.cuda.synchronize()
    assert granted.tolist() == [1] + [0] * 33 + [1]
    assert int(err) == Bd.DEV_CAPACITY and int(left) == 61
    assert refs.tolist() == [1, 1, 0, 1] + [0] * 60
    assert table[0, :3].tolist() == [0, 1, -1]
    table[0, :2] = -1
    assert all(int(table[b].max()) == -1 == int(table[b].min()) for b in range(B))
    assert torch.equal(pool, before) and (ws[n:] == 77).all()
