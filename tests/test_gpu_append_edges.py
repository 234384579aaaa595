"""wedlm_append_kv at the edges: rms_eps, pad rows of the window block, positions
past 32 bits, lengths on either side of a page's end."""
import functools

import pytest
import torch

from tests import test_gpu_append_kv as base
from tests.paged_common import PAGE, block_rows, rotate, rotate_bound

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (BF, 64), (FP, 128), (FP, 64)])
@pytest.mark.parametrize("n", [1, 9, 16, 33])
def test_pad_rows_are_zeros_without_an_eps(monkeypatch, dtype, hd, n):
    """A pad row has no mean square to divide by: with rms_eps = 0 it is zeros all
    the same, and the rows are the formula's."""
    monkeypatch.setattr(base, "rotate", functools.partial(rotate, eps=0.0))
    c = base.Case(3, n, 4, 2, hd, dtype, [0, 7, 30], [n, n // 2, 0], True, True, False, seed=n)
    before = c.pool.clone()
    c.call(rms_eps=0.0)
    c.check(before)


@pytest.mark.parametrize("gain", [float("inf"), float("nan")])
def test_pad_rows_are_zeros_whatever_the_gain(gain):
    c = base.Case(2, 5, 4, 2, 128, BF, [3, 20], [5, 2], True, True, False, seed=21)
    c.kn[7] = gain
    c.call()
    assert (block_rows(c.win, 128)[:, :, :, 5:] == 0).all()
    assert torch.isfinite(c.q_out).all()  # the queries have a gain of their own


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("eps,scale", [(0.1, 1.0), (1e-6, 1e-3), (1e-2, 1e-3)])
def test_eps_enters_the_norm(monkeypatch, dtype, hd, eps, scale):
    """Where eps weighs as much as the mean square or more, and rows that are all
    zeros."""
    monkeypatch.setattr(base, "rotate", functools.partial(rotate, eps=eps))
    c = base.Case(3, 9, 4, 2, hd, dtype, [0, 7, 30], [9, 4, 0], True, True, True, seed=22)
    c.qkv[:, :, :-1] *= scale
    c.qkv[0, 2, :-1] = 0
    before = c.pool.clone()
    c.call(rms_eps=eps)
    c.check(before)


def test_positions_past_32_bits():
    """Without `pos` a row's position is seq_len + p, also where that passes 2^31 - 1:
    nothing can be appended there, but the queries are rotated."""
    from serving_wedlm_step_gb300 import binding as Bd
    c = base.Case(2, 3, 4, 2, 128, FP, 0, None, True, False, False, seed=23)
    far = [(1 << 31) - 1, (1 << 31) - 2]
    c.seq_len.copy_(torch.tensor(far, dtype=torch.int32))
    before = c.pool.clone()
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == Bd.DEV_CAPACITY and c.new_len.tolist() == far
    assert torch.equal(c.pool, before)
    for b in range(2):
        t = torch.arange(3, device="cuda") + far[b]
        y, mag = rotate(c.q[b], t, c.theta)
        got = c.q_out[b * 3:(b + 1) * 3].double()
        assert ((got - y).abs() <= rotate_bound(y, mag, FP)).all()
        y, mag = rotate(c.k[b], t, c.theta)
        got = block_rows(c.win[b], 128)[0, :, :3].transpose(0, 1).double()
        assert ((got - y).abs() <= rotate_bound(y, mag, FP)).all()


def test_more_rows_than_a_page_stay_in_their_pages():
    """Lengths on either side of a page's end, one row at a time and many."""
    for n in (1, 2, PAGE, PAGE + 1):
        c = base.Case(4, n, 0, 2, 64, FP, [0, PAGE - 1, PAGE, 2 * PAGE - n % PAGE], None, False,
                      True, False, seed=n)
        before = c.pool.clone()
        c.call()
        c.check(before)
