"""What the binding of the append and the shared-prefix attention refuses for a
pool's shape and for numbers that the C structs do not hold."""
import pytest
import torch

from tests import test_gpu_append_kv as base
from tests.paged_common import PAGE, AttnCase

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def shapes(pages, nkv, hd):
    """Shapes of a pool of these pages."""
    return [(pages, 2, nkv, PAGE * hd), (pages, 2, nkv, PAGE, hd),
            (pages, 2, nkv, 2, hd // 8, 8, 8), (pages, 2, nkv * PAGE * hd),
            (pages, 32 * nkv * hd), (pages * 32 * nkv * hd,)]


def other_shapes(pages, nkv, hd):
    """Shapes of as many values that say something else."""
    return [(pages // 2, 2, 2 * nkv, PAGE * hd),      # twice the kv heads
            (pages * 2, 2, nkv // 2, PAGE * hd),      # half of them
            (pages // 2, 2, nkv, PAGE * 2 * hd),      # twice the head size
            (pages // 2, 2, nkv, PAGE, 2 * hd),
            (pages, nkv, 2, PAGE * hd),               # heads ahead of K and V
            (2, pages, nkv, PAGE * hd),               # K and V apart
            (pages // 2, 64 * nkv * hd)]


def test_append_takes_a_pool_of_its_own_shape_only():
    from serving_wedlm_step_gb300 import binding as Bd
    for want in shapes(1, 4, 64):
        c = base.Case(2, 4, 0, 4, 64, FP, [0, 20], None, False, False, False, seed=31)
        keep = c.pool[:4].clone()
        c.table.clamp_(max=3)
        c.table[0, 0], c.table[1, 1] = 2, 1
        c.pool = keep
        before = keep.clone()
        c.pool = keep.view(4 * want[0], *want[1:]) if len(want) > 1 else keep.view(-1)
        c.call()
        c.pool = keep
        c.check(before)
    for shape in other_shapes(4, 4, 64):
        c.pool = keep.view(*shape)
        before = keep.clone()
        with pytest.raises(Bd.WedlmError) as e:
            c.call()
        torch.cuda.synchronize()
        assert e.value.code == Bd.ERR_INVALID_ARG and torch.equal(keep, before), shape


def test_attention_takes_a_pool_of_its_own_shape_only():
    from serving_wedlm_step_gb300 import binding as Bd
    c = AttnCase([16 * 3 + 5, 16 * 3], 4, 8, 4, 64, 3, BF, seed=32)
    c.pool = torch.cat([c.pool, c.pool[:c.pool.shape[0] % 2]])  # an even number of pages
    pool, want = c.pool, c.call()
    for shape in shapes(pool.shape[0], 4, 64):
        c.pool = pool.view(*shape)
        assert torch.equal(c.call(), want), shape
    for shape in other_shapes(pool.shape[0], 4, 64):
        c.pool, o = pool.view(*shape), c.out()
        with pytest.raises(Bd.WedlmError) as e:
            c.call(o)
        torch.cuda.synchronize()
        assert e.value.code == Bd.ERR_INVALID_ARG and o.isnan().all(), shape


@pytest.mark.parametrize("bad", [dict(rope_theta=1e39), dict(rms_eps=1e39), dict(rope_theta=-1e39),
                                 dict(rope_theta="1e6"), dict(rms_eps=None)])
def test_numbers_that_32_bits_do_not_hold_are_refused(bad):
    from serving_wedlm_step_gb300 import binding as Bd
    c = base.Case(1, 2, 4, 2, 64, FP, 0, None, True, True, False, seed=33)
    before = c.pool.clone()
    with pytest.raises(Bd.WedlmError) as e:
        c.call(**bad)
    torch.cuda.synchronize()
    assert e.value.code == Bd.ERR_INVALID_ARG and torch.equal(c.pool, before)


def test_sizes_that_32_bits_do_not_hold_are_refused():
    """Rows expanded from one, and a page table of 2^31 columns."""
    from serving_wedlm_step_gb300 import binding as Bd
    c = base.Case(1, 1, 0, 2, 64, FP, 0, None, False, False, False, seed=34)
    c.k, c.v = (t.expand(1, 1 << 31, 2, 64) for t in (c.k, c.v))
    with pytest.raises(Bd.WedlmError) as e:
        c.call()
    assert e.value.code == Bd.ERR_INVALID_ARG
    a = AttnCase([16 * 3 + 5], 4, 4, 2, 64, 3, BF, seed=35)
    a.table = torch.empty(1, 1 << 31, dtype=torch.int32, device="cuda")  # 8 GB, not read
    for kw in (dict(), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(Bd.WedlmError) as e:
            a.call(**kw)
        assert e.value.code == Bd.ERR_INVALID_ARG
