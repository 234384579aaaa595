"""Arrays of a call that lie in the pools it writes are refused.  No call here reaches a
kernel: the workspace is stated too small, which is looked at last."""
import ctypes

import pytest

from tests.test_pages_cpu import A, Bd, call, make  # noqa: F401 (Bd is a fixture)

POOL = 40 * 4096  # bytes of each of the two pools of make(), at 64 A and 65 A
ARRAYS = {"reserve": ("page_table", "seq_len", "page_refs", "new_page_table", "new_page_refs", "error",
                      "counts", "granted", "n_free", "workspace"),
          "compact": ("page_table", "page_refs", "new_page_table", "new_page_refs", "error", "page_map",
                      "n_live", "workspace")}
FORMS = (dict(), dict(kv_pools=None, base=64 * A, layer_stride=A))


@pytest.mark.parametrize("pools", FORMS)
@pytest.mark.parametrize("op,name", [(op, n) for op in ARRAYS for n in ARRAYS[op]])
def test_arrays_in_a_pool_are_refused(Bd, op, name, pools):  # noqa: F811
    end = 4 if name != "workspace" else 256
    for at in (64 * A, 65 * A, 65 * A + 4096, 65 * A + POOL - end):
        assert call(Bd, op, make(Bd, op, **{name: at}, workspace_bytes=0, **pools)) == Bd.ERR_INVALID_ARG, at


@pytest.mark.parametrize("pools", FORMS)
@pytest.mark.parametrize("op", ARRAYS)
def test_arrays_beside_and_between_the_pools_are_taken(Bd, op, pools):  # noqa: F811
    for name in ARRAYS[op]:
        for at in (64 * A + POOL, 65 * A - 65536, 65 * A + POOL):
            args = make(Bd, op, **{name: at}, workspace_bytes=0, **pools)
            assert call(Bd, op, args) == Bd.ERR_CAPACITY, (name, at)


def test_a_shared_pool_is_taken(Bd):  # noqa: F811
    """Two layers that share a pool: its pages are copied alike for both."""
    same = (ctypes.c_void_p * 2)(64 * A, 64 * A)
    for pools in (dict(kv_pools=same), dict(kv_pools=None, base=64 * A, layer_stride=0)):
        assert call(Bd, "compact", make(Bd, "compact", workspace_bytes=0, **pools)) == Bd.ERR_CAPACITY


@pytest.mark.parametrize("op", ARRAYS)
def test_pools_over_one_another_are_refused(Bd, op):  # noqa: F811
    """A page of one layer that is part of others of another layer: copies would race."""
    for off in (16, 4096, POOL - 16):
        for parts in ((64 * A, 64 * A + off), (64 * A + off, 64 * A)):
            for pools in (dict(kv_pools=(ctypes.c_void_p * 2)(*parts)),
                          dict(n_layers=3, kv_pools=(ctypes.c_void_p * 3)(parts[0], 66 * A, parts[1])),
                          dict(kv_pools=None, base=64 * A, layer_stride=off)):
                assert call(Bd, op, make(Bd, op, workspace_bytes=0, **pools)) == Bd.ERR_INVALID_ARG
    for pools in (dict(kv_pools=(ctypes.c_void_p * 2)(64 * A, 64 * A + POOL)),
                  dict(kv_pools=None, base=64 * A, layer_stride=POOL),
                  dict(n_layers=1, kv_pools=None, base=64 * A, layer_stride=16)):
        assert call(Bd, op, make(Bd, op, workspace_bytes=0, **pools)) == Bd.ERR_CAPACITY
