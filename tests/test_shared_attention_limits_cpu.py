"""The sizes that wedlm_shared_attention takes, at the ends of its two limits."""
import pytest


@pytest.fixture(scope="module")
def Bd():
    from serving_wedlm_step_gb300.build import build
    build()
    from serving_wedlm_step_gb300 import binding
    return binding


def takes(Bd, batch, window, nq, nkv, hd, dtype, pages, shared=0):
    try:
        return Bd.shared_prefix_workspace(batch, window, nq, nkv, hd, dtype, pages, shared) > 0
    except Bd.WedlmError as e:
        assert e.code == Bd.ERR_INVALID_ARG
        return False


def test_tiles_of_full_tables_stay_below_2_to_31(Bd):
    # 1024 sequences of one token, 16 kv heads: 4 shared units and 1024 private ones a
    # head; 16 * (4 * (1 + 0) + 1024 * (1 + T)) < 2^31 for T = 131070, not 131071
    a = (1024, 1, 16, 16, 64, Bd.BF16)
    assert takes(Bd, *a, 131070 * 8 - 1)
    assert not takes(Bd, *a, 131070 * 8)
    # with 64 shared pages, 4 * (1 + 8) a head
    assert takes(Bd, *a, 131070 * 8 - 1, 64)
    # fp32: units of 64 rows; 16 * (16 + 1024 * (1 + T)), the same T
    f = (1024, 1, 16, 16, 64, Bd.FP32)
    assert takes(Bd, *f, 131070 * 8 - 1)
    assert not takes(Bd, *f, 131070 * 8)
    # the shared range alone: 8 kv heads, 64 units a head (1024 x 16 rows): 2^26 shared
    # pages are 2^23 tiles, and 8 * 64 * 2^23 passes 2^31
    assert not takes(Bd, 1024, 16, 8, 8, 64, Bd.BF16, 8, 1 << 26)
    assert takes(Bd, 1024, 16, 8, 8, 64, Bd.BF16, 8, 1 << 24)


def test_units_stay_within_2_to_24(Bd):
    # 32 q heads to a kv head: 256 rows a unit, 8 units a window of 64, 8192 of the batch;
    # 1024 * (8192 + 1024 * 8) = 2^24
    assert takes(Bd, 1024, 64, 32 * 1024, 1024, 64, Bd.BF16, 1)
    # 33: 6 tokens (198 rows) a unit, 11 a window
    assert not takes(Bd, 1024, 64, 33 * 1024, 1024, 64, Bd.BF16, 1)
    # fp32, 64 rows a unit: 8 q heads to a kv head reach it, 9 pass it
    assert takes(Bd, 1024, 64, 8 * 1024, 1024, 64, Bd.FP32, 1)
    assert not takes(Bd, 1024, 64, 9 * 1024, 1024, 64, Bd.FP32, 1)
