"""wedlm_shared_attention where the page tables are so wide that the split counts
every tile and every unit's ends as 1."""
import pytest
import torch

from tests.paged_common import AttnCase

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,W,nq,nkv,hd,S,own,cols", [
    # 32 units of 256 rows a sequence, 1.25M tiles a full table: above 2^31 at 28 a tile
    (BF, 64, 128, 1, 64, 9, [5, 300], 10_000_000),
    (BF, 64, 128, 1, 128, 0, [130, 0], 10_000_000),
    # single tokens of 64 sequences with 8 kv heads, 16 a tile
    (BF, 1, 32, 8, 128, 20, [40 * (b % 7) for b in range(64)], 2_200_000),
    # 128 units of 64 rows a sequence, at 4 a tile
    (FP, 64, 128, 1, 64, 9, [5, 300], 17_000_000),
    (FP, 64, 128, 1, 128, 3, [0, 129], 17_000_000),
])
def test_matches_formula(dtype, W, nq, nkv, hd, S, own, cols):
    B = len(own)
    # weight of full tables as the split first counts it: it must not fit
    rows = W * nq // nkv
    tile = (28 if W * nq // nkv > 128 else 16) if dtype == BF else (4 if rows > 16 else 2)
    units = (rows + 255) // 256 if dtype == BF else (rows + 63) // 64
    assert nkv * B * units * (cols // 8) * tile > 1 << 31
    c = AttnCase([16 * S + n for n in own], W, nq, nkv, hd, S, dtype, seed=S, extra_cols=cols)
    o = c.call()
    c.check(o)
    assert int(c.err) == 0
    assert torch.equal(o, c.call())
