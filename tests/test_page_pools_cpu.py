"""The binding's reading of the pools' tensors, on host tensors (whose device is -1)."""
import pytest
import torch

HOST = -1


@pytest.fixture(scope="module")
def Bd():
    from serving_wedlm_step_gb300.build import build
    build()
    from serving_wedlm_step_gb300 import binding
    return binding


@pytest.mark.parametrize("layers,pages", [(1, 6), (1, 1), (3, 1), (3, 6)])
def test_page_bytes_follow_the_shape(Bd, layers, pages):
    """Strides of dimensions of one element mean nothing: a pool laid out pages first,
    with one layer, is contiguous whatever its layer stride is."""
    shape, es = (2, 2, 16 * 8), 2
    page = 2 * 2 * 16 * 8 * es
    pool = torch.zeros(layers, pages, *shape, dtype=torch.bfloat16)
    for p in (pool, torch.zeros(pages, layers, *shape, dtype=torch.bfloat16).transpose(0, 1)):
        if not p.is_contiguous():
            with pytest.raises(Bd.WedlmError):
                Bd._page_pools(p, HOST, pages)
            continue
        (n, page_bytes, _, base, step), _ = Bd._page_pools(p, HOST, pages)
        assert (n, page_bytes, base, step) == (layers, page, p.data_ptr(), pages * page)
    (n, page_bytes, _, _, _), _ = Bd._page_pools(list(pool), HOST, pages)
    assert (n, page_bytes) == (layers, page)


@pytest.mark.parametrize("pools", [torch.zeros(2, 0, 64), torch.zeros(0, 0, 64), torch.zeros(0, 4, 64),
                                   torch.zeros(2, 4, 0), [torch.zeros(0, 64)], [torch.zeros(4, 0)], [],
                                   [torch.zeros(4, 64), torch.zeros(0, 64)]])
@pytest.mark.parametrize("N", [0, 4])
def test_empty_pools_are_refused(Bd, pools, N):
    with pytest.raises(Bd.WedlmError) as e:
        Bd._page_pools(pools, HOST, N)
    assert e.value.code == Bd.ERR_INVALID_ARG
