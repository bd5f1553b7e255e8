"""What the operators on the paged cache ask of the cache's handle (no GPU
needed): at least one page where new tokens attend to it, and the device that
its tensors are on.  Addresses are never dereferenced."""
import pytest
import torch

import test_layer_abi as abi
from bit_weight_delta_bd_gb300 import bitdelta as bd


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return bd.load()


# ------------------------------------------------------------------------------- a cache without pages

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [1, 4096])
@pytest.mark.parametrize("pages", [abi.pages, abi.pages8])
def test_attention_refuses_a_cache_without_pages(lib, pages, max_new, dim):
    """There is no page that could stand in for a bad one, and no array for a tensor map to describe."""
    call = dict(qs=4 * dim, max_new=max_new)
    assert abi.attention(lib, cache=pages(n_pages=0, dim=dim), **call) == bd.BD_ERR_UNSUPPORTED_SHAPE
    assert abi.attention(lib, cache=pages(n_pages=0, dim=dim), T=0, **call) == bd.BD_OK
    assert abi.attention(lib, cache=pages(n_pages=0, dim=dim), n_seq=0, **call) == bd.BD_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a usable GPU")
@pytest.mark.parametrize("entry", [abi.rope, abi.read])
def test_append_and_read_take_a_cache_without_pages(lib, entry):
    """Slots of -1 write nothing, and rows of pages that do not exist are zeros: both look before they access.  (A call
    that passes every check reaches the CUDA runtime, which fails here.)"""
    assert entry(lib, cache=abi.pages(n_pages=0)) == bd.BD_ERR_CUDA
