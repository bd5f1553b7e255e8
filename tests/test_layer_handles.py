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


# ------------------------------------------------------------------------------- a cache of another device

class OnDevice:
    """A tensor as far as the binding's checks look at one: its device, shape, type and an address."""
    is_cuda = True

    def __init__(self, index, *shape, dtype=torch.bfloat16):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), dtype

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return abi.at(self.device.index)


class Library:
    """Accepts every call and notes down its name."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            return bd.BD_OK
        return call


@pytest.mark.parametrize("made,used", [(0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("entry", ["append", "read", "attention"])
def test_a_cache_is_used_on_its_own_device(monkeypatch, entry, made, used):
    device, library = [made], Library()
    monkeypatch.setattr(bd, "_device", lambda: device[0])
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device[0])
    monkeypatch.setattr(bd, "load", lambda *path: library)
    cache = bd.KvPages(OnDevice(made, 10, 2, 16, 64), OnDevice(made, 10, 2, 16, 64))
    device[0] = used
    heads, ints = lambda n: OnDevice(used, 3, n, 64), lambda *n: OnDevice(used, *n, dtype=torch.int32)  # noqa: E731
    ws = OnDevice(used, 4096, dtype=torch.uint8)
    calls = {
        "append": lambda: bd.bd_rope_append(heads(4), heads(2), heads(2), None, None, ints(3), cache, heads(4), ws),
        "read": lambda: bd.bd_kv_read(cache, ints(1, 4), ints(2), heads(2), heads(2), ws),
        "attention": lambda: bd.bd_attention(heads(4), ints(2), cache, ints(1, 4), ints(1), 0.1, 3, heads(4), ws)}
    if made == used:
        calls[entry]()
        assert len(library.called) == 1
    else:
        with pytest.raises(ValueError, match=f"cache is on cuda:{made}"):
            calls[entry]()
        assert not library.called
