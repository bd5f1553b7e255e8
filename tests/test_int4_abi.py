"""Host-side refusals of the norms around a block and of the 4-bit cache (no GPU
needed): what bd_block_norm and the calls on a BD_KV_INT4 cache turn away, with
addresses that are never dereferenced, and the binding's own checks."""
import ctypes

import pytest
import torch

import test_layer_abi as abi
import test_layer_handles as handles
from bit_weight_delta_bd_gb300 import bitdelta as bd
from test_layer_abi import ALIGN, BAD, INF, NAN, SHAPE, WS, at

NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a usable GPU")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return bd.load()


# ------------------------------------------------------------------------------- the norms around a block

def norm(lib, x=at(0), res=at(1), T=4, d=64, post=at(2), ptab=(at(3), at(4)), gate=at(5), rows=3, idx=at(6), bs=0.5,
         rs=1.0, gain=at(7), tab=(at(8), at(9)), vid=at(10), V=2, eps=1e-5, ro=at(1), out=at(11), dt=bd.BD_OUT_BF16,
         scale=0, ws=at(12), wsn=4096):
    t, p = ((ctypes.c_void_p * max(len(v), 1))(*v) if v is not None else None for v in (tab, ptab))
    return lib.bd_block_norm(x, res, T, d, post, p, gate, rows, idx, bs, rs, gain, t, vid, V, eps, ro, out, dt, scale,
                             ws, wsn, None)


@pytest.mark.parametrize("args,want", [
    (dict(T=0), bd.BD_OK), (dict(T=0, x=0, res=0, gain=0, out=0), bd.BD_OK),
    (dict(T=-1), SHAPE), (dict(T=2 ** 31), SHAPE), (dict(d=0), SHAPE), (dict(d=-8), SHAPE), (dict(d=60), SHAPE),
    (dict(rows=-1), SHAPE), (dict(rows=2 ** 31), SHAPE),
    (dict(dt=3), BAD), (dict(dt=-1), BAD), (dict(V=-1), BAD), (dict(V=65), BAD), (dict(eps=-1e-5), BAD),
    (dict(eps=NAN), BAD), (dict(bs=INF), BAD), (dict(bs=NAN), BAD), (dict(rs=-INF), BAD), (dict(rs=NAN), BAD),
    (dict(ws=0), WS), (dict(wsn=8), WS), (dict(ws=at(12, 64)), ALIGN),
    (dict(x=0), BAD), (dict(res=0, ro=0), BAD), (dict(gain=0), BAD), (dict(out=0), BAD), (dict(tab=None), BAD),
    (dict(ptab=None), BAD), (dict(tab=(at(8), 0)), BAD), (dict(ptab=(0, at(4))), BAD),
    (dict(gate=0), BAD),  # rows are looked up in a gate that is not there
    (dict(rows=0), BAD), (dict(idx=0), BAD),  # three gates for four tokens
    (dict(dt=bd.BD_OUT_E4M3), BAD), (dict(scale=at(13)), BAD),
    (dict(x=at(0, 8)), ALIGN), (dict(res=at(1, 8), ro=0), ALIGN), (dict(ro=at(13, 4)), ALIGN),
    (dict(gain=at(7, 2)), ALIGN), (dict(post=at(2, 8)), ALIGN), (dict(gate=at(5, 8)), ALIGN), (dict(idx=at(6, 2)), ALIGN),
    (dict(out=at(11, 8)), ALIGN), (dict(vid=at(10, 1)), ALIGN), (dict(tab=(at(8), at(9, 8))), ALIGN),
    (dict(ptab=(at(3, 2), at(4))), ALIGN), (dict(dt=bd.BD_OUT_E4M3, scale=at(13, 2)), ALIGN),
    (dict(out=at(0)), BAD), (dict(out=at(1)), BAD), (dict(out=at(2)), BAD), (dict(out=at(3, 112)), BAD),
    (dict(out=at(5, 368)), BAD), (dict(out=at(6, -496)), BAD), (dict(out=at(7)), BAD), (dict(out=at(8, -16)), BAD),
    (dict(out=at(10)), BAD), (dict(out=at(12)), BAD), (dict(ro=at(0, 16)), BAD), (dict(ro=at(1, 16)), BAD),
    (dict(ro=at(2)), BAD), (dict(ro=at(4)), BAD), (dict(ro=at(5)), BAD), (dict(ro=at(6)), BAD), (dict(ro=at(9)), BAD),
    (dict(ro=at(11)), BAD), (dict(ro=at(12)), BAD), (dict(dt=bd.BD_OUT_E4M3, scale=at(11, 16)), BAD),
    (dict(dt=bd.BD_OUT_E4M3, scale=at(10)), BAD), (dict(dt=bd.BD_OUT_E4M3, scale=at(6)), BAD),
    (dict(dt=bd.BD_OUT_E4M3, scale=at(1, 16)), BAD)])
def test_block_norm_refusals(lib, args, want):
    assert norm(lib, **args) == want


@NO_GPU
@pytest.mark.parametrize("args", [
    {}, dict(ro=at(0)), dict(ro=0), dict(ro=at(13)), dict(post=0, ptab=None), dict(gate=0, rows=0, idx=0),
    dict(rows=1, idx=0), dict(rows=4, idx=0), dict(V=0, tab=None, ptab=None), dict(vid=0, V=0, tab=None, ptab=None),
    dict(dt=bd.BD_OUT_F32), dict(dt=bd.BD_OUT_E4M3, scale=at(13)), dict(x=at(1), ro=0), dict(x=at(1)), dict(bs=0.0, rs=-1.0),
    # neighbours that just do not meet
    dict(out=at(5, 384)), dict(out=at(6, -512)), dict(out=at(8, 128))])
def test_what_the_norm_lets_through(lib, args):
    """A call that passes every check reaches the CUDA runtime, which fails here."""
    assert norm(lib, **args) == bd.BD_ERR_CUDA


# ------------------------------------------------------------------------------- a cache of 4-bit codes

def pages4(**kw):
    return abi.pages8(**{"dtype": bd.BD_KV_INT4, **kw})


@pytest.mark.parametrize("entry", [abi.rope, abi.read, abi.attention])
@pytest.mark.parametrize("cache,want", [
    (pages4(ks=0), BAD), (pages4(vs=0), BAD), (pages4(k=0), BAD), (pages4(dtype=3), BAD), (pages4(dim=32), SHAPE),
    (pages4(dim=96), SHAPE), (pages4(page=8), SHAPE), (pages4(n_pages=2 ** 31 // 16), SHAPE), (pages4(n_kv=0), SHAPE),
    (pages4(k=at(20, 8)), ALIGN), (pages4(v=at(21, 4)), ALIGN), (pages4(ks=at(22, 8)), ALIGN),
    (pages4(vs=at(23, 4)), ALIGN)])
def test_cache_refusals(lib, entry, cache, want):
    assert entry(lib, cache=cache) == want


# 10 pages x 2 heads x 16 tokens: codes of 32 bytes and two words of scales for each vector of 64
CODES, PAIRS = 320 * 32, 320 * 8


@pytest.mark.parametrize("entry,args", [
    (abi.read, lambda a: dict(ko=a)), (abi.read, lambda a: dict(vo=a)), (abi.attention, lambda a: dict(out=a)),
    (abi.attention, lambda a: dict(lse=a)), (abi.rope, lambda a: dict(k=a)), (abi.rope, lambda a: dict(qo=a, qos=256))])
def test_buffers_meet_the_cache_to_its_last_byte(lib, entry, args):
    for base, size in ((20, CODES), (21, CODES), (22, PAIRS), (23, PAIRS)):
        assert entry(lib, cache=pages4(), **args(at(base, size - 16))) == BAD
        if not torch.cuda.is_available():  # the first byte behind it is free
            assert entry(lib, cache=pages4(), **args(at(base, size))) == bd.BD_ERR_CUDA


@NO_GPU
@pytest.mark.parametrize("entry,args", [
    (abi.rope, {}), (abi.read, {}), (abi.attention, {}), (abi.attention, dict(max_new=1)),
    (abi.rope, dict(n_q=0, q=0, qo=0)), (abi.read, dict(cache=pages4(n_pages=0))),
    (abi.rope, dict(cache=pages4(n_pages=0))), (abi.read, dict(cache=pages4(page=128, dim=128)))])
def test_what_the_checks_let_through(lib, entry, args):
    assert entry(lib, **{"cache": pages4(), **args}) == bd.BD_ERR_CUDA


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [1, 4096])
def test_attention_refuses_a_cache_without_pages(lib, max_new, dim):
    handles.test_attention_refuses_a_cache_without_pages(lib, pages4, max_new, dim)


# ------------------------------------------------------------------------------- the binding's own checks

def test_binding_refuses_caches(lib):
    z, bf, u8 = torch.zeros, torch.bfloat16, torch.uint8
    k = z(4, 2, 16, 32, dtype=u8)
    pair = z(4, 2, 16, 2, 2, dtype=bf)
    for args in ((k, k), (k, k, pair), (k, k, pair, pair[..., 0]), (k, k, z(4, 2, 16), z(4, 2, 16)),
                 (k, k, z(4, 2, 16, 2, dtype=bf), z(4, 2, 16, 2, dtype=bf)), (k, k, pair[:, :, :8], pair[:, :, :8])):
        with pytest.raises(ValueError, match="scales"):
            bd.KvPages(*args)
    with pytest.raises(ValueError, match="one dtype"):
        bd.KvPages(k, z(4, 2, 16, 64, dtype=u8), pair, pair)
    with pytest.raises(ValueError, match="one dtype"):
        bd.KvPages(k, k.to(torch.int8), pair, pair)


@pytest.fixture
def fake(monkeypatch):
    library = handles.Library()
    monkeypatch.setattr(bd, "_device", lambda: 0)
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(bd, "load", lambda *path: library)
    return library


def tensor(*shape, dtype=torch.bfloat16, index=0):
    return handles.OnDevice(index, *shape, dtype=dtype)


def test_binding_takes_a_cache_of_pairs(fake):
    u8, f32 = torch.uint8, torch.float32
    c = bd.KvPages(tensor(4, 2, 16, 64, dtype=u8), tensor(4, 2, 16, 64, dtype=u8), tensor(4, 2, 16, 4, 2),
                   tensor(4, 2, 16, 4, 2))
    assert (c.head_dim, c.page_size, c.n_kv, c.n_pages, c._c.dtype) == (128, 16, 2, 4, bd.BD_KV_INT4)
    with pytest.raises(ValueError, match="k_scale has dtype"):
        bd.KvPages(tensor(4, 2, 16, 64, dtype=u8), tensor(4, 2, 16, 64, dtype=u8), tensor(4, 2, 16, 4, 2, dtype=f32),
                   tensor(4, 2, 16, 4, 2, dtype=f32))


def block_norm(**kw):
    i32 = torch.int32
    a = dict(x=tensor(5, 64), residual=tensor(5, 64), gain=tensor(64), eps=1e-5, out=tensor(5, 64),
             ws=tensor(4096, dtype=torch.uint8), post_gain=tensor(64), gate=tensor(3, 64), gate_idx=tensor(5, dtype=i32),
             vid=tensor(5, dtype=i32), gain_list=(), post_gain_list=())
    bd.bd_block_norm(**{**a, **kw})


def test_binding_refuses_norms(fake):
    host = torch.zeros(64, dtype=torch.bfloat16)
    e4m3, f16, i64 = torch.float8_e4m3fn, torch.float16, torch.int64
    for kw, match in (
            (dict(gain=tensor(32)), "gain"), (dict(residual=tensor(4, 64)), "residual"), (dict(out=tensor(5, 32)), "out"),
            (dict(residual_out=tensor(5, 65)), "residual_out"), (dict(post_gain=tensor(1, 64)), "post_gain"),
            (dict(scale=tensor(4, dtype=torch.float32), out=tensor(5, 64, dtype=e4m3)), "scale"),
            (dict(vid=tensor(4, dtype=torch.int32)), "vid"), (dict(gate=tensor(3, 32)), "gate"),
            (dict(gate=tensor(3, 1, 64)), "gate"), (dict(gate=None), "gate"), (dict(gate=tensor()), "gate"),
            (dict(gate_idx=tensor(4, dtype=torch.int32)), "gate_idx"), (dict(gate_idx=tensor(5, dtype=i64)), "gate_idx"),
            (dict(post_gain_list=[tensor(64)]), "differ in length"),
            (dict(gain_list=[host], post_gain_list=[host]), "gain"), (dict(out=tensor(5, 64, dtype=f16)), "dtype"),
            (dict(x=tensor(5, 64, dtype=torch.float32)), "dtype"), (dict(gate=tensor(3, 64, index=1)), "gate")):
        with pytest.raises(ValueError, match=match):
            block_norm(**kw)
    assert not fake.called
    block_norm()
    block_norm(gate=tensor(64), gate_idx=None)
    block_norm(gate=None, gate_idx=None, post_gain=None, post_gain_list=(), vid=None, gain_list=())
    assert fake.called == ["bd_block_norm"] * 3
