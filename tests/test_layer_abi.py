"""Host-side refusals of the operators between a layer's linears (no GPU
needed): every argument that bd_rms_norm, bd_rope_append, bd_kv_read and
bd_attention turn away, with addresses that are never dereferenced, and the
binding's own checks of shapes and types."""
import ctypes

import pytest
import torch

from bit_weight_delta_bd_gb300 import bitdelta as bd

G = 1 << 30
A = 1 << 40  # buffers lie G apart, far above any size below
BAD, SHAPE, ALIGN, WS = (bd.BD_ERR_INVALID_ARG, bd.BD_ERR_UNSUPPORTED_SHAPE, bd.BD_ERR_MISALIGNED,
                         bd.BD_ERR_WORKSPACE)
INF, NAN = float("inf"), float("nan")


def at(i, off=0):
    return A + i * G + off


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return bd.load()


def pages(k=at(20), v=at(21), ks=0, vs=0, n_pages=10, page=16, n_kv=2, dim=64, dtype=bd.BD_KV_BF16):
    return bd._KvPages(k, v, ks, vs, n_pages, page, n_kv, dim, dtype)


def pages8(**kw):
    return pages(**{"ks": at(22), "vs": at(23), "dtype": bd.BD_KV_INT8, **kw})


BAD_CACHES = [
    (pages(dim=96), SHAPE), (pages(dim=256), SHAPE), (pages(page=8), SHAPE), (pages(page=48), SHAPE),
    (pages(page=256), SHAPE), (pages(page=0), SHAPE), (pages(page=-16), SHAPE), (pages(n_kv=0), SHAPE),
    (pages(n_kv=1025), SHAPE), (pages(n_pages=-1), SHAPE), (pages(n_pages=2 ** 31 // 16), SHAPE),
    (pages(dtype=2), BAD), (pages(dtype=-1), BAD), (pages(k=0), BAD), (pages(v=0), BAD), (pages8(ks=0), BAD),
    (pages8(vs=0), BAD), (pages(k=at(20, 8)), ALIGN), (pages(v=at(21, 2)), ALIGN), (pages8(ks=at(22, 4)), ALIGN),
    (pages8(vs=at(23, 8)), ALIGN)]


def norm(lib, x=at(0), res=at(1), T=4, d=64, gain=at(2), vid=at(3), V=2, tab=(at(4), at(5)), eps=1e-5, ro=at(1),
         out=at(6), dt=bd.BD_OUT_BF16, scale=0, ws=at(7), wsn=4096):
    t = (ctypes.c_void_p * max(len(tab), 1))(*tab) if tab is not None else None
    return lib.bd_rms_norm(x, res, T, d, gain, vid, V, t, eps, ro, out, dt, scale, ws, wsn, None)


@pytest.mark.parametrize("args,want", [
    (dict(T=0), bd.BD_OK), (dict(T=0, x=0, gain=0, out=0), bd.BD_OK),
    (dict(T=-1), SHAPE), (dict(T=2 ** 31), SHAPE), (dict(d=0), SHAPE), (dict(d=-8), SHAPE), (dict(d=60), SHAPE),
    (dict(dt=3), BAD), (dict(dt=-1), BAD), (dict(V=-1), BAD), (dict(V=65), BAD), (dict(eps=-1e-5), BAD),
    (dict(eps=NAN), BAD), (dict(ws=0), WS), (dict(wsn=8), WS), (dict(ws=at(7, 64)), ALIGN),
    (dict(x=0), BAD), (dict(gain=0), BAD), (dict(out=0), BAD), (dict(tab=None), BAD), (dict(tab=(at(4), 0)), BAD),
    (dict(dt=bd.BD_OUT_E4M3), BAD),  # its scale is missing
    (dict(scale=at(8)), BAD),  # a scale that nothing writes
    (dict(x=at(0, 8)), ALIGN), (dict(res=at(1, 8), ro=0), ALIGN), (dict(ro=at(9, 4)), ALIGN), (dict(gain=at(2, 2)), ALIGN),
    (dict(out=at(6, 8)), ALIGN), (dict(vid=at(3, 2)), ALIGN), (dict(tab=(at(4), at(5, 8))), ALIGN),
    (dict(dt=bd.BD_OUT_E4M3, scale=at(8, 2)), ALIGN),
    (dict(out=at(0)), BAD), (dict(out=at(1)), BAD), (dict(out=at(2)), BAD), (dict(out=at(3, -16)), BAD),
    (dict(out=at(4, 112)), BAD), (dict(out=at(7)), BAD), (dict(ro=at(0, 16)), BAD), (dict(ro=at(1, 16)), BAD),
    (dict(ro=at(2)), BAD), (dict(ro=at(5)), BAD), (dict(ro=at(7)), BAD), (dict(ro=at(6)), BAD),
    (dict(dt=bd.BD_OUT_E4M3, scale=at(6, 16)), BAD), (dict(dt=bd.BD_OUT_E4M3, scale=at(3)), BAD)])
def test_norm_refusals(lib, args, want):
    assert norm(lib, **args) == want


def rope(lib, q=at(0), qs=1024, k=at(1), ks=1024, v=at(2), vs=1024, T=4, n_q=4, pos=at(3), axes=1, aop=None,
         tab=at(4), n_pos=8, rot=32, slot=at(5), cache=None, qo=at(6), qos=1024, ws=at(7), wsn=4096):
    c = pages() if cache is None else cache
    return lib.bd_rope_append(q, qs, k, ks, v, vs, T, n_q, pos, axes, aop, tab, n_pos, rot, 0, slot,
                              ctypes.addressof(c), qo, qos, ws, wsn, None)


@pytest.mark.parametrize("args,want", [
    (dict(T=0), bd.BD_OK), (dict(T=-1), SHAPE), (dict(n_q=-1), SHAPE), (dict(n_q=65537, qs=65537 * 64, qos=65537 * 64), SHAPE),
    (dict(rot=-16), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(ks=120), SHAPE), (dict(vs=120), SHAPE),
    (dict(ks=1028), SHAPE), (dict(vs=1025), SHAPE), (dict(qs=248), SHAPE), (dict(qs=1020), SHAPE),
    (dict(qos=248), SHAPE), (dict(qos=1022), SHAPE), (dict(axes=0), BAD), (dict(axes=5), BAD),
    (dict(axes=2, aop=bytes([0, 1] * 7 + [2, 0])), BAD), (dict(ws=0), WS), (dict(wsn=0), WS), (dict(ws=at(7, 16)), ALIGN),
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(slot=0), BAD), (dict(q=0), BAD), (dict(qo=0), BAD), (dict(pos=0), BAD),
    (dict(tab=0), BAD), (dict(n_pos=0), BAD), (dict(q=at(0, 8)), ALIGN), (dict(k=at(1, 8)), ALIGN),
    (dict(v=at(2, 2)), ALIGN), (dict(qo=at(6, 4)), ALIGN), (dict(tab=at(4, 8)), ALIGN), (dict(pos=at(3, 2)), ALIGN),
    (dict(slot=at(5, 1)), ALIGN), (dict(k=at(20)), BAD), (dict(v=at(21, 16)), BAD), (dict(q=at(20)), BAD),
    (dict(qo=at(21)), BAD), (dict(slot=at(20)), BAD), (dict(pos=at(21)), BAD), (dict(tab=at(20)), BAD),
    (dict(ws=at(20)), BAD), (dict(qo=at(0, 16)), BAD), (dict(qo=at(0), qos=512), BAD), (dict(qo=at(1)), BAD),
    (dict(qo=at(3, -16)), BAD), (dict(qo=at(4)), BAD), (dict(qo=at(5)), BAD), (dict(qo=at(7)), BAD),
    # slices of one product, q in place, but k's columns meet q's
    (dict(qo=at(0), k=at(0, 496), v=at(0, 1024)), BAD)])
def test_rope_refusals(lib, args, want):
    assert rope(lib, **args) == want


def read(lib, cache=None, table=at(0), max_pages=4, off=at(1), n_seq=3, rows=100, ko=at(2), vo=at(3), ws=at(4),
         wsn=4096):
    c = pages() if cache is None else cache
    return lib.bd_kv_read(ctypes.addressof(c), table, max_pages, off, n_seq, rows, ko, vo, ws, wsn, None)


@pytest.mark.parametrize("args,want", [
    (dict(n_seq=0), bd.BD_OK), (dict(rows=0), bd.BD_OK), (dict(n_seq=-1), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=2 ** 31), SHAPE), (dict(max_pages=-1), SHAPE), (dict(max_pages=2 ** 31 // 16), SHAPE),
    (dict(ws=0), WS), (dict(wsn=255), WS), (dict(table=0), BAD), (dict(off=0), BAD), (dict(ko=0), BAD), (dict(vo=0), BAD),
    (dict(ko=at(2, 8)), ALIGN), (dict(vo=at(3, 2)), ALIGN), (dict(table=at(0, 2)), ALIGN), (dict(off=at(1, 1)), ALIGN),
    (dict(ko=at(20)), BAD), (dict(vo=at(21, 16)), BAD), (dict(ko=at(0)), BAD), (dict(vo=at(1)), BAD),
    (dict(ko=at(4)), BAD), (dict(vo=at(2, 16)), BAD), (dict(cache=pages8(), ko=at(23)), BAD)])
def test_read_refusals(lib, args, want):
    assert read(lib, **args) == want


def attention(lib, q=at(0), qs=1024, off=at(1), T=7, n_seq=3, max_new=4, n_q=4, cache=None, table=at(2), max_pages=4,
              kv_len=at(3), scale=0.1, out=at(4), lse=at(5), ws=at(6), wsn=G):
    c = pages() if cache is None else cache
    return lib.bd_attention(q, qs, off, T, n_seq, max_new, n_q, ctypes.addressof(c), table, max_pages, kv_len, scale,
                            1, out, lse, ws, wsn, None)


@pytest.mark.parametrize("args,want", [
    (dict(T=0), bd.BD_OK), (dict(n_seq=0), bd.BD_OK), (dict(n_q=0), SHAPE), (dict(n_q=3), SHAPE), (dict(T=-1), SHAPE),
    (dict(n_q=65538, qs=65538 * 64), SHAPE), (dict(n_seq=-1), SHAPE), (dict(max_new=-1), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(max_pages=2 ** 31 // 16), SHAPE), (dict(T=2 ** 29), SHAPE), (dict(qs=248), SHAPE),
    (dict(qs=1028), SHAPE), (dict(scale=INF), BAD), (dict(scale=NAN), BAD), (dict(ws=0), WS), (dict(wsn=256), WS),
    (dict(ws=at(6, 128)), ALIGN), (dict(q=0), BAD), (dict(off=0), BAD), (dict(kv_len=0), BAD), (dict(out=0), BAD),
    (dict(table=0), BAD), (dict(q=at(0, 8)), ALIGN), (dict(out=at(4, 8)), ALIGN), (dict(off=at(1, 2)), ALIGN),
    (dict(kv_len=at(3, 1)), ALIGN), (dict(table=at(2, 2)), ALIGN), (dict(lse=at(5, 2)), ALIGN), (dict(out=at(0)), BAD),
    (dict(out=at(1)), BAD), (dict(out=at(2)), BAD), (dict(out=at(3)), BAD), (dict(out=at(6)), BAD), (dict(out=at(20)), BAD),
    (dict(lse=at(4)), BAD), (dict(lse=at(0)), BAD), (dict(lse=at(21)), BAD), (dict(ws=at(20)), BAD), (dict(ws=at(0)), BAD),
    (dict(ws=at(2)), BAD), (dict(cache=pages8(), out=at(22)), BAD)])
def test_attention_refusals(lib, args, want):
    assert attention(lib, **args) == want


@pytest.mark.parametrize("entry", [rope, read, attention])
def test_cache_refusals(lib, entry):
    for i, (cache, want) in enumerate(BAD_CACHES):
        assert entry(lib, cache=cache) == want, i
    assert lib.bd_kv_read(None, at(0), 4, at(1), 3, 100, at(2), at(3), at(4), 4096, None) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a usable GPU")
@pytest.mark.parametrize("entry,args", [
    (norm, {}), (norm, dict(res=0, ro=0, vid=0, V=0, tab=None)), (norm, dict(ro=at(0))), (norm, dict(V=0, tab=None)),
    (norm, dict(dt=bd.BD_OUT_E4M3, scale=at(8))), (rope, {}), (rope, dict(n_q=0, q=0, qo=0)),
    (rope, dict(rot=0, pos=0, tab=0, n_pos=0)), (rope, dict(axes=2, aop=bytes([0, 1] * 8))),
    (rope, dict(qo=at(0))), (rope, dict(qo=at(0), k=at(0, 512), v=at(0, 768))), (rope, dict(cache=pages8())), (read, {}),
    (read, dict(cache=pages8(page=128, dim=128))), (attention, {}), (attention, dict(lse=0)),
    (attention, dict(max_pages=0, table=0)), (attention, dict(scale=-1.0)), (attention, dict(max_new=0))])
def test_what_the_checks_let_through(lib, entry, args):
    """A call that passes every check reaches the CUDA runtime, which fails here."""
    assert entry(lib, **args) == bd.BD_ERR_CUDA


def test_workspace_sizes(lib):
    for n in (bd.bd_rms_norm_workspace_size(4096, 8192), bd.bd_rope_append_workspace_size(4096),
              bd.bd_kv_read_workspace_size(10 ** 6)):
        assert n >= 256 and n % 256 == 0
    small = bd.bd_attention_workspace_size(1, 1, 8, 8, 64)
    large = bd.bd_attention_workspace_size(4096, 64, 64, 8, 128)
    assert 256 <= small <= large and small % 256 == 0 and large % 256 == 0
    assert bd.bd_attention_workspace_size(-1, 1, 8, 8, 64) == 256


def test_status_names(lib):
    assert bd.BD_ERR_BAD_INDEX == 11 and bd.status_string(11).startswith("BD_ERR_BAD_INDEX")


# ------------------------------------------------------------------------------- the binding's own checks

def test_binding_refuses_shapes_and_types(lib):
    bf, z = torch.bfloat16, torch.zeros
    k = z(4, 2, 16, 64, dtype=bf)
    with pytest.raises(ValueError, match="n_pages"):
        bd.KvPages(k, z(4, 2, 16, 128, dtype=bf))
    with pytest.raises(ValueError, match="scales"):
        bd.KvPages(k, k, z(4, 2, 16), z(4, 2, 16))
    with pytest.raises(ValueError, match="scales"):
        bd.KvPages(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="scales"):
        bd.KvPages(k.to(torch.int8), k.to(torch.int8), z(4, 2, 8), z(4, 2, 8))
    if not torch.cuda.is_available():
        with pytest.raises(ValueError, match="CUDA"):
            bd.KvPages(k, k)


def test_rope_table_values():
    t = bd.rope_table(50, 32, 10000.0, "cpu")
    assert t.shape == (50, 16, 2) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.tensor([1.0, 0.0]).expand(16, 2))
    want = torch.tensor([7 * 10000.0 ** (-2 * 3 / 32)], dtype=torch.float64)
    assert abs(float(t[7, 3, 0]) - float(want.cos())) <= 2 ** -25 and abs(float(t[7, 3, 1]) - float(want.sin())) <= 2 ** -25
