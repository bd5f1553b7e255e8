"""The paged KV cache in 4 bits on the GPU, against plain 64-bit definitions
(int4_oracle.py): rotary positions with the write, and reading it back -- odd
sizes, groups that straddle the turned part of a head, strided inputs, values
that are not finite -- and what they report."""
import math

import pytest
import torch

import int4_oracle as ref4
import layer_oracle as ref
from bit_weight_delta_bd_gb300 import bitdelta as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cache_on(c, dev):
    on = {n: c[n].to(dev) for n in ("k", "v", "ks", "vs", "table")}
    return bd.KvPages(on["k"], on["v"], on["ks"], on["vs"]), on["table"]


def empty_cache(n_pages, n_kv, page, dim, dev, fill=0x5A, pair=3.0):
    return bd.KvPages(*(torch.full((n_pages, n_kv, page, dim // 2), fill, device=dev, dtype=torch.uint8) for _ in range(2)),
                      *(torch.full((n_pages, n_kv, page, dim // 32, 2), pair, device=dev, dtype=torch.bfloat16)
                        for _ in range(2)))


# ------------------------------------------------------------------------------- the write

@pytest.mark.parametrize("T,n_q,n_kv,dim,page,axes,rot,inter,packed", [
    (1, 8, 1, 128, 16, 1, 128, False, False), (33, 64, 8, 128, 64, 1, 128, False, True),
    (50, 3, 3, 64, 32, 3, 48, True, True), (17, 5, 1, 64, 128, 2, 32, False, True),
    (129, 14, 2, 128, 16, 4, 64, False, False), (9, 0, 4, 128, 16, 1, 0, False, False),
    (700, 10, 5, 64, 16, 1, 64, True, True), (21, 2, 2, 64, 16, 1, 48, False, False),
    (40, 1, 1, 128, 32, 2, 112, False, True), (13, 7, 7, 128, 16, 1, 16, False, False),
    (65, 4, 3, 64, 64, 1, 16, True, False), (300, 9, 3, 128, 128, 1, 96, False, True), (5, 1, 1, 64, 16, 1, 64, False, False)])
def test_append(dev, T, n_q, n_kv, dim, page, axes, rot, inter, packed):
    g = gen(T)
    x = torch.randn(T, n_q + 2 * n_kv, dim, generator=g).to(torch.bfloat16)
    n_pos, pairs = 500, rot // 2
    tab = bd.rope_table(n_pos, rot, 10000.0, "cpu") if rot else None
    pos = torch.randint(0, n_pos, (T, axes), generator=g, dtype=torch.int32)
    axis = torch.randint(0, axes, (pairs,), generator=g).tolist()
    n_pages = -(-T // page) + 4
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    if T > 1:
        slot[T // 2] = -1
    q, k, v = x[:, :n_q], x[:, n_q: n_q + n_kv], x[:, n_q + n_kv:]
    xd = x.to(dev)
    parts = (xd[:, :n_q], xd[:, n_q: n_q + n_kv], xd[:, n_q + n_kv:])
    qd, kd, vd = parts if packed else tuple(t.contiguous() for t in parts)
    cache = empty_cache(n_pages, n_kv, page, dim, dev)
    ws = bd.new_workspace(bd.bd_rope_append_workspace_size(T), dev)
    qo = torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16) if n_q else None
    bd.bd_rope_append(qd if n_q else None, kd, vd, pos.to(dev), tab.to(dev) if rot else None, slot.to(dev), cache, qo,
                      ws, axis_of_pair=axis if rot else None, interleaved=inter)
    assert bd.bd_check_async(ws) == bd.BD_OK
    # operation by operation in fp32: equal bit for bit
    if rot:
        cs = tab[pos.long()[:, axis], torch.arange(pairs)]
        tq, tk = (ref.turn(t.float(), cs[..., 0], cs[..., 1], rot, inter) for t in (q, k))
    else:
        tq, tk = q.float(), k.float()
    if n_q:
        assert torch.equal(qo.cpu(), tq.to(torch.bfloat16))
    live = slot >= 0
    pg, at = slot[live].long() // page, slot[live].long() % page
    for pool, pairs_of, val in ((cache.k, cache.k_scale, tk), (cache.v, cache.v_scale, v.float())):
        want = torch.full(pool.shape, 0x5A, dtype=torch.uint8)
        want_pairs = torch.full(pairs_of.shape, 3.0, dtype=torch.bfloat16)
        want[pg, :, at], want_pairs[pg, :, at] = ref4.codes(val[live])
        assert torch.equal(pairs_of.cpu(), want_pairs)
        assert torch.equal(pool.cpu(), want)
        # and the values themselves: half a step, what the rounded scale leaves past 15 steps, and the lowest value's rounding
        got = ref4.values(pool.cpu()[pg, :, at], pairs_of.cpu()[pg, :, at])
        scale = want_pairs[pg, :, at][..., 0].double().repeat_interleave(32, -1)
        low = want_pairs[pg, :, at][..., 1].double().repeat_interleave(32, -1)
        assert ((got - val[live].double()).abs() <= scale * (0.5 + 16 * 2.0 ** -8) + low.abs() * 2.0 ** -8).all()


def test_groups_of_one_value_zeros_and_extremes(dev):
    """Scales of groups whose elements are equal, zero, tiny or huge, and of groups that are not finite."""
    dim = 64
    v = torch.randn(8, 1, dim, generator=gen(4))
    v[0] = 0
    v[1] = -2.5
    v[2] *= 1e-20
    v[3] *= 1e20
    v[4, 0, 5] = math.nan
    v[5, 0, 40] = math.inf
    v[6, 0, 3] = -math.inf
    v[7, 0, :32] = torch.where(torch.arange(32) % 2 == 0, 3e38, -3e38)
    v = v.to(torch.bfloat16)
    cache = empty_cache(1, 1, 16, dim, dev)
    ws, slot = bd.new_workspace(256, dev), torch.arange(8, dtype=torch.int32, device=dev)
    bd.bd_rope_append(None, v.to(dev), v.to(dev), None, None, slot, cache, None, ws)
    for pool, pair in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        byte, pr = pool.cpu()[0, 0, :8], pair.cpu()[0, 0, :8]
        want_byte, want_pair = ref4.codes(v[:, 0].float())
        assert torch.equal(pr[:4], want_pair[:4]) and torch.equal(byte[:4], want_byte[:4])
        back = ref4.values(byte, pr)
        assert (back[0] == 0).all() and torch.equal(back[1].float(), torch.full((dim,), -2.5))
        assert (back[2:4].isfinite()).all()
        assert not pr[4, 0, 0].isfinite() and pr[4, 1].isfinite().all()
        assert not pr[5, 1, 0].isfinite() and pr[5, 0].isfinite().all()
        assert not pr[6, 0, 0].isfinite() and not pr[7, 0, 0].isfinite() and pr[7, 1].isfinite().all()


def test_append_reports_bad_indices(dev):
    T, dim, page = 4, 64, 16
    x = torch.randn(T, 3, dim, generator=gen(3)).to(torch.bfloat16).to(dev)
    cache, ws = empty_cache(2, 1, page, dim, dev), bd.new_workspace(256, dev)
    tab, qo = bd.rope_table(10, dim, 10000.0, dev), torch.empty(T, 1, dim, device=dev, dtype=torch.bfloat16)
    for slots, positions in (([0, 1, 32, 3], [0, 1, 2, 3]), ([0, 1, -2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 1, 10, 3])):
        bd.bd_rope_append(x[:, :1], x[:, 1:2], x[:, 2:], torch.tensor(positions, dtype=torch.int32, device=dev), tab,
                          torch.tensor(slots, dtype=torch.int32, device=dev), cache, qo, ws)
        assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX


# ------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("lens,n_kv,dim,page", [
    ([1], 1, 64, 16), ([0, 17, 0, 64, 3], 3, 128, 16), ([300, 1, 129], 8, 128, 128), ([1000, 0], 2, 64, 32), ([0], 1, 64, 16),
    ([40] * 60, 1, 64, 16), ([5, 700], 33, 128, 16), ([9], 600, 64, 16), ([20000], 1, 128, 64)])
def test_read(dev, lens, n_kv, dim, page):
    c = ref4.paged([0] * len(lens), lens, n_kv, dim, page, seed=len(lens))
    cache, table = cache_on(c, dev)
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    rows = sum(lens) + 5
    for start in (0, 8):  # outputs on whole sectors, and on half ones
        room = [torch.full((rows * n_kv * dim + 8,), 3.0, device=dev, dtype=torch.bfloat16) for _ in range(2)]
        ko, vo = (t[start: start + rows * n_kv * dim].view(rows, n_kv, dim) for t in room)
        ws = bd.new_workspace(bd.bd_kv_read_workspace_size(rows), dev)
        bd.bd_kv_read(cache, table, off, ko, vo, ws)
        assert bd.bd_check_async(ws) == bd.BD_OK
        for out, name, whole in ((ko, "k", room[0]), (vo, "v", room[1])):
            # a value is one fp32 sum of an exact product, rounded to bf16: bit for bit
            want = torch.cat([x.float() for x in c["vals"][name]] + [torch.full((5, n_kv, dim), 3.0)]).to(torch.bfloat16)
            assert torch.equal(out.cpu(), want)
            assert (whole[:start] == 3).all() and (whole[start + rows * n_kv * dim:] == 3).all()


def test_read_reports_bad_pages(dev):
    cache, ws = empty_cache(2, 1, 16, 64, dev, fill=0, pair=1.0), bd.new_workspace(256, dev)
    ko, vo = (torch.empty(20, 1, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
    for table, n in (([[0, 2]], 20), ([[-1, 1]], 20), ([[0]], 20), ([[0, 1]], 21)):
        off = torch.tensor([0, n], dtype=torch.int32, device=dev)
        bd.bd_kv_read(cache, torch.tensor(table, dtype=torch.int32, device=dev), off, ko, vo, ws)
        assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX
    bd.bd_kv_read(cache, torch.tensor([[0, 2]], dtype=torch.int32, device=dev),
                  torch.tensor([0, 20], dtype=torch.int32, device=dev), ko, vo, ws)
    assert (ko[:16] == 1).all() and (ko[16:] == 0).all()
