"""The operators between a layer's linears on the GPU, against plain 64-bit
definitions (layer_oracle.py): RMS norm with the residual's addition, rotary
positions with the write into the paged cache, reading it back, and attention
of new tokens over it -- at odd sizes, empty rows, pages that end inside a
tile, strided inputs, NaN past the lengths, another stream -- and what they
refuse."""
import math

import pytest
import torch

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


def within(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float((err / bound).nan_to_num(posinf=9e9).max()):.3g} times"


# ------------------------------------------------------------------------------- norm

def run_norm(dev, T, d, V, out_dtype, residual=True, seed=0, in_place=False, eps=1e-5):
    g = gen(seed)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    r = (2 * torch.randn(T, d, generator=g)).to(torch.bfloat16) if residual else None
    gains = (1 + 0.2 * torch.randn(V + 1, d, generator=g)).to(torch.bfloat16)
    vid = torch.randint(-1, V, (T,), generator=g, dtype=torch.int32) if V else None
    which = (vid + 1).long() if V else torch.zeros(T, dtype=torch.long)
    h, y = ref.rms_norm(x, r, gains, which, eps)
    xd, gd = x.to(dev), gains.to(dev)
    rd = r.to(dev) if residual else None
    out = torch.empty(T, d, device=dev, dtype=out_dtype)
    scale = torch.empty(T, device=dev) if out_dtype == torch.float8_e4m3fn else None
    ho = (rd if in_place else torch.empty_like(xd)) if residual else None
    ws = bd.new_workspace(bd.bd_rms_norm_workspace_size(T, d), dev)
    bd.bd_rms_norm(xd, gd[0], eps, out, ws, residual=rd, residual_out=ho, scale=scale,
                   vid=vid.to(dev) if V else None, gain_list=[gd[v + 1] for v in range(V)])
    assert bd.bd_check_async(ws) == bd.BD_OK
    return h, y, ho, out, scale


@pytest.mark.parametrize("T,d,V,residual,in_place", [
    (1, 8, 0, False, False), (3, 128, 2, True, False), (32, 8192, 14, True, False), (5, 8200, 0, True, True),
    (7, 16384, 64, True, False), (2, 33000, 1, True, True), (2, 40000, 3, False, False), (257, 1000, 5, True, False)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_rms_norm(dev, T, d, V, residual, in_place, out_dtype):
    h, y, ho, out, _ = run_norm(dev, T, d, V, out_dtype, residual, seed=d, in_place=in_place)
    bound = y.abs() * ref.norm_rel(d)
    if out_dtype == torch.bfloat16:
        bound = bound + ref.half_ulp_bf16(y.abs() + bound)
    within(out, y, bound, "norm")
    if residual:
        within(ho, h, ref.half_ulp_bf16(h) + h.abs() * 2 * ref.U32, "residual")


@pytest.mark.parametrize("T,d,V", [(1, 8, 0), (9, 8192, 3), (2, 40008, 0), (33, 5128, 0)])
def test_rms_norm_e4m3(dev, T, d, V):
    _, y, _, out, scale = run_norm(dev, T, d, V, torch.float8_e4m3fn, True, seed=T)
    s = y.abs().amax(1).clamp_min(1e-30) / 448
    rel = ref.norm_rel(d) + 4 * ref.U32
    within(scale, s, s * rel, "scale")
    z = (y / s[:, None]).abs()
    half_step = torch.where(z >= 2.0 ** -6, torch.pow(2.0, torch.floor(torch.log2(z.clamp_min(2.0 ** -6))) - 4),
                            torch.full_like(z, 2.0 ** -10))
    within(out.float().cpu().double() * scale.cpu().double()[:, None], y,
           s[:, None] * half_step * (1 + 2.0 ** -10) + y.abs() * 4 * rel, "codes")


def test_rms_norm_zero_and_nonfinite_rows(dev):
    d = 256
    x = torch.randn(4, d, generator=gen(1)).to(torch.bfloat16)
    x[0] = 0
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    ws = bd.new_workspace(256, dev)
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    out = torch.empty(4, d, device=dev)
    bd.bd_rms_norm(x.to(dev), gain, 1e-5, out, ws)
    o = out.cpu()
    assert (o[0] == 0).all() and o[1].isnan().all() and o[2, 9].isnan() and o[3].isfinite().all()
    o8, sc = torch.empty(4, d, device=dev, dtype=torch.float8_e4m3fn), torch.empty(4, device=dev)
    bd.bd_rms_norm(x.to(dev), gain, 1e-5, o8, ws, scale=sc)
    assert (o8[0].float() == 0).all() and sc[0] > 0 and not sc[1].isfinite() and not sc[2].isfinite()
    assert sc[3].isfinite() and o8[3].float().isfinite().all()


def test_rms_norm_bad_variant(dev):
    d = 64
    x = torch.randn(3, d, generator=gen(2)).to(torch.bfloat16).to(dev)
    gains = torch.stack([torch.full((d,), 1.0), torch.full((d,), 3.0)]).to(torch.bfloat16).to(dev)
    out, base = (torch.empty(3, d, device=dev) for _ in range(2))
    ws = bd.new_workspace(256, dev)
    bd.bd_rms_norm(x, gains[0], 1e-5, base, ws)
    vid = torch.tensor([0, 5, -2], dtype=torch.int32, device=dev)
    bd.bd_rms_norm(x, gains[0], 1e-5, out, ws, vid=vid, gain_list=[gains[1]])
    assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_VARIANT
    assert bd.bd_check_async(ws) == bd.BD_OK
    assert torch.equal(out[1:], base[1:]) and not torch.equal(out[0], base[0])


# ------------------------------------------------------------------------------- rotary positions, cache

@pytest.mark.parametrize("T,n_q,n_kv,dim,page,int8,axes,rot,inter,packed", [
    (1, 8, 1, 128, 16, False, 1, 128, False, False),
    (33, 64, 8, 128, 64, True, 1, 128, False, True),
    (50, 3, 3, 64, 32, True, 3, 48, True, True),
    (17, 5, 1, 64, 128, False, 2, 32, False, True),
    (129, 14, 2, 128, 16, True, 4, 64, False, False),
    (9, 0, 4, 128, 16, True, 1, 0, False, False),
    (700, 10, 5, 64, 16, False, 1, 64, True, True)])
def test_rope_append(dev, T, n_q, n_kv, dim, page, int8, axes, rot, inter, packed):
    g = gen(T)
    heads = n_q + 2 * n_kv
    x = torch.randn(T, heads, dim, generator=g).to(torch.bfloat16)
    n_pos, pairs = 500, rot // 2
    tab = bd.rope_table(n_pos, rot, 10000.0, "cpu") if rot else None
    pos = torch.randint(0, n_pos, (T, axes), generator=g, dtype=torch.int32)
    axis = torch.randint(0, axes, (pairs,), generator=g).tolist()
    n_pages = -(-T // page) + 4
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slot[T // 2] = -1
    q, k, v = x[:, :n_q], x[:, n_q: n_q + n_kv], x[:, n_q + n_kv:]
    xd = x.to(dev)
    parts = (xd[:, :n_q], xd[:, n_q: n_q + n_kv], xd[:, n_q + n_kv:])
    qd, kd, vd = parts if packed else tuple(t.contiguous() for t in parts)
    shape = (n_pages, n_kv, page, dim)
    fill = 99 if int8 else 7.0
    kp, vp = (torch.full(shape, fill, device=dev, dtype=torch.int8 if int8 else torch.bfloat16) for _ in range(2))
    ks, vs = (torch.full(shape[:3], 5.0, device=dev) if int8 else None for _ in range(2))
    cache = bd.KvPages(kp, vp, ks, vs)
    ws = bd.new_workspace(256, dev)
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
    for pool, sc, val in ((kp, ks, tk), (vp, vs, v.float())):
        want = torch.full(shape, fill, dtype=pool.dtype)
        if int8:
            wsc = torch.full(shape[:3], 5.0)
            want[pg, :, at], wsc[pg, :, at] = ref.codes(val[live])
            assert torch.equal(sc.cpu(), wsc)
        else:
            want[pg, :, at] = val[live].to(torch.bfloat16)
        assert torch.equal(pool.cpu(), want)
    # and the angles themselves, in 64 bits
    if rot and n_q:
        f = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        ang = pos.double()[:, axis] * f
        want = ref.turn(q.double(), ang.cos(), ang.sin(), rot, inter)
        bound = 6 * ref.U32 * q.double().abs().amax(-1, keepdim=True) + ref.half_ulp_bf16(want) * (1 + 2.0 ** -8)
        within(qo, want, bound, "turned q")
    # in place, where q is one tensor or a slice of the packed rows
    if n_q:
        bd.bd_rope_append(qd, kd, vd, pos.to(dev), tab.to(dev), slot.to(dev), cache, qd, ws, axis_of_pair=axis,
                          interleaved=inter)
        assert torch.equal(qd, qo)


def test_rope_append_reports_bad_indices(dev):
    T, dim, page = 4, 64, 16
    x = torch.randn(T, 3, dim, generator=gen(3)).to(torch.bfloat16).to(dev)
    kp, vp = (torch.zeros(2, 1, page, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    cache, ws = bd.KvPages(kp, vp), bd.new_workspace(256, dev)
    tab, qo = bd.rope_table(10, dim, 10000.0, dev), torch.empty(T, 1, dim, device=dev, dtype=torch.bfloat16)
    args = (x[:, :1], x[:, 1:2], x[:, 2:])
    pos = torch.zeros(T, dtype=torch.int32, device=dev)
    for slots, positions in (([0, 1, 32, 3], [0, 1, 2, 3]), ([0, 1, -2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 1, 10, 3]),
                             ([0, 1, 2, 3], [0, 1, -1, 3])):
        pos.copy_(torch.tensor(positions, dtype=torch.int32))
        bd.bd_rope_append(*args, pos, tab, torch.tensor(slots, dtype=torch.int32, device=dev), cache, qo, ws)
        assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX
    assert bd.bd_check_async(ws) == bd.BD_OK


def test_int8_codes_of_zero_and_nonfinite_vectors(dev):
    dim = 64
    v = torch.randn(4, 1, dim, generator=gen(4)).to(torch.bfloat16)
    v[0] = 0
    v[1, 0, 5] = math.nan
    v[2, 0, 6] = math.inf
    kp, vp = (torch.zeros(1, 1, 16, dim, device=dev, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.zeros(1, 1, 16, device=dev) for _ in range(2))
    cache, ws = bd.KvPages(kp, vp, ks, vs), bd.new_workspace(256, dev)
    slot = torch.arange(4, dtype=torch.int32, device=dev)
    bd.bd_rope_append(None, v.to(dev), v.to(dev), None, None, slot, cache, None, ws)
    assert (vp[0, 0, 0] == 0).all() and vs[0, 0, 0] > 0 and vs[0, 0, 3].isfinite()
    assert not vs[0, 0, 1].isfinite() and not vs[0, 0, 2].isfinite()


@pytest.mark.parametrize("lens,n_kv,dim,page,int8", [
    ([1], 1, 64, 16, False), ([0, 17, 0, 64, 3], 3, 128, 16, True), ([300, 1, 129], 8, 128, 128, False),
    ([1000, 0], 2, 64, 32, True), ([0], 1, 64, 16, True)])
def test_kv_read(dev, lens, n_kv, dim, page, int8):
    c = ref.paged([0] * len(lens), lens, n_kv, dim, page, int8, seed=len(lens))
    on = {n: c[n].to(dev) if c[n] is not None else None for n in ("k", "v", "ks", "vs", "table")}
    cache = bd.KvPages(on["k"], on["v"], on["ks"], on["vs"])
    off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    rows = sum(lens) + 5
    ko, vo = (torch.full((rows, n_kv, dim), 3.0, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ws = bd.new_workspace(256, dev)
    bd.bd_kv_read(cache, on["table"], off, ko, vo, ws)
    assert bd.bd_check_async(ws) == bd.BD_OK
    for out, name in ((ko, "k"), (vo, "v")):
        want = torch.cat(c["vals"][name] + [torch.full((5, n_kv, dim), 3.0, dtype=torch.float64)])
        # code * scale is one fp32 product, rounded to bf16: bit for bit
        assert torch.equal(out.cpu(), want.float().to(torch.bfloat16))


def test_kv_read_reports_bad_pages(dev):
    kp, vp = (torch.ones(2, 1, 16, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
    cache, ws = bd.KvPages(kp, vp), bd.new_workspace(256, dev)
    ko, vo = (torch.empty(20, 1, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
    for table, n in (([[0, 2]], 20), ([[-1, 1]], 20), ([[0]], 20)):
        off = torch.tensor([0, n], dtype=torch.int32, device=dev)
        bd.bd_kv_read(cache, torch.tensor(table, dtype=torch.int32, device=dev), off, ko, vo, ws)
        assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX
    bad = torch.tensor([[0, 2]], dtype=torch.int32, device=dev)
    bd.bd_kv_read(cache, bad, torch.tensor([0, 20], dtype=torch.int32, device=dev), ko, vo, ws)
    assert (ko[:16] == 1).all() and (ko[16:] == 0).all()


# ------------------------------------------------------------------------------- attention

def run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, causal=True, seed=0, scale=None, packed=False,
                  q_scale=1.0, max_new=None):
    c = ref.paged(n_new, kv_len, n_kv, dim, page, int8, seed=seed)
    on = {n: c[n].to(dev) if c[n] is not None else None for n in ("k", "v", "ks", "vs", "table")}
    cache = bd.KvPages(on["k"], on["v"], on["ks"], on["vs"])
    T = sum(n_new)
    q = (q_scale * torch.randn(T, n_q + (2 * n_kv if packed else 0), dim, generator=gen(seed + 1))).to(torch.bfloat16)
    qd = q.to(dev)[:, :n_q]
    q = q[:, :n_q]
    q_off = [0]
    for n in n_new:
        q_off.append(q_off[-1] + n)
    out = torch.full((T, n_q, dim), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.empty(T, n_q, device=dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, len(n_new), n_q, n_kv, dim), dev)
    scale = scale if scale is not None else dim ** -0.5
    off_d = torch.tensor(q_off, dtype=torch.int32, device=dev)
    len_d = torch.tensor(kv_len, dtype=torch.int32, device=dev)
    bd.bd_attention(qd, off_d, cache, on["table"], len_d, scale, max(n_new) if max_new is None else max_new, out, ws,
                    causal=causal, lse=lse)
    assert bd.bd_check_async(ws) == bd.BD_OK
    want = ref.attention(q, q_off, c["vals"]["k"], c["vals"]["v"], kv_len, scale, causal)
    b_out, b_lse = ref.attention_bounds(*want, max(kv_len + [1]))
    within(out, want[0], b_out, "attention")
    assert torch.equal(lse.cpu() == -math.inf, want[1] == -math.inf)
    fin = want[1] > -math.inf
    within(lse.cpu()[fin], want[1][fin], b_lse[fin], "log-sum-exp")
    # the same call again gives the same bits, without the log-sum-exp too
    out2 = torch.empty_like(out)
    bd.bd_attention(qd, off_d, cache, on["table"], len_d, scale, max(n_new) if max_new is None else max_new, out2, ws,
                    causal=causal)
    assert torch.equal(out, out2)
    return out, qd, on, off_d, len_d


DECODE = [
    ([1], [1], 1, 1, 64, 16), ([1], [500], 64, 8, 128, 16), ([1, 1, 1], [0, 1, 63], 8, 2, 128, 16),
    ([1] * 9, [64, 65, 127, 128, 129, 16, 15, 17, 2000], 16, 8, 128, 32), ([1, 0, 1], [300, 5, 1000], 5, 1, 64, 128),
    ([1, 1], [3001, 1], 32, 2, 64, 64), ([1] * 70, [(37 * i) % 300 for i in range(70)], 7, 7, 64, 16),
    ([1], [6000], 24, 1, 128, 64)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", DECODE)
def test_attention_decode(dev, n_new, kv_len, n_q, n_kv, dim, page, int8):
    run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, seed=len(n_new), packed=len(n_new) % 2 == 1)


CHUNK = [
    ([5], [5], 4, 2, 64, 16, True), ([2, 3, 1], [2, 300, 77], 8, 1, 128, 16, True),
    ([130], [130], 8, 8, 64, 32, True), ([65, 1, 200, 0], [65, 700, 333, 9], 16, 4, 128, 64, True),
    ([33], [1100], 12, 4, 64, 128, False), ([257], [300], 5, 1, 128, 16, True), ([300], [1300], 8, 2, 128, 128, False),
    ([40, 7], [10, 0], 6, 2, 64, 16, True),  # more new tokens than keys: the first rows see nothing
    ([129, 128, 127], [129, 1024, 640], 14, 2, 64, 64, True)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page,causal", CHUNK)
def test_attention_chunk(dev, n_new, kv_len, n_q, n_kv, dim, page, causal, int8):
    run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, causal=causal, seed=n_new[0], packed=n_new[0] % 2 == 1)


def test_attention_max_new_changes_no_meaning(dev):
    """A host that does not know the longest chunk still gets the same answer (within the bounds)."""
    for max_new in (0, 1, 5000):
        run_attention(dev, [70, 1], [150, 260], 8, 2, 128, 16, False, seed=5, max_new=max_new)
        run_attention(dev, [1, 1], [150, 260], 8, 2, 128, 16, True, seed=6, max_new=max_new)


@pytest.mark.parametrize("int8", [False, True])
def test_attention_large_scores(dev, int8):
    """Scores in the hundreds: the running maximum has to carry."""
    run_attention(dev, [1, 20], [700, 900], 8, 2, 64, 32, int8, seed=9, q_scale=12.0, scale=1.0)
    run_attention(dev, [1, 200], [1, 300], 8, 2, 128, 32, int8, seed=9, q_scale=0.0)


def test_attention_nan_query_stays_in_its_rows(dev):
    for n_new in ([1, 1], [40, 1]):
        out, qd, on, off, ln = run_attention(dev, n_new, [90, 90], 4, 2, 64, 16, False, seed=3)
        q = qd.clone()
        q[0, 1] = math.nan
        out2 = torch.empty_like(out)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(q.shape[0], 2, 4, 2, 64), dev)
        bd.bd_attention(q, off, bd.KvPages(on["k"], on["v"]), on["table"], ln, 0.125, max(n_new), out2, ws)
        assert out2[0, 1].isnan().all()
        out2[0, 1] = out[0, 1]
        assert torch.equal(out2, out)


def test_attention_reports_bad_indices(dev):
    kp, vp = (torch.ones(3, 1, 16, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
    cache = bd.KvPages(kp, vp)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    for n in (2, 40):
        q = torch.ones(n, 4, 64, device=dev, dtype=torch.bfloat16)
        out = torch.empty_like(q)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(n, 1, 4, 1, 64), dev)
        for table, off, length in (([[0, 3]], [0, n], [32]), ([[-7, 0]], [0, n], [32]), ([[0, 1]], [0, n], [33]),
                                   ([[0, 1]], [0, n], [-1]), ([[0, 1]], [0, n + 1], [32]), ([[0, 1]], [1, 0], [32])):
            bd.bd_attention(q, i32(off), cache, i32(table), i32(length), 0.125, n, out, ws)
            assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX, (table, off, length)
        bd.bd_attention(q, i32([0, n]), cache, i32([[0, 1]]), i32([32]), 0.125, n, out, ws)
        assert bd.bd_check_async(ws) == bd.BD_OK


def test_attention_workspace_may_hold_anything(dev):
    """Scratch past the error word needs no clearing between calls of different kinds."""
    ws_size = bd.bd_attention_workspace_size(300, 3, 16, 2, 128)
    ws = bd.new_workspace(ws_size, dev)
    ws[256:] = 0xFF
    c = ref.paged([1, 100, 3], [900, 333, 50], 2, 128, 16, False, seed=1)
    on = {n: c[n].to(dev) for n in ("k", "v", "table")}
    q = torch.randn(104, 16, 128, generator=gen(8)).to(torch.bfloat16)
    out = torch.empty(104, 16, 128, device=dev, dtype=torch.bfloat16)
    off = torch.tensor([0, 1, 101, 104], dtype=torch.int32, device=dev)
    bd.bd_attention(q.to(dev), off, bd.KvPages(on["k"], on["v"]), on["table"],
                    torch.tensor([900, 333, 50], dtype=torch.int32, device=dev), 0.1, 100, out, ws)
    assert bd.bd_check_async(ws) == bd.BD_OK
    want = ref.attention(q, [0, 1, 101, 104], c["vals"]["k"], c["vals"]["v"], [900, 333, 50], 0.1, True)
    within(out, want[0], ref.attention_bounds(*want, 900)[0], "attention")


# ------------------------------------------------------------------------------- streams and graphs

def test_layer_on_another_stream_and_in_a_graph(dev):
    """norm -> rotary and append -> attention -> read on a side stream, then captured and replayed."""
    T, n_q, n_kv, dim, page = 3, 8, 2, 128, 16
    d = (n_q + 2 * n_kv) * dim
    g = gen(11)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).to(dev)
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    n = torch.empty_like(x)
    kp, vp = (torch.randn(12, n_kv, page, dim, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    cache = bd.KvPages(kp, vp)
    table = torch.arange(12, dtype=torch.int32, device=dev).view(3, 4)
    kv_len = torch.tensor([20, 33, 64], dtype=torch.int32, device=dev)
    slot = torch.tensor([19, 4 * page + 32, 8 * page + 63], dtype=torch.int32, device=dev)
    pos = torch.tensor([19, 32, 63], dtype=torch.int32, device=dev)
    off = torch.arange(4, dtype=torch.int32, device=dev)
    kv_off = torch.tensor([0, 20, 53, 117], dtype=torch.int32, device=dev)
    tab = bd.rope_table(64, dim, 10000.0, dev)
    qo, out = (torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ko, vo = (torch.empty(117, n_kv, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 3, n_q, n_kv, dim), dev)

    def layer():
        bd.bd_rms_norm(x, gain, 1e-5, n, ws)
        h = n.view(T, n_q + 2 * n_kv, dim)
        bd.bd_rope_append(h[:, :n_q], h[:, n_q: n_q + n_kv], h[:, n_q + n_kv:], pos, tab, slot, cache, qo, ws)
        bd.bd_attention(qo, off, cache, table, kv_len, dim ** -0.5, 1, out, ws)
        bd.bd_kv_read(cache, table, kv_off, ko, vo, ws)

    layer()
    torch.cuda.synchronize()
    first = [t.clone() for t in (n, qo, out, ko, vo)]
    side = torch.cuda.Stream()
    for t in (n, qo, out, ko, vo):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (n, qo, out, ko, vo)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for t in (n, qo, out, ko, vo):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (n, qo, out, ko, vo)))
    assert bd.bd_check_async(ws) == bd.BD_OK
