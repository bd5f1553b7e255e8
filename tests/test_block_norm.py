"""The norms around a block with its gate, on the GPU, against the plain 64-bit
definition: odd and long rows, variants, gates of every kind, outputs in place,
rows of zeros, rows that are not finite, sums that cancel, streams and graphs --
and what the entry point refuses."""
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


def definition(x, r, post, gate, gain, bs, rs, eps):
    """(h, y, and the sum of the magnitudes of h's two terms), in float64; gains and gate a row per token, or None."""
    n = x.double()
    if post is not None:
        n = n / (n.pow(2).mean(1, keepdim=True) + eps).sqrt() * post.double()
    if gate is not None:
        n = n * gate.double()
    h = rs * r.double() + bs * n
    size = (rs * r.double()).abs() + (bs * n).abs()
    return h, h / (h.pow(2).mean(1, keepdim=True) + eps).sqrt() * gain.double(), size


def tolerance(h, y, size, gain, eps):
    """Bounds of h and y.  h's terms carry the first norm's relative error (as bd_rms_norm's output) and four more
    roundings; y that of h, of its mean of squares (whose change is at most that of h's 2-norm) and the second norm's."""
    d = h.shape[1]
    dh = size * (ref.norm_rel(d) + 6 * ref.U32)
    mean = h.pow(2).mean(1, keepdim=True) + eps
    turn = dh.pow(2).mean(1, keepdim=True).sqrt() / mean.sqrt()
    dy = dh / mean.sqrt() * gain.double().abs() + y.abs() * (ref.norm_rel(d) + turn)
    return dh, dy * (1 + 2.0 ** -10) + 1e-40


def make(T, d, V, post, gate, seed, spread=1.0):
    g = gen(seed)
    x = (spread * torch.randn(T, d, generator=g)).to(torch.bfloat16)
    r = (2 * torch.randn(T, d, generator=g)).to(torch.bfloat16)
    gains = (1 + 0.2 * torch.randn(V + 1, d, generator=g)).to(torch.bfloat16)
    posts = (1 + 0.2 * torch.randn(V + 1, d, generator=g)).to(torch.bfloat16) if post else None
    vid = torch.randint(-1, V, (T,), generator=g, dtype=torch.int32) if V else None
    rows = {"none": 0, "row": 1, "token": T, "pick": 5}[gate]
    gates = torch.randn(rows, d, generator=g).to(torch.bfloat16) if rows else None
    idx = torch.randint(0, rows, (T,), generator=g, dtype=torch.int32) if gate == "pick" else None
    return x, r, gains, posts, vid, gates, idx


def run(dev, T, d, V, post, gate, out_dtype, seed=0, in_place=None, bs=0.7071, rs=-0.9, eps=1e-5, spread=1.0):
    x, r, gains, posts, vid, gates, idx = make(T, d, V, post, gate, seed, spread)
    which = (vid + 1).long() if V else torch.zeros(T, dtype=torch.long)
    row_gate = None if gates is None else gates[idx.long()] if idx is not None else gates.expand(T, d) if gate == "row" else gates
    bs32, rs32 = float(torch.tensor(bs)), float(torch.tensor(rs))
    h, y, size = definition(x, r, posts[which] if post else None, row_gate, gains[which], bs32, rs32, float(torch.tensor(eps)))
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    xd, rd, gd, pd = on(x), on(r), on(gains), on(posts)
    out = torch.empty(T, d, device=dev, dtype=out_dtype)
    scale = torch.empty(T, device=dev) if out_dtype == torch.float8_e4m3fn else None
    ho = {None: torch.empty_like(xd), "residual": rd, "x": xd}[in_place]
    ws = bd.new_workspace(bd.bd_block_norm_workspace_size(T, d), dev)
    bd.bd_block_norm(xd, rd, gd[0], eps, out, ws, residual_out=ho, post_gain=pd[0] if post else None,
                     gate=on(gates[0] if gate == "row" and T % 2 else gates), gate_idx=on(idx), block_scale=bs,
                     residual_scale=rs, scale=scale, vid=on(vid), gain_list=[gd[v + 1] for v in range(V)],
                     post_gain_list=[pd[v + 1] for v in range(V)] if post else ())
    assert bd.bd_check_async(ws) == bd.BD_OK
    dh, dy = tolerance(h, y, size, gains[which], eps)
    within(ho, h, dh + ref.half_ulp_bf16(h.abs() + dh), "residual")
    return y, dy, out, scale


CASES = [
    (1, 8, 0, True, "none", None), (3, 128, 2, True, "row", None), (32, 8192, 14, True, "row", None),
    (5, 8200, 0, False, "token", "residual"), (7, 16384, 64, True, "pick", None), (2, 33000, 1, True, "pick", "residual"),
    (2, 40000, 3, False, "none", "x"), (3, 40000, 0, True, "token", None), (257, 1000, 5, True, "token", "x"),
    (400, 256, 3, True, "pick", None), (700, 512, 0, False, "row", "residual"), (333, 504, 2, True, "none", None),
    (310, 8192, 0, True, "row", "x"), (420, 4104, 2, False, "pick", None), (1000, 1000, 2, True, "pick", "residual"),
    (320, 20480, 2, True, "token", None), (900, 64, 1, False, "none", None), (2000, 40, 64, True, "token", None)]


@pytest.mark.parametrize("T,d,V,post,gate,in_place", CASES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_block_norm(dev, T, d, V, post, gate, in_place, out_dtype):
    y, dy, out, _ = run(dev, T, d, V, post, gate, out_dtype, seed=d, in_place=in_place)
    within(out, y, dy + ref.half_ulp_bf16(y.abs() + dy) if out_dtype == torch.bfloat16 else dy, "norm")


@pytest.mark.parametrize("T,d,V,post,gate,in_place", CASES)
def test_block_norm_e4m3(dev, T, d, V, post, gate, in_place):
    y, dy, out, scale = run(dev, T, d, V, post, gate, torch.float8_e4m3fn, seed=T, in_place=in_place)
    amax = y.abs().amax(1)
    rel = (dy / y.abs().amax(1, keepdim=True)).amax(1) + 4 * ref.U32
    s = amax.clamp_min(1e-30) / 448
    within(scale, s, s * rel, "scale")
    z = (y / s[:, None]).abs()
    # (a value next to a power of two may be rounded with the step above it)
    half_step = torch.where(z >= 2.0 ** -6, torch.pow(2.0, torch.floor(torch.log2((z * 1.001).clamp_min(2.0 ** -6))) - 4),
                            torch.full_like(z, 2.0 ** -10))
    within(out.float().cpu().double() * scale.cpu().double()[:, None], y,
           s[:, None] * half_step * (1 + 2.0 ** -10) + dy + y.abs() * 2 * rel[:, None], "codes")


def test_sums_that_cancel(dev):
    """h is what is left of two large terms: its norm has to be that of what is left."""
    T, d = 5, 2048
    g = gen(3)
    r = (100 * torch.randn(T, d, generator=g)).to(torch.bfloat16)
    x = -r.clone()
    x[:, ::7] += 0.5 * torch.randn(T, len(range(0, d, 7)), generator=g).to(torch.bfloat16)
    gain = torch.ones(d, dtype=torch.bfloat16)
    h, y, size = definition(x, r, None, None, gain.expand(T, d), 1.0, 1.0, 1e-5)
    out, ws = torch.empty(T, d, device=dev), bd.new_workspace(256, dev)
    bd.bd_block_norm(x.to(dev), r.to(dev), gain.to(dev), 1e-5, out, ws)
    within(out, y, y.abs() * (ref.norm_rel(d) + 4 * ref.U32), "norm")  # (the sum itself is exact)


def test_zero_and_nonfinite_rows(dev):
    d = 256
    x = torch.randn(6, d, generator=gen(1)).to(torch.bfloat16)
    r = torch.randn(6, d, generator=gen(2)).to(torch.bfloat16)
    x[0], r[0] = 0, 0
    x[1, 7] = math.nan
    r[2, 9] = math.inf
    x[3] = 0
    r[4] = 0
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    ws = bd.new_workspace(256, dev)
    for post in (gain, None):
        out, ho = torch.empty(6, d, device=dev), torch.empty(6, d, device=dev, dtype=torch.bfloat16)
        bd.bd_block_norm(x.to(dev), r.to(dev), gain, 1e-5, out, ws, residual_out=ho, post_gain=post)
        o = out.cpu()
        assert (o[0] == 0).all() and (ho[0] == 0).all() and o[1].isnan().all() and o[2, 9].isnan()
        assert o[3:].isfinite().all() and torch.equal(ho[3].cpu(), r[3])
        o8, sc = torch.empty(6, d, device=dev, dtype=torch.float8_e4m3fn), torch.empty(6, device=dev)
        bd.bd_block_norm(x.to(dev), r.to(dev), gain, 1e-5, o8, ws, scale=sc, post_gain=post)
        assert (o8[0].float() == 0).all() and sc[0] > 0 and not sc[1].isfinite() and not sc[2].isfinite()
        assert sc[3:].isfinite().all() and o8[3:].float().isfinite().all()


def test_bad_variants_and_gate_rows(dev):
    """Ids and rows out of range are reported, and take the base's gains and the first row."""
    T, d = 4, 64
    x, r, gains, posts, _, gates, _ = make(T, d, 1, True, "pick", 2)
    on = [t.to(dev) for t in (x, r, gains, posts, gates)]
    xd, rd, gd, pd, gg = on
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    out, base = (torch.empty(T, d, device=dev) for _ in range(2))
    ws = bd.new_workspace(256, dev)
    lists = dict(gain_list=[gd[1]], post_gain_list=[pd[1]])

    def call(to, vid, idx, gate=gg):
        bd.bd_block_norm(xd, rd, gd[0], 1e-5, to, ws, post_gain=pd[0], gate=gate, gate_idx=i32(idx), vid=i32(vid), **lists)

    call(base, [-1] * 4, [0] * 4)
    assert bd.bd_check_async(ws) == bd.BD_OK
    call(out, [0, 1, -2, -1], [0, 0, 0, 0])
    assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_VARIANT and bd.bd_check_async(ws) == bd.BD_OK
    assert torch.equal(out[1:], base[1:]) and not torch.equal(out[0], base[0])
    call(out, [-1] * 4, [1, 5, -1, 0])
    assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX and bd.bd_check_async(ws) == bd.BD_OK
    assert torch.equal(out[1:], base[1:]) and not torch.equal(out[0], base[0])
    call(out, [-1] * 4, [0, 1, -1, 0], gate=gg[:1])
    assert bd.bd_check_async(ws) == bd.BD_ERR_BAD_INDEX
    assert torch.equal(out, base)


def test_as_rms_norm(dev):
    """Without gate, scales and norm after the block it is bd_rms_norm with a residual, bit for bit."""
    for T, d in ((33, 8192), (500, 512), (400, 1000), (2, 40000)):
        x, r, gains, _, vid, _, _ = (t.to(dev) if t is not None else None for t in make(T, d, 3, False, "none", T))
        a, b = (torch.empty(T, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
        ha, hb = torch.empty_like(a), torch.empty_like(b)
        ws = bd.new_workspace(256, dev)
        bd.bd_rms_norm(x, gains[0], 1e-5, a, ws, residual=r, residual_out=ha, vid=vid, gain_list=list(gains[1:]))
        bd.bd_block_norm(x, r, gains[0], 1e-5, b, ws, residual_out=hb, vid=vid, gain_list=list(gains[1:]))
        assert torch.equal(ha, hb)
        assert (a.float() - b.float()).abs().max() <= a.float().abs().max() * 2.0 ** -8


def test_same_bits_in_a_graph_and_on_a_stream(dev):
    for T, d in ((4, 8192), (600, 512), (700, 8192)):
        x, r, gains, posts, vid, gates, _ = (t.to(dev) if t is not None else None for t in make(T, d, 2, True, "token", T))
        out, ho = torch.empty(T, d, device=dev), torch.empty_like(x)
        ws = bd.new_workspace(256, dev)

        def call():
            bd.bd_block_norm(x, r, gains[0], 1e-5, out, ws, residual_out=ho, post_gain=posts[0], gate=gates, vid=vid,
                             gain_list=list(gains[1:]), post_gain_list=list(posts[1:]))

        call()
        torch.cuda.synchronize()
        first = out.clone(), ho.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        out.zero_(), ho.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(ho, first[1])
        side = torch.cuda.Stream()
        out.zero_(), ho.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(ho, first[1])


def test_no_rows(dev):
    e = torch.empty(0, 64, device=dev, dtype=torch.bfloat16)
    bd.bd_block_norm(e, e, torch.ones(64, device=dev, dtype=torch.bfloat16), 1e-5, torch.empty_like(e),
                     bd.new_workspace(256, dev))
