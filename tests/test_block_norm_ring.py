"""The norms around a block where there are many rows (GPU): the kernel whose rows
come through a ring, by warps and by blocks, with two stages and with more, on its
rare paths -- rows of zeros, rows that are not finite, sums that cancel, ids and
gate rows out of range in the first and in later turns of the ring, 8-bit rows so
small that their factor leaves fp32's range -- against the plain 64-bit definition."""
import math

import pytest
import torch

import layer_oracle as ref
from bit_weight_delta_bd_gb300 import bitdelta as bd
from test_block_norm import definition, dev, gen, tolerance, within  # noqa: F401  (dev is a fixture)

pytestmark = pytest.mark.gpu

# by warps with 1, 2 and 4 groups a thread, by blocks with three stages or more and with two
SHAPES = [(700, 256), (20000, 256), (700, 504), (700, 1000), (20000, 1000), (400, 5120), (400, 8192), (3000, 8192), (400, 16384)]


def data(T, d, seed, dev):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(seed)
    return [torch.randn(T, d, generator=g, device=dev).to(torch.bfloat16) for _ in range(2)]


def spread(T, n):
    """n rows from the first to the last, of every turn of the ring."""
    return torch.linspace(0, T - 1, n).long()


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("post", [True, False])
def test_zero_and_nonfinite_rows(dev, T, d, post):  # noqa: F811
    """A row that is not finite leaves every other as it is, those of the same warp, block and stage too."""
    x, r = data(T, d, 1, dev)
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    rows = spread(T, 60)
    zero, nan, inf, ninf = rows[0::4], rows[1::4], rows[2::4], rows[3::4]
    hit = torch.zeros(T, dtype=torch.bool)
    hit[rows] = True
    ws = bd.new_workspace(256, dev)
    results = []
    for bad in (False, True):
        if bad:
            x[zero], r[zero] = 0, 0
            x[nan, d - 1] = math.nan
            r[inf, 7] = math.inf
            x[ninf, d // 2] = -math.inf
        out, ho = torch.empty(T, d, device=dev), torch.empty_like(x)
        o16, o8, sc = torch.empty_like(x), torch.empty(T, d, device=dev, dtype=torch.float8_e4m3fn), torch.empty(T, device=dev)
        for o, s in ((out, None), (o16, None), (o8, sc)):
            bd.bd_block_norm(x, r, gain, 1e-5, o, ws, residual_out=ho, scale=s, post_gain=gain if post else None)
        assert bd.bd_check_async(ws) == bd.BD_OK
        results.append([t.cpu() for t in (out, ho, o16, o8.float(), sc)])
    for a, b in zip(*results):
        assert torch.equal(a[~hit], b[~hit])
    out, ho, o16, o8, sc = results[1]
    for t in (out, ho, o16, o8):
        assert (t[zero] == 0).all()
    assert (sc[zero] == torch.tensor(1e-30) / torch.tensor(448.0)).all()
    assert out[nan].isnan().all() and o16[nan].isnan().all() and not sc[nan].isfinite().any()
    assert out[inf, 7].isnan().all() and (ho[inf, 7] == math.inf).all() and not sc[inf].isfinite().any()
    # (-infinity over a norm that is infinite is NaN, in the norm after the block already)
    assert not sc[ninf].isfinite().any() and not ho[ninf, d // 2].isfinite().any() and out[ninf, d // 2].isnan().all()


@pytest.mark.parametrize("T,d", SHAPES)
def test_sums_that_cancel(dev, T, d):  # noqa: F811
    """h is what is left of two large terms: its norm has to be that of what is left."""
    g = torch.Generator(device=dev).manual_seed(3)
    r = (100 * torch.randn(T, d, generator=g, device=dev)).to(torch.bfloat16)
    x = -r.clone()
    x[:, ::7] += 0.5 * torch.randn(T, len(range(0, d, 7)), generator=g, device=dev).to(torch.bfloat16)
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    out, ws = torch.empty(T, d, device=dev), bd.new_workspace(256, dev)
    bd.bd_block_norm(x, r, gain, 1e-5, out, ws)
    h, y, _ = definition(x.cpu(), r.cpu(), None, None, gain.cpu().expand(T, d), 1.0, 1.0, 1e-5)
    within(out, y, y.abs() * (ref.norm_rel(d) + 4 * ref.U32), "norm")  # (the sum itself is exact)


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("post", [True, False])
def test_bad_variants_and_gate_rows(dev, T, d, post):  # noqa: F811
    """Ids and rows out of range are reported, one at a time, and take the base's gains and the first row."""
    x, r = data(T, d, 2, dev)
    g = torch.Generator(device=dev).manual_seed(5)
    gains, posts, gates = (torch.randn(n, d, generator=g, device=dev).to(torch.bfloat16) for n in (3, 3, 4))
    out, base = (torch.empty(T, d, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ws = bd.new_workspace(256, dev)
    vid, idx = (torch.randint(lo, hi, (T,), generator=g, device=dev, dtype=torch.int32) for lo, hi in ((-1, 2), (0, 4)))

    def call(to, vid, idx, gate=gates):
        bd.bd_block_norm(x, r, gains[0], 1e-5, to, ws, post_gain=posts[0] if post else None, gate=gate, gate_idx=idx,
                         vid=vid, gain_list=list(gains[1:]), post_gain_list=list(posts[1:]) if post else ())
        return bd.bd_check_async(ws)

    for i, at in enumerate(spread(T, 9).tolist() + [min(T - 1, 304 * 8 + 3)]):
        v, w = vid.clone(), idx.clone()
        v[at], w[at] = -1, 0
        assert call(base, v, w) == bd.BD_OK
        v[at] = (2, -2, 2 ** 31 - 1, -2 ** 31)[i % 4]
        assert call(out, v, w) == bd.BD_ERR_BAD_VARIANT and torch.equal(out, base)
        v[at], w[at] = -1, (4, -1, -2 ** 31, 2 ** 31 - 1)[i % 4]
        assert call(out, v, w) == bd.BD_ERR_BAD_INDEX and torch.equal(out, base)
        zeros = torch.zeros_like(idx)
        assert call(base, v, zeros, gates[:1]) == bd.BD_OK
        zeros[at] = (1, -1)[i % 2]
        assert call(out, v, zeros, gates[:1]) == bd.BD_ERR_BAD_INDEX and torch.equal(out, base)


@pytest.mark.parametrize("T,d", [(300, 1000), (700, 256), (700, 504), (700, 1000), (400, 5120), (400, 8192), (400, 16384)])
@pytest.mark.parametrize("small,gain_size,eps", [
    (2.0 ** -60, 2.0 ** -62, 2.0 ** -70),   # |h gain| near 2^-122: 448 over it is past fp32's range
    (2.0 ** -62, 2.0 ** -60, 0.0),          # the same without eps: the factor is near 2^62
    (2.0 ** -60, 2.0 ** -62, 2.0 ** -40),   # |y| near 2^-102: it counts as 1e-30
    (2.0 ** -60, 2.0 ** -60, 2.0 ** -47),   # near 2^-96, next to that border
    (1.0, 1.0, 1e-5)])
def test_e4m3_of_tiny_rows(dev, T, d, small, gain_size, eps):  # noqa: F811
    """Codes and scale are the definition's wherever |h gain| is a normal number (elements below 2^-126 may be off by
    2^-149, the step of numbers there)."""
    g = gen(9)
    r = (small * torch.randn(T, d, generator=g)).to(torch.bfloat16)
    gain = (gain_size * (1 + 0.2 * torch.randn(d, generator=g))).to(torch.bfloat16)
    x = torch.zeros_like(r)
    out, sc = torch.empty(T, d, device=dev, dtype=torch.float8_e4m3fn), torch.empty(T, device=dev)
    ws = bd.new_workspace(256, dev)
    bd.bd_block_norm(x.to(dev), r.to(dev), gain.to(dev), eps, out, ws, scale=sc)
    assert bd.bd_check_async(ws) == bd.BD_OK
    h, y, size = definition(x, r, None, None, gain.expand(T, d), 1.0, 1.0, eps)
    amax = y.abs().amax(1)
    s = amax.clamp_min(1e-30) / 448
    rel = ref.norm_rel(d) + 8 * ref.U32
    mult = (h.pow(2).mean(1, keepdim=True) + eps).rsqrt()  # of h gain, whose last bit may be 2^-149
    within(sc, s, s * rel + mult[:, 0] * 2.0 ** -149 / 448, "scale")
    z = (y / s[:, None]).abs()
    half_step = torch.where(z >= 2.0 ** -6, torch.pow(2.0, torch.floor(torch.log2((z * 1.001).clamp_min(2.0 ** -6))) - 4),
                            torch.full_like(z, 2.0 ** -10))
    step = mult * 2.0 ** -149
    within(out.float().cpu().double(), y / s[:, None],
           half_step * (1 + 2.0 ** -10) + z * 3 * rel + (1 + z / 448) * step / s[:, None], "codes")


@pytest.mark.parametrize("T,d", [(300, 1000), (700, 256), (700, 1000), (400, 8192), (400, 16384)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("x_size,post_size,r_size,block_scale,residual_scale", [
    (2.0 ** -58, 2.0 ** -22, 1.0, 2.0 ** 72, 2.0 ** 50),  # block_scale over x's root mean square is past fp32's range
    (2.0 ** 50, 2.0 ** 30, 2.0 ** -20, -2.0 ** -85, 2.0 ** -35),  # and here below its normal numbers
    (2.0 ** -58, 1.0, 1.0, 2.0 ** 40, 2.0 ** 40), (2.0 ** 50, 1.0, 1.0, 2.0 ** -50, 2.0 ** -50)])
def test_block_scales_of_any_size(dev, T, d, gated, x_size, post_size, r_size, block_scale, residual_scale):  # noqa: F811
    """Wherever the formula's own factors, and the squares that it sums, are in fp32's range, so is the result."""
    g = gen(T + d)
    x, r, post, gate = ((n * torch.randn(*m, generator=g)).to(torch.bfloat16)
                        for n, m in ((x_size, (T, d)), (r_size, (T, d)), (post_size, (d,)), (1.0, (T, d))))
    gain = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    out, ho = torch.empty(T, d, device=dev), torch.empty(T, d, device=dev, dtype=torch.bfloat16)
    ws = bd.new_workspace(256, dev)
    bd.bd_block_norm(x.to(dev), r.to(dev), gain.to(dev), 0.0, out, ws, residual_out=ho, post_gain=post.to(dev),
                     gate=gate.to(dev) if gated else None, block_scale=block_scale, residual_scale=residual_scale)
    assert bd.bd_check_async(ws) == bd.BD_OK
    h, y, size = definition(x, r, post.expand(T, d), gate if gated else None, gain.expand(T, d), block_scale, residual_scale, 0.0)
    dh, dy = tolerance(h, y, size, gain.expand(T, d), 0.0)
    within(ho, h, dh + ref.half_ulp_bf16(h.abs() + dh), "residual")
    within(out, y, dy, "norm")


@pytest.mark.parametrize("T,d", SHAPES + [(33, 8192), (2, 40000)])
def test_elements_as_rms_norm(dev, T, d):  # noqa: F811
    """Without gate, scales and norm after the block each element is bd_rms_norm's with a residual but for the order of
    sums and products in fp32: at most a step of bf16 apart, and mostly equal."""
    x, r = data(T, d, 6, dev)
    gain = torch.randn(d, generator=torch.Generator(device=dev).manual_seed(7), device=dev).to(torch.bfloat16)
    a, b, ha, hb = (torch.empty_like(x) for _ in range(4))
    ws = bd.new_workspace(256, dev)
    bd.bd_rms_norm(x, gain, 1e-5, a, ws, residual=r, residual_out=ha)
    bd.bd_block_norm(x, r, gain, 1e-5, b, ws, residual_out=hb)
    assert torch.equal(ha, hb)
    near = (a.float() - b.float()).abs()
    # both are within norm_rel of the formula before they are rounded, and a step of bf16 is 2^-7 at most
    assert bool((near <= 2.0 ** -7 * (1 + 2.0 ** -8) * a.float().abs()).all())
    assert float((near > 0).float().mean()) <= 2 * 2 * ref.norm_rel(d) * 2.0 ** 8
