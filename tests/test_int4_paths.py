"""The 4-bit cache and the norms around a block where they are used whole (GPU):
buffers whose offsets pass 32 bits, wide strides, 16-byte boundaries, masks and
scales of any sign, two streams and two graphs of one workspace, results that do
not depend on the run, the bounds-checked build, and the example's block."""
import math
import os
import subprocess
import sys

import pytest
import torch

import int4_oracle as ref4
import layer_oracle as ref
import test_int4_attention as att
import test_layer_large as large
from bit_weight_delta_bd_gb300 import bitdelta as bd
from test_int4_attention import cache_on, dev, gen, within  # noqa: F401  (dev is a fixture)

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def ints(values, dev):  # noqa: F811
    return torch.tensor(values, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------------------- masks and scales

FEW = [([1, 2, 1], [900, 300, 1], 16, 2, 128, 16), ([2, 0, 8], [70, 9, 4100], 4, 2, 64, 64), ([16], [1], 3, 3, 128, 32)]
MANY = [([40, 1], [300, 65], 16, 2, 128, 16), ([129, 3], [129, 1000], 4, 1, 64, 64), ([600], [700], 2, 2, 128, 32)]


@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", FEW + MANY)
def test_without_a_causal_mask(dev, n_new, kv_len, n_q, n_kv, dim, page):  # noqa: F811
    att.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, causal=False, seed=sum(kv_len) % 91)


@pytest.mark.parametrize("scale", [-0.1, 0.0, -1.0])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", FEW + MANY)
def test_scales_of_any_sign(dev, n_new, kv_len, n_q, n_kv, dim, page, scale):  # noqa: F811
    att.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, scale=scale, seed=sum(kv_len) % 83)


@pytest.mark.parametrize("n_new,max_new", [([1, 300, 1, 2], 300), ([1, 300, 1, 2], 1), ([16, 17, 1, 0], 2 ** 62)])
@pytest.mark.parametrize("dim,n_q,n_kv", [(128, 8, 1), (64, 4, 4)])
def test_any_mixture_and_hint(dev, n_new, max_new, dim, n_q, n_kv):  # noqa: F811
    """(Which kernel a sequence takes is not the test's to know: the bounds are the wider ones of both.)"""
    att.run_attention(dev, n_new, [900, 1200, 5, 64], n_q, n_kv, dim, 16, seed=dim + n_new[0], max_new=max_new,
                      coded_rel=ref4.U11, value_rel=2 * ref.U16)


@pytest.mark.parametrize("n_new", [1, 40])
@pytest.mark.parametrize("gap", [4, 8, 12])
def test_small_probabilities(dev, n_new, gap):  # noqa: F811
    """One key has all the weight but what `gap` (in units of the exponential) leaves to the others, and values of 0,
    code and lowest value, in every group but the first: there the others' products are the result.  They lie 2^-17.3 at
    most below the largest product of the row, where the few rows' fp16 still has 11 bits."""
    dim, length, page = 64, 120, 16
    g = gen(gap + n_new)
    c = ref4.paged([n_new], [length], 1, dim, page, 5, spare=0)
    pg = c["table"][0, : -(-length // page)].long()
    c["k"][:] = 0
    c["ks"][..., 0], c["ks"][..., 1] = 1.0, 0.0
    c["v"][:] = torch.randint(0, 256, c["v"].shape, generator=g, dtype=torch.uint8)
    c["vs"][..., 0], c["vs"][..., 1] = 0.125, 0.0
    c["k"][pg[0], 0, 3, 0] = 15  # element 0 of key 3
    c["vs"][pg[0], 0, 3, 1, 0] = 0.0
    q = torch.zeros(n_new, 1, dim)
    q[..., 0] = gap / 15
    q = q.to(torch.bfloat16)
    k, v = (ref4.values(c[n][pg], c[n + "s"][pg]).transpose(1, 2).flatten(0, 1)[:length] for n in "kv")
    cache, table = cache_on(c, dev)
    out = torch.empty(n_new, 1, dim, device=dev, dtype=torch.bfloat16)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(n_new, 1, 1, 1, dim), dev)
    bd.bd_attention(q.to(dev), ints([0, n_new], dev), cache, table, ints([length], dev), 1.0, n_new, out, ws)
    assert bd.bd_check_async(ws) == bd.BD_OK
    want = ref.attention(q, [0, n_new], [k], [v], [length], 1.0, True)
    # scores of one product each; probability (times scale) and value rounded to 8 bits at worst, sums in fp32
    bound = want[0].abs() * (2 * ref.U16 + gap * 2.0 ** -20 + (length + 64) * 2.0 ** -21)
    within(out, want[0], bound + ref.half_ulp_bf16(want[0].abs() + bound), "attention")


# ------------------------------------------------------------------------------- sizes far apart

SIZES = [  # of token j's key and value, and the scale
    (lambda j: 2.0 ** (20 * (j % 3) - 20), lambda j: 1.0, 0.02),
    (lambda j: 1.0, lambda j: 2.0 ** (20 * (j % 3) - 20), 0.1),
    (lambda j: 2.0 ** (-30 if j % 5 else 0), lambda j: 2.0 ** (30 if j % 7 else -40), 0.1),
    (lambda j: 1.0, lambda j: 2.0 ** (60 if 100 <= j < 110 else -60), 0.1),  # a tile of each kind
    (lambda j: 1.0, lambda j: 2.0 ** (-60 if j < 128 else 60 if j < 256 else 0), 0.1)]


@pytest.mark.parametrize("sizes", range(len(SIZES)))
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", [
    ([1, 2], [300, 129], 8, 2, 64, 16), ([300], [333], 8, 2, 128, 16), ([40, 130], [300, 200], 4, 2, 64, 64),
    ([20, 5], [400, 77], 4, 2, 128, 32)])
def test_magnitudes_in_every_kernel(dev, n_new, kv_len, n_q, n_kv, dim, page, sizes):  # noqa: F811
    """Few rows, pairs, single blocks: keys and values of neighbouring tokens, and of tiles, far apart.  (fp16's bits
    reach 2^-25 below a row's largest product; the bound is 8 bits of all products together.)"""
    key_of, value_of, scale = SIZES[sizes]
    c = att.scaled_cache(n_new, kv_len, n_kv, dim, page, 7, key_of, value_of)
    att.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, seed=7, scale=scale, c=c, coded_rel=ref.U16,
                      value_rel=2 * ref.U16)


@pytest.mark.parametrize("what", [2.0 ** 40, 2.0 ** 80, -2.0 ** 80])
@pytest.mark.parametrize("n_new,n_q,dim", [(2, 8, 128), (40, 8, 128), (300, 8, 128), (40, 4, 64)])
def test_hidden_values_of_any_size(dev, n_new, n_q, dim, what):  # noqa: F811
    """Values that a causal row does not see, however large, leave it what it was to the bounds of its own."""
    length = n_new + 30
    c = ref4.paged([n_new], [length], 2, dim, 16, 3)
    pg, at = c["table"][0, (length - 1) // 16].long(), (length - 1) % 16
    c["vs"][pg, :, at, :, 1] = what  # the last token's, which its own rows alone see
    c["vals"]["v"][0][-1] = ref4.values(c["v"][pg, :, at], c["vs"][pg, :, at])
    att.run_attention(dev, [n_new], [length], n_q, 2, dim, 16, seed=3, c=c, coded_rel=ref.U16, value_rel=2 * ref.U16)


@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("n_new,max_new,dim", [([1, 1], 1, 64), ([40, 1], 40, 64), ([300, 2], 300, 128), ([30, 1], 30, 128)])
def test_values_that_are_not_finite_stay_in_their_group(dev, n_new, max_new, dim, part, what):  # noqa: F811
    """A scale or lowest value of a seen value that is not finite reaches the dims of its group, of the rows that see
    it; the key's other groups, larger than every other token's, are what they were."""
    lens = [n + 90 for n in n_new]
    c = ref4.paged(n_new, lens, 2, dim, 16, 3)
    pg, at = c["table"][0, 10 // 16].long(), 10 % 16  # key 10, before every new token
    c["vs"][pg, 1, at, :, 1] = 100.0
    c["vals"]["v"][0][10] = ref4.values(c["v"][pg, :, at], c["vs"][pg, :, at])
    base, q, _, _, off, ln = att.run_attention(dev, n_new, lens, 4, 2, dim, 16, seed=3, c=c, max_new=max_new,
                                               coded_rel=ref4.U11, value_rel=2 * ref.U16)
    c["vs"][pg, 1, at, 1, part] = what
    cache, table = cache_on(c, dev)
    out = torch.empty_like(base)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(sum(n_new), 2, 4, 2, dim), dev)
    bd.bd_attention(q, off, cache, table, ln, dim ** -0.5, max_new, out, ws)
    hit = torch.zeros_like(base, dtype=torch.bool)
    hit[: n_new[0], 2:, 32:64] = True
    assert not out[hit].isfinite().any()
    # (another factor may have been taken for the tile, or reference for the row: a rounding's width apart)
    near = (out[~hit].float() - base[~hit].float()).abs()
    assert bool((near <= 2.0 ** -7 * base[~hit].float().abs() + 2.0 ** -9).all())


# ------------------------------------------------------------------------------- the ends of the sizes

def test_a_hint_of_no_new_tokens(dev):  # noqa: F811
    att.run_attention(dev, [1, 40], [300, 200], 8, 2, 128, 16, seed=5, max_new=0, coded_rel=ref4.U11, value_rel=2 * ref.U16)


def test_as_many_heads_as_there_may_be(dev):  # noqa: F811
    """1024 kv heads: written, read back, attended to by few rows and by a chunk."""
    for T in (1, 40):
        run, need, (_, _, qo, out, ko, vo) = layer(dev, T, [T], [T + 3], 2048, 1024, 64, 16)
        ws = bd.new_workspace(need, dev)
        run(ws)
        assert bd.bd_check_async(ws) == bd.BD_OK
        want = ref.attention(qo[:, ::194].cpu(), [0, T], [ko[:, ::97].cpu()], [vo[:, ::97].cpu()], [T + 3], 0.125, True)[0]
        assert float((out[:, ::194].double().cpu() - want).norm() / want.norm()) <= 0.02


# ------------------------------------------------------------------------------- past 32 bits

def test_cache_past_32_bits(dev):  # noqa: F811
    """Sequences on the last pages of a cache with more than 2^32 bytes of scales of keys (and four times that of codes)
    give what the same tokens give on the first pages."""
    n_kv, page, dim, n_q = 8, 128, 128, 32
    n_pages = 2 ** 32 // (n_kv * page * dim // 32 * 4) + 12
    cache = bd.KvPages(*(torch.empty(n_pages, n_kv, page, dim // 2, dtype=torch.uint8, device=dev) for _ in range(2)),
                       *(torch.empty(n_pages, n_kv, page, dim // 32, 2, dtype=torch.bfloat16, device=dev) for _ in range(2)))
    lens = [700, 129]
    pages = [[0, 3, 1, 2, 5, 4], [6, 7, 8, 9, 10, 11]]
    T = sum(lens)
    g = gen(9)
    q, k, v = (torch.randn(T, h, dim, generator=g).to(torch.bfloat16).to(dev) for h in (n_q, n_kv, n_kv))
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
    tab = bd.rope_table(1024, dim, 10000.0, dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 2, n_q, n_kv, dim), dev)
    off, one, kv_len = ints([0, lens[0], T], dev), ints([0, 1, 2], dev), ints(lens, dev)
    runs = []
    for first in (0, n_pages - 12):
        table = torch.tensor(pages, dtype=torch.int32) + first
        slot = (table[seq, pos // page] * page + pos % page).to(torch.int32).to(dev)
        table = table.to(dev)
        qo, out = torch.empty_like(q), torch.empty_like(q)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        step = torch.empty(2, n_q, dim, device=dev, dtype=torch.bfloat16)
        bd.bd_rope_append(q, k, v, pos.to(torch.int32).to(dev), tab, slot, cache, qo, ws)
        bd.bd_kv_read(cache, table, off, ko, vo, ws)
        bd.bd_attention(qo, off, cache, table, kv_len, dim ** -0.5, max(lens), out, ws)
        bd.bd_attention(qo[[lens[0] - 1, T - 1]].contiguous(), one, cache, table, kv_len, dim ** -0.5, 1, step, ws)
        assert bd.bd_check_async(ws) == bd.BD_OK
        runs.append([qo, ko, vo, out, step])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    near = ref.attention(runs[0][0].cpu(), [0, lens[0], T], *[
        [t[: lens[0]].cpu(), t[lens[0]:].cpu()] for t in (runs[0][1], runs[0][2])], lens, dim ** -0.5, True)[0]
    assert float((runs[0][3].double().cpu() - near).norm() / near.norm()) <= 0.02


def test_strides_past_32_bits(dev):  # noqa: F811
    """Rows of q, k and v that lie 2^24 elements apart, past 2^31 elements from the first."""
    T, n_q, n_kv, dim, page, stride = 200, 8, 2, 128, 16, 2 ** 24 + 8
    wide = torch.empty((T - 1) * stride + 2048, dtype=torch.bfloat16, device=dev)
    near = torch.randn(T, n_q + 2 * n_kv, dim, generator=gen(4)).to(torch.bfloat16).to(dev)
    far = wide.as_strided(near.shape, (stride, dim, 1))
    far.copy_(near)
    pos, off = torch.arange(T, dtype=torch.int32, device=dev), ints([0, T], dev)
    table = torch.arange(13, dtype=torch.int32, device=dev).view(1, 13)
    tab = bd.rope_table(T, dim, 10000.0, dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 1, n_q, n_kv, dim), dev)
    runs = []
    for x in (near, far):
        cache = att.empty_cache(13, n_kv, page, dim, dev)
        out = torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16)
        q = x[:, :n_q]
        bd.bd_rope_append(q, x[:, n_q: n_q + n_kv], x[:, n_q + n_kv:], pos, tab, pos, cache, q, ws)  # in place
        bd.bd_attention(q, off, cache, table, ints([T], dev), 0.1, T, out, ws)
        assert bd.bd_check_async(ws) == bd.BD_OK
        runs.append([q.clone(), cache.k, cache.v, cache.k_scale, cache.v_scale, out])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("d", [8192, 1000])
def test_norm_past_32_bits(dev, d):  # noqa: F811
    """Rows whose elements lie past 2^31 equal the same rows at the front, in place and with a gate of their own."""
    T = 2 ** 31 // d + 300
    x = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    x[:64].normal_(generator=torch.Generator(device=dev).manual_seed(3))
    x[64:-64] = 1.0
    x[-64:] = x[:64]
    gain = torch.randn(d, device=dev, generator=torch.Generator(device=dev).manual_seed(4)).to(torch.bfloat16)
    out, gate = torch.zeros_like(x), x.clone()
    ws = bd.new_workspace(bd.bd_block_norm_workspace_size(T, d), dev)
    bd.bd_block_norm(x, x, gain, 1e-5, out, ws, residual_out=x, post_gain=gain, gate=gate)
    assert bd.bd_check_async(ws) == bd.BD_OK
    assert torch.equal(out[-64:], out[:64]) and bool((out[:64] != 0).any())
    assert torch.equal(x[-64:], x[:64]) and not torch.equal(x[:64], gate[:64])


# ------------------------------------------------------------------------------- where buffers lie

def moved(t):
    u = torch.empty(t.numel() + 16 // t.element_size(), device=t.device, dtype=t.dtype)[16 // t.element_size():]
    u.copy_(t.flatten())
    assert u.data_ptr() % 32 == 16
    return u.view(t.shape)


@pytest.mark.parametrize("dim,n_kv", [(128, 2), (64, 1)])
def test_cache_on_16_byte_boundaries(dev, dim, n_kv):  # noqa: F811
    """Buffers 16 bytes off the start of a 32-byte sector give the same bits as ones on it."""
    T, n_q, page = 300, 8, 16
    g = torch.Generator(device=dev).manual_seed(6)
    q, k, v = (torch.randn(T, h, dim, generator=g, device=dev).to(torch.bfloat16) for h in (n_q, n_kv, n_kv))
    pos, off = torch.arange(T, dtype=torch.int32, device=dev), ints([0, T], dev)
    one = ints([0, 1], dev)
    table = torch.arange(20, dtype=torch.int32, device=dev).view(1, 20)
    tab = bd.rope_table(T, dim, 10000.0, dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 1, n_q, n_kv, dim), dev)
    for inter in (False, True):
        runs = []
        for place in (lambda t: t, moved):
            c = att.empty_cache(20, n_kv, page, dim, dev)
            cache = bd.KvPages(*(place(t) for t in (c.k, c.v, c.k_scale, c.v_scale)))
            qo, out, ko, vo = (place(torch.zeros_like(t)) for t in (q, q, k, v))
            step = place(torch.zeros_like(q[:1]))
            bd.bd_rope_append(place(q), place(k), place(v), pos, tab, pos, cache, qo, ws, interleaved=inter)
            bd.bd_kv_read(cache, table, off, ko, vo, ws)
            bd.bd_attention(qo, off, cache, table, off[1:], dim ** -0.5, T, out, ws)
            bd.bd_attention(qo[:1], one, cache, table, off[1:], dim ** -0.5, 1, step, ws)
            assert bd.bd_check_async(ws) == bd.BD_OK
            runs.append([cache.k, cache.v, cache.k_scale, cache.v_scale, qo, ko, vo, out, step])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("T,d", [(5, 8200), (400, 1000), (400, 8192), (3, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn])
def test_norm_on_16_byte_boundaries_and_in_place(dev, T, d, dtype):  # noqa: F811
    """The same bits wherever the buffers lie, and where the residual stream takes h's place or is x itself."""
    g = torch.Generator(device=dev).manual_seed(7)
    x, r, gate = (torch.randn(T, d, generator=g, device=dev).to(torch.bfloat16) for _ in range(3))
    gain = torch.randn(d, generator=g, device=dev).to(torch.bfloat16)
    ws = bd.new_workspace(256, dev)

    def run(x, r, gate, gain, ro, place=lambda t: t):
        out = place(torch.zeros(T, d, device=dev, dtype=dtype))
        scale = torch.zeros(T, device=dev) if dtype == torch.float8_e4m3fn else None
        bd.bd_block_norm(x, r, gain, 1e-5, out, ws, residual_out=ro, post_gain=gain, gate=gate, scale=scale)
        assert bd.bd_check_async(ws) == bd.BD_OK
        return [out.view(torch.uint8), ro, *([scale] if scale is not None else [])]

    first = run(x, r, gate, gain, torch.zeros_like(x))
    xs, rs = x.clone(), r.clone()
    for again in (run(*map(moved, (x, r, gate, gain, x)), moved), run(x, rs, gate, gain, rs), run(xs, r, gate, gain, xs)):
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    both = x.clone()
    first = run(x, x, gate, gain, torch.zeros_like(x))
    assert all(torch.equal(a, b) for a, b in zip(first, run(both, both, gate, gain, both)))


# ------------------------------------------------------------------------------- one result

def layer(dev, seed, news, lens, n_q, n_kv, dim, page):  # noqa: F811
    """One layer's calls over a cache, its inputs, and what they write."""
    g = gen(seed)
    T, d = sum(news), (n_q + 2 * n_kv) * dim
    c = ref4.paged(news, lens, n_kv, dim, page, seed)
    cache, table = cache_on(c, dev)
    x, r = (torch.randn(T, d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).to(dev)
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(news, lens)])
    seq = torch.cat([torch.full((m,), s) for s, m in enumerate(news)])
    slot = (c["table"][seq, pos // page] * page + pos % page).to(torch.int32).to(dev)
    off = ints([sum(news[:s]) for s in range(len(news) + 1)], dev)
    kv_off = ints([sum(lens[:s]) for s in range(len(lens) + 1)], dev)
    kv_len, pos = ints(lens, dev), pos.to(torch.int32).to(dev)
    tab = bd.rope_table(max(lens), dim, 10000.0, dev)
    n, h = torch.zeros_like(x), torch.zeros_like(x)
    qo, out = (torch.zeros(T, n_q, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ko, vo = (torch.zeros(sum(lens), n_kv, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    need = bd.bd_attention_workspace_size(T, len(news), n_q, n_kv, dim)

    def run(ws):
        bd.bd_block_norm(x, r, gain, 1e-5, n, ws, residual_out=h, post_gain=gain)
        heads = n.view(T, n_q + 2 * n_kv, dim)
        bd.bd_rope_append(heads[:, :n_q], heads[:, n_q: n_q + n_kv], heads[:, n_q + n_kv:], pos, tab, slot, cache, qo, ws)
        bd.bd_attention(qo, off, cache, table, kv_len, dim ** -0.5, max(news), out, ws)
        bd.bd_kv_read(cache, table, kv_off, ko, vo, ws)

    return run, need, (n, h, qo, out, ko, vo)


BATCHES = [([1] * 5, [900, 33, 1, 2000, 512], 16, 2, 128, 16), ([300, 1, 40], [800, 700, 40], 4, 2, 64, 32)]


def test_two_streams_at_once(dev):  # noqa: F811
    """Batches on streams and workspaces of their own, in flight together, give what each gives alone."""
    made = [layer(dev, i, *b) for i, b in enumerate(BATCHES)]
    spaces = [bd.new_workspace(need, dev) for _, need, _ in made]
    for (run, _, _), ws in zip(made, spaces):
        run(ws)
    torch.cuda.synchronize()
    first = [[t.clone() for t in outs] for _, _, outs in made]
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(20):
        for s, (run, _, _), ws in zip(streams, made, spaces):
            with torch.cuda.stream(s):
                run(ws)
    torch.cuda.synchronize()
    assert all(bd.bd_check_async(ws) == bd.BD_OK for ws in spaces)
    assert all(torch.equal(a, b) for f, (_, _, outs) in zip(first, made) for a, b in zip(f, outs))


def test_two_graphs_of_one_workspace(dev):  # noqa: F811
    """Two captured batches that share a workspace, replayed in turn on one stream."""
    made = [layer(dev, 7 + i, *b) for i, b in enumerate(BATCHES)]
    ws = bd.new_workspace(max(need for _, need, _ in made), dev)
    for run, _, _ in made:
        run(ws)
    torch.cuda.synchronize()
    first = [[t.clone() for t in outs] for _, _, outs in made]
    graphs = []
    for run, _, outs in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(ws)
        for t in outs:
            t.zero_()
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert bd.bd_check_async(ws) == bd.BD_OK
    assert all(torch.equal(a, b) for f, (_, _, outs) in zip(first, made) for a, b in zip(f, outs))


@pytest.mark.parametrize("batch", BATCHES + [([700, 300, 64], [3200, 1777, 64], 16, 2, 128, 32)])
def test_results_do_not_depend_on_the_run(dev, batch):  # noqa: F811
    run, need, outs = layer(dev, 3, *batch)
    ws = bd.new_workspace(need, dev)
    run(ws)
    first = [t.clone() for t in outs]
    for _ in range(20):
        run(ws)
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
    assert bd.bd_check_async(ws) == bd.BD_OK


# ------------------------------------------------------------------------------- the bounds-checked build

def test_bounds_checked_build(dev):  # noqa: F811
    """The operators' tests through the library that checks each access (conftest.py asks it after every test)."""
    from bit_weight_delta_bd_gb300 import build

    lib = build.build(debug_bounds=True)
    files = [os.path.join(HERE, f) for f in ("test_int4_cache.py", "test_int4_attention.py", "test_block_norm.py")]
    p = subprocess.run([sys.executable, "-m", "pytest", *files, "-m", "gpu", "-x", "-q"], cwd=os.path.dirname(HERE),
                       env=dict(os.environ, BD_LIBRARY=lib), capture_output=True, text=True, timeout=1200)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-2000:]


# ------------------------------------------------------------------------------- the example

@pytest.mark.parametrize("int4,post_norm", [(True, False), (True, True), (False, True)])
def test_example_block(dev, int4, post_norm):  # noqa: F811
    """Prompts, then single tokens on top of them, against the dense block.  A 4-bit code is off by at most a 30th of
    its group's range, some 6 times the typical value for 32 of them: 0.115 of a vector's norm at most if it is uniform
    within its step.  K's moves a score by as much (q has the norm of 8 that the scale divides by), V's the mean by as
    much; together 0.163 of the attention's norm, whose share of the residual stream's is at most three quarters: 2^-3.
    (8 bits: 2^-5, of which the roundings to bf16 are most.)"""
    m = large.example()
    block = m.DecoderBlock(hidden=512, n_q=8, n_kv=2, head_dim=64, variants=3, n_seq=3, max_len=96, page=16,
                           int8=not int4, int4=int4, post_norm=post_norm, max_tokens=256, device=dev)
    g = gen(21)
    prompts, steps = [70, 1, 33], 4
    total = [p + steps for p in prompts]
    streams = [torch.randn(n, 512, generator=g).to(torch.bfloat16).to(dev) for n in total]
    variant = ints([1, -1, 2], dev)
    got_h, got_n = [[] for _ in total], [[] for _ in total]
    have = [0, 0, 0]
    for new in [prompts] + [[1, 1, 1]] * steps:
        off, kv_len, pos, slot, seq = m.batch(block, new, have, dev)
        x = torch.cat([s[a: a + n] for s, a, n in zip(streams, have, new)]).clone()
        n = block.forward(x, variant[seq.long()], off, kv_len, pos, slot, max(new), block.new_buffers(len(x)))
        for s in range(3):
            a, b = int(off[s]), int(off[s + 1])
            got_h[s].append(x[a:b].clone())
            got_n[s].append(n[a:b].clone())
        have = [h + k for h, k in zip(have, new)]
    assert bd.bd_check_async(block.ws) == bd.BD_OK
    which = torch.cat([torch.full((n,), int(variant[s]) + 1, device=dev) for s, n in enumerate(total)])
    x = torch.cat(streams).double()
    h, n = large.dense_block(block, x, which, total)
    if post_norm:
        def normed(t, gains):
            return t * torch.rsqrt(t.pow(2).mean(1, keepdim=True) + block.eps) * torch.stack(list(gains)).double()[which]

        h = x + block.gates.double()[which] * normed(h - x, block.post_gains)
        n = normed(h, block.gains[1])
    for got, want in ((got_h, h), (got_n, n)):
        got = torch.cat([torch.cat(g) for g in got]).double()
        rel = ((got - want).norm(dim=1) / want.norm(dim=1)).max()
        assert math.isfinite(float(rel)) and float(rel) <= (2 ** -3 if int4 else 2 ** -5), float(rel)
