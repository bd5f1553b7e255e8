"""Attention over a 4-bit cache whose values differ in size from group to group
of one token, while scores climb along the cache (GPU): a row of the query, alone
among its kv head's, meets keys that lie above all before them, and one group of
32 elements outweighs the others, or is nothing.  Every row and every group has
its turn: the pairs of sequence and kv head take them one after the other.

Bounds, beside those of int4_oracle.py (roundings to 11 bits).  Few rows: a
product of probability and scale is rounded to a multiple of 2^-24 where the
row's largest product with a scale or lowest value is 2^11 or more: off by 2^-36
of that at most, 15 times for the code, 15/16 2^-32.  Chunks: a probability is
off by 2^-36 of the largest times its tile's power of two likewise, times values
below 4 of those, and values over it times 2^13 by 15 roundings of the scale, one
of the lowest value and one of the sum to multiples of 2^-24, 17 2^-38; together
33 2^-38.  So each key adds 2^-32 at most of the largest probability times the
largest size, max(16 scale, |lowest value|).
"""
import math

import pytest
import torch

import int4_oracle as ref4
import test_int4_attention as att
from bit_weight_delta_bd_gb300 import bitdelta as bd
from layer_oracle import half_ulp_bf16
from test_int4_attention import cache_on, dev, gen, within  # noqa: F401  (dev is a fixture)
from test_int4_paths import SIZES

pytestmark = pytest.mark.gpu


def refresh(c):
    """The values that the cache's codes and pairs stand for, after they were changed."""
    page, c["steps"] = c["k"].shape[2], []
    for s, length in enumerate(c["kv_len"]):
        at = torch.arange(length)
        pg, off = c["table"][s].long()[at // page], at % page
        for name in "kv":
            pair = c[name + "s"][pg, :, off]
            c["vals"][name][s] = ref4.values(c[name][pg, :, off], pair)
            if name == "k":
                p = pair.double().abs()
                c["steps"].append((15 * p[..., 0] + p[..., 1]).repeat_interleave(32, -1))


def climb(c, q, q_off, scale, keys, first=0):
    """Puts keys along a row's query into the cache: pair i of (sequence, kv head) takes row i + first; keys[j] lies so
    much above what the others reach.  Returns the row's number past each turn of the rows, by pair."""
    n_kv, page = c["k"].shape[1:3]
    group = q.shape[1] // n_kv
    turns = {}
    for s, length in enumerate(c["kv_len"]):
        rows = (q_off[s + 1] - q_off[s]) * group
        for h in range(n_kv):
            i = s * n_kv + h + first
            r = i % rows if rows else 0
            turns[s, h] = i // rows if rows else 0
            for j, above in keys.items():
                if not rows or j >= length - (q_off[s + 1] - q_off[s]):
                    continue
                x = q[q_off[s] + r // group, h * group + r % group].float()
                byte, pair = ref4.codes(x * ((3.5 + above) / (abs(scale) * float(x @ x))))
                pg, at = c["table"][s, j // page].long(), j % page
                c["k"][pg, h, at], c["ks"][pg, h, at] = byte, pair
    return turns


def attend(dev, c, q, n_new, scale, max_new=None, given=None, hit=None):  # noqa: F811
    """Runs the call and holds it to the bounds of the module's head; with another cache than the definition's, but for
    the elements that it may hit, which it has to make infinite or NaN."""
    lens, (T, n_q, dim) = c["kv_len"], q.shape
    cache, table = cache_on(given or c, dev)
    q_off = [0]
    for n in n_new:
        q_off.append(q_off[-1] + n)
    out, lse = torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16), torch.empty(T, n_q, device=dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, len(lens), n_q, cache.n_kv, dim), dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    most = max(n_new) if max_new is None else max_new
    bd.bd_attention(q.to(dev), i32(q_off), cache, table, i32(lens), scale, most, out, ws, lse=lse)
    assert bd.bd_check_async(ws) == bd.BD_OK
    want = ref4.attention(q, q_off, c, scale, True)
    few = most * (n_q // cache.n_kv) <= 16
    mixed = not few and min(n_new) * (n_q // cache.n_kv) <= 16  # either kernel may take its sequences
    b_out, b_lse = ref4.bounds(want, dim, max(lens), ref4.U11 if few or mixed else 0.0, 0.0 if few else 2 * ref4.U11)
    for s, length in enumerate(lens):
        rows = slice(q_off[s], q_off[s + 1])
        if not length or q_off[s] == q_off[s + 1]:
            continue
        at = torch.arange(length)
        pair = c["vs"][c["table"][s].long()[at // c["v"].shape[2]], :, at % c["v"].shape[2]].double().abs()
        size = torch.maximum(16 * pair[..., 0], pair[..., 1]).amax(-1)  # [len][n_kv]
        k = c["vals"]["k"][s].double().repeat_interleave(n_q // cache.n_kv, 1)
        z = torch.einsum("thd,jhd->thj", q[rows].double(), k) * scale
        see = length - (q_off[s + 1] - q_off[s]) + torch.arange(q_off[s + 1] - q_off[s])
        z = z.masked_fill(at[None, None] > see[:, None, None], -math.inf)
        p = torch.exp(z - want[1][rows][..., None]).nan_to_num(0.0)  # (a row that sees no key)
        big = (p * size.T.repeat_interleave(n_q // cache.n_kv, 0)[None]).amax(-1)
        if not few:  # a tile's values share their factor
            big = p.amax(-1) * size.amax(0).repeat_interleave(n_q // cache.n_kv)[None]
        b_out[rows] += (1 + 2.0 ** -7) * length * 2.0 ** -32 * big[..., None]
    if hit is None:
        within(out, want[0], b_out, "attention")
    else:
        assert not out.cpu()[hit].isfinite().any()
        within(out.cpu()[~hit], want[0][~hit], b_out[~hit], "attention")
    assert torch.equal(lse.cpu() == -math.inf, want[1] == -math.inf)
    fin = want[1] > -math.inf
    within(lse.cpu()[fin], want[1][fin], b_lse[fin], "log-sum-exp")


# what the group whose turn it is is times, and what the others are; the lowest values as they are or 0
KINDS = [(2.0, 1.0, True), (2.0, 1.0, False), (8.0, 1.0, False), (16.0, 1.0, True), (2.0 ** 7, 1.0, True),
         (2.0 ** 7, 1.0, False), (2.0 ** 12, 1.0, True), (2.0 ** 20, 1.0, False), (0.0, 1.0, True), (1.0, 0.0, True),
         (1.0, 0.0, False), (2.0 ** -20, 1.0, True)]
# keys that lie above the rest, and by how much (natural units): for the first of a block's four warps that takes
# them, past its first 32 keys, for other blocks of a cluster, and past 1024 keys of a dealt cache
KEYS = {40: 5.0, 100: 2.0, 129: 3.6, 135: 9.0, 170: 5.5, 200: 4.0, 230: 12.0, 300: 6.0, 390: 4.5, 500: 8.0, 650: 10.0,
        777: 3.9, 1100: 5.0, 1290: 7.0, 1700: 11.0, 1950: 12.0} | {2100 + 139 * i: 4.0 + i % 9 for i in range(24)}
FORMS = [
    ([1] * 4, [333, 700, 1300, 2000], 4, 4, 64, 16), ([1] * 4, [333, 700, 1300, 2000], 4, 4, 128, 64),  # 1 row, clusters
    ([3, 1, 3], [2000, 260, 900], 4, 4, 128, 16), ([1] * 3, [2000, 260, 900], 12, 4, 64, 32),  # 3 rows
    ([1] * 4, [333, 700, 1300, 2000], 64, 8, 128, 16), ([1] * 4, [150, 300, 5000, 600], 64, 8, 128, 128),  # 8 rows
    ([1] * 4, [150, 300, 5000, 600], 32, 4, 64, 16),
    ([2] * 4, [2000, 140, 300, 1000], 64, 8, 128, 16), ([4, 2, 4], [2000, 300, 900], 16, 4, 64, 32),  # 16 rows
    ([1] * 4, [5000, 300, 900, 2000], 64, 4, 128, 32)]
DEALT = [  # several tiles to a block
    ([1] * 4, [4400, 3000, 4100, 2500], 32, 16, 128, 64), ([1] * 4, [4400, 3000, 4100, 2500], 16, 16, 64, 16),
    ([4] * 4, [4400, 3000, 4100, 2500], 64, 16, 64, 128)]
CHUNKS = [
    ([20, 40], [400, 1300], 8, 2, 64, 16), ([20, 33], [700, 1300], 4, 2, 128, 32), ([300], [1300], 8, 4, 128, 16),
    ([300, 1, 1, 40, 1], [700, 1500, 300, 777, 900], 16, 2, 128, 16), ([1, 200, 1, 1], [2000, 700, 300, 500], 8, 2, 64, 64)]
LONG = [  # several tiles to a block, and the single tokens' dealt so
    ([40] * 6, [1500, 1400, 1600, 1700, 900, 1100], 8, 8, 64, 16), ([40] * 6, [1500, 1400, 1600, 1700, 900, 1100], 8, 8, 128, 64),
    ([270] * 3, [1500, 1700, 900], 8, 8, 128, 32),
    ([150, 1, 1, 1], [1700, 4400, 3000, 4100], 32, 16, 128, 16), ([150, 1, 1, 1], [1700, 4400, 3000, 4100], 16, 16, 64, 32)]


@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page,kind", [
    (*form, kind) for i, form in enumerate(FORMS + DEALT + CHUNKS + LONG) for kind in range(i % 2, len(KINDS), 2)])
def test_groups_apart_while_scores_climb(dev, n_new, kv_len, n_q, n_kv, dim, page, kind):  # noqa: F811
    times, others, lows = KINDS[kind]
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, 31 + kind)
    q = torch.randn(sum(n_new), n_q, dim, generator=gen(kind)).to(torch.bfloat16)
    q_off = [sum(n_new[:s]) for s in range(len(n_new) + 1)]
    scale = dim ** -0.5 * (-1 if kind % 5 == 4 else 1)
    turns = climb(c, q if scale > 0 else -q, q_off, scale, KEYS, first=kind)
    for (s, h), turn in turns.items():
        pg = c["table"][s, : -(-kv_len[s] // page)].long()
        f = torch.full((dim // 32, 1), others)
        f[(turn + kind) % (dim // 32)] = times
        c["vs"][pg, h] = (c["vs"][pg, h].float() * f).to(torch.bfloat16)
    if not lows:
        c["vs"][..., 1] = 0.0  # (values that are all of one sign)
        for s, length in enumerate(kv_len):  # past the lengths NaN again
            if length % page:
                c["vs"][c["table"][s, length // page].long(), :, length % page:] = math.nan
    refresh(c)
    attend(dev, c, q, n_new, scale)


@pytest.mark.parametrize("part,what", [(0, math.nan), (0, math.inf), (1, math.inf), (1, math.nan)])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", [FORMS[4], FORMS[6], FORMS[7], *DEALT[:2], CHUNKS[0], *LONG[:3]])
def test_a_group_that_is_not_finite_hides_no_other(dev, n_new, kv_len, n_q, n_kv, dim, page, part, what):  # noqa: F811
    """A key that lies above those before it, with a group that is not finite and another that is larger than the rest:
    all dims but the first group's are what they were."""
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, 8)
    q = torch.randn(sum(n_new), n_q, dim, generator=gen(3)).to(torch.bfloat16)
    q_off = [sum(n_new[:s]) for s in range(len(n_new) + 1)]
    climb(c, q, q_off, dim ** -0.5, {200: 6.0, 850: 6.0})
    given, hit = dict(c, vs=None), torch.zeros(q.shape, dtype=torch.bool)
    bad = []
    for s, length in enumerate(kv_len):
        for h in range(n_kv):
            for j in (200, 850):
                if j < length - n_new[s]:
                    group = (s + h + j // 200) % (dim // 32)
                    pg, at = c["table"][s, j // page].long(), j % page
                    c["vs"][pg, h, at, (group + 1) % (dim // 32)] *= 2.0 ** 7
                    bad.append((pg, h, at, group))
                    heads = slice(h * (n_q // n_kv), (h + 1) * (n_q // n_kv))
                    hit[q_off[s]: q_off[s + 1], heads, 32 * group: 32 * group + 32] = True
    refresh(c)
    given["vs"] = c["vs"].clone()
    for pg, h, at, group in bad:
        given["vs"][pg, h, at, group, part] = what
    attend(dev, c, q, n_new, dim ** -0.5, given=given, hit=hit)


@pytest.mark.parametrize("sizes", range(len(SIZES)))
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", DEALT + LONG)
def test_sizes_apart_from_tile_to_tile(dev, n_new, kv_len, n_q, n_kv, dim, page, sizes):  # noqa: F811
    """Keys and values of neighbouring tokens, and of tiles, far apart, where a block takes several tiles."""
    key_of, value_of, scale = SIZES[sizes]
    c = att.scaled_cache(n_new, kv_len, n_kv, dim, page, 7, key_of, value_of)
    q = torch.randn(sum(n_new), n_q, dim, generator=gen(sizes)).to(torch.bfloat16)
    attend(dev, c, q, n_new, scale)


# ------------------------------------------------------------------------------- values of nothing

@pytest.mark.parametrize("zero", ["tile", "tail", "key", "far"])
@pytest.mark.parametrize("written", [True, False])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", [
    ([1, 2], [300, 400], 8, 2, 128, 16), *DEALT[:1], *LONG[:3]])
def test_zeros_among_small_values(dev, n_new, kv_len, n_q, n_kv, dim, page, zero, written):  # noqa: F811
    """Values of 0 say nothing of the size of the others, whatever their probability: a tile of them, single ones, and
    single ones among values far apart; as bd_rope_append writes them (a scale of 2^-104), and with scales of 0."""
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, 17)
    q = torch.randn(sum(n_new), n_q, dim, generator=gen(4)).to(torch.bfloat16)
    tiny = float((torch.tensor(1e-30) / torch.tensor(15.0)).to(torch.bfloat16))
    for s, length in enumerate(kv_len):
        at = torch.arange(length)
        pg, off = c["table"][s].long()[at // page], at % page
        hit = {"tile": at // 128 % 3 == 1, "tail": at >= length // 256 * 128, "key": at % 5 == 2, "far": at % 3 == 2}[zero]
        f = torch.full((length,), 2.0 ** -40)
        if zero == "far":
            f[at % 3 == 1] = 2.0 ** -60
        pair = c["vs"][pg, :, off].float() * f[:, None, None, None]
        pair[hit] = torch.tensor([tiny if written else 0.0, 0.0])
        c["vs"][pg, :, off] = pair.to(torch.bfloat16)
        if written:
            c["v"][pg[hit], :, off[hit]] = 0
    refresh(c)
    attend(dev, c, q, n_new, dim ** -0.5)


# ------------------------------------------------------------------------------- large scores

@pytest.mark.parametrize("score", [2.0 ** 20, -2.0 ** 20, 2.0 ** 19.7, -2.0 ** 17.3])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", [FORMS[0], FORMS[4], FORMS[7], *DEALT[:2], CHUNKS[0], *LONG])
def test_scores_of_a_million(dev, n_new, kv_len, n_q, n_kv, dim, page, score):  # noqa: F811
    """Keys that are all alike, with scores of up to 2^20 in magnitude: every row is the mean of the values that it sees,
    whose groups differ in size.  (All keys have the same score, whatever its rounding.)"""
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, 5)
    q = torch.zeros(sum(n_new), n_q, dim, dtype=torch.bfloat16)
    byte, pair = ref4.codes(torch.randn(n_kv, dim, generator=gen(2)))
    c["k"][:], c["ks"][:] = byte[None, :, None], pair[None, :, None]
    key = ref4.values(byte, pair).repeat_interleave(n_q // n_kv, 0)
    q[:] = (score * key / (0.25 * key.pow(2).sum(-1, keepdim=True))).to(torch.bfloat16)
    for s, length in enumerate(kv_len):
        pg = c["table"][s, : -(-length // page)].long()
        f = 2.0 ** torch.randint(-8, 9, (n_kv, 1, dim // 32, 1), generator=gen(s)).float()
        c["vs"][pg] = (c["vs"][pg].float() * f).to(torch.bfloat16)
    refresh(c)
    cache, table = cache_on(c, dev)
    q_off = [sum(n_new[:s]) for s in range(len(n_new) + 1)]
    out, lse = torch.empty(q.shape, device=dev, dtype=torch.bfloat16), torch.empty(q.shape[:2], device=dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(q.shape[0], len(kv_len), n_q, n_kv, dim), dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    bd.bd_attention(q.to(dev), i32(q_off), cache, table, i32(kv_len), 0.25, max(n_new), out, ws, lse=lse)
    assert bd.bd_check_async(ws) == bd.BD_OK
    z = (q.double() * key[None]).sum(-1) * 0.25
    zmag = (q.double().abs() * key.abs()[None]).sum(-1) * 0.25
    for s, length in enumerate(kv_len):
        at = torch.arange(length)
        pair = c["vs"][c["table"][s].long()[at // page], :, at % page].double()
        sizes = (15 * pair[..., 0].abs()).repeat_interleave(32, -1), pair[..., 1].abs().repeat_interleave(32, -1)
        v = c["vals"]["v"][s].double()
        seen = length - n_new[s] + 1 + torch.arange(n_new[s])
        mean = [(x.cumsum(0)[seen - 1] / seen[:, None, None]).repeat_interleave(n_q // n_kv, 1) for x in (v, *sizes)]
        rows = slice(q_off[s], q_off[s + 1])
        # roundings of probabilities times scales, or of probabilities and values; fp32 sums; the largest size's 2^-32
        bound = (mean[1] + mean[2]) * (2 * ref4.U11 + (length + 64) * 2.0 ** -21)
        bound = bound + 2.0 ** -32 * torch.maximum(16 * pair[..., 0].abs(), pair[..., 1].abs()).max()
        within(out[rows], mean[0], bound + half_ulp_bf16(mean[0].abs() + bound), "attention")
        want = z[rows] + seen.log()[:, None]
        within(lse[rows], want, zmag[rows] * (dim + 8) * 2.0 ** -22 + (length + 64) * 2.0 ** -22, "log-sum-exp")
