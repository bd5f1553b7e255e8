"""Attention over the paged KV cache in 4 bits on the GPU, against plain 64-bit
definitions (int4_oracle.py): single tokens, chunks and mixtures, odd sizes,
empty rows, strided queries, NaN past the lengths, magnitudes far apart, hidden
and non-finite keys and values, streams and graphs -- and what it reports."""
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


def within(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float((err / bound).nan_to_num(posinf=9e9).max()):.3g} times"


def cache_on(c, dev):
    on = {n: c[n].to(dev) for n in ("k", "v", "ks", "vs", "table")}
    return bd.KvPages(on["k"], on["v"], on["ks"], on["vs"]), on["table"]


def empty_cache(n_pages, n_kv, page, dim, dev, fill=0x5A, pair=3.0):
    return bd.KvPages(*(torch.full((n_pages, n_kv, page, dim // 2), fill, device=dev, dtype=torch.uint8) for _ in range(2)),
                      *(torch.full((n_pages, n_kv, page, dim // 32, 2), pair, device=dev, dtype=torch.bfloat16)
                        for _ in range(2)))


# ------------------------------------------------------------------------------- attention

def run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, causal=True, seed=0, scale=None, packed=False, q_scale=1.0,
                  max_new=None, offset=0.0, coded_rel=None, value_rel=None, c=None):
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, seed, offset=offset) if c is None else c
    cache, table = cache_on(c, dev)
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
    most = max(n_new) if max_new is None else max_new
    bd.bd_attention(qd, off_d, cache, table, len_d, scale, most, out, ws, causal=causal, lse=lse)
    assert bd.bd_check_async(ws) == bd.BD_OK
    want = ref4.attention(q, q_off, c, scale, causal)
    few = most * (n_q // n_kv) <= 16
    # few rows: probability times scale enters its product in fp16; chunks: probabilities and V's values in fp16
    b_out, b_lse = ref4.bounds(want, dim, max(kv_len + [1]), (ref4.U11 if few else 0.0) if coded_rel is None else coded_rel,
                               (0.0 if few else 2 * ref4.U11) if value_rel is None else value_rel)
    within(out, want[0], b_out, "attention")
    assert torch.equal(lse.cpu() == -math.inf, want[1] == -math.inf)
    fin = want[1] > -math.inf
    within(lse.cpu()[fin], want[1][fin], b_lse[fin], "log-sum-exp")
    # the same call again gives the same bits, without the log-sum-exp too
    out2 = torch.empty_like(out)
    bd.bd_attention(qd, off_d, cache, table, len_d, scale, most, out2, ws, causal=causal)
    assert torch.equal(out, out2)
    return out, qd, cache, table, off_d, len_d


DECODE = [
    ([1], [1], 1, 1, 64, 16), ([1], [500], 64, 8, 128, 16), ([1, 1, 1], [0, 1, 63], 8, 2, 128, 16),
    ([1] * 9, [64, 65, 127, 128, 129, 16, 15, 17, 2000], 16, 8, 128, 32), ([1, 0, 1], [300, 5, 1000], 5, 1, 64, 128),
    ([1, 1], [3001, 1], 32, 2, 64, 64), ([1] * 70, [(37 * i) % 300 for i in range(70)], 7, 7, 64, 16),
    ([1], [6000], 24, 3, 128, 64), ([2, 1], [900, 33], 16, 2, 128, 16), ([3, 0, 3, 1], [70, 9, 2, 4100], 10, 2, 64, 32)]


@pytest.mark.parametrize("offset", [0.0, 4.0])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", DECODE)
def test_attention_decode(dev, n_new, kv_len, n_q, n_kv, dim, page, offset):
    run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, seed=len(n_new), packed=len(n_new) % 2 == 1, offset=offset)


@pytest.mark.parametrize("n_q,n_kv,dim,page", [(16, 2, 128, 16), (16, 1, 64, 32), (32, 2, 128, 64), (3, 3, 64, 128)])
def test_attention_many_short_and_one_long(dev, n_q, n_kv, dim, page):
    """Sequences of one tile, of two, and of none beside a long one, which makes the batch one that is dealt out: a
    block's segments are shorter than its teams are many."""
    lens = [(i * 97) % 300 for i in range(150)] + [5000] + [1, 0, 128, 129, 256, 257] * 5
    for n_new in ([1] * len(lens), [1, 0, 2] * (len(lens) // 3)):
        run_attention(dev, n_new + [1] * (len(lens) - len(n_new)), lens, n_q, n_kv, dim, page, seed=21)
    small = [1, 5000, 64, 300]  # 64 sequences or fewer: another way to deal
    for n_new in ([1, 1, 1, 1], [2, 1, 0, 1]):
        run_attention(dev, n_new, small, n_q, n_kv, dim, page, seed=22)
    run_attention(dev, [1] * 61, [5000] + [(i * 97) % 300 for i in range(60)], n_q, n_kv, dim, page, seed=23)


CHUNK = [
    ([5], [5], 8, 2, 64, 16, True), ([6, 3, 1], [6, 300, 77], 8, 1, 128, 16, True),
    ([130], [130], 8, 8, 64, 32, True), ([65, 1, 200, 0], [65, 700, 333, 9], 16, 4, 128, 64, True),
    ([33], [1100], 12, 4, 64, 128, False), ([257], [300], 5, 1, 128, 16, True), ([300], [1300], 8, 2, 128, 128, False),
    ([40, 7], [10, 0], 6, 2, 64, 16, True),  # more new tokens than keys: the first rows see nothing
    ([129, 128, 127], [129, 1024, 640], 14, 2, 64, 64, True), ([600, 300], [900, 300], 2, 2, 128, 32, True)]


@pytest.mark.parametrize("offset", [0.0, 4.0])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page,causal", CHUNK)
def test_attention_chunk(dev, n_new, kv_len, n_q, n_kv, dim, page, causal, offset):
    run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, causal=causal, seed=n_new[0], packed=n_new[0] % 2 == 1,
                  offset=offset)


def test_attention_mixed_batch(dev):
    """Chunks with single tokens beside them, which take a launch of their own."""
    run_attention(dev, [300, 1, 1, 40, 1], [300, 1500, 2, 77, 64], 16, 2, 128, 16, seed=2, value_rel=2 * ref.U16,
                  coded_rel=ref4.U11)
    run_attention(dev, [1, 200, 1, 1], [4000, 200, 0, 500], 8, 1, 64, 64, seed=3, value_rel=2 * ref.U16,
                  coded_rel=ref4.U11)


def test_attention_max_new_changes_no_meaning(dev):
    for max_new in (0, 1, 5000):
        loose = dict(coded_rel=ref4.U11, value_rel=2 * ref.U16)
        run_attention(dev, [70, 1], [150, 260], 8, 2, 128, 16, seed=5, max_new=max_new, **loose)
        run_attention(dev, [1, 1], [150, 260], 8, 2, 128, 16, seed=6, max_new=max_new, **loose)


def test_attention_large_scores(dev):
    """Scores in the hundreds: the running maximum has to carry.  (Probabilities span more than fp16 holds: 8 bits.)"""
    run_attention(dev, [1, 2], [700, 900], 8, 2, 64, 32, seed=9, q_scale=12.0, scale=1.0, coded_rel=ref.U16)
    run_attention(dev, [1, 20], [700, 900], 8, 2, 64, 32, seed=9, q_scale=12.0, scale=1.0)
    run_attention(dev, [1, 200], [1, 300], 8, 2, 128, 32, seed=9, q_scale=0.0)
    run_attention(dev, [1, 1], [100, 300], 8, 2, 128, 32, seed=9, scale=-0.3)
    run_attention(dev, [1, 100], [100, 300], 8, 2, 128, 32, seed=9, scale=-0.3)
    run_attention(dev, [1, 1], [100, 300], 8, 2, 128, 32, seed=9, scale=0.0)
    run_attention(dev, [1, 100], [100, 300], 8, 2, 128, 32, seed=9, scale=0.0)


def scaled_cache(n_new, kv_len, n_kv, dim, page, seed, key_of, value_of):
    """A cache whose keys and values of token j are multiplied by key_of(j) and value_of(j), powers of two."""
    c = ref4.paged(n_new, kv_len, n_kv, dim, page, seed)
    c["steps"] = []
    for s, length in enumerate(kv_len):
        at = torch.arange(length)
        pg, off = c["table"][s].long()[at // page], at % page
        for name, of in (("k", key_of), ("v", value_of)):
            f = torch.tensor([of(j) for j in range(length)], dtype=torch.float32)
            pair = c[name + "s"][pg, :, off].float() * f[:, None, None, None]
            c[name + "s"][pg, :, off] = pair.to(torch.bfloat16)
            c["vals"][name][s] = ref4.values(c[name][pg, :, off], c[name + "s"][pg, :, off])
            if name == "k":
                p = pair.double().abs()
                c["steps"].append((15 * p[..., 0] + p[..., 1]).repeat_interleave(32, -1))
    return c


@pytest.mark.parametrize("news", [[1, 1], [2, 60]])
def test_attention_magnitudes(dev, news):
    """Keys and values of very different sizes in neighbouring tokens, tiny ones, and large ones."""
    lens = [200, 333]
    for key_of, value_of, scale in (
            (lambda j: 2.0 ** (j % 7 - 3), lambda j: 2.0 ** (5 * (j % 5) - 10), 0.05),
            (lambda j: 2.0 ** -60, lambda j: 2.0 ** -60, 2.0 ** 57),
            (lambda j: 2.0 ** 60, lambda j: 2.0 ** 60, 2.0 ** -63),
            (lambda j: 2.0 ** (-40 if j % 3 else 0), lambda j: 2.0 ** (40 if j % 11 else -40), 0.1)):
        c = scaled_cache(news, lens, 2, 128, 16, 7, key_of, value_of)
        run_attention(dev, news, lens, 8, 2, 128, 16, seed=7, scale=scale, c=c, coded_rel=ref.U16, value_rel=2 * ref.U16)


def test_attention_of_hidden_keys(dev):
    """What a causal row does not see of K has no influence, whatever it is: huge, infinite or NaN."""
    n_new, lens = [40], [70]
    c = ref4.paged(n_new, lens, 2, 128, 16, 3)
    out = run_attention(dev, n_new, lens, 8, 2, 128, 16, seed=3, c=c)[0]
    for value in (1e30, math.inf, math.nan):
        last = c["table"][0, 69 // 16].long(), 69 % 16
        c["ks"][last[0], :, last[1]] = value  # the key of the last token, which its own rows alone see
        cache, table = cache_on(c, dev)
        q = torch.randn(40, 8, 128, generator=gen(4)).to(torch.bfloat16).to(dev)
        out2 = torch.empty_like(out)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(40, 1, 8, 2, 128), dev)
        bd.bd_attention(q, torch.tensor([0, 40], dtype=torch.int32, device=dev), cache, table,
                        torch.tensor(lens, dtype=torch.int32, device=dev), 128 ** -0.5, 40, out2, ws)
        assert torch.equal(out2[:39], out[:39])
        if value != value:
            assert out2[39].isnan().all()


def test_attention_nonfinite_values_stay_in_their_groups(dev):
    """V of a seen key that is not finite reaches the dims of its own group, of the rows that see it."""
    for n_new in ([1, 1], [40, 1]):
        lens = [90, 90]
        c = ref4.paged(n_new, lens, 2, 64, 16, 3)
        base = run_attention(dev, n_new, lens, 4, 2, 64, 16, seed=3, c=c, max_new=max(n_new))[0]
        pg, at = c["table"][0, 10 // 16].long(), 10 % 16  # key 10, before every new token
        c["vs"][pg, 1, at, 1, 0] = math.nan
        cache, table = cache_on(c, dev)
        T = sum(n_new)
        q = torch.randn(T, 4, 64, generator=gen(4)).to(torch.bfloat16).to(dev)
        out = torch.empty_like(base)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 2, 4, 2, 64), dev)
        off = torch.tensor([0, n_new[0], T], dtype=torch.int32, device=dev)
        bd.bd_attention(q, off, cache, table, torch.tensor(lens, dtype=torch.int32, device=dev), 0.125, max(n_new), out, ws)
        hit = torch.zeros_like(base, dtype=torch.bool)
        hit[: n_new[0], 2:, 32:] = True
        assert out[hit].isnan().all() and out[~hit].isfinite().all()


def test_attention_nan_query_stays_in_its_rows(dev):
    for n_new in ([1, 1], [40, 1]):
        out, qd, cache, table, off, ln = run_attention(dev, n_new, [90, 90], 4, 2, 64, 16, seed=3)
        q = qd.clone()
        q[0, 1] = math.nan
        out2 = torch.empty_like(out)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(q.shape[0], 2, 4, 2, 64), dev)
        bd.bd_attention(q, off, cache, table, ln, 0.125, max(n_new), out2, ws)
        assert out2[0, 1].isnan().all()
        out2[0, 1] = out[0, 1]
        assert torch.equal(out2, out)


def test_attention_reports_bad_indices(dev):
    cache = empty_cache(3, 1, 16, 64, dev, pair=1.0)
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


def test_attention_rows_of_no_sequence_stay(dev):
    """Tokens that no sequence claims, and a workspace full of anything past its error word."""
    c = ref4.paged([1, 30], [64, 100], 2, 128, 16, 1)
    cache, table = cache_on(c, dev)
    q = torch.randn(40, 16, 128, generator=gen(8)).to(torch.bfloat16).to(dev)
    out = torch.full((40, 16, 128), 7.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((40, 16), 7.0, device=dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(40, 2, 16, 2, 128), dev)
    ws[256:] = 0xFF
    for most in (30, 1):
        bd.bd_attention(q, torch.tensor([0, 1, 31], dtype=torch.int32, device=dev), cache, table,
                        torch.tensor([64, 100], dtype=torch.int32, device=dev), 0.1, most, out, ws, lse=lse)
        assert bd.bd_check_async(ws) == bd.BD_OK
        assert (out[31:] == 7).all() and (lse[31:] == 7).all() and (lse[:31] != 7).all()


# ------------------------------------------------------------------------------- all together

def test_write_attend_read_on_a_stream_and_in_a_graph(dev):
    """norms -> rotary and append -> attention -> read on a side stream, then captured and replayed, against the bf16
    cache of the values that are read back."""
    T, n_q, n_kv, dim, page = 3, 8, 2, 128, 16
    d = (n_q + 2 * n_kv) * dim
    g = gen(11)
    x, r = (torch.randn(T, d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    gain = torch.ones(d, dtype=torch.bfloat16, device=dev)
    n, h = torch.empty_like(x), torch.empty_like(x)
    lens = [20, 33, 64]
    c = ref4.paged([1] * 3, lens, n_kv, dim, page, 2)
    cache, table = cache_on(c, dev)
    kv_len = torch.tensor(lens, dtype=torch.int32, device=dev)
    pos = kv_len - 1
    slot = table.gather(1, (pos // page).long()[:, None])[:, 0] * page + pos % page
    slot = slot.to(torch.int32)
    off = torch.arange(4, dtype=torch.int32, device=dev)
    kv_off = torch.tensor([0, 20, 53, 117], dtype=torch.int32, device=dev)
    tab = bd.rope_table(64, dim, 10000.0, dev)
    qo, out = (torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ko, vo = (torch.empty(117, n_kv, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 3, n_q, n_kv, dim), dev)

    def layer():
        bd.bd_block_norm(x, r, gain, 1e-5, n, ws, residual_out=h, post_gain=gain)
        heads = n.view(T, n_q + 2 * n_kv, dim)
        bd.bd_rope_append(heads[:, :n_q], heads[:, n_q: n_q + n_kv], heads[:, n_q + n_kv:], pos, tab, slot, cache, qo, ws)
        bd.bd_attention(qo, off, cache, table, kv_len, dim ** -0.5, 1, out, ws)
        bd.bd_kv_read(cache, table, kv_off, ko, vo, ws)

    layer()
    torch.cuda.synchronize()
    first = [t.clone() for t in (n, h, qo, out, ko, vo)]
    # attention over the same values in a bf16 cache
    kb, vb = (torch.zeros(cache.n_pages, n_kv, page, dim, device=dev, dtype=torch.bfloat16) for _ in range(2))
    for s, (a, b) in enumerate(zip([0, 20, 53], [20, 53, 117])):
        at = torch.arange(b - a, device=dev)
        pg = table[s].long()[at // page]
        kb[pg, :, at % page], vb[pg, :, at % page] = ko[a:b], vo[a:b]
    near = torch.empty_like(out)
    bd.bd_attention(qo, off, bd.KvPages(kb, vb), table, kv_len, dim ** -0.5, 1, near, ws)
    assert (near.float() - out.float()).norm() <= 0.02 * out.float().norm()
    side = torch.cuda.Stream()
    for t in (n, h, qo, out, ko, vo):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (n, h, qo, out, ko, vo)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for t in (n, h, qo, out, ko, vo):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (n, h, qo, out, ko, vo)))
    assert bd.bd_check_async(ws) == bd.BD_OK
