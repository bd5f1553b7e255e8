"""The operators between a layer's linears where they are used whole: buffers
whose offsets pass 32 bits, the bounds-checked build, results that do not
depend on the run, and the example that runs a decoder layer's attention
half."""
import importlib.util
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layer_oracle as ref
import test_layer_ops as ops
from bit_weight_delta_bd_gb300 import bitdelta as bd

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


# ------------------------------------------------------------------------------- past 32 bits

def test_norm_past_32_bits(dev):
    """Rows whose elements lie past 2^31 equal the same rows in a call of their own."""
    T, d = 2 ** 31 // 8192 + 40, 8192
    x = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    x[:64].normal_(generator=torch.Generator(device=dev).manual_seed(3))
    x[64:-64] = 1.0
    x[-64:] = x[:64]
    gain = torch.randn(d, device=dev, generator=torch.Generator(device=dev).manual_seed(4)).to(torch.bfloat16)
    out = torch.zeros_like(x)
    ws = bd.new_workspace(bd.bd_rms_norm_workspace_size(T, d), dev)
    bd.bd_rms_norm(x, gain, 1e-5, out, ws, residual=x, residual_out=x)
    assert bd.bd_check_async(ws) == bd.BD_OK
    assert torch.equal(out[-64:], out[:64]) and bool((out[:64] != 0).any())
    assert torch.equal(x[-64:], x[:64])


@pytest.mark.parametrize("int8", [False, True])
def test_cache_past_32_bits(dev, int8):
    """Sequences on the last pages of a cache with more than 2^32 bytes (and 2^31 elements) of keys: appended, read
    back and attended to, they give what the same tokens give on the first pages."""
    n_kv, page, dim, n_q = 8, 128, 128, 32
    n_pages = (2 ** 32 // (1 if int8 else 2)) // (n_kv * page * dim) + 12
    shape = (n_pages, n_kv, page, dim)
    if int8:
        cache = bd.KvPages(*(torch.empty(shape, dtype=torch.int8, device=dev) for _ in range(2)),
                           *(torch.empty(shape[:3], device=dev) for _ in range(2)))
    else:
        cache = bd.KvPages(*(torch.empty(shape, dtype=torch.bfloat16, device=dev) for _ in range(2)))
    lens = [700, 129]
    pages = [[0, 3, 1, 2, 5, 4], [6, 7, 8, 9, 10, 11]]
    T = sum(lens)
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(T, h, dim, generator=g).to(torch.bfloat16).to(dev) for h in (n_q, n_kv, n_kv))
    pos = torch.cat([torch.arange(n) for n in lens])
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
    tab = bd.rope_table(1024, dim, 10000.0, dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 2, n_q, n_kv, dim), dev)
    off = torch.tensor([0, lens[0], T], dtype=torch.int32, device=dev)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    kv_len = torch.tensor(lens, dtype=torch.int32, device=dev)
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
    want = ref.attention(runs[0][0].cpu(), [0, lens[0], T], *[
        [t[: lens[0]].cpu(), t[lens[0]:].cpu()] for t in (runs[0][1], runs[0][2])], lens, dim ** -0.5, True)
    if not int8:  # (an int8 cache's values are read back rounded, which attention does not do)
        bound = ref.attention_bounds(*want, max(lens))[0]
        assert bool(((runs[0][3].double().cpu() - want[0]).abs() <= bound).all())


# ------------------------------------------------------------------------------- clusters, and the deal

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page,max_new", [
    # clusters with several items each: more rows than max_new lets the host expect
    ([5, 1, 9], [800, 33, 300], 16, 2, 128, 16, 1), ([3, 0, 40], [2000, 7, 500], 8, 1, 64, 64, 2),
    # one row a head, 16 rows, rows that see nothing, blocks without a tile of their own
    ([1], [900], 8, 8, 128, 32, 1), ([16], [1000], 8, 8, 64, 16, 16), ([4, 2], [2, 700], 8, 2, 128, 16, 4),
    ([1, 1], [1, 1000], 8, 1, 64, 128, 1), ([1] * 19, [1023 - 50 * i for i in range(19)], 8, 8, 64, 16, 1),
    ([1], [8192], 8, 1, 128, 64, 1), ([2], [4001], 7, 1, 64, 16, 2),
    # dealt out: caches too long, or too many
    ([1, 1], [20000, 3000], 8, 1, 128, 128, 1), ([1] * 40, [3000 - 70 * i for i in range(40)], 16, 8, 64, 16, 1),
    ([2] * 30, [1500 - 51 * i for i in range(30)], 64, 8, 128, 32, 2), ([1], [9000], 12, 1, 64, 16, 1)])
def test_attention_clusters_and_deal(dev, n_new, kv_len, n_q, n_kv, dim, page, max_new, int8):
    ops.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, seed=sum(kv_len) % 97, max_new=max_new)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page,max_new", [
    # chunks and decode steps in one batch: 16 rows and fewer take the kernel for few rows
    ([1, 300, 1, 1, 40, 2, 3], [900, 800, 33, 1, 400, 1500, 3], 16, 2, 128, 16, 300),
    ([16, 17, 200, 1], [200, 300, 200, 5000], 4, 4, 64, 64, 200), ([1] * 30 + [129], [40 * i for i in range(31)], 12, 1, 128, 32, 129),
    ([1, 1, 1], [700, 0, 64], 8, 1, 64, 16, 50),  # no chunk after all
    ([0, 0, 150], [9, 0, 150], 8, 2, 128, 128, 150), ([1, 30, 2], [50, 30, 700], 8, 2, 128, 16, 2 ** 62), ([600, 8, 1], [600, 1000, 2000], 2, 2, 128, 16, 9)])
def test_attention_mixed_batch(dev, n_new, kv_len, n_q, n_kv, dim, page, max_new, int8):
    ops.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, seed=sum(kv_len) % 89, max_new=max_new)


@pytest.mark.parametrize("n_new", [1, 40])
@pytest.mark.parametrize("gap", [20, 30, 60])
def test_attention_small_probabilities(dev, n_new, gap):
    """One key has all the weight and a value of 0 in every dim but the first: the others hold what is left to the
    keys `gap` (in units of the exponential) below it, to the same relative bound."""
    dim, length, page = 64, 120, 16
    g = torch.Generator().manual_seed(gap + n_new)
    kc = torch.zeros(8, 1, page, dim, dtype=torch.int8)
    vc = torch.randint(-127, 128, (8, 1, page, dim), generator=g).to(torch.int8)
    kc[:, 0, :, 0] = torch.randint(-12, -8, (8, page), generator=g).to(torch.int8)
    kc[0, 0, 3, 0] = 118
    vc[0, 0, 3, 1:] = 0
    ks, vs = torch.full((8, 1, page), 0.5), 0.01 + 0.01 * torch.rand(8, 1, page, generator=g)
    q = torch.zeros(n_new, 1, dim)
    q[:, :, 0] = gap / 64
    q = q.to(torch.bfloat16)
    cache = bd.KvPages(*(t.to(dev) for t in (kc, vc, ks, vs)))
    table = torch.arange(8, dtype=torch.int32, device=dev).view(1, 8)
    out = torch.empty(n_new, 1, dim, device=dev, dtype=torch.bfloat16)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(n_new, 1, 1, 1, dim), dev)
    bd.bd_attention(q.to(dev), torch.tensor([0, n_new], dtype=torch.int32, device=dev), cache, table,
                    torch.tensor([length], dtype=torch.int32, device=dev), 1.0, n_new, out, ws)
    assert bd.bd_check_async(ws) == bd.BD_OK
    k, v = ((c.double() * s.double()[..., None]).transpose(1, 2).reshape(128, 1, dim)[:length]
            for c, s in ((kc, ks), (vc, vs)))
    want = ref.attention(q, [0, n_new], [k], [v], [length], 1.0, True)
    assert float(want[0][:, :, 1:].abs().max()) < 0.01 * 2.0 ** -(gap / 1.5)
    ops.within(out, want[0], ref.attention_bounds(*want, length)[0], "attention")


@pytest.mark.parametrize("int8", [False, True])
def test_buffers_on_16_byte_boundaries(dev, int8):
    """Buffers 16 bytes off the start of a 32-byte sector give the same bits as ones on it."""
    T, n_q, n_kv, dim, page = 300, 8, 2, 128, 16
    g = torch.Generator(device=dev).manual_seed(6)

    def rand(*shape, off=0):
        n = int(np.prod(shape))
        t = torch.empty(n + 8, device=dev, dtype=torch.bfloat16)
        t[off: off + n].normal_(generator=g)
        return t[off: off + n].view(shape)

    def moved(t):
        u = torch.empty(t.numel() + 16 // t.element_size(), device=dev, dtype=t.dtype)[16 // t.element_size():]
        u.copy_(t.flatten())
        assert u.data_ptr() % 32 == 16
        return u.view(t.shape)

    q, k, v = rand(T, n_q, dim), rand(T, n_kv, dim), rand(T, n_kv, dim)
    shape = (20, n_kv, page, dim)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    table = torch.arange(20, dtype=torch.int32, device=dev).view(1, 20)
    off = torch.tensor([0, T], dtype=torch.int32, device=dev)
    tab = bd.rope_table(T, dim, 10000.0, dev)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 1, n_q, n_kv, dim), dev)
    for inter in (False, True):
        runs = []
        for place in (lambda t: t, moved):
            kv = [place(torch.zeros(shape, dtype=torch.int8 if int8 else torch.bfloat16, device=dev)) for _ in range(2)]
            cache = bd.KvPages(*kv, *([torch.zeros(shape[:3], device=dev) for _ in range(2)] if int8 else []))
            qo, out, ko, vo = (place(torch.zeros_like(t)) for t in (q, q, k, v))
            bd.bd_rope_append(place(q), place(k), place(v), pos, tab, pos, cache, qo, ws, interleaved=inter)
            bd.bd_kv_read(cache, table, off, ko, vo, ws)
            bd.bd_attention(qo, off, cache, table, off[1:], dim ** -0.5, T, out, ws)
            assert bd.bd_check_async(ws) == bd.BD_OK
            runs.append([*kv, qo, ko, vo, out])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


# ------------------------------------------------------------------------------- one result

def test_results_do_not_depend_on_the_run(dev):
    g = torch.Generator(device=dev).manual_seed(2)
    n_kv, page, dim, n_q = 2, 32, 128, 16
    kp, vp = (torch.randn(300, n_kv, page, dim, generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
    cache = bd.KvPages(kp, vp)
    table = torch.arange(300, dtype=torch.int32, device=dev).view(3, 100)
    kv_len = torch.tensor([3200, 1777, 64], dtype=torch.int32, device=dev)
    for news in ([1, 1, 1], [700, 300, 64]):
        T = sum(news)
        q = torch.randn(T, n_q, dim, generator=g, device=dev).to(torch.bfloat16)
        off = torch.tensor(np.cumsum([0] + news), dtype=torch.int32, device=dev)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(T, 3, n_q, n_kv, dim), dev)
        outs = [torch.empty_like(q) for _ in range(20)]
        for o in outs:
            bd.bd_attention(q, off, cache, table, kv_len, 0.09, max(news), o, ws)
        assert bd.bd_check_async(ws) == bd.BD_OK
        assert all(torch.equal(outs[0], o) for o in outs[1:])


# ------------------------------------------------------------------------------- the bounds-checked build

def run_with(lib_path, out):
    p = subprocess.run([sys.executable, os.path.join(HERE, "layer_bounds_run.py"), out], cwd=ROOT,
                       env=dict(os.environ, BD_LIBRARY=lib_path), capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-4000:]
    return json.loads(p.stdout.strip().splitlines()[-1])


def test_bounds_checked_build_is_silent_and_bit_identical(dev, tmp_path):
    from bit_weight_delta_bd_gb300 import build

    rn = run_with(build.LIB, str(tmp_path / "normal.npz"))
    rb = run_with(build.build(debug_bounds=True), str(tmp_path / "bounds.npz"))
    assert rn["enabled"] is False and rb["enabled"] is True
    assert rb["status"] == bd.BD_OK and rb["bits"] == 0, f"a bounds check fired in kernels 0x{rb['bits']:x}"
    a, b = np.load(tmp_path / "normal.npz"), np.load(tmp_path / "bounds.npz")
    assert sorted(a.files) == sorted(b.files) and len(a.files) > 60
    assert not [n for n in a.files if not np.array_equal(a[n], b[n])]


# ------------------------------------------------------------------------------- the example

def example():
    spec = importlib.util.spec_from_file_location("decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense_block(block, x, which, news):
    """The block in float64 from the same weights, with a cache that is not quantised."""
    def weights(w, name):
        signs, alpha = block.deltas[name]
        out = [w.double()]
        for s, a in zip(signs, alpha):
            bits = ((s[:, :, None] >> torch.arange(32, device=s.device)) & 1).reshape(w.shape)
            out.append(w.double() + a.double()[:, None] * (2.0 * bits - 1))
        return out

    def normed(h, gains):
        return h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + block.eps) * torch.stack(gains).double()[which]

    def per_token(h, ws):
        return torch.stack([ws[int(w)] @ t for w, t in zip(which, h)])

    n_q, n_kv, dim = block.n_q, block.n_kv, block.dim
    qkv = per_token(normed(x, block.gains[0]), weights(block.w_qkv, "qkv")).view(len(x), n_q + 2 * n_kv, dim)
    att, row = [], 0
    for n in news:
        h = qkv[row: row + n]
        c, s = block.rope[:n, :, 0].double(), block.rope[:n, :, 1].double()
        q, k = (ref.turn(t, c, s, dim, False) for t in (h[:, :n_q], h[:, n_q: n_q + n_kv]))
        k, v = (t.repeat_interleave(n_q // n_kv, 1) for t in (k, h[:, n_q + n_kv:]))
        sc = torch.einsum("ihd,jhd->hij", q, k) * dim ** -0.5
        sc = sc.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -float("inf"))
        att.append(torch.einsum("hij,jhd->ihd", sc.softmax(-1), v))
        row += n
    h = x + per_token(torch.cat(att).reshape(len(x), -1), weights(block.w_o, "o"))
    return h, normed(h, block.gains[1])


@pytest.mark.parametrize("int8", [False, True])
def test_example_block(dev, int8):
    """Prompts, then single tokens on top of them, against the dense block.  Each value passes about eight roundings
    to bf16 (2^-9 of it at most, independent) and, in an int8 cache, one of 2^-7.6 of its vector's largest value, some
    three times its typical one: within 2^-5 of the result's norm with room to spare."""
    m = example()
    block = m.DecoderBlock(hidden=512, n_q=8, n_kv=2, head_dim=64, variants=3, n_seq=3, max_len=96, page=16, int8=int8,
                           max_tokens=256, device=dev)
    g = torch.Generator().manual_seed(21)
    prompts, steps = [70, 1, 33], 4
    total = [p + steps for p in prompts]
    streams = [torch.randn(n, 512, generator=g).to(torch.bfloat16).to(dev) for n in total]
    variant = torch.tensor([1, -1, 2], dtype=torch.int32, device=dev)
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
    h, n = dense_block(block, torch.cat(streams).double(), which, total)
    for got, want in ((got_h, h), (got_n, n)):
        got = torch.cat([torch.cat(g) for g in got]).double()
        rel = ((got - want).norm(dim=1) / want.norm(dim=1)).max()
        assert float(rel) <= 2 ** -5, float(rel)
