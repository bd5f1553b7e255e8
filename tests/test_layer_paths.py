"""The operators between a layer's linears on the paths that sizes and hints
choose between: clusters with many items, CTA pairs over ragged chunks, norms
of many rows and of every row length's kernel, attention without a causal mask
in few rows, and scales of any sign -- against the 64-bit definitions of
layer_oracle.py, with its bounds."""
import os
import subprocess
import sys

import pytest
import torch

import layer_oracle as ref
import test_layer_ops as ops
from bit_weight_delta_bd_gb300 import bitdelta as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def again(run, out, times):
    """The call repeated: the same bits each time."""
    outs = [torch.empty_like(out) for _ in range(times)]
    for o in outs:
        run(o)
    assert all(torch.equal(out, o) for o in outs)


# ------------------------------------------------------------------------------- clusters

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", [
    ([64], [1100], 8, 1, 64, 16), ([50, 3, 21], [500, 400, 30], 16, 1, 128, 16), ([33, 1], [260, 900], 7, 1, 128, 64)])
def test_clusters_of_many_items(dev, n_new, kv_len, n_q, n_kv, dim, page, int8):
    """A host that expects one token a sequence gets clusters, whose blocks join item after item."""
    out, q, on, off, lens = ops.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, seed=sum(n_new), max_new=1)
    cache = bd.KvPages(on["k"], on["v"], on["ks"], on["vs"])
    ws = bd.new_workspace(bd.bd_attention_workspace_size(len(q), len(n_new), n_q, n_kv, dim), dev)
    again(lambda o: bd.bd_attention(q, off, cache, on["table"], lens, dim ** -0.5, 1, o, ws), out, 50)
    assert bd.bd_check_async(ws) == bd.BD_OK


# ------------------------------------------------------------------------------- pairs

@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,page", [
    # lengths that end inside a tile, in either half of its keys, on pages of every size; what lies past is NaN
    ([300, 77, 513], [300, 1001, 1500], 8, 2, 16), ([257, 1, 400, 90], [257, 33, 830, 95], 8, 1, 64),
    ([130, 600], [1111, 601], 4, 1, 128), ([80] * 9, [80 + 29 * i for i in range(9)], 32, 4, 32)])
def test_pairs_over_ragged_chunks(dev, n_new, kv_len, n_q, n_kv, page, int8):
    """Both CTAs' rows, values past the lengths and converted tiles reach the products: many short items, again and
    again, with the same bits."""
    out, q, on, off, lens = ops.run_attention(dev, n_new, kv_len, n_q, n_kv, 128, page, int8, seed=len(n_new))
    cache = bd.KvPages(on["k"], on["v"], on["ks"], on["vs"])
    ws = bd.new_workspace(bd.bd_attention_workspace_size(len(q), len(n_new), n_q, n_kv, 128), dev)
    again(lambda o: bd.bd_attention(q, off, cache, on["table"], lens, 128 ** -0.5, max(n_new), o, ws), out, 100)
    assert bd.bd_check_async(ws) == bd.BD_OK


# ------------------------------------------------------------------------------- offsets of a read

@pytest.mark.parametrize("n_seq", [1, 3, 700])
def test_kv_read_reports_bad_offsets(dev, n_seq):
    """Offsets that run backwards, start past 0, or end past the output's rows; what has a place is read."""
    pool = torch.arange(16, dtype=torch.float32, device=dev).view(1, 1, 16, 1).expand(2, 1, 16, 64)
    pool = pool.to(torch.bfloat16).contiguous()
    cache, ws = bd.KvPages(pool, pool.clone()), bd.new_workspace(256, dev)
    table = torch.zeros(n_seq, 1, dtype=torch.int32, device=dev)
    good = [min(5 * s, 12) for s in range(n_seq + 1)]
    rows = good[-1]

    def read(off, rows):
        ko, vo = (torch.full((rows, 1, 64), 3.0, device=dev, dtype=torch.bfloat16) for _ in range(2))
        bd.bd_kv_read(cache, table, torch.tensor(off, dtype=torch.int32, device=dev), ko, vo, ws)
        return bd.bd_check_async(ws), ko

    want = torch.tensor([r - max(o for o in good if o <= r) for r in range(rows)], dtype=torch.float32)
    status, ko = read(good, rows)
    assert status == bd.BD_OK and torch.equal(ko[:, 0, 0].float().cpu(), want)
    status, ko = read(good, rows - 1)
    assert status == bd.BD_ERR_BAD_INDEX and torch.equal(ko[:, 0, 0].float().cpu(), want[:-1])
    assert read([1] + good[1:], rows)[0] == bd.BD_ERR_BAD_INDEX
    assert read([-2] + good[1:], rows)[0] == bd.BD_ERR_BAD_INDEX
    if n_seq > 1:
        back = list(good)
        back[n_seq // 2] = good[-1] + 1
        assert read(back, rows)[0] == bd.BD_ERR_BAD_INDEX
    assert read(good, rows)[0] == bd.BD_OK


# ------------------------------------------------------------------------------- norms of every kernel

OUT = [torch.bfloat16, torch.float32, torch.float8_e4m3fn]


def check_norm(dev, T, d, V, out_dtype, seed, residual=True, in_place=False):
    h, y, ho, out, scale = ops.run_norm(dev, T, d, V, out_dtype, residual, seed=seed, in_place=in_place)
    if residual:
        ops.within(ho, h, ref.half_ulp_bf16(h) + h.abs() * 2 * ref.U32, "residual")
    bound = y.abs() * ref.norm_rel(d)
    if out_dtype == torch.bfloat16:
        bound = bound + ref.half_ulp_bf16(y.abs() + bound)
    if out_dtype != torch.float8_e4m3fn:
        return ops.within(out, y, bound, "norm")
    # the scale is off by the norm's error; a code by half its step and by the scale's error
    s = y.abs().amax(1).clamp_min(1e-30) / 448
    rel = ref.norm_rel(d) + 4 * ref.U32
    ops.within(scale, s, s * rel, "scale")
    z = (y / s[:, None]).abs()
    half_step = torch.pow(2.0, torch.floor(torch.log2(z.clamp_min(2.0 ** -6))) - 4)
    ops.within(out.float().cpu().double() * scale.cpu().double()[:, None], y,
               s[:, None] * half_step * (1 + 2.0 ** -10) + y.abs() * 4 * rel, "codes")


@pytest.mark.parametrize("out_dtype", OUT)
@pytest.mark.parametrize("T,d,V", [
    # more rows than the GPU has places for: a warp a row up to 512, then one, two, four groups a thread, and
    # rows that are read twice
    (700, 8, 0), (1001, 248, 3), (700, 256, 0), (901, 264, 14), (701, 512, 64), (320, 520, 0), (1300, 4096, 5),
    (4096, 8192, 14), (700, 16384, 0), (305, 16392, 2), (400, 20480, 3), (310, 32768, 0), (306, 33000, 1),
    # few rows of the same lengths
    (5, 16392, 2), (3, 20480, 0), (2, 32768, 1)])
def test_norm_kernels(dev, T, d, V, out_dtype):
    check_norm(dev, T, d, V, out_dtype, seed=T + d)


@pytest.mark.parametrize("T,d", [(700, 504), (900, 8192), (400, 20480), (308, 32776)])
def test_norm_many_rows_in_place(dev, T, d):
    check_norm(dev, T, d, 2, torch.bfloat16, seed=T, in_place=True)
    check_norm(dev, T, d, 0, torch.float32, seed=T + 1, residual=False)


# ------------------------------------------------------------------------------- masks and scales of attention

FEW = [  # clusters, and caches that are dealt out; 2 to 16 rows a head
    ([2], [300], 1, 1, 64, 16), ([3, 1], [70, 900], 8, 2, 128, 16), ([16], [513], 4, 4, 64, 64),
    ([2, 5], [9000, 40], 8, 8, 128, 128), ([1] * 20 + [2], [1200 - 50 * i for i in range(21)], 16, 8, 64, 32),
    ([2, 2], [0, 1], 8, 1, 128, 32)]
MANY = [([40, 7], [130, 7], 8, 2, 64, 16), ([300, 1, 33], [700, 90, 33], 8, 2, 128, 64), ([9], [400], 4, 1, 128, 16),
        ([70, 70], [0, 1], 4, 1, 64, 32)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", FEW)
def test_few_rows_without_a_causal_mask(dev, n_new, kv_len, n_q, n_kv, dim, page, int8):
    ops.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, causal=False, seed=len(n_new) + dim)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("scale", [-0.1, 0.0, -1.0])
@pytest.mark.parametrize("n_new,kv_len,n_q,n_kv,dim,page", FEW + MANY)
def test_scales_of_any_sign(dev, n_new, kv_len, n_q, n_kv, dim, page, scale, int8):
    """Below zero the largest products weigh least; at zero every key that a row sees weighs the same."""
    causal = sum(kv_len) % 3 != 0
    ops.run_attention(dev, n_new, kv_len, n_q, n_kv, dim, page, int8, causal=causal, seed=sum(kv_len) % 83, scale=scale)


@pytest.mark.parametrize("n_new", [[1, 1], [40, 1]])
def test_nan_query_stays_in_its_rows_int8(dev, n_new):
    out, qd, on, off, ln = ops.run_attention(dev, n_new, [90, 90], 4, 2, 128, 16, True, seed=3)
    q = qd.clone()
    q[0, 1] = float("nan")
    out2 = torch.empty_like(out)
    ws = bd.new_workspace(bd.bd_attention_workspace_size(len(q), 2, 4, 2, 128), dev)
    cache = bd.KvPages(on["k"], on["v"], on["ks"], on["vs"])
    bd.bd_attention(q, off, cache, on["table"], ln, 128 ** -0.5, max(n_new), out2, ws)
    assert out2[0, 1].isnan().all()
    # (the rows of an item share the type of a step's products: the others keep their bounds, not their bits)
    c = ref.paged(n_new, [90, 90], 2, 128, 16, True, seed=3)
    want = ref.attention(qd.cpu(), off.tolist(), c["vals"]["k"], c["vals"]["v"], [90, 90], 128 ** -0.5, True)
    out2[0, 1] = out[0, 1]
    ops.within(out2, want[0], ref.attention_bounds(*want, 90)[0], "attention")


# ------------------------------------------------------------------------------- the bounds-checked build

def test_bounds_checked_build_on_these_paths(dev):
    """The same tests through the library that checks each access (conftest.py asks it after every test)."""
    from bit_weight_delta_bd_gb300 import build

    lib = build.build(debug_bounds=True)
    p = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-m", "gpu", "-x", "-q", "-k",
                        "norm_kernels or norm_many or many_items or ragged_chunks or bad_offsets"],
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       env=dict(os.environ, BD_LIBRARY=lib), capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-2000:]
