"""The operators between a layer's linears on the paths that sizes and hints
choose between: clusters with many items, CTA pairs over ragged chunks, norms
of many rows and of every row length's kernel, attention without a causal mask
in few rows, and scales of any sign -- against the 64-bit definitions of
layer_oracle.py, with its bounds."""
import numpy as np
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
