"""Runs the operators between a layer's linears once per kernel on cuda:0 and
saves each output's bits to an .npz file, for the bounds-checked build's test,
which runs this script through both libraries (BD_LIBRARY) and compares.

Usage: python tests/layer_bounds_run.py OUT.npz

The cases take every kernel: norms of short and long rows in each output type,
rotary appends of both cache types, reads, and attention by whole rows, by
split rows with their join, and by chunks in one piece and in several."""
from __future__ import annotations

import json
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_delta_bd_gb300 import bitdelta as bd  # noqa: E402


def run(path: str) -> dict:
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    g = torch.Generator().manual_seed(5)
    res: dict[str, np.ndarray] = {}
    bf = torch.bfloat16

    def rand(*shape):
        return torch.randn(*shape, generator=g).to(bf).to(dev)

    def keep(name, *tensors):
        for i, t in enumerate(tensors):
            res[f"{name}_{i}"] = t.detach().contiguous().view(torch.uint8).cpu().numpy()

    def clean(ws):
        assert bd.bd_check_async(ws) == bd.BD_OK

    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731

    for T, d in ((1, 8), (7, 1000), (37, 520), (130, 8192), (3, 20480)):
        x, r, gains = rand(T, d), rand(T, d), [rand(d) for _ in range(4)]
        vid = ints((torch.arange(T) % 4 - 1).tolist())
        for dt in (bf, torch.float32, torch.float8_e4m3fn):
            out, ro = torch.zeros(T, d, dtype=dt, device=dev), torch.zeros_like(x)
            scale = torch.zeros(T, device=dev) if dt == torch.float8_e4m3fn else None
            ws = bd.new_workspace(bd.bd_rms_norm_workspace_size(T, d), dev)
            bd.bd_rms_norm(x, gains[0], 1e-5, out, ws, residual=r, residual_out=ro, scale=scale, vid=vid,
                           gain_list=gains[1:])
            clean(ws)
            keep(f"norm_{T}_{d}_{str(dt)[6:]}", out, ro, *([scale] if scale is not None else []))

    for int8, dim, page, n_q, n_kv in ((False, 128, 16, 8, 2), (True, 128, 64, 8, 2), (False, 64, 128, 6, 6),
                                       (True, 64, 32, 8, 1)):
        lens = [700, 33, 1, 1500]
        maxp = -(-max(lens) // page)
        shape = (len(lens) * maxp, n_kv, page, dim)
        if int8:
            cache = bd.KvPages(*(torch.zeros(shape, dtype=torch.int8, device=dev) for _ in range(2)),
                               *(torch.zeros(shape[:3], device=dev) for _ in range(2)))
        else:
            cache = bd.KvPages(*(torch.zeros(shape, dtype=bf, device=dev) for _ in range(2)))
        table = torch.randperm(shape[0], generator=g).to(torch.int32).view(len(lens), maxp)
        pos = torch.cat([torch.arange(n) for n in lens])
        seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)])
        slot = table[seq, pos // page] * page + pos % page
        T = len(pos)
        tab = bd.rope_table(2048, dim, 10000.0, dev)
        packed = rand(T, n_q + 2 * n_kv, dim)
        qo = torch.zeros(T, n_q, dim, dtype=bf, device=dev)
        ws = bd.new_workspace(bd.bd_attention_workspace_size(T, len(lens), n_q, n_kv, dim), dev)
        bd.bd_rope_append(packed[:, :n_q], packed[:, n_q: n_q + n_kv], packed[:, n_q + n_kv:], ints(pos.tolist()), tab,
                          ints(slot.tolist()), cache, qo, ws)
        clean(ws)
        name = f"i8{int(int8)}_{dim}"
        keep(f"append_{name}", qo, cache.k, cache.v, *([cache.k_scale, cache.v_scale] if int8 else []))
        td = table.to(dev)
        ko, vo = (torch.zeros(T + 3, n_kv, dim, dtype=bf, device=dev) for _ in range(2))
        bd.bd_kv_read(cache, td, ints([0] + np.cumsum(lens).tolist()), ko, vo, ws)
        clean(ws)
        keep(f"read_{name}", ko, vo)
        # single tokens, a few (speculative), chunks of one and several tiles, short caches alone
        for news, ln in (([1] * 4, lens), ([3, 1, 1, 2], lens), ([600, 33, 1, 40], lens), ([1] * 4, [70, 33, 1, 200]),
                         ([1500, 0, 0, 0], [1500, 5, 0, 9])):
            n = sum(news)
            q, out = rand(n, n_q, dim), torch.zeros(n, n_q, dim, dtype=bf, device=dev)
            lse = torch.zeros(n, n_q, device=dev)
            short = -(-max(ln) // page)
            bd.bd_attention(q, ints([0] + np.cumsum(news).tolist()), cache, td[:, :short].contiguous(), ints(ln),
                            dim ** -0.5, max(news), out, ws, lse=lse)
            clean(ws)
            keep(f"attention_{name}_{n}_{ln[0]}", out, lse)

    torch.cuda.synchronize()
    st, bits = bd.bd_debug_bounds_check()
    np.savez(path, **res)
    return {"status": st, "bits": bits, "enabled": bd.bd_debug_bounds_enabled(), "arrays": len(res)}


if __name__ == "__main__":
    print(json.dumps(run(sys.argv[1])))
