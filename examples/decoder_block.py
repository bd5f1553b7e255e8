"""The attention half of a decoder layer, served to many variants at once out
of one paged KV cache: norm -> packed q, k, v product -> rotary positions and
the write into the cache -> attention -> output product -> norm with the
residual's addition.  Every step is an entry point of the library; a batch
holds prompts and single tokens of any mixture of variants, and what a variant
has of its own (the gains and the deltas of its linears) is picked per token.

    python examples/decoder_block.py [--hidden 8192] [--kv int8] [--steps 32]

The weights are random.  The first call takes the sequences' prompts in one
batch, the others one token of each sequence, replayed as a CUDA graph."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_delta_bd_gb300 import bitdelta as bd  # noqa: E402


class DecoderBlock:
    """Weights, cache and workspaces of one layer's attention half.  Sequence s owns the pages page_table[s]."""

    def __init__(self, hidden=8192, n_q=64, n_kv=8, head_dim=128, variants=14, n_seq=16, max_len=1024, page=64,
                 int8=True, max_tokens=4096, theta=10000.0, seed=0, device="cuda"):
        self.hidden, self.n_q, self.n_kv, self.dim, self.page = hidden, n_q, n_kv, head_dim, page
        self.n_seq, self.eps = n_seq, 1e-5
        g = torch.Generator(device=device).manual_seed(seed)
        rows = (n_q + 2 * n_kv) * head_dim
        self.w_qkv, self.w_o = (torch.randn(o, i, generator=g, device=device).mul_(i ** -0.5).to(torch.bfloat16)
                                for o, i in ((rows, hidden), (hidden, n_q * head_dim)))
        self.deltas = {}
        for name, w in (("qkv", self.w_qkv), ("o", self.w_o)):
            o, i = w.shape
            signs = [torch.randint(-2 ** 31, 2 ** 31, (o, i // 32), generator=g, device=device).to(torch.int32)
                     for _ in range(variants)]
            alpha = [torch.rand(o, generator=g, device=device).mul_(0.2 * i ** -0.5) for _ in range(variants)]
            self.deltas[name] = (signs, alpha)
        self.gains = [[(1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16)
                       for _ in range(variants + 1)] for _ in range(2)]  # two norms; the base's gain first
        self.max_pages = -(-max_len // page)
        shape = (n_seq * self.max_pages, n_kv, page, head_dim)
        if int8:
            self.cache = bd.KvPages(*(torch.zeros(shape, dtype=torch.int8, device=device) for _ in range(2)),
                                    *(torch.zeros(shape[:3], device=device) for _ in range(2)))
        else:
            self.cache = bd.KvPages(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        # pages in an order of their own, as an allocator would leave them
        self.page_table = torch.randperm(shape[0], generator=g, device=device).to(torch.int32).view(n_seq, -1)
        self.rope = bd.rope_table(max_len, head_dim, theta, device)
        T, V = max_tokens, variants
        self.ws = bd.new_workspace(max(
            bd.bd_rms_norm_workspace_size(T, hidden), bd.bd_linear_multi_workspace_size(T, V, rows, hidden),
            bd.bd_linear_multi_workspace_size(T, V, hidden, n_q * head_dim), bd.bd_rope_append_workspace_size(T),
            bd.bd_attention_workspace_size(T, n_seq, n_q, n_kv, head_dim)), device)

    def slots(self, seq, pos):
        """Where token pos[t] of sequence seq[t] lies in the cache."""
        page = self.page_table[seq.long(), (pos // self.page).long()]
        return page * self.page + pos % self.page

    def new_buffers(self, T):
        dev, bf = self.w_o.device, torch.bfloat16
        return {"n": torch.empty(T, self.hidden, device=dev, dtype=bf),
                "qkv": torch.empty(T, (self.n_q + 2 * self.n_kv) * self.dim, device=dev, dtype=bf),
                "att": torch.empty(T, self.n_q, self.dim, device=dev, dtype=bf),
                "y": torch.empty(T, self.hidden, device=dev, dtype=bf)}

    def forward(self, x, vid, q_off, kv_len, pos, slot, max_new, buf):
        """x [T][hidden] is the residual stream, and becomes it plus the block's output; returns the second norm's
        result, which the feed-forward half takes.  vid[t] is token t's variant (-1: the base model)."""
        b, ws = buf, self.ws
        n_q, n_kv = self.n_q, self.n_kv
        first, second = self.gains
        bd.bd_rms_norm(x, first[0], self.eps, b["n"], ws, vid=vid, gain_list=first[1:])
        bd.bd_linear_multi(b["n"], vid, *self.deltas["qkv"], bd.BD_ALPHA_PER_ROW, self.w_qkv, b["qkv"], ws)
        heads = b["qkv"].view(x.shape[0], n_q + 2 * n_kv, self.dim)
        q, k, v = heads[:, :n_q], heads[:, n_q: n_q + n_kv], heads[:, n_q + n_kv:]
        bd.bd_rope_append(q, k, v, pos, self.rope, slot, self.cache, q, ws)  # q turns in place
        bd.bd_attention(q, q_off, self.cache, self.page_table, kv_len, self.dim ** -0.5, max_new, b["att"], ws)
        bd.bd_linear_multi(b["att"].view(x.shape[0], -1), vid, *self.deltas["o"], bd.BD_ALPHA_PER_ROW, self.w_o,
                           b["y"], ws)
        bd.bd_rms_norm(b["y"], second[0], self.eps, b["n"], ws, residual=x, residual_out=x, vid=vid,
                       gain_list=second[1:])
        return b["n"]


def batch(block, new, have, device):
    """(q_off, kv_len, pos, slot) of new[s] tokens for each sequence, which has have[s] in the cache already."""
    seq = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(new)])
    pos = torch.cat([torch.arange(h, h + n, dtype=torch.int32) for n, h in zip(new, have)])
    off = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
    kv_len = torch.tensor([n + h for n, h in zip(new, have)], dtype=torch.int32)
    seq, pos = seq.to(device), pos.to(device)
    return off.to(device), kv_len.to(device), pos, block.slots(seq, pos), seq


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--kv", choices=("int8", "bf16"), default="int8")
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    V, S = 14, a.sequences
    block = DecoderBlock(hidden=a.hidden, n_q=a.heads, n_kv=a.kv_heads, variants=V, n_seq=S, int8=a.kv == "int8",
                         max_len=300 + a.steps, max_tokens=300 * S, device=dev)
    g = torch.Generator().manual_seed(1)
    prompts = torch.randint(1, 300, (S,), generator=g).tolist()
    variant = torch.randint(-1, V, (S,), generator=g, dtype=torch.int32).to(dev)

    off, kv_len, pos, slot, seq = batch(block, prompts, [0] * S, dev)
    x = torch.randn(sum(prompts), a.hidden, generator=g).to(torch.bfloat16).to(dev)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    block.forward(x, variant[seq.long()], off, kv_len, pos, slot, max(prompts), block.new_buffers(len(x)))
    end.record()
    torch.cuda.synchronize()
    print(f"prompts: {len(x)} tokens of {S} sequences in {start.elapsed_time(end):.3f} ms (first call)")

    # single tokens: the buffers stay, so that the step is captured once and replayed
    off, kv_len, pos, slot, seq = batch(block, [1] * S, prompts, dev)
    x = torch.randn(S, a.hidden, generator=g).to(torch.bfloat16).to(dev)
    buf = block.new_buffers(S)
    block.forward(x.clone(), variant, off, kv_len, pos, slot, 1, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, variant, off, kv_len, pos, slot, 1, buf)
    start.record()
    for _ in range(a.steps):
        graph.replay()
        kv_len += 1
        pos += 1
        slot.copy_(block.slots(seq, pos))
    end.record()
    torch.cuda.synchronize()
    print(f"single tokens: {a.steps} steps of {S} sequences, {start.elapsed_time(end) / a.steps * 1e3:.1f} us a step")
    st = bd.bd_check_async(block.ws)
    print("status:", bd.status_string(st))
    assert st == bd.BD_OK and bool(torch.isfinite(x.float()).all())


if __name__ == "__main__":
    main()
