"""Plain definitions of the 4-bit cache (CPU tensors) for the tests, and the
bounds that attention over it is held to.

A value is code * scale + low, with a bf16 scale and lowest value for each group
of 32 elements.  A score formed group by group adds products of magnitude |q|
(15 scale + |low|), whatever the value they make, so its rounding error is held
to (dim + 8) 2^-22 times their sum."""
from __future__ import annotations

import math

import torch

import layer_oracle as ref

U11 = 2.0 ** -11  # fp16's unit roundoff


def pack(code):
    """[..., dim] codes as bytes [..., dim / 2]: element 8 w + 2 i + j in bits 16 j + 4 i of word w."""
    w = code.long().reshape(*code.shape[:-1], code.shape[-1] // 8, 4, 2)
    words = sum(w[..., i, j] << (16 * j + 4 * i) for i in range(4) for j in range(2))
    return torch.stack([(words >> (8 * b)) & 255 for b in range(4)], -1).flatten(-2).to(torch.uint8)


def unpack(byte):
    words = sum(byte.long().reshape(*byte.shape[:-1], byte.shape[-1] // 4, 4)[..., b] << (8 * b) for b in range(4))
    return torch.stack([(words >> (16 * j + 4 * i)) & 15 for i in range(4) for j in range(2)], -1).flatten(-2)


def codes(x):
    """(bytes, pairs [..., dim / 32, 2] bf16) of float32 vectors, operation by operation."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    lo, hi = g.amin(-1), g.amax(-1)
    scale = ((hi - lo).clamp_min(1e-30) / torch.tensor(15.0)).to(torch.bfloat16)
    low = lo.to(torch.bfloat16)
    c = torch.round((g - low.float()[..., None]) / scale.float()[..., None]).clamp(0, 15)
    return pack(c.flatten(-2)), torch.stack([scale, low], -1)


def values(byte, pairs, dtype=torch.float64):
    """[..., dim] values: in float32 as they are read back, in float64 as they are defined."""
    c = unpack(byte).to(dtype)
    per = [pairs[..., i].to(dtype).repeat_interleave(32, -1) for i in range(2)]
    return c * per[0] + per[1]


def paged(n_new, kv_len, n_kv, dim, page, seed, spare=3, offset=0.0):
    """A 4-bit cache of the sequences on pages in random order (CPU tensors): groups past each length and on spare
    pages have scales and lowest values of NaN, unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_len]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((len(kv_len), max(need + [1]) + 1), -1, dtype=torch.int32)
    c = {"n_new": n_new, "kv_len": kv_len, "table": table, "vals": {"k": [], "v": []}, "steps": []}
    for name in "kv":
        c[name] = torch.randint(0, 256, (n_pages, n_kv, page, dim // 2), generator=g, dtype=torch.uint8)
        c[name + "s"] = torch.full((n_pages, n_kv, page, dim // 32, 2), math.nan, dtype=torch.bfloat16)
    used = 0
    for s, length in enumerate(kv_len):
        ids = perm[used: used + need[s]]
        used += need[s]
        table[s, : need[s]] = ids.to(torch.int32)
        at = torch.arange(length)
        pg, off = (ids[at // page], at % page) if length else (at, at)
        for name in "kv":
            x = torch.randn(length, n_kv, dim, generator=g) + offset * torch.randn(n_kv, dim, generator=g)
            byte, pair = codes(x)
            c[name][pg, :, off], c[name + "s"][pg, :, off] = byte, pair
            c["vals"][name].append(values(byte, pair))
            if name == "k":  # what a score's products may amount to
                p = pair.double().abs()
                c["steps"].append((15 * p[..., 0] + p[..., 1]).repeat_interleave(32, -1))
    return c


def attention(q, q_off, c, scale, causal):
    """float64: (out, lse) of layer_oracle.attention over the values; the sums of p |v|; those of p times what the
    codes may add to the lowest value; and, of each row, the largest sum of its scores' products in magnitude."""
    out, lse, mag, _ = ref.attention(q, q_off, c["vals"]["k"], c["vals"]["v"], c["kv_len"], scale, causal)
    spans = []
    for s, length in enumerate(c["kv_len"]):
        pg = c["table"][s, : -(-length // c["k"].shape[2])].long()
        pair = c["vs"][pg].transpose(1, 2).flatten(0, 1)[:length].double()
        spans.append((15 * pair[..., 0].abs()).repeat_interleave(32, -1))
    coded = ref.attention(q, q_off, c["vals"]["k"], spans, c["kv_len"], scale, causal)[0]
    z = torch.zeros_like(lse)
    for s, length in enumerate(c["kv_len"]):
        rows = slice(q_off[s], q_off[s + 1])
        if length and q_off[s + 1] > q_off[s]:
            big = c["steps"][s].repeat_interleave(q.shape[1] // c["steps"][s].shape[1], 1)  # [len][n_q][dim]
            z[rows] = torch.einsum("thd,jhd->thj", q[rows].double().abs(), big).amax(-1) * abs(scale)
    return out, lse, mag, coded, z


def bounds(want, dim, n_keys, coded_rel, value_rel):
    """Elementwise bounds of the bf16 output and of the log-sum-exp: coded_rel times what V's codes may amount to,
    value_rel times V's values, and what an error of the scores, formed in fp32, makes of both."""
    out_ref, lse, mag, coded, z = want
    sums = (n_keys + 64) * 2.0 ** -22
    err = z * (dim + 8) * 2.0 ** -22
    out = coded * coded_rel + mag * value_rel + (mag + coded) * (torch.expm1(2 * err)[..., None] + 2 * sums)
    out = out + ref.half_ulp_bf16(out_ref.abs() + out)
    return out, err + sums + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -22 + 1e-6
