"""Plain 64-bit definitions of the operators between a layer's linears (CPU,
torch float64), the inputs of their tests, and the bounds that their results
are held to.

Bounds.  u32 = 2^-24 is fp32's unit roundoff, u16 = 2^-8 bf16's.  A sum of
squares of n terms, added in chains of at most n / 1024 + 8 terms and a tree
of 10 levels, is off by at most (n / 1024 + 20) u32 relative (all terms are
positive); its inverse root by half of that and two roundings, the products
by two more.  A tensor-core dot product of n terms is held to (n + 4) 2^-22
times the sum of the terms' magnitudes, as the linears are (helpers.py).  In
attention a score's error e (times scale) changes each probability by a factor
within exp(+-e), numerator and denominator alike; probabilities enter their
product with V rounded to bf16, which adds u16 times sum_j p_j |v_j|.
"""
from __future__ import annotations

import math

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8


def half_ulp_bf16(y: torch.Tensor) -> torch.Tensor:
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -126)))
    return torch.pow(2.0, e - 8)


def rms_norm(x, residual, gains, which, eps):
    """(h, y) in float64; gains [V + 1][d] with the base's first, which [T] rows of it."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / (h.pow(2).mean(1, keepdim=True) + eps).sqrt() * gains.double()[which]
    return h, y


def norm_rel(d: int) -> float:
    return (0.5 * (d / 1024 + 20) + 6) * U32


def turn(x, cos, sin, rot, interleaved):
    """x [T][heads][dim] turned by cos, sin [T][rot/2], in x's own dtype, operation by operation."""
    y = x.clone()
    half = rot // 2
    ia = [2 * i if interleaved else i for i in range(half)]
    ib = [2 * i + 1 if interleaved else i + half for i in range(half)]
    a, b, c, s = x[..., ia], x[..., ib], cos[:, None], sin[:, None]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def codes(x):
    """Int8 codes and scales of float32 vectors, operation by operation."""
    scale = x.abs().amax(-1).clamp_min(1e-30) / torch.tensor(127.0)
    return torch.round(x / scale[..., None]).clamp(-127, 127).to(torch.int8), scale


def attention(q, q_off, k, v, kv_len, scale, causal):
    """(out, lse, weight, score error, largest |v| sums) in float64.  k, v: lists of [len][n_kv][dim] per sequence."""
    T, n_q, dim = q.shape
    out = torch.zeros(T, n_q, dim, dtype=torch.float64)
    mag = torch.zeros(T, n_q, dim, dtype=torch.float64)
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64)
    err = torch.zeros(T, n_q, dtype=torch.float64)
    for s in range(len(kv_len)):
        n, length = q_off[s + 1] - q_off[s], kv_len[s]
        if n == 0 or length == 0:
            continue
        group = n_q // k[s].shape[1]
        for h in range(n_q):
            kk, vv = k[s][:, h // group].double(), v[s][:, h // group].double()
            qq = q[q_off[s]: q_off[s + 1], h].double()
            z = qq @ kk.T * scale
            zmag = qq.abs() @ kk.abs().T * abs(scale)
            if causal:
                i = torch.arange(n)[:, None]
                hide = torch.arange(length)[None, :] > length - n + i
                z = z.masked_fill(hide, -math.inf)
                zmag = zmag.masked_fill(hide, 0.0)
            norm = torch.logsumexp(z, 1)
            p = torch.where(z == -math.inf, torch.zeros_like(z), torch.exp(z - norm[:, None]))
            rows = slice(q_off[s], q_off[s + 1])
            out[rows, h], mag[rows, h], lse[rows, h] = p @ vv, p @ vv.abs(), norm
            err[rows, h] = zmag.amax(1) * (dim + 8) * 2.0 ** -22
    return out, lse, mag, err


def attention_bounds(ref, lse, mag, err, n_keys):
    """Elementwise bounds of the bf16 output and of the log-sum-exp."""
    sums = (n_keys + 64) * 2.0 ** -22
    rel = U16 + torch.expm1(2 * err)[..., None] + 2 * sums
    out = mag * rel
    out = out + half_ulp_bf16(ref.abs() + out)
    return out, err + sums + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -22 + 1e-6


def paged(n_new, kv_len, n_kv, dim, page, int8, seed, spare=3, rot_fill=True):
    """A cache of the sequences on pages in random order (CPU tensors): values past each length, spare pages and
    unused table entries hold NaN (int8: NaN scales) and -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_len]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g)
    width = max(need + [1]) + 1
    table = torch.full((len(kv_len), width), -1, dtype=torch.int32)
    c = {"n_new": n_new, "kv_len": kv_len, "table": table}
    shape = (n_pages, n_kv, page, dim)
    for name in "kv":
        if int8:
            c[name] = torch.full(shape, 77, dtype=torch.int8)
            c[name + "s"] = torch.full(shape[:3], math.nan)
        else:
            c[name] = torch.full(shape, math.nan, dtype=torch.bfloat16)
            c[name + "s"] = None
    used = 0
    c["vals"] = {"k": [], "v": []}
    for s, length in enumerate(kv_len):
        ids = perm[used: used + need[s]]
        used += need[s]
        table[s, : need[s]] = ids.to(torch.int32)
        at = torch.arange(length)
        pg, off = (ids[at // page], at % page) if length else (at, at)
        for name in "kv":
            val = torch.randn(length, n_kv, dim, generator=g)
            if int8:
                cd = torch.randint(-127, 128, (length, n_kv, dim), generator=g, dtype=torch.int8)
                sc = (0.5 + torch.rand(length, n_kv, generator=g)) * 0.02
                c[name][pg, :, off], c[name + "s"][pg, :, off] = cd, sc
                c["vals"][name].append(cd.double() * sc.double()[..., None])
            else:
                val = val.to(torch.bfloat16)
                c[name][pg, :, off] = val
                c["vals"][name].append(val.double())
    return c
