"""The operators between a layer's linears, as cases that can be timed and checked.

Four operators of the serving path around the BitDelta linears: the RMS norm
with the residual's addition, rotary positions with the write into the paged
KV cache, reading the cache back, and attention of new tokens over the paged
cache.  ``run`` makes one call of one of them on prepared inputs: with ``own``
false in plain torch operations in 32 bits, with ``own`` true through the
library's entry points.  Sizes follow the 70B-shaped decoder layer of the
slice workload (d = 8192, 14 variants, 32 decode tokens) and generic ones
around it.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5
THETA = 500000.0


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of the slice workload: 32 tokens of 14 variants, each with its own gain; latency
        {"name": "norm decode 14 variants", "op": "norm", "T": 32, "d": 8192, "V": 14, "out": "bf16"},
        # a prompt of 4096 tokens, output in 8 bits for products that take e4m3
        {"name": "norm prompt e4m3", "op": "norm", "T": 4096, "d": 8192, "V": 0, "out": "e4m3"},
        # one decode step: 32 sequences get one token each, 64 query and 8 kv heads
        {"name": "append decode bf16", "op": "append", "n_seq": 32, "new": 1, "ctx": 15, "n_kv": 8, "group": 8,
         "dim": 128, "kv": "bf16", "page": 16, "axes": 1, "rot": 128, "interleaved": False, "ragged": 1},
        # a prompt written in 8 bits and read back as the values it stands for (a prefix that is handed on)
        {"name": "append prompt int8 and read", "op": "append", "n_seq": 1, "new": 4096, "ctx": 0, "n_kv": 8,
         "group": 8, "dim": 128, "kv": "int8", "page": 64, "axes": 1, "rot": 128, "interleaved": False, "ragged": 0},
        # image and video tokens: positions in time, height and width, small heads, ragged batch
        {"name": "append three axes bf16", "op": "append", "n_seq": 5, "new": 1201, "ctx": 77, "n_kv": 16, "group": 1,
         "dim": 64, "kv": "bf16", "page": 32, "axes": 3, "rot": 48, "interleaved": True, "ragged": 3},
        # moving eight sequences off the device, 8-bit cache
        {"name": "read int8 batch", "op": "read", "n_seq": 8, "ctx": 8192, "n_kv": 8, "dim": 128, "kv": "int8",
         "page": 64, "ragged": 2},
        # two short sequences with small heads; latency
        {"name": "read bf16 short", "op": "read", "n_seq": 2, "ctx": 300, "n_kv": 4, "dim": 64, "kv": "bf16",
         "page": 16, "ragged": 4},
        # the smallest call: one sequence, one token, a short cache
        {"name": "attention one token", "op": "attention", "n_seq": 1, "new": 1, "ctx": 500, "n_kv": 8, "group": 8,
         "dim": 128, "kv": "bf16", "page": 16, "lse": False, "ragged": 0},
        # a decode step of a batch with caches of different lengths
        {"name": "attention decode batch", "op": "attention", "n_seq": 32, "new": 1, "ctx": 8192, "n_kv": 8,
         "group": 8, "dim": 128, "kv": "bf16", "page": 64, "lse": False, "ragged": 5},
        # few sequences with long 8-bit caches; the log-sum-exp is kept to join a shared prefix
        {"name": "attention long int8", "op": "attention", "n_seq": 4, "new": 1, "ctx": 65537, "n_kv": 8, "group": 8,
         "dim": 128, "kv": "int8", "page": 64, "lse": True, "ragged": 6},
        # a chunk of a long prompt over what is already in the cache
        {"name": "attention chunk bf16", "op": "attention", "n_seq": 1, "new": 4096, "ctx": 8192, "n_kv": 8,
         "group": 8, "dim": 128, "kv": "bf16", "page": 64, "lse": False, "ragged": 0},
        # chunks and single tokens of several sequences in one call, 8-bit cache
        {"name": "attention mixed chunks int8", "op": "attention", "n_seq": 8, "new": 700, "ctx": 8300, "n_kv": 8,
         "group": 4, "dim": 128, "kv": "int8", "page": 32, "lse": False, "ragged": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    d = 8 * _log(rng, 16, 2048)
    return d + 8 if d % 1024 == 0 else d


def draw(rng):
    op = rng.choice(["norm", "append", "read", "attention", "attention"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "d": rng.choice([8192, _width(rng)]), "V": rng.choice([0, 0, 1, 5, 14, 64]),
                "out": rng.choice(["bf16", "e4m3"])}
    c = {"op": op, "n_seq": _log(rng, 1, 64), "n_kv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
         "kv": rng.choice(["bf16", "int8"]), "page": rng.choice([16, 32, 64, 128]), "ragged": rng.randrange(1, 1 << 20)}
    if op == "read":
        c["ctx"] = _log(rng, 1, max(2, 262144 // c["n_seq"]))
        return c
    c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    if op == "append":
        c["new"] = rng.choice([1, _log(rng, 1, max(2, 8192 // c["n_seq"]))])
        c["ctx"] = rng.randrange(0, 200)
        c["axes"] = rng.choice([1, 2, 3])
        c["rot"] = rng.choice([c["dim"], c["dim"] // 2, 48])
        c["interleaved"] = rng.random() < 0.5
        return c
    c["new"] = rng.choice([1, 1, rng.randrange(2, 9), _log(rng, 9, 2048)])
    c["ctx"] = _log(rng, 1, 65536)
    while c["n_seq"] > 1 and c["n_seq"] * (c["ctx"] + c["new"]) * max(c["n_kv"] * c["group"] * c["new"] / 2000.0,
                                                                      c["n_kv"] / 8.0) > 400000:
        c["n_seq"] = (c["n_seq"] + 1) // 2
    while (c["ctx"] + c["new"]) * c["n_kv"] * c["group"] * c["new"] > 8e8:
        c["new"] = (c["new"] + 1) // 2
        c["ctx"] = (c["ctx"] + 1) // 2
    c["lse"] = rng.random() < 0.3
    return c


def _lengths(case):
    """(new tokens, tokens already in the cache) of each sequence: full length first, the others ragged."""
    n, new, ctx = case["n_seq"], case.get("new", 0), case["ctx"]
    if not case["ragged"]:
        return [new] * n, [ctx] * n
    r = random.Random(case["ragged"])
    news = [new] + [1 if r.random() < 0.25 else r.randint((new + 1) // 2, new) for _ in range(n - 1)] if new else [0] * n
    ctxs = [ctx] + [r.randint(ctx // 2, ctx) for _ in range(n - 1)]
    return news, ctxs


# ------------------------------------------------------------------------------- inputs

def _pages(case, news, ctxs, g, dev):
    """A paged cache that holds the sequences' tokens on pages in random order, with a few pages of others."""
    page, n_kv, dim = case["page"], case["n_kv"], case["dim"]
    need = [max(1, -(-(a + b) // page)) for a, b in zip(news, ctxs)]
    total = sum(need)
    n_pages = total + total // 8 + 3
    perm = torch.randperm(n_pages, generator=g, device=dev)[:total].to(torch.int32)
    off = torch.zeros(case["n_seq"] + 1, dtype=torch.int64)
    off[1:] = torch.tensor(need).cumsum(0)
    width = max(need)
    at = torch.arange(width)[None, :] + off[:-1, None]
    live = (torch.arange(width)[None, :] < torch.tensor(need)[:, None]).to(dev)
    table = torch.where(live, perm[at.clamp_max(total - 1).to(dev)], torch.zeros((), dtype=torch.int32, device=dev))
    shape = (n_pages, n_kv, page, dim)
    st = {"table": table.contiguous(), "max_kv": width * page}
    for name in ("k", "v"):
        if case["kv"] == "int8":
            codes = torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)
            amax = 2.5 + 1.5 * torch.rand(shape[:3], generator=g, device=dev)
            st[name + "_pages"], st[name + "_scale"] = codes, amax / 127
        else:
            st[name + "_pages"] = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
            st[name + "_scale"] = None
    return st


def _offsets(lens, dev):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    st = {"case": case}
    if case["op"] == "norm":
        T, d, V = case["T"], case["d"], case["V"]
        st["x"], st["residual"] = normal(T, d), normal(T, d) * 2
        gains = (1 + 0.1 * torch.randn(V + 1, d, generator=g, device=dev)).to(torch.bfloat16)
        st["gain"], st["gain_list"] = gains[0].clone(), [gains[v + 1].clone() for v in range(V)]
        st["vid"] = torch.randint(-1, V, (T,), generator=g, device=dev, dtype=torch.int32) if V else None
        e4m3 = case["out"] == "e4m3"
        st["out"] = torch.empty(T, d, device=dev, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        st["scale"] = torch.empty(T, device=dev) if e4m3 else None
        st["residual_out"] = torch.empty_like(st["x"])
        return st

    news, ctxs = _lengths(case)
    n_kv, dim, page = case["n_kv"], case["dim"], case["page"]
    st |= _pages(case, news, ctxs, g, dev)
    T, total = sum(news), sum(news) + sum(ctxs)
    st["kv_len"] = torch.tensor([a + b for a, b in zip(news, ctxs)], dtype=torch.int32).to(dev)
    st["kv_off"] = _offsets([a + b for a, b in zip(news, ctxs)], dev)
    if case["op"] != "attention" and (case["op"] == "read" or case["kv"] == "int8"):
        st["k_out"] = torch.empty(total, n_kv, dim, device=dev, dtype=torch.bfloat16)
        st["v_out"] = torch.empty_like(st["k_out"])
    if case["op"] == "read":
        return st

    n_q = n_kv * case["group"]
    st["q_off"] = _offsets(news, dev)
    st["out"] = torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16)
    if case["op"] == "attention":
        st["q"] = normal(T, n_q, dim)
        st["max_new"] = max(news)
        st["lse"] = torch.empty(T, n_q, device=dev) if case["lse"] else None
        return st

    # append: the packed output of one q/k/v product, as a caller with stacked weights has it
    qkv = normal(T, (n_q + 2 * n_kv) * dim)
    st["qkv"] = qkv
    st["q"] = qkv[:, : n_q * dim].view(T, n_q, dim)
    st["k"] = qkv[:, n_q * dim: (n_q + n_kv) * dim].view(T, n_kv, dim)
    st["v"] = qkv[:, (n_q + n_kv) * dim:].view(T, n_kv, dim)
    seq = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news)).to(dev)
    at = torch.arange(T, device=dev) - st["q_off"].long()[seq] + torch.tensor(ctxs, device=dev)[seq]
    st["slot"] = (st["table"][seq, at // page].long() * page + at % page).to(torch.int32)
    pairs = case["rot"] // 2
    n_pos = 8192
    if case["axes"] == 1:
        st["pos"] = (at % n_pos).to(torch.int32).view(T, 1)
    else:  # time, height, width (or height, width) of patches on a 32-wide grid
        parts = [at // 1024, at // 32 % 32, at % 32][3 - case["axes"]:]
        st["pos"] = torch.stack(parts, 1).to(torch.int32).contiguous()
    st["axis_of_pair"] = [i * case["axes"] // pairs for i in range(pairs)]
    st["axis"] = torch.tensor(st["axis_of_pair"], device=dev)
    freq = THETA ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
    angle = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * freq
    st["rope_table"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
    return st


# ------------------------------------------------------------------------------- the plain form

def _plain_norm(st):
    h = st["x"].float() + st["residual"].float()
    gain = st["gain"].float() if st["vid"] is None else torch.stack([st["gain"], *st["gain_list"]])[st["vid"].long() + 1].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * gain
    if st["scale"] is None:
        return {"out": y.to(torch.bfloat16), "residual": h.to(torch.bfloat16)}
    amax = y.abs().amax(-1, keepdim=True).clamp_min(1e-30)
    return {"out": (y * (448.0 / amax)).to(torch.float8_e4m3fn), "scale": (amax / 448.0)[:, 0],
            "residual": h.to(torch.bfloat16)}


def _plain_turn(x, cs, rot, interleaved):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_codes(x):
    scale = x.abs().amax(-1).clamp_min(1e-30) / 127.0
    return torch.round(x / scale[..., None]).clamp(-127, 127).to(torch.int8), scale


def _plain_append(st):
    case = st["case"]
    pairs = case["rot"] // 2
    cs = st["rope_table"][st["pos"].long()[:, st["axis"]], torch.arange(pairs, device=st["pos"].device)]
    q = _plain_turn(st["q"], cs, case["rot"], case["interleaved"]).to(torch.bfloat16)
    k = _plain_turn(st["k"], cs, case["rot"], case["interleaved"])
    v = st["v"].float()
    page, at = st["slot"].long() // case["page"], st["slot"].long() % case["page"]
    if case["kv"] == "bf16":
        st["k_pages"][page, :, at] = k.to(torch.bfloat16)
        st["v_pages"][page, :, at] = v.to(torch.bfloat16)
        return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    st["k_pages"][page, :, at], st["k_scale"][page, :, at] = _plain_codes(k)
    st["v_pages"][page, :, at], st["v_scale"][page, :, at] = _plain_codes(v)
    return {"q": q, **_plain_read(st)}


def _plain_read(st):
    n, page = st["k_out"].shape[0], st["case"]["page"]
    row = torch.arange(n, device=st["kv_off"].device, dtype=torch.int32)
    seq = torch.bucketize(row, st["kv_off"][1:], right=True)
    at = (row - st["kv_off"][seq]).long()
    pg, at = st["table"][seq, at // page].long(), at % page
    k, v = st["k_pages"][pg, :, at].float(), st["v_pages"][pg, :, at].float()
    if st["k_scale"] is not None:
        k, v = k * st["k_scale"][pg, :, at][..., None], v * st["v_scale"][pg, :, at][..., None]
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _plain_heads(pages, scale, table):
    """[n_seq, n_kv, keys, dim] in 32 bits out of the pages."""
    x = pages[table.long()].float()
    if scale is not None:
        x = x * scale[table.long()][..., None]
    n, p, h, t, d = x.shape
    return x.transpose(1, 2).reshape(n, h, p * t, d)


def _plain_attention(st):
    q, case = st["q"], st["case"]
    T, n_q, dim = q.shape
    n_kv, group, new, dev = case["n_kv"], case["group"], st["max_new"], st["q"].device
    k = _plain_heads(st["k_pages"], st["k_scale"], st["table"])
    v = _plain_heads(st["v_pages"], st["v_scale"], st["table"])
    n_seq, _, keys, _ = k.shape
    first, length = st["q_off"][:-1, None], st["kv_len"][:, None, None]
    n_new = (st["q_off"][1:, None] - first)[..., None]
    i = torch.arange(new, device=dev, dtype=torch.int32)[None, :, None]
    j = torch.arange(keys, device=dev, dtype=torch.int32)[None, None, :]
    seen = (j < length) & (j <= length - n_new + i)  # [n_seq, new, keys]
    qp = q[(first + i[..., 0]).clamp_max(T - 1).long()].float()  # [n_seq, new, n_q, dim]
    qp = qp.view(n_seq, new, n_kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n_seq, n_kv, new * group, dim)
    s = (torch.matmul(qp, k.transpose(-1, -2)) * (1 / math.sqrt(dim))).view(n_seq, n_kv, new, group, keys)
    s = s.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n_seq, n_kv, new * group, keys), v).view(n_seq, n_kv, new, group, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log())[..., 0]
    t = torch.arange(T, device=dev, dtype=torch.int32)
    seq = torch.bucketize(t, st["q_off"][1:], right=True)
    at = (t - st["q_off"][seq]).long()
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(n_seq, new, n_q, dim)[seq, at].to(torch.bfloat16)}
    if st["lse"] is not None:
        out["lse"] = lse.permute(0, 2, 1, 3).reshape(n_seq, new, n_q)[seq, at]
    return out


# ------------------------------------------------------------------------------- the library's calls

def _handles(st):
    """What a serving program keeps beside its inputs: the cache's handle and a workspace."""
    from bit_weight_delta_bd_gb300 import bitdelta as bd

    if "ws" not in st:
        need = 0
        if st["case"]["op"] == "attention":
            need = bd.bd_attention_workspace_size(st["q"].shape[0], st["case"]["n_seq"], st["q"].shape[1],
                                                  st["case"]["n_kv"], st["case"]["dim"])
        st["ws"] = bd.new_workspace(need, "cuda")
        if "k_pages" in st:
            st["cache"] = bd.KvPages(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
    return bd


def _own_norm(st):
    bd = _handles(st)
    bd.bd_rms_norm(st["x"], st["gain"], EPS, st["out"], st["ws"], residual=st["residual"],
                   residual_out=st["residual_out"], scale=st["scale"], vid=st["vid"], gain_list=st["gain_list"])
    got = {"out": st["out"], "residual": st["residual_out"]}
    return got if st["scale"] is None else {**got, "scale": st["scale"]}


def _own_append(st):
    bd, case = _handles(st), st["case"]
    bd.bd_rope_append(st["q"], st["k"], st["v"], st["pos"], st["rope_table"], st["slot"], st["cache"], st["out"],
                      st["ws"], axis_of_pair=st["axis_of_pair"], interleaved=case["interleaved"])
    if case["kv"] == "bf16":
        return {"q": st["out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    return {"q": st["out"], **_own_read(st)}


def _own_read(st):
    bd = _handles(st)
    bd.bd_kv_read(st["cache"], st["table"], st["kv_off"], st["k_out"], st["v_out"], st["ws"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_attention(st):
    bd = _handles(st)
    bd.bd_attention(st["q"], st["q_off"], st["cache"], st["table"], st["kv_len"], 1 / math.sqrt(st["case"]["dim"]),
                    st["max_new"], st["out"], st["ws"], lse=st["lse"])
    return {"out": st["out"]} if st["lse"] is None else {"out": st["out"], "lse": st["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "read": _own_read, "attention": _own_attention}[op](state)
    return {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attention": _plain_attention}[op](state)


# ------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        out = 1 if case["out"] == "e4m3" else 2
        return {"bytes": T * d * (6 + out) + 2 * d * (case["V"] + 1) + 4 * T, "flops": 7 * T * d}
    news, ctxs = _lengths(case)
    T, total = sum(news), sum(news) + sum(ctxs)
    n_kv, dim = case["n_kv"], case["dim"]
    n_q = n_kv * case.get("group", 0)
    token = 2 * n_kv * (2 * dim if case["kv"] == "bf16" else dim + 4)  # a token's K and V in the cache
    if case["op"] == "read":
        return {"bytes": total * (token + 4 * n_kv * dim), "flops": 2 * total * n_kv * dim}
    if case["op"] == "append":
        moved = T * (4 * n_q * dim + 4 * n_kv * dim + token + 4 * case["axes"] + 4 * case["rot"] + 4)
        if case["kv"] == "int8":
            moved += total * (token + 4 * n_kv * dim)
        return {"bytes": moved, "flops": 3 * T * (n_q + n_kv) * case["rot"]}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(news, ctxs))
    return {"bytes": total * token + 4 * T * n_q * dim + (4 * T * n_q if case["lse"] else 0),
            "flops": 4 * pairs * n_q * dim}


# ------------------------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(st):
    h = st["x"].double() + st["residual"].double()
    out, scales = torch.empty_like(h), torch.empty(h.shape[0], dtype=torch.float64, device=h.device)
    gains = torch.stack([st["gain"], *st["gain_list"]]).double()
    which = torch.zeros(h.shape[0], dtype=torch.long, device=h.device) if st["vid"] is None else st["vid"].long() + 1
    for v in range(gains.shape[0]):
        rows = which == v
        hv = h[rows]
        out[rows] = hv * gains[v] / (hv.pow(2).sum(1, keepdim=True) / hv.shape[1] + EPS).sqrt()
    if st["scale"] is None:
        return {"out": out, "residual": h}
    scales = out.abs().max(1).values / 448
    # the code is a rounding to 4 significant bits (3 below 2^-6): kept as a rounding of the exact quotient
    z = out / scales[:, None]
    e = torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    return {"out": (torch.round(z / step) * step).clamp(-448, 448), "scale": scales, "residual": h}


def _exact_turn(x, st):
    case = st["case"]
    pairs, y = case["rot"] // 2, x.double()
    out = y.clone()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
        w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                        st["pos"][:, st["axis_of_pair"][i]].double() * THETA ** (-i / pairs))
        z = torch.complex(y[..., a], y[..., b]) * w[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_read(st, k_new=None, v_new=None):
    """Values of every token; those of `slot` come from k_new, v_new, coded on 255 levels."""
    case, page = st["case"], st["case"]["page"]
    off, got = st["kv_off"].tolist(), {}
    for name, new in (("k", k_new), ("v", v_new)):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        flat = pages.double() if scale is None else pages.double() * scale.double()[..., None]
        flat = flat.permute(0, 2, 1, 3).reshape(-1, case["n_kv"], case["dim"])
        if new is not None:
            step = new.abs().max(-1, keepdim=True).values / 127
            flat[st["slot"].long()] = torch.round(new / step) * step
        rows = []
        for s in range(case["n_seq"]):
            at = torch.arange(off[s + 1] - off[s], device=pages.device)
            rows.append(flat[st["table"][s].long()[at // page] * page + at % page])
        got[name] = torch.cat(rows)
    return got


def _exact_append(st):
    case = st["case"]
    q, k, v = _exact_turn(st["q"], st), _exact_turn(st["k"], st), st["v"].double()
    if case["kv"] == "int8":
        return {"q": q, **_exact_read(st, k, v)}
    got = {"q": q}
    for name, new in (("k", k), ("v", v)):
        pages = st[name + "_pages"].double()
        flat = pages.permute(0, 2, 1, 3).reshape(-1, case["n_kv"], case["dim"])
        flat[st["slot"].long()] = new
        got[name + "_pages"] = flat.view(pages.shape[0], case["page"], case["n_kv"], case["dim"]).permute(0, 2, 1, 3).contiguous()
    return got


def _exact_attention(st):
    case = st["case"]
    T, n_q, dim = st["q"].shape
    group = case["group"]
    out = torch.zeros(T, n_q, dim, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(T, n_q, dtype=torch.float64, device=st["q"].device)
    off, lens = st["q_off"].tolist(), st["kv_len"].tolist()
    for s in range(case["n_seq"]):
        n, length = off[s + 1] - off[s], lens[s]
        pages = st["table"][s, : -(-length // case["page"])].long()
        last = torch.arange(length - n, length, device=out.device)[:, None]  # the last key that each new token sees
        hidden = torch.arange(length, device=out.device)[None, :] > last
        for h in range(case["n_kv"]):
            k, v = (st[x + "_pages"][pages, h].double() for x in "kv")
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"][pages, h].double()[..., None], v * st["v_scale"][pages, h].double()[..., None]
            k, v = k.reshape(-1, dim)[:length], v.reshape(-1, dim)[:length]
            for j in range(h * group, (h + 1) * group):
                z = st["q"][off[s]: off[s + 1], j].double() @ k.T / dim ** 0.5
                z.masked_fill_(hidden, -math.inf)
                norm = torch.logsumexp(z, 1)
                out[off[s]: off[s + 1], j] = torch.exp(z - norm[:, None]) @ v
                lse[off[s]: off[s + 1], j] = norm
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_read(st) if case["op"] == "read" else _exact_attention(st)
