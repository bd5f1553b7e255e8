"""A decoder layer's attention half over a KV cache in 4 bits, as cases that can be timed and checked.

Four operators of the serving path around the BitDelta linears: rotary
positions with the write into a paged cache of 4-bit codes, that cache read
back, attention of new tokens over it, and the norms after a block and before
the next one with the block's gate, its scale and the residual's.  ``run``
makes one call of one of them on prepared inputs: with ``own`` false in plain
torch operations in 32 bits, with ``own`` true through the library's entry
points.  Sizes follow the 70B-shaped decoder layer of the slice workload (d =
8192, 14 variants, 32 decode tokens) and generic ones around it.

The 4-bit cache.  32 neighbouring elements of a head make a group with a scale
and a lowest value, both bf16; an element is code * scale + low, code 0 .. 15:
    low = bf16(min x),  scale = bf16(max(max x - min x, 1e-30) / 15),
    code = round-half-even((x - low) / scale), kept within 0 .. 15.
Element 8 w + 2 i of a head lies in bits 4 i of its 32-bit word w, element
8 w + 2 i + 1 in bits 16 + 4 i.
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
        # one decode step of the slice workload: 32 tokens of 14 variants, each with its own gains of both norms; latency
        {"name": "norms decode 14 variants", "op": "norms", "T": 32, "d": 8192, "V": 14, "post": True, "gate": "row",
         "out": "bf16"},
        # a prompt of 4096 tokens; a gate for each token, output in 8 bits for products that take e4m3
        {"name": "norms prompt gated e4m3", "op": "norms", "T": 4096, "d": 8192, "V": 0, "post": True, "gate": "token",
         "out": "e4m3"},
        # many short rows of an odd width, of sequences with gates of their own
        {"name": "norms short rows", "op": "norms", "T": 20011, "d": 1000, "V": 5, "post": True, "gate": "pick",
         "out": "bf16"},
        # one decode step: 32 sequences get one token each, 64 query and 8 kv heads; read back for the comparison
        {"name": "append decode", "op": "append", "n_seq": 32, "new": 1, "ctx": 15, "n_kv": 8, "group": 8,
         "dim": 128, "page": 16, "axes": 1, "rot": 128, "interleaved": False, "ragged": 1},
        # a prompt written in 4 bits and read back as the values it stands for (a prefix that is handed on)
        {"name": "append prompt and read", "op": "append", "n_seq": 1, "new": 4096, "ctx": 0, "n_kv": 8,
         "group": 8, "dim": 128, "page": 64, "axes": 1, "rot": 128, "interleaved": False, "ragged": 0},
        # moving eight sequences off the device
        {"name": "read batch", "op": "read", "n_seq": 8, "ctx": 8192, "n_kv": 8, "dim": 128, "page": 64, "ragged": 2},
        # two short sequences with small heads; latency
        {"name": "read short", "op": "read", "n_seq": 2, "ctx": 300, "n_kv": 4, "dim": 64, "page": 16, "ragged": 4},
        # the smallest attention: one sequence, one token, a short cache
        {"name": "attention one token", "op": "attention", "n_seq": 1, "new": 1, "ctx": 500, "n_kv": 8, "group": 8,
         "dim": 128, "page": 16, "lse": False, "ragged": 0},
        # a decode step of a batch with caches of different lengths
        {"name": "attention decode batch", "op": "attention", "n_seq": 32, "new": 1, "ctx": 8192, "n_kv": 8,
         "group": 8, "dim": 128, "page": 64, "lse": False, "ragged": 5},
        # few sequences with long caches; the log-sum-exp is kept to join a shared prefix
        {"name": "attention long", "op": "attention", "n_seq": 4, "new": 1, "ctx": 65537, "n_kv": 8, "group": 8,
         "dim": 128, "page": 64, "lse": True, "ragged": 6},
        # a chunk of a long prompt over what is already in the cache
        {"name": "attention chunk", "op": "attention", "n_seq": 1, "new": 4096, "ctx": 8192, "n_kv": 8,
         "group": 8, "dim": 128, "page": 64, "lse": False, "ragged": 0},
        # chunks and single tokens of several sequences in one call, small heads
        {"name": "attention mixed chunks", "op": "attention", "n_seq": 8, "new": 700, "ctx": 8300, "n_kv": 8,
         "group": 4, "dim": 64, "page": 32, "lse": True, "ragged": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norms", "append", "read", "attention", "attention"])
    if op == "norms":
        return {"op": op, "T": _log(rng, 1, 8192), "d": rng.choice([8192, 8 * _log(rng, 16, 2048)]),
                "V": rng.choice([0, 0, 1, 5, 14, 64]), "post": rng.random() < 0.8,
                "gate": rng.choice(["none", "row", "token", "pick"]), "out": rng.choice(["bf16", "f32", "e4m3"])}
    c = {"op": op, "n_seq": _log(rng, 1, 64), "n_kv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
         "page": rng.choice([16, 32, 64, 128]), "ragged": rng.randrange(1, 1 << 20)}
    if op == "read":
        c["ctx"] = _log(rng, 1, max(2, 262144 // c["n_seq"]))
        return c
    c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    if op == "append":
        c["new"] = rng.choice([1, _log(rng, 1, max(2, 8192 // c["n_seq"]))])
        c["ctx"] = rng.randrange(0, 200)
        c["axes"] = rng.choice([1, 2, 3])
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 48])
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


# ------------------------------------------------------------------------------- the 4-bit form

def _quantise(x):
    """(codes [..., dim / 2] uint8, scale and low [..., dim / 32, 2] bf16) of fp32 heads."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.amin(-1), g.amax(-1)
    # (a tensor of 15s: by a plain number torch multiplies with its reciprocal, which is another rounding)
    pair = torch.stack([(hi - lo).clamp_min(1e-30) / torch.full_like(lo, 15.0), lo], -1).to(torch.bfloat16)
    scale, low = pair[..., 0].float()[..., None], pair[..., 1].float()[..., None]
    code = torch.round((g - low) / scale).clamp_(0, 15).to(torch.int32)
    w = code.reshape(*x.shape[:-1], -1, 4, 2)
    # a byte holds elements 8 w + 4 b + {0, 2} (b = 0, 1), then 8 w + 4 b + {1, 3}
    even, odd = w[..., 0], w[..., 1]
    halves = [h[..., 0::2] + 16 * h[..., 1::2] for h in (even, odd)]
    return torch.cat(halves, -1).to(torch.uint8).flatten(-2), pair


def _values(codes, pair):
    """fp32 heads out of codes [..., dim / 2] and scale and low."""
    b = codes.reshape(*codes.shape[:-1], -1, 2, 2)  # [word][odd][byte]
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).transpose(-1, -2)  # [word][i][odd]
    c = c.reshape(*codes.shape[:-1], -1, 32).float()
    v = c * pair[..., 0].float()[..., None] + pair[..., 1].float()[..., None]
    return v.flatten(-2)


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
    st = {"table": table.contiguous()}
    shape = (n_pages, n_kv, page)
    per = max(1, (1 << 25) // (n_kv * page * dim))  # pages at a time
    for name in ("k", "v"):
        codes = torch.empty(*shape, dim // 2, device=dev, dtype=torch.uint8)
        pair = torch.empty(*shape, dim // 32, 2, device=dev, dtype=torch.bfloat16)
        # keys have channels that lie far from zero in every token
        mean = torch.randn(n_kv, 1, dim, generator=g, device=dev).pow(3) * (0.5 if name == "k" else 0.0)
        for p in range(0, n_pages, per):
            n = min(per, n_pages - p)
            x = torch.randn(n, *shape[1:], dim, generator=g, device=dev)
            codes[p: p + n], pair[p: p + n] = _quantise(x + mean)
        st[name + "_pages"], st[name + "_scale"] = codes, pair
    return st


def _offsets(lens, dev):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(dev)


def _prepare_norms(case, g, dev):
    T, d, V = case["T"], case["d"], case["V"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    st = {"case": case, "x": normal(T, d), "residual": normal(T, d) * 2}
    for name in ("gain", "post_gain"):
        gains = (1 + 0.1 * torch.randn(V + 1, d, generator=g, device=dev)).to(torch.bfloat16)
        if name == "gain" or case["post"]:
            st[name], st[name + "_list"] = gains[0].clone(), [gains[v + 1].clone() for v in range(V)]
        else:
            st[name], st[name + "_list"] = None, []
    st["vid"] = torch.randint(-1, V, (T,), generator=g, device=dev, dtype=torch.int32) if V else None
    # a learned scale of each channel; a gate of each token; or gates of sequences, which their tokens pick
    rows = {"none": 0, "row": 1, "token": T, "pick": 1 + T // 64}[case["gate"]]
    gate = torch.sigmoid(torch.randn(rows, d, generator=g, device=dev)).to(torch.bfloat16)
    st["gate"] = gate if rows else None
    pick = case["gate"] == "pick"
    st["gate_idx"] = torch.sort(torch.randint(0, rows, (T,), generator=g, device=dev, dtype=torch.int32))[0] if pick else None
    st["block_scale"], st["residual_scale"] = 0.7071, 0.95
    dt = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[case["out"]]
    st["out"] = torch.empty(T, d, device=dev, dtype=dt)
    st["scale"] = torch.empty(T, device=dev) if case["out"] == "e4m3" else None
    st["residual_out"] = torch.empty_like(st["x"])
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    if case["op"] == "norms":
        return _prepare_norms(case, g, dev)

    st = {"case": case}
    news, ctxs = _lengths(case)
    n_kv, dim, page = case["n_kv"], case["dim"], case["page"]
    st |= _pages(case, news, ctxs, g, dev)
    T, total = sum(news), sum(news) + sum(ctxs)
    st["kv_len"] = torch.tensor([a + b for a, b in zip(news, ctxs)], dtype=torch.int32).to(dev)
    st["kv_off"] = _offsets([a + b for a, b in zip(news, ctxs)], dev)
    if case["op"] != "attention":
        st["k_out"] = torch.empty(total, n_kv, dim, device=dev, dtype=torch.bfloat16)
        st["v_out"] = torch.empty_like(st["k_out"])
    if case["op"] == "read":
        return st

    n_q = n_kv * case["group"]
    st["q_off"] = _offsets(news, dev)
    st["out"] = torch.empty(T, n_q, dim, device=dev, dtype=torch.bfloat16)
    if case["op"] == "attention":
        st["q"] = torch.randn(T, n_q, dim, generator=g, device=dev, dtype=torch.bfloat16)
        st["max_new"] = max(news)
        st["lse"] = torch.empty(T, n_q, device=dev) if case["lse"] else None
        return st

    # append: the packed output of one q/k/v product, as a caller with stacked weights has it
    qkv = torch.randn(T, (n_q + 2 * n_kv) * dim, generator=g, device=dev, dtype=torch.bfloat16)
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

def _rstd(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_norms(st):
    which = None if st["vid"] is None else st["vid"].long() + 1

    def gain_of(name):
        return st[name].float() if which is None else torch.stack([st[name], *st[name + "_list"]])[which].float()

    n = st["x"].float()
    if st["post_gain"] is not None:
        n = n * _rstd(n) * gain_of("post_gain")
    if st["gate"] is not None:
        n = n * (st["gate"] if st["gate_idx"] is None else st["gate"][st["gate_idx"].long()]).float()
    h = st["residual_scale"] * st["residual"].float() + st["block_scale"] * n
    y = h * _rstd(h) * gain_of("gain")
    if st["scale"] is None:
        return {"out": y.to(st["out"].dtype), "residual": h.to(torch.bfloat16)}
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


def _plain_append(st):
    case = st["case"]
    pairs = case["rot"] // 2
    cs = st["rope_table"][st["pos"].long()[:, st["axis"]], torch.arange(pairs, device=st["pos"].device)]
    q = _plain_turn(st["q"], cs, case["rot"], case["interleaved"]).to(torch.bfloat16)
    k = _plain_turn(st["k"], cs, case["rot"], case["interleaved"])
    page, at = st["slot"].long() // case["page"], st["slot"].long() % case["page"]
    st["k_pages"][page, :, at], st["k_scale"][page, :, at] = _quantise(k)
    st["v_pages"][page, :, at], st["v_scale"][page, :, at] = _quantise(st["v"].float())
    return {"q": q, **_plain_read(st)}


def _plain_read(st):
    n, page = st["k_out"].shape[0], st["case"]["page"]
    row = torch.arange(n, device=st["kv_off"].device, dtype=torch.int32)
    seq = torch.bucketize(row, st["kv_off"][1:], right=True)
    at = (row - st["kv_off"][seq]).long()
    pg, at = st["table"][seq, at // page].long(), at % page
    return {x: _values(st[x + "_pages"][pg, :, at], st[x + "_scale"][pg, :, at]).to(torch.bfloat16) for x in "kv"}


def _plain_heads(pages, pair, table):
    """[n_seq, n_kv, keys, dim] in 32 bits out of the pages."""
    x = _values(pages[table.long()], pair[table.long()])
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


def _own_norms(st):
    bd = _handles(st)
    bd.bd_block_norm(st["x"], st["residual"], st["gain"], EPS, st["out"], st["ws"], residual_out=st["residual_out"],
                     post_gain=st["post_gain"], gate=st["gate"], gate_idx=st["gate_idx"],
                     block_scale=st["block_scale"], residual_scale=st["residual_scale"], scale=st["scale"],
                     vid=st["vid"], gain_list=st["gain_list"], post_gain_list=st["post_gain_list"])
    got = {"out": st["out"], "residual": st["residual_out"]}
    return got if st["scale"] is None else {**got, "scale": st["scale"]}


def _own_append(st):
    bd, case = _handles(st), st["case"]
    bd.bd_rope_append(st["q"], st["k"], st["v"], st["pos"], st["rope_table"], st["slot"], st["cache"], st["out"],
                      st["ws"], axis_of_pair=st["axis_of_pair"], interleaved=case["interleaved"])
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
        return {"norms": _own_norms, "append": _own_append, "read": _own_read, "attention": _own_attention}[op](state)
    return {"norms": _plain_norms, "append": _plain_append, "read": _plain_read, "attention": _plain_attention}[op](state)


# ------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norms":
        T, d = case["T"], case["d"]
        out = {"bf16": 2, "f32": 4, "e4m3": 1}[case["out"]]
        gains = (case["V"] + 1) * (2 if case["post"] else 1)
        gates = {"none": 0, "row": 1, "token": T, "pick": 1 + T // 64}[case["gate"]]
        return {"bytes": T * d * (6 + out) + 2 * d * (gains + gates) + 8 * T, "flops": 14 * T * d}
    news, ctxs = _lengths(case)
    T, total = sum(news), sum(news) + sum(ctxs)
    n_kv, dim = case["n_kv"], case["dim"]
    n_q = n_kv * case.get("group", 0)
    token = 2 * n_kv * (dim // 2 + dim // 8)  # a token's K and V in the cache
    if case["op"] == "read":
        return {"bytes": total * (token + 4 * n_kv * dim), "flops": 4 * total * n_kv * dim}
    if case["op"] == "append":
        moved = T * (4 * n_q * dim + 4 * n_kv * dim + token + 4 * case["axes"] + 4 * case["rot"] + 4)
        moved += total * (token + 4 * n_kv * dim)
        return {"bytes": moved, "flops": 3 * T * (n_q + n_kv) * case["rot"] + 8 * (T + total) * n_kv * dim}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(news, ctxs))
    return {"bytes": total * token + 4 * T * n_q * dim + (4 * T * n_q if case["lse"] else 0),
            "flops": 4 * pairs * n_q * dim}


# ------------------------------------------------------------------------------- the definitions in 64 bits

def _exact_norms(st):
    T, d = st["x"].shape
    which = torch.zeros(T, dtype=torch.long, device=st["x"].device) if st["vid"] is None else st["vid"].long() + 1

    def normed(z, base, others):
        out = torch.empty_like(z)
        for v, w in enumerate([base, *others]):
            rows = which == v
            zv = z[rows]
            out[rows] = zv / (zv.pow(2).sum(1, keepdim=True) / d + EPS).sqrt() * w.double()
        return out

    n = st["x"].double()
    if st["post_gain"] is not None:
        n = normed(n, st["post_gain"], st["post_gain_list"])
    if st["gate"] is not None:
        g = st["gate"].double()
        n = g[st["gate_idx"].long()] * n if st["gate_idx"] is not None else g * n
    h = n * st["block_scale"] + st["residual"].double() * st["residual_scale"]
    out = normed(h, st["gain"], st["gain_list"])
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


def _eight_bits(x):
    """Rounded to 8 significant bits, as bf16 is."""
    m, _ = torch.frexp(x)  # 0.5 <= |m| < 1
    unit = torch.where(m == 0, torch.ones_like(x), x / m)  # a power of two
    return torch.round(m * 256) / 256 * unit


def _exact_on_levels(x):
    """What is left of x once each group of 32 lies on its 16 levels."""
    out = torch.empty_like(x)
    for d in range(0, x.shape[-1], 32):
        g = x[..., d: d + 32]
        low = g.min(-1, keepdim=True).values
        step = _eight_bits((g.max(-1, keepdim=True).values - low) / torch.full_like(low, 15))
        low = _eight_bits(low)
        out[..., d: d + 32] = low + step * torch.round((g - low) / step).clamp(0, 15)
    return out


def _exact_pages(st, name):
    """[n_pages][n_kv][page][dim]: element by element out of the words."""
    words = st[name + "_pages"].contiguous().view(torch.int32)
    pair = st[name + "_scale"].double()
    dim = 8 * words.shape[-1]
    out = torch.empty(*words.shape[:-1], dim, dtype=torch.float64, device=words.device)
    for e in range(8):
        shift = 16 * (e % 2) + 4 * (e // 2)
        out[..., e::8] = torch.bitwise_and(torch.bitwise_right_shift(words, shift), 15).double()
    for d in range(0, dim, 32):
        out[..., d: d + 32] *= pair[..., d // 32, 0:1]
        out[..., d: d + 32] += pair[..., d // 32, 1:2]
    return out


def _exact_read(st, k_new=None, v_new=None):
    case, page = st["case"], st["case"]["page"]
    off, got = st["kv_off"].tolist(), {}
    for name, new in (("k", k_new), ("v", v_new)):
        flat = _exact_pages(st, name).permute(0, 2, 1, 3).reshape(-1, case["n_kv"], case["dim"])
        if new is not None:
            flat[st["slot"].long()] = _exact_on_levels(new)
        rows = []
        for s in range(case["n_seq"]):
            at = torch.arange(off[s + 1] - off[s], device=flat.device)
            rows.append(flat[st["table"][s].long()[at // page] * page + at % page])
        got[name] = torch.cat(rows)
    return got


def _exact_append(st):
    q, k = _exact_turn(st["q"], st), _exact_turn(st["k"], st)
    return {"q": q, **_exact_read(st, k, st["v"].double())}


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
            part = {x + y: st[x + y][pages, h] for x in "kv" for y in ("_pages", "_scale")}
            k, v = (_exact_pages(part, x).reshape(-1, dim)[:length] for x in "kv")
            for j in range(h * group, (h + 1) * group):
                z = st["q"][off[s]: off[s + 1], j].double() @ k.T / dim ** 0.5
                z.masked_fill_(hidden, -math.inf)
                norm = torch.logsumexp(z, 1)
                out[off[s]: off[s + 1], j] = torch.exp(z - norm[:, None]) @ v
                lse[off[s]: off[s + 1], j] = norm
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norms":
        return _exact_norms(st)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_read(st) if case["op"] == "read" else _exact_attention(st)
