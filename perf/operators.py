"""Cases of the operators between a decoder block's q/k/v linear and its o linear:

  rotate  per-head RMSNorm of q and k with the position rotation, in one pass
  append  the same pass writing K and V to a quantized paged cache (or the write alone), and the
          written tokens read back
  read    a quantized paged cache read back as 16-bit rows (prefix reuse, chunked prefill)
  tree    attention of one token, a chain or a tree of drafted tokens over that cache

`run` computes them with elementary torch operations, or (own = True) with the library's entry points.
A cache holds int8 codes, E4M3 codes or packed 4-bit codes (element 2i in the low nibble), pages of
[heads][tokens][head size], and one scale per token and head (U4: fp16 scale and zero-point).
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
_FLOOR = 2.0 ** -64  # the smallest scale of an int8 or E4M3 row


def listed():
    return [
        # one decode step's token far into a long conversation: only latency counts
        {"name": "rotate one token", "op": "rotate", "dtype": "bf16", "tokens": 1, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "norm": True, "inter": False, "far": 131071},
        # a prefill chunk, q and k as views of the fused q/k/v rows
        {"name": "rotate prefill", "op": "rotate", "dtype": "bf16", "tokens": 8192, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "norm": True, "inter": False, "far": 8192},
        # a decode step of 64 sequences: one token each joins its sequence's cache
        {"name": "append decode step", "op": "append", "fmt": "e4m3", "dtype": "bf16", "seqs": 64, "new": 1,
         "ctx": 4096, "spread": 1, "hq": 32, "hk": 8, "d": 128, "rot": 128, "norm": True, "inter": False, "page": 64},
        # ragged prefill chunks of a 4096-wide model whose keys and values have all 32 heads
        {"name": "append ragged chunks", "op": "append", "fmt": "int8", "dtype": "fp16", "seqs": 5, "new": 1367,
         "ctx": 1000, "spread": 2, "hq": 32, "hk": 32, "d": 128, "rot": 64, "norm": False, "inter": True, "page": 16},
        # keys and values that are ready (rotated before) into 4 bits, heads of 64
        {"name": "write four bits", "op": "append", "fmt": "u4", "dtype": "bf16", "seqs": 2, "new": 1025,
         "ctx": 33, "spread": 3, "hq": 0, "hk": 8, "d": 64, "rot": 0, "norm": False, "inter": False, "page": 32},
        # one short cached prompt taken up again
        {"name": "read one prefix", "op": "read", "fmt": "int8", "dtype": "fp16", "seqs": 1, "ctx": 777, "spread": 0,
         "hk": 32, "d": 128, "page": 16},
        # long prefixes of a batch for a prefill that needs 16-bit rows
        {"name": "read long prefixes", "op": "read", "fmt": "e4m3", "dtype": "bf16", "seqs": 8, "ctx": 32768,
         "spread": 4, "hk": 8, "d": 128, "page": 64},
        # one token over a short context, all heads their own: latency
        {"name": "decode short", "op": "tree", "fmt": "int8", "dtype": "fp16", "seqs": 1, "nodes": 1, "ctx": 500,
         "spread": 0, "hq": 32, "hk": 32, "d": 128, "page": 16, "tree": False},
        # a serving step: 64 sequences of very different lengths, one token each
        {"name": "decode ragged batch", "op": "tree", "fmt": "e4m3", "dtype": "bf16", "seqs": 64, "nodes": 1,
         "ctx": 8191, "spread": 5, "hq": 32, "hk": 8, "d": 128, "page": 64, "tree": False},
        # one user, a tree of 26 drafted tokens over a very long context in 4 bits
        {"name": "tree long context", "op": "tree", "fmt": "u4", "dtype": "bf16", "seqs": 1, "nodes": 26,
         "ctx": 131001, "spread": 0, "hq": 32, "hk": 8, "d": 128, "page": 64, "tree": True},
        # wide trees: so many rows for each cached token that the products bound it
        {"name": "tree wide", "op": "tree", "fmt": "int8", "dtype": "fp16", "seqs": 16, "nodes": 64, "ctx": 8192,
         "spread": 6, "hq": 64, "hk": 8, "d": 128, "page": 32, "tree": True},
        # a large batch of ordinary trees over long contexts
        {"name": "tree large batch", "op": "tree", "fmt": "e4m3", "dtype": "bf16", "seqs": 32, "nodes": 16,
         "ctx": 32768, "spread": 7, "hq": 32, "hk": 8, "d": 128, "page": 64, "tree": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "tree", "tree"])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    hk = rng.choice([1, 2, 4, 8, 8, 32])
    hq = hk * rng.choice([g for g in (1, 2, 4, 5, 8) if g * hk <= 64])
    d = rng.choice([64, 128, 128, 128, 256])
    if (hq + 2 * hk) * d == 3072 or (hq + hk) * d == 3072 or hq * d == 3072:
        hq, hk, d = 20, 4, 128
    rot = rng.choice([d, d, d // 2])
    inter, norm = rng.random() < 0.3, rng.random() < 0.6
    if op != "rotate":
        case["fmt"] = rng.choice(["int8", "e4m3", "u4"])
        case["page"] = rng.choice([16, 32, 64, 128])
        case["spread"] = rng.randrange(8, 1 << 20)
    case |= {"hk": hk, "d": d}
    if op == "rotate":
        case |= {"tokens": _log(rng, 1, 8192 * 40 * 128 // ((hq + hk) * d)), "hq": hq, "rot": rot, "norm": norm,
                 "inter": inter, "far": _log(rng, 1, 1 << 20)}
    elif op == "append":
        if case["fmt"] == "u4" or rng.random() < 0.2:  # the write alone
            hq, rot, norm, inter = 0, 0, False, False
        seqs = _log(rng, 1, 64)
        case |= {"seqs": seqs, "new": _log(rng, 1, max(1, (1 << 23) // ((hq + 2 * hk) * d * seqs))),
                 "ctx": _log(rng, 1, 4096), "hq": hq, "rot": rot, "norm": norm, "inter": inter}
    elif op == "read":
        seqs = _log(rng, 1, 16)
        case |= {"seqs": seqs, "ctx": _log(rng, 1, max(1, (1 << 27) // (hk * d * seqs)))}
    else:
        nodes = rng.choice([1, _log(rng, 1, 64)])
        case |= {"hq": hq, "seqs": _log(rng, 1, 64), "nodes": nodes, "ctx": _log(rng, 1, 131072),
                 "tree": nodes > 1 and rng.random() < 0.8}
        most = work(listed()[-1])
        while work(case)["bytes"] > most["bytes"] or work(case)["flops"] > most["flops"]:
            case["ctx"] = case["ctx"] * 2 // 3
            case["seqs"] = max(1, case["seqs"] * 4 // 5)
    for key in ("tokens", "new", "ctx"):
        if case.get(key) == 3072:
            case[key] += 1
    return case


# ---- the lengths of a case's sequences: from the case alone ------------------------------------------------------


def _lens(case):
    """(new tokens or nodes, cached tokens before them) of each sequence; with a spread they differ."""
    r = random.Random(case.get("spread", 0) * 7919 + 13)
    most = case.get("nodes", case.get("new", 0))
    new, ctx = [], []
    for b in range(case["seqs"]):
        spread = case.get("spread", 0) and b
        new.append(r.randint(max(1, most // 2), most) if spread and most else most)
        ctx.append(r.randint(case["ctx"] // 16, case["ctx"]) if spread else case["ctx"])
    return new, ctx


def _row_bytes(fmt, d):
    return (d // 2 if fmt == "u4" else d) + 4


def work(case):
    op, d, hk = case["op"], case["d"], case["hk"]
    if op == "rotate":
        n = case["tokens"] * (case["hq"] + hk) * d
        return {"bytes": 4 * n + 8 * case["tokens"], "flops": 10 * n}
    new, ctx = _lens(case)
    rb = _row_bytes(case["fmt"], d)
    if op == "append":  # q, k, v in; q, codes and the values of the codes out
        t = sum(new)
        return {"bytes": t * (4 * case["hq"] * d + 2 * hk * (4 * d + rb) + 16), "flops": 12 * t * (case["hq"] + 2 * hk) * d}
    if op == "read":
        t = sum(ctx)
        return {"bytes": 2 * t * hk * (rb + 2 * d), "flops": 2 * t * hk * d}
    tokens, pairs = sum(new) + sum(ctx), sum(n * (n + c) for n, c in zip(new, ctx))
    return {"bytes": 2 * tokens * hk * rb + sum(new) * case["hq"] * (4 * d + 4), "flops": 4 * case["hq"] * d * pairs}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _heads(g, n, h, d, dtype):
    """Rows as a projection gives them: channels of different sizes, a few large ones."""
    size = torch.exp(0.4 * torch.randn(h, d, generator=g, device="cuda"))
    size[:, torch.randperm(d, generator=g, device="cuda")[: max(1, d // 64)]] *= 4
    return (torch.randn(n, h, d, generator=g, device="cuda") * size).to(dtype)


def _rotation(case, g, pos):
    d, dt = case["d"], _DT[case["dtype"]]
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    s = {"pos": pos, "freq": 500000.0 ** (-2.0 * i / max(1, case["rot"])), "eps": 1e-6, "inter": case["inter"],
         "gq": None, "gk": None}
    if case["norm"]:
        s["gq"], s["gk"] = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2))
    return s


def _cache(case, g, total):
    """A cache whose pages lie in no order: [pages][heads][page][bytes] twice, scales, and each sequence's pages.
    Places that no sequence has reached hold what an earlier one left: any codes, and scales that are not numbers."""
    fmt, page, hk, d = case["fmt"], case["page"], case["hk"], case["d"]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(total), max(need) + 1), pages - 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    width = d // 2 if fmt == "u4" else d
    kind = torch.int8 if fmt == "int8" else torch.uint8
    s = {"fmt": fmt, "page": page, "table": table}
    for w in ("k", "v"):
        s[w + "c"] = torch.randint(0, 126, (pages, hk, page, width), generator=g, device="cuda", dtype=torch.int32).to(kind)
        s[w + "s"] = torch.full((pages, hk, page, 2), math.nan, dtype=torch.float16, device="cuda") if fmt == "u4" else \
            torch.full((pages, hk, page), math.nan, device="cuda")
    return s


def _fill(case, g, s, total):
    """Every place that a sequence has reached gets the codes of some row."""
    page, hk, d = case["page"], case["hk"], case["d"]
    left = torch.full((s["kc"].shape[0],), 0, dtype=torch.int64, device="cuda")  # tokens of each page in use
    for b, t in enumerate(total):
        n = -(-t // page)
        used = torch.full((n,), page, dtype=torch.int64, device="cuda")
        if n:
            used[-1] = t - (n - 1) * page
        left[s["table"][b, :n].long()] = used
    inside = torch.arange(page, device="cuda")[None, None, :] < left[:, None, None]
    step = max(1, (1 << 27) // (hk * page * d))
    for w in ("k", "v"):
        size = torch.exp(0.4 * torch.randn(hk, 1, d, generator=g, device="cuda"))
        if w == "k":
            size[:, :, :: max(1, d // 3)] *= 4
        for a in range(0, s["kc"].shape[0], step):
            m = min(step, s["kc"].shape[0] - a)
            x = torch.randn(m, hk, page, d, generator=g, device="cuda") * size
            x *= torch.exp(0.3 * torch.randn(m, hk, page, 1, generator=g, device="cuda"))
            codes, scale = _quantize(x.to(_DT[case["dtype"]]).float(), case["fmt"])
            here = inside[a: a + m].expand(m, hk, page)
            s[w + "c"][a: a + m] = torch.where(here[..., None], codes, s[w + "c"][a: a + m])
            s[w + "s"][a: a + m] = torch.where(here if scale.dim() == 3 else here[..., None], scale, s[w + "s"][a: a + m])


def _ints(v, dtype):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _starts(v):
    return _ints([0] + list(np.cumsum(v)), torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, d, hk, dt = case["op"], case["d"], case["hk"], _DT[case["dtype"]]
    s = {"op": op, "dtype": dt, "kept": {}}
    if op == "rotate":
        t, hq = case["tokens"], case["hq"]
        qkv = _heads(g, t, hq + 2 * hk, d, dt)
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq: hq + hk], "q_out": torch.empty(t, hq, d, dtype=dt, device="cuda"),
              "k_out": torch.empty(t, hk, d, dtype=dt, device="cuda")}
        first = torch.randint(0, case["far"] + 1, (1,), generator=g, device="cuda") if t > 1 else _ints([case["far"]], torch.int64)
        return s | _rotation(case, g, torch.arange(t, device="cuda") + first)
    new, ctx = _lens(case)
    if op == "append":
        t, hq = sum(new), case["hq"]
        s |= _cache(case, g, [n + c for n, c in zip(new, ctx)])
        qkv = _heads(g, t, hq + 2 * hk, d, dt)
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq: hq + hk], "v": qkv[:, hq + hk:], "alone": hq == 0,
              "starts": _ints(ctx, torch.int32), "indptr": _starts(new)}
        pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, ctx)]).cuda()
        seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        s["slots"] = s["table"][seq, pos // s["page"]].long() * s["page"] + pos % s["page"]
        s |= {"q_out": torch.empty(t, hq, d, dtype=dt, device="cuda")} | \
            {w: torch.empty(t, hk, d, dtype=dt, device="cuda") for w in ("k_out", "v_out")}
        return s | _rotation(case, g, pos)
    s |= _cache(case, g, [n + c for n, c in zip(new, ctx)])
    _fill(case, g, s, [n + c for n, c in zip(new, ctx)])
    if op == "read":
        t = sum(ctx)
        return s | {"starts": _ints([0] * len(ctx), torch.int32), "indptr": _starts(ctx)} | \
            {w: torch.empty(t, hk, d, dtype=dt, device="cuda") for w in ("k_out", "v_out")}
    t, hq = sum(new), case["hq"]
    s |= {"q": 1.5 * torch.randn(t, hq, d, generator=g, device="cuda").to(dt), "indptr": _starts(new),
          "ctx": _ints(ctx, torch.int32), "nodes": max(new), "most": max(n + c for n, c in zip(new, ctx)),
          "scale": d ** -0.5, "out": torch.empty(t, hq, d, dtype=dt, device="cuda"),
          "lse": torch.empty(t, hq, device="cuda"), "mask": None}
    if case["tree"]:  # node i sees itself and its ancestors; parents come before their children
        r = np.random.default_rng(seed)
        rows = []
        for n in new:
            seen = []
            for i in range(n):
                parent = int(r.integers(max(0, i - 6), i)) if i else -1
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
            rows += seen
        s["mask"] = torch.from_numpy(np.array(rows, dtype=np.uint64).view(np.int64)[:, None]).cuda()
    return s


# ---- the plain form ------------------------------------------------------------------------------------------------


def _quantize(x, fmt):
    """Codes and scales of float32 rows: quotients and roundings in 32 bits, ties to even."""
    if fmt == "u4":
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        span = (hi - lo).clamp(min=1e-5)
        scale = (span / torch.full_like(span, 15)).clamp(max=65504).half()  # a quotient: a plain number would be multiplied by its inverse
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
        n = (torch.round(x / scale.float()[..., None]) + zero[..., None]).clamp(0, 15).to(torch.uint8)
        return n[..., ::2] | n[..., 1::2] << 4, torch.stack([scale, zero.half()], -1)
    amax = x.abs().amax(-1)
    scale = (amax / torch.full_like(amax, 127 if fmt == "int8" else 448)).clamp(min=_FLOOR)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    n = x / scale[..., None]
    if fmt == "int8":
        return torch.round(n).to(torch.int8), scale
    return n.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _values(codes, scale, fmt):
    """The float32 values that codes stand for."""
    if fmt == "u4":
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        return (n - scale[..., 1:].float()) * scale[..., :1].float()
    n = codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    return n * scale[..., None]


def _norm_rotate(x, gamma, s):
    x = x.float()
    if gamma is not None:
        x = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])) * gamma.float()
    h = s["freq"].numel()
    if not h:
        return x
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    turn, rest = x[..., : 2 * h], x[..., 2 * h:]
    a, b = (turn[..., ::2], turn[..., 1::2]) if s["inter"] else (turn[..., :h], turn[..., h:])
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([u, w], -1).flatten(-2) if s["inter"] else torch.cat([u, w], -1), rest], -1)


def _plain(s):
    dt = s["dtype"]
    if s["op"] == "rotate":
        return {"q": _norm_rotate(s["q"], s["gq"], s).to(dt), "k": _norm_rotate(s["k"], s["gk"], s).to(dt)}
    fmt, page = s["fmt"], s["page"]
    if s["op"] == "append":
        k, v = _norm_rotate(s["k"], s["gk"], s), s["v"].float()
        at = (s["slots"] // page, slice(None), s["slots"] % page)
        out = {}
        for w, x in (("k", k), ("v", v)):
            s[w + "c"][at], s[w + "s"][at] = _quantize(x, fmt)
            out[w] = _values(s[w + "c"][at], s[w + "s"][at], fmt).to(dt)
        return out if s["alone"] else out | {"q": _norm_rotate(s["q"], s["gq"], s).to(dt)}
    if s["op"] == "read":
        t = torch.arange(s["indptr"].numel() - 1, device="cuda")
        count = (s["indptr"][1:] - s["indptr"][:-1]).long()
        seq = torch.repeat_interleave(t, count, output_size=s["k_out"].shape[0])
        pos = torch.arange(s["k_out"].shape[0], device="cuda") - s["indptr"].long()[seq] + s["starts"].long()[seq]
        at = (s["table"][seq, pos // page].long(), slice(None), pos % page)
        return {w: _values(s[w + "c"][at], s[w + "s"][at], fmt).to(dt) for w in ("k", "v")}
    # tree: sequences padded to the longest, queries to the most nodes
    count = (s["indptr"][1:] - s["indptr"][:-1]).long()
    seqs, most, nodes, hk = count.numel(), s["most"], s["nodes"], s["kc"].shape[1]
    table = s["table"][:, : -(-most // page)].long()
    k, v = (_values(s[w + "c"][table], s[w + "s"][table], fmt).transpose(1, 2).flatten(2, 3)[:, :, :most] for w in ("k", "v"))
    node = torch.arange(nodes, device="cuda")
    row = (s["indptr"].long()[:-1, None] + node).clamp(max=s["q"].shape[0] - 1)
    place = torch.arange(most, device="cuda")
    behind = place - s["ctx"].long()[:, None]
    v = torch.where((behind < count[:, None])[:, None, :, None], v, 0.0)
    if s["mask"] is None:
        seen = behind[:, None] <= node[:, None]
    else:
        bits = s["mask"][row, 0][:, :, None] >> behind[:, None].clamp(0, 63) & 1
        seen = (behind[:, None] < 0) | ((bits == 1) & (behind < count[:, None])[:, None])
    d = s["q"].shape[2]
    q = s["q"][row].float().unflatten(2, (hk, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seq][hk][node * group][d]
    group = q.shape[2] // nodes
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    score = torch.where(seen.repeat_interleave(group, 1)[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    mine = (node < count[:, None]).nonzero(as_tuple=True)
    o, lse = (x.unflatten(2, (nodes, group)).transpose(1, 2)[mine].flatten(1, 2) for x in (o, lse))
    return {"out": o.to(dt), "lse": lse}


# ---- the library's entry points --------------------------------------------------------------------------------------


def _calls(s):
    """The calls of one pass, their arguments checked and marshalled once, as a decode loop keeps them."""
    import quantized_linear_layer_gb300 as q
    op = s["op"]
    turn = {} if op in ("read", "tree") else {"q_gamma": s["gq"], "k_gamma": s["gk"], "eps": s["eps"], "interleaved": s["inter"]}
    if op == "rotate":
        return [q.qlin_qk_norm_rope_prepare(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["freq"], **turn)]
    fmt = {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[s["fmt"]]
    cache = q.qlin_kv_cache(s["kc"], s["vc"], s["ks"], s["vs"], fmt)
    if op == "tree":
        space = torch.empty(q.qlin_tree_attention_workspace_bytes(cache, s["q"].shape[1], s["nodes"], s["ctx"].numel()), dtype=torch.uint8, device="cuda")
        return [q.qlin_tree_attention_prepare(s["q"], cache, s["table"], s["indptr"], s["ctx"], s["mask"], s["out"], space,
                                              s["nodes"], scale=s["scale"], lse=s["lse"])]
    read = q.qlin_kv_cache_read_prepare(cache, s["table"], s["starts"], s["indptr"], s["k_out"], s["v_out"])
    if op == "read":
        return [read]
    if s["alone"]:
        return [q.qlin_kv_cache_write_prepare(s["k"], s["v"], s["slots"], cache), read]
    return [q.qlin_qk_norm_rope_cache_prepare(s["q"], s["k"], s["v"], s["q_out"], s["pos"], s["freq"], s["slots"], cache, **turn),
            read]


def run(state):
    s = state
    if not own:
        return _plain(s)
    calls = s["kept"].get("calls")
    if calls is None:
        calls = s["kept"]["calls"] = _calls(s)
    for c in calls:
        c.run()
    if s["op"] == "tree":
        return {"out": s["out"], "lse": s["lse"]}
    out = {"k": s["k_out"]}
    if s["op"] != "rotate":
        out["v"] = s["v_out"]
    if s["op"] == "rotate" or (s["op"] == "append" and not s["alone"]):
        out["q"] = s["q_out"]
    return out


# ---- 64 bits ---------------------------------------------------------------------------------------------------------


def _f32(x):
    return x.float().double()


def _stored64(x, fmt):
    """What reading gives back for rows x (64 bits): scales and quotients are 32-bit (U4 scales 16-bit) numbers by
    definition, their roundings written out here."""
    if fmt == "u4":
        low = torch.minimum(x.min(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
        high = torch.maximum(x.max(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
        span = torch.maximum(_f32(high - low), _f32(torch.tensor(1e-5, device=x.device)))
        scale = torch.minimum(_f32(span / 15), torch.tensor(65504.0, dtype=x.dtype, device=x.device)).half().double()[..., None]
        zero = _f32(-low[..., None] / scale).round().clamp(0, 15)
        return scale * ((_f32(x / scale).round() + zero).clamp(0, 15) - zero)
    big = x.abs().max(-1, keepdim=True).values
    scale = _f32(big / {"int8": 127, "e4m3": 448}[fmt]).clamp_min(_FLOOR)
    scale[big == 0] = 1
    n = _f32(x / scale)
    if fmt == "int8":
        return scale * n.round()
    n = n.clamp(-448, 448)
    grid = torch.exp2(torch.log2(n.abs().clamp_min(2.0 ** -6)).floor() - 3)  # three bits behind the leading one
    return scale * (torch.round(n / grid) * grid)


def _rotated64(x, gamma, s):
    x = x.double()
    if gamma is not None:
        x = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * gamma.double()
    h = s["freq"].numel()
    y = x.clone()
    first = torch.arange(h, device="cuda") * (2 if s["inter"] else 1)
    second = first + (1 if s["inter"] else h)
    turned = torch.polar(torch.ones_like(s["freq"]).expand(x.shape[0], h), torch.outer(s["pos"].double(), s["freq"]))
    z = torch.complex(x[..., first], x[..., second]) * turned[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _cached64(s, b, upto):
    """K and V of sequence b's first tokens, [heads][tokens][d]."""
    pages = s["table"][b, : -(-upto // s["page"])].long()
    got = []
    for w in ("k", "v"):
        c, f = (s[w + x][pages].transpose(0, 1).flatten(1, 2)[:, :upto] for x in ("c", "s"))
        if s["fmt"] == "u4":
            n = torch.empty(*c.shape[:2], 2 * c.shape[2], dtype=torch.float64, device="cuda")
            n[..., 0::2], n[..., 1::2] = (c % 16).double(), (c // 16).double()
            got.append(f[..., 0:1].double() * (n - f[..., 1:2].double()))
        else:
            n = c.double() if s["fmt"] == "int8" else c.view(torch.float8_e4m3fn).double()
            got.append(n * f.double()[..., None])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rotate":
        return {"q": _rotated64(s["q"], s["gq"], s), "k": _rotated64(s["k"], s["gk"], s)}
    if s["op"] == "append":
        out = {"k": _stored64(_rotated64(s["k"], s["gk"], s), s["fmt"]), "v": _stored64(s["v"].double(), s["fmt"])}
        return out if s["alone"] else out | {"q": _rotated64(s["q"], s["gq"], s)}
    new, ctx = _lens(case)
    if s["op"] == "read":
        rows = [_cached64(s, b, c) for b, c in enumerate(ctx)]
        return {w: torch.cat([r[i].transpose(0, 1) for r in rows]) for i, w in ((0, "k"), (1, "v"))}
    out, lse, at = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), s["lse"].double(), 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        k, v = _cached64(s, b, n + c)
        hk = k.shape[0]
        q = s["q"][at: at + n].double().reshape(n, hk, -1, case["d"])
        hide = torch.zeros(n, n + c, dtype=torch.bool, device="cuda")
        for i in range(n):
            bits = (2 << i) - 1 if s["mask"] is None else int(s["mask"][at + i, 0]) & (1 << 64) - 1
            hide[i, c:] = torch.tensor([not bits >> j & 1 for j in range(n)], device="cuda")
        for h in range(hk):
            score = torch.einsum("ngd,ld->ngl", q[:, h], k[h]) * s["scale"]
            score.masked_fill_(hide[:, None], -math.inf)
            total = torch.logsumexp(score, -1)
            p = torch.exp(score - total[..., None]).nan_to_num(0.0)
            g = q.shape[2]
            out[at: at + n, h * g: (h + 1) * g] = torch.einsum("ngl,ld->ngd", p, v[h])
            lse[at: at + n, h * g: (h + 1) * g] = total
        at += n
    return {"out": out, "lse": lse}
