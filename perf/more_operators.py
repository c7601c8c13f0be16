"""Cases of the operators of a serving step around the quantized paged cache:

  pages   block tables, row bounds, positions and slots of a step from the sequences' lengths, the pages
          taken from and given back to a stack of free ones
  chunk   attention of a chunk of new tokens over the cache: causal, with a prefix that all see, a window,
          scores capped by a tanh, a bias by distance
  verify  drafted tokens (a chain or a tree) verified against the target's probabilities, and the next token
  keep    the accepted path of a tree of drafts moved to the end of its sequence in the cache, read back

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


def listed():
    return [
        # one decode step of 64 conversations: a token each, now and then a page
        {"name": "pages decode step", "op": "pages", "seqs": 64, "new": 1, "ctx": 8191, "spread": 1, "page": 64, "join": 0,
         "rows": 64, "depths": False, "room": 1.0},
        # prompts taken in beside running sequences with trees of drafts, into a pool that is too small for all of them
        {"name": "pages admission", "op": "pages", "seqs": 600, "new": 24, "ctx": 4096, "spread": 2, "page": 16, "join": 77,
         "rows": 65536, "depths": True, "room": 0.9},
        # one token of one conversation, scores capped: only latency counts
        {"name": "chunk one token", "op": "chunk", "fmt": "int8", "dtype": "fp16", "seqs": 1, "new": 1, "ctx": 2047, "spread": 0,
         "hq": 32, "hk": 8, "d": 128, "page": 16, "cap": 30.0, "slopes": False, "window": 0, "prefix": 0},
        # the usual prefill: chunks of several prompts behind what is cached of them
        {"name": "chunk prompts", "op": "chunk", "fmt": "e4m3", "dtype": "bf16", "seqs": 4, "new": 2048, "ctx": 8192, "spread": 3,
         "hq": 32, "hk": 8, "d": 128, "page": 64, "cap": 0.0, "slopes": False, "window": 0, "prefix": 0},
        # 4-bit cache, all heads of 64 their own, bias by distance: ragged chunks
        {"name": "chunk biased four bits", "op": "chunk", "fmt": "u4", "dtype": "fp16", "seqs": 6, "new": 777, "ctx": 3001,
         "spread": 4, "hq": 32, "hk": 32, "d": 64, "page": 32, "cap": 0.0, "slopes": True, "window": 0, "prefix": 0},
        # capped scores in a window, a shared prefix that everybody sees, heads of 256
        {"name": "chunk capped window", "op": "chunk", "fmt": "int8", "dtype": "bf16", "seqs": 3, "new": 2049, "ctx": 6000,
         "spread": 5, "hq": 16, "hk": 8, "d": 256, "page": 64, "cap": 50.0, "slopes": False, "window": 2048, "prefix": 700},
        # a long document by large chunks: the largest products
        {"name": "chunk long document", "op": "chunk", "fmt": "int8", "dtype": "fp16", "seqs": 1, "new": 8192, "ctx": 16384,
         "spread": 0, "hq": 32, "hk": 8, "d": 128, "page": 64, "cap": 0.0, "slopes": False, "window": 0, "prefix": 0},
        # one conversation, four drafted tokens, a vocabulary of 32000: latency
        {"name": "verify one chain", "op": "verify", "seqs": 1, "nodes": 5, "vocab": 32000, "draft": True, "fan": 1, "agree": 0.8,
         "spread": 0},
        # a serving step: 64 conversations with chains of drafts from a small model, a large vocabulary
        {"name": "verify chains", "op": "verify", "seqs": 64, "nodes": 6, "vocab": 128256, "draft": True, "fan": 1, "agree": 0.7,
         "spread": 6},
        # trees whose nodes are the draft's likeliest tokens (no probabilities of theirs), an odd vocabulary
        {"name": "verify trees", "op": "verify", "seqs": 32, "nodes": 26, "vocab": 50257, "draft": False, "fan": 4, "agree": 0.6,
         "spread": 7},
        # one conversation keeps a path of its tree
        {"name": "keep one path", "op": "keep", "fmt": "int8", "dtype": "fp16", "seqs": 1, "nodes": 26, "most": 6, "ctx": 4000,
         "spread": 0, "hk": 8, "d": 128, "page": 16},
        # a large batch of wide trees, each with its own path
        {"name": "keep large batch", "op": "keep", "fmt": "e4m3", "dtype": "bf16", "seqs": 192, "nodes": 64, "most": 9, "ctx": 2000,
         "spread": 8, "hk": 32, "d": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "chunk", "chunk", "verify", "keep"])
    case = {"op": op, "spread": rng.randrange(8, 1 << 20)}
    if op == "pages":
        seqs = _log(rng, 1, 600)
        new = _log(rng, 1, max(1, 16384 // seqs))
        case |= {"seqs": seqs, "new": new, "ctx": _log(rng, 1, 16384), "page": rng.choice([16, 32, 64, 128, 256]),
                 "join": rng.choice([0, seqs // 4]), "rows": seqs * new + rng.choice([0, 0, 100]), "depths": rng.random() < 0.5,
                 "room": rng.choice([1.0, 1.0, 0.9])}
        return case
    if op == "verify":
        vocab = rng.choice([_log(rng, 500, 262144), 32000, 128256])
        nodes = _log(rng, 1, 64)
        fan = rng.choice([1, 1, 2, 4])
        case |= {"seqs": _log(rng, 1, max(1, min(64, 300_000_000 // (vocab * nodes * 2)))), "nodes": nodes, "vocab": vocab,
                 "draft": rng.random() < 0.6, "fan": fan, "agree": rng.choice([0.3, 0.6, 0.8])}
        return case
    hk = rng.choice([1, 2, 4, 8, 8, 32])
    d = rng.choice([64, 128, 128, 128, 256])
    case |= {"fmt": rng.choice(["int8", "e4m3", "u4"]), "dtype": rng.choice(["fp16", "bf16"]), "hk": hk, "d": d,
             "page": rng.choice([16, 32, 64, 128])}
    if op == "keep":
        nodes = _log(rng, 2, 64)
        case |= {"seqs": _log(rng, 1, max(1, 192 * 32 * 128 // (hk * d))), "nodes": nodes, "most": rng.randint(1, max(1, nodes // 2)),
                 "ctx": _log(rng, 1, 2000)}
        case["seqs"] = min(case["seqs"], 192)
        return case
    hq = hk * rng.choice([g for g in (1, 2, 4, 5, 8) if g * hk <= 64])
    if hq * d == 3072:
        hq = hk
    kind = rng.choice(["plain", "plain", "cap", "slopes", "window", "prefix", "all"])
    case |= {"hq": hq, "seqs": _log(rng, 1, 32), "new": _log(rng, 1, 8192), "ctx": _log(rng, 1, 65536),
             "cap": rng.choice([20.0, 50.0]) if kind in ("cap", "all") else 0.0, "slopes": kind in ("slopes", "all"),
             "window": _log(rng, 16, 8192) if kind in ("window", "all") else 0,
             "prefix": _log(rng, 16, 4096) if kind in ("prefix", "all") else 0}
    most = {"flops": max(work(c)["flops"] for c in listed()), "bytes": 2 ** 31}
    while work(case)["flops"] > most["flops"] or work(case)["bytes"] > most["bytes"]:
        case["seqs"] = max(1, case["seqs"] * 4 // 5)
        case["new"] = max(1, case["new"] * 4 // 5)
        case["ctx"] = max(1, case["ctx"] * 4 // 5)
    return case


# ---- the lengths of a case's sequences: from the case alone ------------------------------------------------------


def _lens(case):
    """(new tokens, cached tokens before them) of each sequence; with a spread they differ."""
    r = random.Random(case["spread"] * 7919 + 13)
    most = case.get("nodes", case.get("new", 0))
    new, ctx = [], []
    for b in range(case["seqs"]):
        spread = case["spread"] and b
        new.append(r.randint(max(1, most // 2), most) if spread else most)
        ctx.append(r.randint(case.get("ctx", 0) // 16, case.get("ctx", 0)) if spread else case.get("ctx", 0))
    for b in range(case.get("join", 0)):  # prompts that begin: nothing cached, a chunk of many tokens
        i = b * case["seqs"] // case["join"]
        new[i], ctx[i] = r.randint(1, 512 if case["rows"] > 30000 else 2 * most), 0
    return new, ctx


def _row_bytes(fmt, d):
    return (d // 2 if fmt == "u4" else d) + 4


def _pairs(case):
    """Query rows times tokens that a row sees, and the tokens that some row sees, over all sequences."""
    r = random.Random(case["spread"] + 5)
    pairs = tokens = 0
    for n, c in zip(*_lens(case)):
        prefix = min(r.randint(0, case["prefix"]), n + c) if case["prefix"] else 0
        p = np.arange(c, c + n, dtype=np.int64)
        low = np.maximum(p - case["window"] + 1, 0) if case["window"] else np.zeros_like(p)
        # what lies in the window, and of the prefix what does not
        pairs += int((p - low + 1 + np.minimum(low, prefix) + np.maximum(prefix - p - 1, 0)).sum())
        tokens += c + n - max(0, int(low[0]) - prefix)
    return pairs, tokens


def _depth(case):
    """About how many drafted tokens a sequence has one behind the other."""
    return case["nodes"] - 1 if case["fan"] == 1 else int(math.log(1 + (case["nodes"] - 1) * (case["fan"] - 1), case["fan"]))


def work(case):
    op = case["op"]
    if op == "pages":
        new, ctx = _lens(case)
        taken = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for n, c in zip(new, ctx))
        b, t = case["seqs"], case["rows"]
        # lengths and page counts in, bounds out; slots and positions out (and depths in); pages taken and given back; each
        # row's page number; the same lengths once more when the step is taken back
        return {"bytes": 28 * b + t * (16 + (4 if case["depths"] else 0)) + 16 * taken + 4 * sum(new), "flops": 10 * (t + b)}
    if op == "verify":
        rows = 1 + (1 - case["agree"] ** _depth(case) if case["draft"] else 0)  # the target's row where it ends, the draft's unless all were accepted
        n = case["seqs"] * case["vocab"] * rows
        return {"bytes": int(4 * n) + case["seqs"] * case["nodes"] * 24, "flops": int(4 * n)}
    d, hk = case["d"], case["hk"]
    rb = _row_bytes(case["fmt"], d)
    if op == "keep":  # codes and scales from one place to another; the same read and written as 16-bit rows
        t = sum(_counts(case))
        return {"bytes": t * 2 * hk * (3 * rb + 2 * d), "flops": t * 2 * hk * d}
    pairs, tokens = _pairs(case)
    return {"bytes": 2 * tokens * hk * rb + sum(_lens(case)[0]) * case["hq"] * (4 * d + 4), "flops": 4 * case["hq"] * d * pairs}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _starts(v):
    return _ints([0] + list(np.cumsum(v)))


def _cache(case, g, total):
    """A cache whose pages lie in no order: [pages][heads][page][bytes] twice, scales, and each sequence's pages.
    Places that no sequence has reached hold what an earlier one left: any codes, and scales that are not numbers."""
    fmt, page, hk, d = case["fmt"], case["page"], case["hk"], case["d"]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(total), max(need) + 1), pages - 1, dtype=torch.int32, device="cuda")
    left = torch.zeros(pages, dtype=torch.int64, device="cuda")  # tokens of each page in use
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        left[order[at: at + n].long()] = page
        left[order[at + n - 1].long()] = total[b] - (n - 1) * page
        at += n
    width = d // 2 if fmt == "u4" else d
    kind = torch.int8 if fmt == "int8" else torch.uint8
    s = {"fmt": fmt, "page": page, "table": table}
    inside = torch.arange(page, device="cuda")[None, None, :] < left[:, None, None]
    step = max(1, (1 << 27) // (hk * page * d))
    for w in ("k", "v"):
        s[w + "c"] = torch.randint(0, 126, (pages, hk, page, width), generator=g, device="cuda", dtype=torch.int32).to(kind)
        s[w + "s"] = torch.full((pages, hk, page, 2), math.nan, dtype=torch.float16, device="cuda") if fmt == "u4" else \
            torch.full((pages, hk, page), math.nan, device="cuda")
        size = torch.exp(0.4 * torch.randn(hk, 1, d, generator=g, device="cuda"))
        if w == "k":
            size[:, :, :: max(1, d // 3)] *= 4
        for a in range(0, pages, step):
            m = min(step, pages - a)
            x = torch.randn(m, hk, page, d, generator=g, device="cuda") * size
            x *= torch.exp(0.3 * torch.randn(m, hk, page, 1, generator=g, device="cuda"))
            codes, scale = _quantize(x, fmt)
            here = inside[a: a + m].expand(m, hk, page)
            s[w + "c"][a: a + m] = torch.where(here[..., None], codes, s[w + "c"][a: a + m])
            s[w + "s"][a: a + m] = torch.where(here if scale.dim() == 3 else here[..., None], scale, s[w + "s"][a: a + m])
    return s


def _quantize(x, fmt):
    """Codes and scales as a cache write leaves them."""
    if fmt == "u4":
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        scale = ((hi - lo).clamp(min=1e-5) / 15).half()
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
        n = (torch.round(x / scale.float()[..., None]) + zero[..., None]).clamp(0, 15).to(torch.uint8)
        return n[..., ::2] | n[..., 1::2] << 4, torch.stack([scale, zero.half()], -1)
    scale = x.abs().amax(-1) / (127 if fmt == "int8" else 448)
    n = x / scale[..., None]
    if fmt == "int8":
        return torch.round(n).clamp(-127, 127).to(torch.int8), scale
    return n.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _counts(case):
    """How many nodes of its tree each sequence keeps, the root among them."""
    r = random.Random(case["spread"] * 31 + 1)
    return [r.randint(1, min(case["most"], max(1, n // 2))) if case["spread"] and b else case["most"]
            for b, n in enumerate(_lens(case)[0])]


def _prepare_pages(case, g):
    new, ctx = _lens(case)
    page = case["page"]
    held = [-(-c // page) for c in ctx]
    want = [-(-(c + n) // page) for n, c in zip(new, ctx)]
    spare = int(case["room"] * (sum(want) - sum(held)))
    spare = spare if case["room"] < 1 else spare + 5
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], max(want) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at: at + n]
        at += n
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = order[at:]
    t = case["rows"]
    s = {"page": page, "pages": pages, "table": table, "held": _ints(held), "free": free, "count": _ints([spare]),
         "ctx": _ints(ctx), "new": _ints(new), "none": torch.zeros(case["seqs"], dtype=torch.int32, device="cuda"), "rows": t,
         "depths": torch.randint(0, 12, (t,), generator=g, device="cuda", dtype=torch.int32) if case["depths"] else None}
    for name in ("", "2"):
        s |= {"indptr" + name: torch.zeros(case["seqs"] + 1, dtype=torch.int32, device="cuda"),
              "positions" + name: torch.zeros(t, dtype=torch.int64, device="cuda"),
              "slots" + name: torch.zeros(t, dtype=torch.int64, device="cuda")}
    return s


def _prepare_verify(case, g):
    new, _ = _lens(case)
    rows, v = sum(new), case["vocab"]
    parents = []
    for n in new:
        parents += [(i - 1) // case["fan"] for i in range(n)]
    target = torch.empty(rows, v, device="cuda")
    draft = torch.empty(rows, v, device="cuda") if case["draft"] else None
    noise = 3.0 * (1 - case["agree"])
    likely = torch.empty(rows, case["fan"], dtype=torch.int64, device="cuda")
    step = max(1, (1 << 27) // v)
    for a in range(0, rows, step):
        m = min(step, rows - a)
        x = 2.5 * torch.randn(m, v, generator=g, device="cuda")
        target[a: a + m] = torch.softmax(x + 0.5 * noise * torch.randn(m, v, generator=g, device="cuda"), -1)
        q = torch.softmax(x, -1)
        if draft is None:
            likely[a: a + m] = q.topk(case["fan"], -1).indices
        else:
            draft[a: a + m] = q
            likely[a: a + m] = torch.multinomial(q, case["fan"], replacement=True, generator=g)
    start = np.concatenate([[0], np.cumsum(new)])
    up = np.concatenate([[start[b] + max(0, (i - 1) // case["fan"]) for i in range(n)] for b, n in enumerate(new)])
    which = np.concatenate([[(i - 1) % case["fan"] for i in range(n)] for n in new])
    tokens = likely[torch.from_numpy(up).cuda(), torch.from_numpy(which).cuda()]
    return {"target": target, "draft": draft, "tokens": tokens,
            "parents": None if case["fan"] == 1 else _ints([-1 if p < 0 else p for p in parents]), "indptr": _starts(new),
            "nodes": max(new), "accept": torch.rand(rows, generator=g, device="cuda"),
            "sample": torch.rand(case["seqs"], generator=g, device="cuda"),
            "path": torch.zeros(case["seqs"], max(new), dtype=torch.int32, device="cuda"),
            "kept": torch.zeros(case["seqs"], dtype=torch.int32, device="cuda"),
            "next": torch.zeros(case["seqs"], dtype=torch.int64, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op, "calls": {}}
    if op == "pages":
        return s | _prepare_pages(case, g)
    if op == "verify":
        return s | _prepare_verify(case, g)
    new, ctx = _lens(case)
    dt, d, hk = _DT[case["dtype"]], case["d"], case["hk"]
    s |= _cache(case, g, [n + c for n, c in zip(new, ctx)]) | {"dtype": dt, "ctx": _ints(ctx), "lens": (new, ctx)}
    if op == "keep":
        # a path's later nodes lie behind as many nodes as it keeps, as the levels of a wide tree do
        r = random.Random(seed)
        counts, paths = _counts(case), torch.full((case["seqs"], max(new)), -1, dtype=torch.int32)
        for b, (n, k) in enumerate(zip(new, counts)):
            paths[b, :k] = torch.tensor([0] + sorted(r.sample(range(k, n), k - 1)), dtype=torch.int32)
        t = sum(counts)
        return s | {"path": paths.cuda(), "kept": _ints(counts), "indptr": _starts(counts), "counts": counts,
                    "after": torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")} | \
            {w: torch.empty(t, hk, d, dtype=dt, device="cuda") for w in ("k_out", "v_out")}
    t, hq = sum(new), case["hq"]
    s |= {"q": 1.5 * torch.randn(t, hq, d, generator=g, device="cuda").to(dt), "indptr": _starts(new), "most": max(new),
          "scale": d ** -0.5, "cap": case["cap"], "window": case["window"], "slopes": None, "prefix": None, "prefixes": [0] * len(new),
          "out": torch.empty(t, hq, d, dtype=dt, device="cuda"), "lse": torch.empty(t, hq, device="cuda")}
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    if case["prefix"]:
        r = random.Random(case["spread"] + 5)
        s["prefixes"] = [min(r.randint(0, case["prefix"]), n + c) for n, c in zip(new, ctx)]
        s["prefix"] = _ints(s["prefixes"])
    return s


# ---- the plain form ------------------------------------------------------------------------------------------------


def _assign_plain(s, ctx, new, name):
    """One step's pages: what sequences no longer need goes to the stack, what they need comes from its top."""
    page, pages, cols = s["page"], s["pages"], s["table"].shape[1]
    ctx, new, held = ctx.long(), new.long(), s["held"].long()
    need = (ctx + new + page - 1) // page
    give, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    top = s["count"].long()
    col = torch.arange(cols, device="cuda")
    # the last sequence's last page goes first, so that giving back what was just taken restores the stack
    before = torch.cumsum(give, 0) - give
    at = top + give.sum() - 1 - (before[:, None] + col - need[:, None])
    at = torch.where((col >= need[:, None]) & (col < held[:, None]), at, pages)
    free = torch.cat([s["free"], s["free"][:1]]).scatter(0, at.flatten(), s["table"].flatten())[:pages]
    top = top + give.sum()
    served = ((take == 0) | (torch.cumsum(take, 0) <= top)) & ((new == 0) | (torch.cumsum(new, 0) <= s["rows"]))
    take, new = torch.where(served, take, 0), torch.where(served, new, 0)
    before = torch.cumsum(take, 0) - take
    at = top - 1 - (before[:, None] + col - held[:, None])
    mine = (col >= held[:, None]) & (col < (held + take)[:, None])
    s["table"].copy_(torch.where(mine, free[at.clamp(0, pages - 1)], s["table"]))
    s["free"].copy_(free)
    s["count"].copy_(top - take.sum())
    s["held"].copy_(held - give + take)
    s["indptr" + name][1:] = torch.cumsum(new, 0)
    row = torch.arange(s["rows"], device="cuda")
    end = s["indptr" + name][1:].long()
    seq = torch.searchsorted(end, row, right=True)
    live = seq < end.numel()
    seq = seq.clamp(max=end.numel() - 1)
    i = row - s["indptr" + name].long()[seq]
    at = ctx[seq] + i
    slot = s["table"][seq, (at // page).clamp(max=cols - 1)].long() * page + at % page
    s["slots" + name].copy_(torch.where(live, slot, -1))
    s["positions" + name].copy_(torch.where(live, ctx[seq] + (i if s["depths"] is None else s["depths"].long()), 0))


def _values(codes, scale, fmt):
    """The float32 values that codes stand for."""
    if fmt == "u4":
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        return (n - scale[..., 1:].float()) * scale[..., :1].float()
    n = codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    return n * scale[..., None]


def _chunk_plain(s):
    hk, page = s["kc"].shape[1], s["page"]
    t, hq, d = s["q"].shape
    group, first = hq // hk, 0
    for b, (n, c) in enumerate(zip(*s["lens"])):
        length = n + c
        table = s["table"][b, : -(-length // page)].long()
        k, v = (_values(s[w + "c"][table], s[w + "s"][table], s["fmt"]).transpose(0, 1).flatten(1, 2)[:, :length] for w in ("k", "v"))
        place = torch.arange(length, device="cuda")
        step = max(1, (1 << 28) // (hq * length))
        for a in range(0, n, step):
            m = min(step, n - a)
            rows = slice(first + a, first + a + m)
            at = torch.arange(c + a, c + a + m, device="cuda")[:, None]
            q = s["q"][rows].float().unflatten(1, (hk, group)).permute(1, 2, 0, 3).flatten(1, 2)  # [hk][group * m][d]
            score = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).unflatten(1, (group, m))
            if s["cap"]:
                score = s["cap"] * torch.tanh(score / s["cap"])
            if s["slopes"] is not None:
                score = score - s["slopes"].view(hk, group, 1, 1) * (at - place).abs()
            seen = place <= at
            if s["window"]:
                seen = seen & (at - place < s["window"])
            if s["prefix"] is not None:
                seen = seen | (place < s["prefix"][b])
            score = torch.where(seen, score, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.flatten(1, 2), v).unflatten(1, (group, m)) / total
            s["out"][rows] = o.permute(2, 0, 1, 3).flatten(1, 2).to(s["dtype"])
            s["lse"][rows] = (top + torch.log(total)).squeeze(-1).permute(2, 0, 1).flatten(1, 2)
        first += n
    return {"out": s["out"], "lse": s["lse"]}


def _verify_plain(s):
    """Nodes in their order: the child of the node reached last is accepted or takes the draft's share away."""
    seqs, nodes = s["path"].shape
    first, count = s["indptr"][:-1].long(), (s["indptr"][1:] - s["indptr"][:-1]).long()
    rows = torch.arange(seqs, device="cuda")
    at = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    length = torch.ones_like(at)
    s["path"].fill_(-1)
    s["path"][:, 0] = 0
    gone = torch.zeros(seqs, dtype=torch.float64, device="cuda")  # the share of the draft taken away from the target so far
    weight = torch.ones_like(gone)
    out = torch.zeros(seqs, s["target"].shape[1], dtype=torch.bool, device="cuda")  # tokens rejected at this node

    def left():
        p = s["target"][first + at].double()
        if s["draft"] is None:
            return torch.where(out, 0.0, p)
        return (p - gone[:, None] * s["draft"][first + at].double()).clamp(min=0)

    last = s["target"].shape[0] - 1
    for i in range(1, nodes):
        node = (first + i).clamp(max=last)
        here = (i < count) & ((i - 1 if s["parents"] is None else s["parents"][node].long()) == at)
        x = s["tokens"][node]
        p = s["target"][first + at, x].double()
        u = s["accept"][node].double()
        if s["draft"] is None:
            w = torch.where(out[rows, x], 0.0, p)
            good = here & (u * weight < w)
            rest = weight - w
        else:
            q = s["draft"][first + at, x].double()
            w = (p - gone * q).clamp(min=0)
            good = here & (u * weight * q < w)
        bad = here & ~good
        if s["draft"] is None:
            weight = torch.where(bad, rest.clamp(min=0), weight)
            out[rows, x] |= bad
        else:
            gone = torch.where(bad, gone + weight, gone)
            weight = torch.where(bad, left().sum(-1), weight)
        at = torch.where(good, i, at)
        gone, weight = torch.where(good, 0.0, gone), torch.where(good, 1.0, weight)
        out &= ~good[:, None]
        s["path"][rows, length.clamp(max=nodes - 1)] = torch.where(good, i, s["path"][rows, length.clamp(max=nodes - 1)].long()).int()
        length = length + good
    w = left()
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, s["target"][first + at].double())
    upto = torch.cumsum(w, -1)
    s["next"].copy_((upto <= s["sample"].double()[:, None] * upto[:, -1:]).sum(-1))
    s["kept"].copy_(length)
    return {"path": s["path"], "kept": s["kept"], "next": s["next"]}


def _keep_plain(s):
    page, most = s["page"], s["path"].shape[1]
    step = torch.arange(most, device="cuda")
    seq, i = (step < s["kept"][:, None]).nonzero(as_tuple=True)
    c = s["ctx"].long()[seq]

    def places(j):
        return s["table"][seq, (c + j) // page].long(), slice(None), (c + j) % page

    src, dst = places(s["path"][seq, i].long()), places(i)
    for x in ("kc", "vc", "ks", "vs"):
        s[x][dst] = s[x][src]
    s["after"].copy_(s["ctx"] + s["kept"])
    return {w: _values(s[w + "c"][dst], s[w + "s"][dst], s["fmt"]).to(s["dtype"]) for w in ("k", "v")} | {"lens": s["after"]}


# ---- the library's entry points --------------------------------------------------------------------------------------


def _calls(s):
    """The calls of one pass, their arguments checked and marshalled once, as a decode loop keeps them."""
    import quantized_linear_layer_gb300 as q
    op = s["op"]
    if op == "pages":
        pages = q.qlin_kv_pages(s["table"], s["held"], s["free"], s["count"], s["page"])
        return [q.qlin_kv_pages_assign_prepare(pages, s["ctx"], new, s["indptr" + x], s["positions" + x], s["slots" + x], s["depths"])
                for new, x in ((s["new"], ""), (s["none"], "2"))]
    if op == "verify":
        return [q.qlin_verify_drafts_prepare(s["target"], s["draft"], s["parents"], s["tokens"], s["indptr"], s["accept"], s["sample"],
                                             s["path"], s["kept"], s["next"])]
    fmt = {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[s["fmt"]]
    cache = q.qlin_kv_cache(s["kc"], s["vc"], s["ks"], s["vs"], fmt)
    if op == "keep":
        return [q.qlin_kv_cache_keep_prepare(cache, s["table"], s["ctx"], s["path"], s["kept"], s["after"]),
                q.qlin_kv_cache_read_prepare(cache, s["table"], s["ctx"], s["indptr"], s["k_out"], s["v_out"])]
    size = q.qlin_chunk_attention_workspace_bytes(cache, s["q"].shape[1], s["most"], s["ctx"].numel())
    space = torch.empty(size, dtype=torch.uint8, device="cuda")
    return [q.qlin_chunk_attention_prepare(s["q"], cache, s["table"], s["indptr"], s["ctx"], s["out"], space, s["most"],
                                           scale=s["scale"], softcap=s["cap"], slopes=s["slopes"], window=s["window"],
                                           prefix_lens=s["prefix"], lse=s["lse"])]


def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "pages":
            _assign_plain(s, s["ctx"], s["new"], "")
            _assign_plain(s, s["ctx"], s["none"], "2")
        else:
            return {"chunk": _chunk_plain, "verify": _verify_plain, "keep": _keep_plain}[op](s)
    else:
        if "own" not in s["calls"]:
            s["calls"]["own"] = _calls(s)
        for c in s["calls"]["own"]:
            c.run()
    if op == "pages":
        return {x: s[x] for x in ("indptr", "positions", "slots", "indptr2", "positions2", "slots2", "table", "held", "free", "count")}
    if op == "verify":
        return {"path": s["path"], "kept": s["kept"], "next": s["next"]}
    if op == "keep":
        return {"k": s["k_out"], "v": s["v_out"], "lens": s["after"]}
    return {"out": s["out"], "lse": s["lse"]}


# ---- 64 bits ---------------------------------------------------------------------------------------------------------


def _assign_exact(s, table, held, stack, ctx, new):
    """The same step over Python lists: `stack` ends at its top."""
    page, rows = s["page"], s["rows"]
    for b in reversed(range(len(ctx))):
        need = -(-(ctx[b] + new[b]) // page)
        while held[b] > need:
            held[b] -= 1
            stack.append(table[b][held[b]])
    room, asked, taken = len(stack), 0, 0
    bounds, positions, slots = [0], [], []
    depths = None if s["depths"] is None else s["depths"].tolist()
    for b, (c, n) in enumerate(zip(ctx, new)):
        more = max(0, -(-(c + n) // page) - held[b])
        taken, asked = taken + more, asked + n
        if not ((more and taken > room) or (n and asked > rows)):
            for _ in range(more):
                table[b][held[b]] = stack.pop()
                held[b] += 1
            for i in range(n):
                positions.append(c + (i if depths is None else depths[len(positions)]))
                slots.append(table[b][(c + i) // page] * page + (c + i) % page)
        bounds.append(len(slots))
    return _ints(bounds), _ints(positions + [0] * (rows - len(slots)), torch.int64), _ints(slots + [-1] * (rows - len(slots)), torch.int64)


def _exact_pages(s):
    table, held, ctx = s["table"].tolist(), s["held"].tolist(), s["ctx"].tolist()
    stack = s["free"][: int(s["count"])].tolist()
    got = {}
    for new, x in ((s["new"], ""), (s["none"], "2")):
        got["indptr" + x], got["positions" + x], got["slots" + x] = _assign_exact(s, table, held, stack, ctx, new.tolist())
    return got | {"table": _ints(table), "held": _ints(held), "free": _ints(stack + s["free"].tolist()[len(stack):]),
                  "count": _ints([len(stack)])}


def _exact_verify(s):
    bounds, tokens = s["indptr"].tolist(), s["tokens"].tolist()
    accept, sample = s["accept"].tolist(), s["sample"].tolist()
    paths, kept, after = [], [], []
    for b in range(len(sample)):
        a, n = bounds[b], bounds[b + 1] - bounds[b]
        parent = list(range(-1, n - 1)) if s["parents"] is None else s["parents"][a: a + n].tolist()
        path = [0]
        while True:
            here = path[-1]
            p = s["target"][a + here].cpu().numpy().astype(np.float64)
            rest, total, moved = p, 1.0, False
            q = None if s["draft"] is None else s["draft"][a + here].cpu().numpy().astype(np.float64)
            drawn = 0.0
            for child in [i for i in range(here + 1, n) if parent[i] == here]:
                x = tokens[a + child]
                if accept[a + child] * total * (1.0 if q is None else q[x]) < rest[x]:
                    path.append(child)
                    moved = True
                    break
                if q is None:
                    rest = rest.copy()
                    total, rest[x] = max(0.0, total - rest[x]), 0.0
                else:
                    drawn += total
                    rest = np.maximum(p - drawn * q, 0.0)
                    total = math.fsum(rest)
            if not moved:
                break
        sums = np.cumsum(rest if rest.any() else p, dtype=np.longdouble)
        after.append(int(np.searchsorted(sums, np.longdouble(sample[b]) * sums[-1], side="right")))
        kept.append(len(path))
        paths.append(path + [-1] * (s["path"].shape[1] - len(path)))
    return {"path": _ints(paths), "kept": _ints(kept), "next": _ints(after, torch.int64)}


def _cached64(s, b, places):
    """K and V of tokens `places` of sequence b, [heads][tokens][d]."""
    pages, offsets = s["table"][b][places // s["page"]].long(), places % s["page"]
    got = []
    for w in ("k", "v"):
        c, f = (s[w + x][pages, :, offsets].transpose(0, 1) for x in ("c", "s"))
        if s["fmt"] == "u4":
            n = torch.empty(*c.shape[:2], 2 * c.shape[2], dtype=torch.float64, device="cuda")
            n[..., 0::2], n[..., 1::2] = (c % 16).double(), (c // 16).double()
            got.append(f[..., 0:1].double() * (n - f[..., 1:2].double()))
        else:
            n = c.double() if s["fmt"] == "int8" else c.contiguous().view(torch.float8_e4m3fn).double()
            got.append(n * f.double()[..., None])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "pages":
        return _exact_pages(s)
    if s["op"] == "verify":
        return _exact_verify(s)
    new, ctx = _lens(case)
    if s["op"] == "keep":
        rows = [_cached64(s, b, c + s["path"][b, :k].long()) for b, (c, k) in enumerate(zip(ctx, s["counts"]))]
        return {w: torch.cat([r[i].transpose(0, 1) for r in rows]) for i, w in ((0, "k"), (1, "v"))} | \
            {"lens": _ints([c + k for c, k in zip(ctx, s["counts"])])}
    if work(case)["flops"] > 4e12:
        return None
    out, lse, first = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), s["lse"].double(), 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        k, v = _cached64(s, b, torch.arange(n + c, device="cuda"))
        group = case["hq"] // k.shape[0]
        step = max(1, (1 << 26) // (n + c))
        for h in range(case["hq"]):
            for a in range(0, n, step):
                rows = torch.arange(a, min(n, a + step), device="cuda")
                score = torch.mm(s["q"][first + rows, h].double(), k[h // group].T).mul_(s["scale"])
                if s["cap"]:
                    score = torch.tanh(score / s["cap"]) * s["cap"]
                gap = (c + rows)[:, None] - torch.arange(n + c, device="cuda")
                if s["slopes"] is not None:
                    score -= s["slopes"][h].double() * gap.abs()
                hide = gap < 0
                if s["window"]:
                    hide |= gap >= s["window"]
                hide[:, : s["prefixes"][b]] = False
                score.masked_fill_(hide, -math.inf)
                total = torch.logsumexp(score, -1)
                out[first + rows, h] = torch.mm(torch.exp(score - total[:, None]), v[h // group])
                lse[first + rows, h] = total
        first += n
    return {"out": out, "lse": lse}
