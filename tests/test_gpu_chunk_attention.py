"""Attention of a chunk of new tokens over the paged, quantized cache, against the
64-bit oracle on the same codes.

Tolerances.  The codes and the rows of q enter exactly.  A score's error e_ij (the
oracle's chunk_attention says what it adds up) moves p_ij by e_ij and by the error of the
sum, sum p e, relative.  Rounding a probability to fp16 moves it by 2^-11, and by 2^-34 of
the row's largest where it becomes subnormal; sums over L tokens in float32 add at most L 2^-24,
exp, log and the scales a few 2^-22.  So out is within
  sum p e |v| + (sum p e + 2^-11 + (L + 64) 2^-24) sum p |v| + L 2^-34 max |v|
plus the final rounding, and lse within sum p e + (L + 64) 2^-24 + 2^-22 |lse|."""

import numpy as np
import pytest
import torch

from oracle import attention as kv
from oracle import serving as ref

pytestmark = pytest.mark.gpu

KIND = {"int8": torch.int8, "e4m3": torch.uint8, "u4": torch.uint8}


class Problem:
    """Sequences of (ctx, new) over a paged cache whose unused places hold NaN scales and any codes."""

    def __init__(self, q, seqs, hq, hk, d, page, fmt, dtype, seed=0, wide=0.5, softcap=0.0, slopes=None, window=0, prefix=None,
                 scale=None, spare_rows=0, size=1.5):
        gen = torch.Generator().manual_seed(seed * 1000 + d + page)
        self.q_, self.seqs, self.fmt, self.page, self.dtype = q, seqs, fmt, page, dtype
        per = [-(-(c + n) // page) for c, n in seqs]
        pages = sum(per) + 2
        order = torch.randperm(pages, generator=gen).int()
        self.table = torch.full((len(seqs), max(per, default=0) + 1), -3, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        x = torch.randn(2, pages, hk, page, d, generator=gen)
        x[0, ..., 1] *= 5
        x *= torch.exp(wide * torch.randn(2, pages, hk, page, 1, generator=gen))
        self.codes, self.scales = kv.kv_quantize(x.numpy(), fmt)
        live = np.zeros((pages, page), bool)
        for b, (c, n) in enumerate(seqs):
            p = np.arange(c + n)
            live[self.table[b, p // page].numpy(), p % page] = True
        dead = self.scales.copy()
        dead[:, np.broadcast_to(~live[:, None, :], (pages, hk, page))] = np.nan
        garbage = np.random.default_rng(seed).integers(0, 256, self.codes.shape).astype(self.codes.dtype)
        self.t = [torch.from_numpy(v.copy()).cuda() for v in (*np.where(live[None, :, None, :, None], self.codes, garbage), *dead)]
        self.cache = q.qlin_kv_cache(*self.t, {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[fmt])
        self.tq = sum(n for _, n in seqs)
        self.q = (size * torch.randn(self.tq + spare_rows, hq, d, generator=gen)).to(dtype)
        self.most = max([n for _, n in seqs] + [1])
        self.scale = d ** -0.5 if scale is None else scale
        self.how = dict(softcap=softcap, window=window, slopes=slopes, prefix=prefix)
        self.indptr = torch.tensor([0] + list(np.cumsum([n for _, n in seqs])), dtype=torch.int32)
        self.ctx = torch.tensor([c for c, _ in seqs], dtype=torch.int32)
        self.out = torch.full(self.q.shape, 3.0, dtype=dtype, device="cuda")
        self.lse = torch.full(self.q.shape[:2], 3.0, device="cuda")

    def prepare(self, q_dev=None, out=None, most=None):
        h, most = self.how, most or self.most
        n = self.q_.qlin_chunk_attention_workspace_bytes(self.cache, self.q.shape[1], most, len(self.seqs))
        self.dev = [t.cuda() for t in (self.table, self.indptr, self.ctx)]
        return self.q_.qlin_chunk_attention_prepare(
            self.q.cuda() if q_dev is None else q_dev, self.cache, *self.dev, self.out if out is None else out,
            torch.full((n,), 0xff, dtype=torch.uint8, device="cuda"), most, self.scale, h["softcap"],
            None if h["slopes"] is None else torch.tensor(h["slopes"], dtype=torch.float32, device="cuda"), h["window"],
            None if h["prefix"] is None else torch.tensor(h["prefix"], dtype=torch.int32, device="cuda"), self.lse)

    def run(self, **kw):
        self.prepare(**kw).run()
        torch.cuda.synchronize()
        assert self.q_.qlin_get_device_error() == 0
        return self

    def values(self, b):
        c, n = self.seqs[b]
        p = np.arange(c + n)
        pages = self.table[b, p // self.page].numpy()
        return [kv.kv_values(self.codes[i][pages, :, p % self.page], self.scales[i][pages, :, p % self.page], self.fmt) for i in range(2)]

    def check(self, only=None, out=None):
        out, lse = (self.out if out is None else out).double().cpu().numpy(), self.lse.double().cpu().numpy()
        half = torch.finfo(self.dtype).eps / 2
        for b, (c, n) in enumerate(self.seqs):
            if n == 0 or (only is not None and b not in only):
                continue
            k, v = self.values(b)
            a, h = int(self.indptr[b]), self.how
            prefix = 0 if h["prefix"] is None else min(max(h["prefix"][b], 0), c + n)
            o, l, w, moved, err = ref.chunk_attention(self.q[a:a + n].double().numpy(), k, v, c, self.scale, h["softcap"], h["slopes"],
                                                      h["window"], prefix)
            s = (c + n + 64) * 2.0 ** -24
            tol = moved + (err[..., None] + 2.0 ** -11 + s) * w + (c + n) * 2.0 ** -34 * np.abs(v).max()
            tol = tol + half * (np.abs(o) + tol) + 2.0 ** -25
            bad = ~(np.abs(out[a:a + n] - o) <= tol)
            assert not bad.any(), (b, c, n, np.argwhere(bad)[:4], np.abs(out[a:a + n] - o).max(), bad.sum())
            bad = ~(np.abs(lse[a:a + n] - l) <= err + s + 2.0 ** -22 * np.abs(l))
            assert not bad.any(), (b, c, n, np.argwhere(bad)[:4], np.abs(lse[a:a + n] - l).max())
        assert (out[self.tq:] == 3).all() and (lse[self.tq:] == 3).all()   # rows behind the last sequence
        return self


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hk,d,page", [(1, 1, 64, 16), (4, 4, 128, 32), (8, 2, 128, 64), (10, 2, 64, 128), (8, 1, 256, 16), (3, 3, 256, 256)])
def test_shapes(qlin_gpu, fmt, dtype, hq, hk, d, page):
    """Every format, type, group and head size; lengths around a tile's borders, one token and none among them."""
    seqs = [(0, 1), (0, 130), (127, 1), (128, 65), (5, 0), (300, 257), (255, 3)]
    Problem(qlin_gpu, seqs, hq, hk, d, page, fmt, dtype, spare_rows=3).run().check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("how", [dict(softcap=5.0), dict(window=1), dict(window=100), dict(prefix=[0, 129, 600, 7, -5]),
                                 dict(window=37, prefix=[1, 260, 10 ** 6, 64, 0]), dict(slopes=[0.5, 0.03]),
                                 dict(softcap=20.0, slopes=[-0.01, 1.0], window=200, prefix=[50, 5, 5, 400, 3])])
def test_scores(qlin_gpu, fmt, d, how):
    """Caps, windows, prefixes and biases, alone and together."""
    seqs = [(0, 140), (200, 70), (10, 300), (515, 33), (129, 1)]
    dtype = torch.bfloat16 if d == 128 else torch.float16
    Problem(qlin_gpu, seqs, 2, 1, d, 32, fmt, dtype, seed=d, **how).run().check()


@pytest.mark.parametrize("fmt,d,hq,hk", [("int8", 128, 8, 2), ("u4", 64, 4, 4), ("e4m3", 256, 4, 2)])
def test_longer(qlin_gpu, fmt, d, hq, hk):
    """Chunks of many tiles, split among blocks, beside single tokens over long contexts."""
    Problem(qlin_gpu, [(1000, 700), (5003, 1), (0, 1500), (3000, 17)], hq, hk, d, 64, fmt, torch.bfloat16).run().check()


def test_few_rows_over_long_contexts(qlin_gpu):
    for seqs in ([(20000, 1)], [(20000, 3), (1, 1)]):
        Problem(qlin_gpu, seqs, 4, 2, 128, 64, "int8", torch.float16, slopes=[0.001, 0.0, -0.0001, 0.1]).run().check()


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -9, 2.0 ** 6, 2.0 ** 40])
def test_rows_of_any_size(qlin_gpu, size):
    """bf16 rows far beyond fp16's range, with the scale that makes scores of them ordinary ones."""
    Problem(qlin_gpu, [(100, 140)], 4, 2, 128, 16, "e4m3", torch.bfloat16, size=1.5 * size, scale=0.09 / size).run().check()


def test_scores_far_apart(qlin_gpu):
    """Scores of some hundreds: one token takes all of a row, the reference moves far and often."""
    Problem(qlin_gpu, [(900, 200)], 4, 2, 128, 16, "int8", torch.float16, scale=2.0, wide=1.0).run().check()


def test_strided_rows(qlin_gpu):
    """q as part of fused q/k/v rows, out as heads-first storage."""
    p = Problem(qlin_gpu, [(50, 200), (0, 31)], 8, 2, 128, 32, "int8", torch.float16)
    whole = torch.zeros(p.tq, 12, 128, dtype=torch.float16, device="cuda")
    whole[:, :8] = p.q.cuda()
    out = torch.full((8, p.tq, 128), 3.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    p.run(q_dev=whole[:, :8], out=out).check(out=out)


def test_odd_scales(qlin_gpu):
    """Value and key scales of zero, below zero, very small and very large."""
    for fmt in ("int8", "e4m3", "u4"):
        p = Problem(qlin_gpu, [(200, 150)], 4, 2, 128, 16, fmt, torch.bfloat16, window=90, prefix=[20])
        r = np.random.default_rng(1)
        for i in range(2):
            s = p.scales[i][..., 0] if fmt == "u4" else p.scales[i]
            pick = r.random(s.shape)
            s[pick < 0.1] *= -1
            s[(pick > 0.1) & (pick < 0.15)] = 0
            s[(pick > 0.15) & (pick < 0.2)] *= 2.0 ** -12
        p.t = [torch.from_numpy(v.copy()).cuda() for v in (*p.codes, *p.scales)]
        p.cache = qlin_gpu.qlin_kv_cache(*p.t, p.cache.fmt)
        p.run().check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_what_is_not_seen_does_not_reach_a_row(qlin_gpu, fmt, which):
    """Scales (zero-points, E4M3 value codes) that are not numbers: rows that see such a token are NaN, others are not touched."""
    p = Problem(qlin_gpu, [(130, 200)], 4, 2, 128, 16, fmt, torch.float16, window=60, prefix=[9]).run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    bad = [40, 131, 132, 250, 329]
    kinds = ["scale"] + (["zero"] if fmt == "u4" else []) + (["code"] if fmt == "e4m3" else [])
    at, j = 130 + np.arange(200)[:, None], np.array(bad)
    hit = torch.from_numpy(((j <= at) & (at - j < 60)).any(1)).cuda()
    for kind in kinds:
        t = [x.clone() for x in p.t]
        i = 0 if which == "k" else 1
        for token in bad:
            page, off = int(p.table[0, token // 16]), token % 16
            if kind == "code":
                t[i][page, :, off, 5] = 0x7f if token % 2 else 0xff
            elif fmt == "u4":
                t[2 + i][page, :, off, 0 if kind == "scale" else 1] = float("nan") if kind == "scale" else 7.5
            else:
                t[2 + i][page, :, off] = float("nan")
        p.cache = qlin_gpu.qlin_kv_cache(*t, p.cache.fmt)
        p.run()
        assert bool(torch.isnan(p.out[hit]).flatten(1).any(1).all())
        assert torch.equal(p.out[~hit], clean[~hit]) and torch.equal(p.lse[~hit], clean_lse[~hit])


def test_pages_out_of_range_are_zeros(qlin_gpu):
    """Tokens on a page that is none count as keys and values of zero, and are recorded."""
    p = Problem(qlin_gpu, [(100, 60), (40, 9)], 4, 2, 128, 16, "int8", torch.float16)
    page = int(p.table[0, 3])
    p.codes[:, page] = 0
    p.table[0, 3] = 10 ** 6
    p.prepare().run()
    torch.cuda.synchronize()
    assert qlin_gpu.qlin_get_device_error() == 0x2000
    p.table[0, 3] = page
    p.check()


@pytest.mark.parametrize("change", ["ctx", "long", "order", "past", "most"])
def test_bounds_that_do_not_fit(qlin_gpu, change):
    """A sequence whose bounds are out of range is recorded and left out; the others are as they were."""
    p = Problem(qlin_gpu, [(20, 30), (100, 40), (7, 50)], 4, 2, 64, 16, "int8", torch.float16)
    want, most = [0, 2], p.most
    if change == "ctx":
        p.ctx[1] = -1
    elif change == "long":
        p.ctx[1] = 16 * p.table.shape[1] - 39
    elif change == "order":
        p.indptr[2], want = 10, [0]
    elif change == "past":
        p.indptr[3], want = 121, [0, 1]
    else:
        most, want = 40, [0, 1]
    p.prepare(most=most).run()
    torch.cuda.synchronize()
    assert qlin_gpu.qlin_get_device_error() == 0x2000
    p.ctx[1] = 100
    p.indptr = torch.tensor([0, 30, 70, 120], dtype=torch.int32)
    p.check(only=want)
    if change != "order":
        left = ({0, 1, 2} - set(want)).pop()
        assert (p.out[p.indptr[left]:p.indptr[left + 1]] == 3).all() and (p.lse[p.indptr[left]:p.indptr[left + 1]] == 3).all()


def test_the_same_twice(qlin_gpu):
    p = Problem(qlin_gpu, [(1000, 300), (77, 1), (0, 513)], 8, 2, 128, 64, "int8", torch.bfloat16)
    a = p.run().out.clone()
    for _ in range(3):
        p.out.fill_(3.0)
        assert torch.equal(a, p.run().out)


def test_replays_with_other_lengths_and_another_stream(qlin_gpu):
    """A captured call reads lengths, bounds and pages at every replay; a prepared one runs on any stream."""
    q = qlin_gpu
    first = Problem(q, [(300, 200), (10, 40), (0, 60)], 4, 2, 128, 16, "int8", torch.float16, seed=1, window=150, prefix=[3, 0, 8])
    call = first.prepare()
    dev, side = first.dev, torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.run(side)
    torch.cuda.current_stream().wait_stream(side)
    first.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for seqs in ([(0, 100), (33, 100), (200, 100)], [(470, 1), (0, 0), (1, 100)]):
        first.out.fill_(3.0)
        first.lse.fill_(3.0)
        first.seqs, first.tq = seqs, sum(n for _, n in seqs)
        first.indptr = torch.tensor([0] + list(np.cumsum([n for _, n in seqs])), dtype=torch.int32)
        first.ctx = torch.tensor([c for c, _ in seqs], dtype=torch.int32)
        # one table for all: the first sequence's pages
        first.table = first.table[:1].expand(3, -1).contiguous()
        dev[0].copy_(first.table)
        dev[1].copy_(first.indptr)
        dev[2].copy_(first.ctx)
        graph.replay()
        torch.cuda.synchronize()
        assert q.qlin_get_device_error() == 0
        first.check()


def test_as_attention_of_a_chain(qlin_gpu):
    """Up to 256 new tokens it answers as tree attention of chains does, within both tolerances' roundings."""
    q = qlin_gpu
    p = Problem(q, [(500, 100), (64, 7)], 8, 2, 128, 16, "e4m3", torch.float16).run().check()
    out, lse = torch.zeros_like(p.out), torch.zeros_like(p.lse)
    ws = torch.empty(q.qlin_tree_attention_workspace_bytes(p.cache, 8, 100, 2), dtype=torch.uint8, device="cuda")
    q.qlin_tree_attention(p.q.cuda(), p.cache, *p.dev, None, out, ws, 100, scale=p.scale, lse=lse)
    p.out, p.lse = out, lse
    p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("hq,hk,d,most", [(8, 8, 128, 1), (8, 2, 128, 4), (32, 2, 64, 1), (10, 2, 256, 3), (10, 2, 256, 4), (3, 1, 64, 6), (8, 2, 128, 9),
                                            (8, 8, 64, 64), (8, 8, 128, 65)])
def test_few_rows(qlin_gpu, fmt, hq, hk, d, most):
    """Single tokens and a few of them, as a decode step has them, on both sides of 16 and of 64 rows per key head."""
    seqs = [(0, 1), (700, most), (16, 0), (127, 1), (128, most), (2100, 1), (5, most)]
    for dtype in (torch.float16, torch.bfloat16):
        Problem(qlin_gpu, seqs, hq, hk, d, 16, fmt, dtype, spare_rows=2).run().check()
    # a call planned for more, and one with a window that takes everything
    Problem(qlin_gpu, seqs, hq, hk, d, 16, fmt, torch.float16, spare_rows=2).run(most=300).check()
    Problem(qlin_gpu, seqs, hq, hk, d, 16, fmt, torch.float16, spare_rows=2, window=2 ** 31 - 1).run().check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("hq,hk,d,most,page", [(4, 4, 128, 1, 64), (8, 2, 64, 4, 16), (5, 1, 256, 3, 128), (2, 1, 128, 8, 32)])
@pytest.mark.parametrize("how", [dict(softcap=5.0), dict(window=1), dict(window=100), dict(window=33, prefix=[1, 260, 10 ** 6, 64, 0, 30, 95]),
                                 dict(prefix=[0, 2100, 3, 7, -5, 1, 96]), dict(slopes=True), dict(window=64, prefix=[0, 64, 128, 0, 32, 0, 128]),
                                 dict(softcap=20.0, slopes=True, window=700, prefix=[50, 5, 5, 400, 3, 0, 1000])])
def test_scores_of_few_rows(qlin_gpu, fmt, hq, hk, d, most, page, how):
    """Caps, windows, prefixes and biases of a decode step's rows; windows that leave whole tiles out, behind a prefix and without."""
    seqs = [(0, most), (2100, most), (127, 1), (600, most), (16, 0), (31, 1), (999, most)]
    how = dict(how, slopes=[0.3 * (-0.5) ** h for h in range(hq)]) if how.get("slopes") else how
    for dtype in (torch.float16, torch.bfloat16):
        Problem(qlin_gpu, seqs, hq, hk, d, page, fmt, dtype, seed=most, spare_rows=1, **how).run().check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_what_a_window_of_few_rows_hides(qlin_gpu, fmt, which):
    """Tokens that are no numbers on either side of a window's edge, in a tile that rows see part of; pages of whole tiles
    that nobody sees are not looked at."""
    p = Problem(qlin_gpu, [(300, 4)], 4, 2, 128, 16, fmt, torch.float16, window=60, prefix=[9]).run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    at, bad = 300 + np.arange(4)[:, None], np.array([20, 241, 242, 302])
    for kind in ["scale"] + (["zero"] if fmt == "u4" else []) + (["code"] if fmt == "e4m3" else []):
        for token in bad.tolist():
            t = [x.clone() for x in p.t]
            i, (page, off) = 0 if which == "k" else 1, (int(p.table[0, token // 16]), token % 16)
            if kind == "code":
                t[i][page, :, off, 5] = 0x7f
            elif fmt == "u4":
                t[2 + i][page, :, off, 0 if kind == "scale" else 1] = float("nan") if kind == "scale" else 7.5
            else:
                t[2 + i][page, :, off] = float("nan")
            p.cache = qlin_gpu.qlin_kv_cache(*t, p.cache.fmt)
            p.run()
            hit = torch.from_numpy(((token <= at) & (at - token < 60))[:, 0]).cuda()
            assert bool(torch.isnan(p.out[hit]).flatten(1).any(1).all()), (kind, token)
            assert torch.equal(p.out[~hit], clean[~hit]) and torch.equal(p.lse[~hit], clean_lse[~hit]), (kind, token)
    p.cache = qlin_gpu.qlin_kv_cache(*p.t, p.cache.fmt)
    p.table[0, 3:14] = -7   # tokens 48 .. 223
    p.run()
    assert torch.equal(p.out, clean) and torch.equal(p.lse, clean_lse)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_what_few_rows_do_not_see(qlin_gpu, fmt, which):
    """As above for calls of few rows: a token that is no number reaches the rows from its own on."""
    p = Problem(qlin_gpu, [(130, 5)], 4, 2, 128, 16, fmt, torch.float16).run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    for kind in ["scale"] + (["zero"] if fmt == "u4" else []) + (["code"] if fmt == "e4m3" else []):
        t = [x.clone() for x in p.t]
        i, (page, off) = 0 if which == "k" else 1, (int(p.table[0, 132 // 16]), 132 % 16)
        if kind == "code":
            t[i][page, :, off, 5] = 0x7f
        elif fmt == "u4":
            t[2 + i][page, :, off, 0 if kind == "scale" else 1] = float("nan") if kind == "scale" else 7.5
        else:
            t[2 + i][page, :, off] = float("nan")
        p.cache = qlin_gpu.qlin_kv_cache(*t, p.cache.fmt)
        p.run()
        assert bool(torch.isnan(p.out[2:]).flatten(1).any(1).all()), kind
        assert torch.equal(p.out[:2], clean[:2]) and torch.equal(p.lse[:2], clean_lse[:2]), kind


@pytest.mark.parametrize("seqs,new", [(200, 1), (200, 9), (33, 70), (1, 1)])
def test_many_sequences(qlin_gpu, seqs, new):
    """Batches whose sequences a block counts side by side, long and short ones in turn; also those with none at all."""
    r = np.random.default_rng(seqs + new)
    which = [(int(r.integers(0, 400)), int(r.integers(0, new + 1)) if b % 17 else 260) for b in range(seqs)]
    Problem(qlin_gpu, which, 8, 2, 64, 32, "int8", torch.float16, window=0 if new > 1 else 300, spare_rows=1).run().check()


def test_no_new_tokens(qlin_gpu):
    p = Problem(qlin_gpu, [(100, 3), (40, 5)], 4, 2, 128, 16, "int8", torch.float16, window=50)
    p.indptr = torch.zeros(3, dtype=torch.int32)
    p.run()
    assert (p.out == 3).all() and (p.lse == 3).all()


@pytest.mark.parametrize("fmt", ["int8", "u4"])
def test_scales_of_the_scores(qlin_gpu, fmt):
    """Zero and negative scales; the widest window; a prefix of everything; a row far behind the first of a long chunk."""
    for scale in (0.0, -0.05):
        Problem(qlin_gpu, [(100, 140)], 4, 2, 128, 16, fmt, torch.bfloat16, scale=scale, softcap=3.0).run().check()
    Problem(qlin_gpu, [(1, 700)], 4, 2, 64, 16, fmt, torch.float16, window=2 ** 31 - 65537, prefix=[701]).run().check()


@pytest.mark.parametrize("d,most", [(128, 1), (256, 60), (64, 300)])
def test_two_calls_on_two_streams(qlin_gpu, d, most):
    """Calls with workspaces of their own run side by side; a captured and a plain one of the same data too."""
    q = qlin_gpu
    a = Problem(q, [(900, most), (30, 1)], 8, 2, d, 16, "int8", torch.float16, seed=1)
    b = Problem(q, [(5, 1), (1500, most)], 8, 2, d, 16, "e4m3", torch.bfloat16, seed=2)
    calls, streams = [a.prepare(), b.prepare()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls[0].run()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        calls[1].run(streams[1])
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
    a.check()
    b.check()


def test_rows_of_infinity(qlin_gpu):
    """A row of q with an infinity or a NaN reaches no other row."""
    for dtype in (torch.float16, torch.bfloat16):
        p = Problem(qlin_gpu, [(60, 150)], 4, 2, 128, 16, "int8", dtype).run()
        clean, clean_lse = p.out.clone(), p.lse.clone()
        p.q[7, 1, 5], p.q[80, 3, 0], p.q[149, 0, 127] = float("inf"), float("nan"), -float("inf")
        p.run()
        hit = torch.zeros(p.q.shape[:2], dtype=torch.bool)
        hit[7, 1] = hit[80, 3] = hit[149, 0] = True
        assert torch.equal(p.out[~hit.cuda()], clean[~hit.cuda()]) and torch.equal(p.lse[~hit.cuda()], clean_lse[~hit.cuda()])
        assert not torch.isfinite(p.out[hit.cuda()]).all()


def test_a_cache_beyond_32_bits(qlin_gpu):
    """Pages whose bytes and scales lie beyond 2^32 bytes, at the end of a large cache."""
    q, hk, d, page, n = qlin_gpu, 2, 128, 64, 70
    pages = (2 ** 32 + 2 ** 28) // (hk * page * d)
    kv_ = [torch.zeros(pages, hk, page, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    sc = [torch.zeros(pages, hk, page, device="cuda") for _ in range(2)]
    p = Problem(q, [(300, n), (17, 1)], 8, hk, d, page, "int8", torch.float16)
    some = p.t[0].shape[0]
    first = pages - some
    for big, small in zip((*kv_, *sc), p.t):
        big[first:] = small
    p.cache = q.qlin_kv_cache(*kv_, *sc, q.QLIN_KV_INT8)
    near = p.table.clone()
    p.table = torch.where(near >= 0, near + first, near)
    p.run()
    p.table = near
    p.check()


@pytest.mark.parametrize("d,n", [(128, 1), (64, 5), (256, 30), (128, 200)])
def test_the_longest_sequence(qlin_gpu, d, n):
    """A window and a prefix at the end of a sequence of 2^31 - 2^16 tokens, which seven pages hold in turn: the same as
    those tokens alone; one token more is recorded."""
    q, page, window, prefix, length = qlin_gpu, 256, 300, 5, 0x7fff0000
    p = Problem(q, [(prefix + window - 1, n)], 2, 1, d, page, "int8", torch.float16, window=window, prefix=[prefix])
    ctx = length - n
    # the same tokens, each where the long sequence has it: seven pages, filled from the short one's
    j = np.concatenate([np.arange(prefix), ctx - window + 1 + np.arange(window - 1 + n)])
    at = np.arange(prefix + window - 1 + n)
    src = p.table[0, at // page].numpy(), at % page
    t = []
    for x in (*p.codes, *p.scales):
        y = np.zeros((7,) + x.shape[1:], x.dtype)
        y[(j // page) % 7, :, j % page] = x[src[0], :, src[1]]
        t.append(torch.from_numpy(y).cuda())
    assert len(set(zip((j // page % 7).tolist(), (j % page).tolist()))) == len(j)
    p.cache = q.qlin_kv_cache(*t, q.QLIN_KV_INT8)
    short, seqs = p.table, p.seqs
    p.table = (torch.arange(-(-(length + 1) // page), dtype=torch.int32) % 7)[None]
    p.ctx = torch.tensor([ctx], dtype=torch.int32)
    p.run()
    p.table, p.seqs = short, seqs
    p.check()
    p.ctx[0] = ctx + 1
    p.table = (torch.arange(-(-(length + 1) // page), dtype=torch.int32) % 7)[None]
    p.prepare().run()
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0x2000


@pytest.mark.parametrize("fmt,seqs,slopes", [("e4m3", [(700, 257), (311, 130), (64, 200)], None), ("int8", [(6000, 9)], [0.2, 0.1, 0.3, 0.4]),
                                             ("u4", [(900, 33), (5, 70), (2000, 40)], None)])
def test_streams_without_rows(qlin_gpu, fmt, seqs, slopes):
    """Tiles of which one of the two halves of rows has none, or none that sees the tile, over and over: no wait runs out and
    every pass gives the same."""
    p = Problem(qlin_gpu, seqs, 4, 1, 128, 16, fmt, torch.float16, slopes=slopes)
    call = p.prepare()
    call.run()
    torch.cuda.synchronize()
    p.check()
    want = p.out.clone()
    for _ in range(20):
        for _ in range(50):
            call.run()
        torch.cuda.synchronize()
        assert qlin_gpu.qlin_get_device_error() == 0 and torch.equal(p.out, want)


# Batches of which every segment is one block's (many sequences of one tile, or several tiles a block), and such as are cut
# between blocks; of rows beyond those that the kernel of few rows takes, and of its own.
CUTS = [([(0, 100)], 100), ([(0, 70)] * 3 + [(3, 66)], 70), ([(0, 40), (20, 65)] * 150, 65), ([(700, 300)], 300), ([(0, 4), (200, 3)], 4)]


def _with_key(p, token, value, code=None):
    """The cache with another scale (and code) of sequence 0's key `token`, all heads."""
    t = [x.clone() for x in p.t]
    page, off = int(p.table[0, token // p.page]), token % p.page
    if p.fmt == "u4":
        t[2][page, :, off, 0] = value
    else:
        t[2][page, :, off] = value
    if code is not None:
        t[0][page, :, off] = code
    return p.q_.qlin_kv_cache(*t, p.cache.fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("seqs,most", CUTS)
def test_rows_that_are_no_numbers(qlin_gpu, fmt, d, seqs, most):
    """A row whose only scores are NaN is NaN, out and lse, whoever has its segment: from its q, from a key that it sees alone."""
    for window, hit_of in ((0, "q"), (0, "key"), (1, "key")):
        p = Problem(qlin_gpu, seqs, 4, 2, d, 16, fmt, torch.float16, window=window).run()
        clean, clean_lse = p.out.clone(), p.lse.clone()
        c, n = seqs[0]
        hit = torch.zeros(p.q.shape[:2], dtype=torch.bool)
        if hit_of == "q":
            p.q[0, 0, 3] = p.q[n - 1, 1, d - 1] = p.q[n // 2, 3, 0] = p.q[p.tq - 1, 2, 1] = float("nan")
            hit[0, 0] = hit[n - 1, 1] = hit[n // 2, 3] = hit[p.tq - 1, 2] = True
        else:
            token = c + (n // 2 if window else 0)        # (without a window and a context: all that row 0 sees)
            p.cache = _with_key(p, token, float("nan"))
            hit[token - c:token - c + 1 if window else n] = True
        p.run()
        hit = hit.cuda()
        assert bool(torch.isnan(p.out[hit]).all()) and bool(torch.isnan(p.lse[hit]).all())
        assert torch.equal(p.out[~hit], clean[~hit]) and torch.equal(p.lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("seqs,most", CUTS)
def test_rows_of_minus_infinity(qlin_gpu, d, seqs, most):
    """A row whose only score is -infinity: 0 and -infinity, whoever has its segment."""
    p = Problem(qlin_gpu, seqs, 4, 2, d, 16, "int8", torch.float16, window=1)
    p.q.abs_()
    p.run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    c, n = seqs[0]
    for row in (0, n // 2, n - 1):
        p.cache = _with_key(p, c + row, float("inf"), -7)
        p.run()
        hit = torch.zeros(len(p.q), dtype=torch.bool, device="cuda")
        hit[row] = True
        assert not p.out[hit].any() and bool((p.lse[hit] == -float("inf")).all())
        assert torch.equal(p.out[~hit], clean[~hit]) and torch.equal(p.lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap", [256.0, 257.0, 1e3, 3e4, 1e6])
def test_large_caps(qlin_gpu, fmt, d, cap):
    """Caps far above the scores leave them as they are, to float32's own precision; scores around the cap, and beyond it.  Tiles of
    rows, and few rows."""
    for scale in (None, 0.2 * cap * d ** -0.5, 2 * cap * d ** -0.5):
        if scale is not None and cap > 1e3:
            continue      # (float32 products of that size say nothing)
        for seqs in ([(0, 140), (200, 70), (515, 33)], [(300, 3), (0, 2)]):
            Problem(qlin_gpu, seqs, 2, 1, d, 32, fmt, torch.float16, seed=d, softcap=cap, scale=scale,
                    slopes=[0.5, 0.03] if d == 64 else None, wide=0.2, size=0.5).run().check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("d,n", [(64, 200), (128, 200), (256, 200), (128, 4)])
@pytest.mark.parametrize("page", [16, 64])
def test_what_every_window_has_left(qlin_gpu, fmt, d, n, page):
    """Tokens between a prefix and the first row's window, on pages that may hold anything by now: scales of any size change
    nothing, and page numbers that are none are not looked at (in a tile of which rows see a part)."""
    seqs = [(200, n), (300, n)]
    p = Problem(qlin_gpu, seqs, 4, 2, d, page, fmt, torch.bfloat16, window=60, prefix=[9, 0]).run().check()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    left = [(b, j // page) for b, (c, _) in enumerate(seqs) for j in range(0, c - 59 - page + 1, page) if j >= p.how["prefix"][b]]
    assert len(left) >= 4
    for scale in ([6e4, -6e4] if fmt == "u4" else [2.0 ** 40, 3e38, -3e38]):
        t = [x.clone() for x in p.t]
        for b, i in left:
            x = t[3][int(p.table[b, i])]
            (x[..., 0] if fmt == "u4" else x).fill_(scale)
        p.cache = qlin_gpu.qlin_kv_cache(*t, p.cache.fmt)
        p.run().check()
        assert torch.equal(p.out, clean) and torch.equal(p.lse, clean_lse)
    for b, i in left:
        p.table[b, i] = -5
    p.prepare().run()
    torch.cuda.synchronize()
    assert torch.equal(p.out, clean) and qlin_gpu.qlin_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("up", [6, 12, 18])
def test_large_scales_that_only_later_rows_see(qlin_gpu, fmt, d, up):
    """A value scale 2^up above the others': rows before its token keep theirs down to 2^-34 of the largest value of the tile."""
    p = Problem(qlin_gpu, [(130, 200)], 4, 2, d, 16, fmt, torch.bfloat16)
    for token in (230, 231, 300):
        page, off = int(p.table[0, token // 16]), token % 16
        p.scales[1][page, :, off] *= 2.0 ** up
    t = [x.clone() for x in p.t]
    t[3] = torch.from_numpy(p.scales[1].copy()).cuda()
    p.cache = qlin_gpu.qlin_kv_cache(*t, p.cache.fmt)
    p.run().check()
