"""Attention of new tokens (one, a chain, a tree of drafts) over the paged,
quantized cache, against the 64-bit oracle on the same codes.

Tolerances.  The codes enter exactly.  A score is a float32 sum of D products
(at most D roundings of 2^-24 of sum |q k|) times float32 scales; its error e
moves a probability by 2 e relative (numerator and denominator).  Rounding a
probability to fp16 moves it by 2^-11.  Sums over L tokens in float32 add at
most L 2^-24, exp and the scales a few 2^-22.  So out is within
(2^-11 + 2 e + (L + 64) 2^-24) sum p |v|, plus the final rounding, and lse
within e + (L + 64) 2^-24 + 2^-22 |lse|."""

import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

KIND = {"int8": torch.int8, "e4m3": torch.uint8, "u4": torch.uint8}


def _fmt(q, fmt):
    return {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[fmt]


class Problem:
    """Sequences of (ctx, nodes) over a paged cache whose unused places hold NaN scales and arbitrary codes."""

    def __init__(self, q, seqs, hq, hk, d, page, fmt, dtype, mask="tree", seed=0, wide=1.0, max_nodes=None, spare=2):
        gen = torch.Generator().manual_seed(seed * 1000 + d + page)
        self.q_, self.seqs, self.fmt, self.page, self.dtype = q, seqs, fmt, page, dtype
        per = [-(-(c + n) // page) for c, n in seqs]
        pages = sum(per) + spare
        order = torch.randperm(pages, generator=gen).int()
        self.table = torch.full((len(seqs), max(per, default=0) + 1), -3, dtype=torch.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        x = torch.randn(2, pages, hk, page, d, generator=gen)
        x[0, ..., 1] *= 5
        x *= torch.exp(wide * torch.randn(2, pages, hk, page, 1, generator=gen) * 0.5)
        self.codes, self.scales = ref.kv_quantize(x.numpy(), fmt)
        # what no sequence has reached: scales that are not numbers
        live = np.zeros((pages, page), bool)
        for b, (c, n) in enumerate(seqs):
            p = np.arange(c + n)
            live[self.table[b, p // page].numpy(), p % page] = True
        dead = self.scales.copy()
        dead[:, np.broadcast_to(~live[:, None, :], (pages, hk, page))] = np.nan
        garbage = np.random.default_rng(seed).integers(0, 256, self.codes.shape).astype(self.codes.dtype)
        self.codes_dev = np.where(live[None, :, None, :, None], self.codes, garbage)
        self.t = [torch.from_numpy(v.copy()).cuda() for v in (*self.codes_dev, *dead)]
        self.cache = q.qlin_kv_cache(*self.t, _fmt(q, fmt))
        tq = sum(n for _, n in seqs)
        self.nodes = max_nodes or max([n for _, n in seqs] + [1])
        self.q = (1.5 * torch.randn(tq, hq, d, generator=gen)).to(dtype)
        words = (self.nodes + 63) // 64
        self.bits = None
        if mask != "chain":
            self.bits = np.zeros((tq, words * 64), bool)
            r = np.random.default_rng(seed + 5)
            row = 0
            for _, n in seqs:
                for i in range(n):
                    if mask == "tree":
                        par = int(r.integers(max(0, i - 5), i)) if i else -1
                        if par >= 0:
                            self.bits[row + i] = self.bits[row + par]
                        self.bits[row + i, i] = True
                    elif mask == "random":
                        self.bits[row + i, :n] = r.random(n) < 0.4
                        self.bits[row + i, n:] = True       # bits of nodes that are not there mean nothing
                    elif mask == "none" and i % 2:
                        self.bits[row + i, i] = True        # every other node sees no node at all
                row += n
        self.mask = None if self.bits is None else torch.from_numpy(
            np.packbits(self.bits, axis=1, bitorder="little").view(np.int64).copy()).cuda()
        self.indptr = torch.tensor([0] + list(np.cumsum([n for _, n in seqs])), dtype=torch.int32)
        self.ctx = torch.tensor([c for c, _ in seqs], dtype=torch.int32)
        self.scale = d ** -0.5

    def run(self, q_dev=None, out=None, stream=None, lse=True):
        q = self.q_
        qd = self.q.cuda() if q_dev is None else q_dev
        self.out = torch.full(self.q.shape, 3.0, dtype=self.dtype, device="cuda") if out is None else out
        self.lse = torch.full(self.q.shape[:2], 3.0, device="cuda") if lse else None
        ws = torch.full((q.qlin_tree_attention_workspace_bytes(self.cache, qd.shape[1], self.nodes, len(self.seqs)),), 255,
                        dtype=torch.uint8, device="cuda")
        self.call = q.qlin_tree_attention_prepare(qd, self.cache, self.table.cuda(), self.indptr.cuda(), self.ctx.cuda(),
                                                  self.mask, self.out, ws, self.nodes, scale=self.scale, lse=self.lse)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        self.call.run(stream)
        torch.cuda.synchronize()
        return self.out, self.lse

    def check(self, error=0):
        assert self.q_.qlin_get_device_error() == error
        row = 0
        eps = torch.finfo(self.dtype).eps / 2
        tiny = torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps
        out = self.out.double().cpu().numpy()
        lse = None if self.lse is None else self.lse.double().cpu().numpy()
        for b, (c, n) in enumerate(self.seqs):
            p = np.arange(c + n)
            pg = self.table[b, p // self.page].numpy()
            k, v = (ref.kv_values(self.codes[i][pg, :, p % self.page], self.scales[i][pg, :, p % self.page], self.fmt) for i in range(2))
            seen = np.ones((n, c + n), bool)
            seen[:, c:] = np.tril(np.ones((n, n), bool)) if self.bits is None else self.bits[row:row + n, :n]
            o, l, w, spread = ref.tree_attention(self.q[row:row + n].double().numpy(), k, v, seen, self.scale)
            e = self.q.shape[2] * 2.0 ** -24 * spread
            s = (c + n + 64) * 2.0 ** -24
            tol = (2.0 ** -11 + 2 * e + s)[..., None] * w + eps * np.abs(o) + tiny
            bad = ~(np.abs(out[row:row + n] - o) <= tol)
            assert not bad.any(), "sequence %d (%d, %d): %d outputs off, worst %g of a tolerance" % (
                b, c, n, bad.sum(), np.nanmax(np.abs(out[row:row + n] - o) / tol))
            if lse is not None:
                y = lse[row:row + n]
                with np.errstate(invalid="ignore"):
                    near = (np.abs(y - l) <= e + s + 2.0 ** -22 * np.abs(l)) | (y == l)
                assert near.all(), "sequence %d: lse off by %g" % (b, np.nanmax(np.abs(y - l)))
            row += n


SHAPES = [  # (sequences of (ctx, nodes)), hq, hk, d, page
    ([(0, 1)], 1, 1, 64, 16),
    ([(1, 1)], 8, 8, 128, 16),
    ([(500, 1)], 32, 4, 128, 16),
    ([(63, 1), (64, 1), (65, 1), (0, 1), (127, 1), (128, 1)], 8, 2, 128, 64),
    ([(1000, 5)], 5, 1, 128, 32),
    ([(77, 16), (3, 1), (300, 9), (0, 16)], 8, 2, 64, 32),
    ([(131, 33)], 16, 2, 128, 128),
    ([(40, 64), (700, 50)], 16, 2, 128, 16),
    ([(90, 7), (2, 20)], 6, 2, 256, 256),
    ([(200, 3)], 4, 4, 256, 64),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(qlin_gpu, fmt, dtype, shape):
    seqs, hq, hk, d, page = SHAPES[shape]
    p = Problem(qlin_gpu, seqs, hq, hk, d, page, fmt, dtype, "tree", shape)
    p.run()
    p.check()


@pytest.mark.parametrize("mask", ["chain", "random", "none"])
@pytest.mark.parametrize("d,nodes", [(64, 13), (128, 64), (128, 65), (128, 200), (256, 30)])
def test_masks(qlin_gpu, mask, d, nodes):
    """Chains, arbitrary masks, nodes that see no node; without cached tokens some rows see nothing at all."""
    p = Problem(qlin_gpu, [(0, nodes), (100, nodes - 1), (0, 1), (64, nodes)], 8, 2, d, 32, "int8", torch.float16, mask, nodes)
    out, lse = p.run()
    p.check()
    if mask == "none":
        assert not (out[0] != 0).any() and torch.isneginf(lse[0]).all()


def test_empty_problems(qlin_gpu):
    """Sequences without nodes between others; no rows; no sequences; more room for nodes than there are."""
    p = Problem(qlin_gpu, [(10, 0), (300, 2), (0, 0), (5, 0), (70, 1)], 4, 2, 128, 16, "e4m3", torch.float16, "tree", 1, max_nodes=100)
    p.run()
    p.check()
    p = Problem(qlin_gpu, [(10, 0), (3, 0)], 4, 2, 128, 16, "e4m3", torch.float16, "chain", 1)
    p.run()
    p.check()


def test_long_context(qlin_gpu):
    """Many pieces of one sequence joined; a key far above the rest at either end."""
    p = Problem(qlin_gpu, [(9001, 3), (4000, 1)], 4, 1, 128, 64, "int8", torch.bfloat16, "tree", 8)
    p.run()
    p.check()
    for at in (0, 9002):
        p = Problem(qlin_gpu, [(9001, 3)], 4, 1, 128, 64, "e4m3", torch.float16, "random", 9)
        page, off = int(p.table[0, at // 64]), at % 64
        for s in (p.scales, ):
            s[0][page, :, off] *= 30
            s[1][page, :, off] *= 2.0 ** -12         # its value row is tiny beside the others'
        p.t[2][page, :, off] *= 30
        p.t[3][page, :, off] *= 2.0 ** -12
        p.run()
        p.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
def test_what_is_hidden_does_not_matter(qlin_gpu, fmt):
    """A node whose key and value rows are NaN reaches only the rows that see it."""
    p = Problem(qlin_gpu, [(45, 9), (10, 2)], 8, 2, 128, 16, fmt, torch.float16, "chain", 4)
    bits = np.zeros((11, 64), bool)
    bits[:, 0] = True
    bits[np.arange(9), np.arange(9)] = True
    bits[9:, 0] = bits[10, 1] = True
    bits[5, 4] = True                                 # node 5 sees node 4, whose rows are not numbers
    p.bits = bits
    p.mask = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int64).copy()).cuda()
    clean, _ = p.run()
    p.check()
    clean = clean.clone()
    at = 45 + 4
    for t in p.t[2:]:
        t[int(p.table[0, at // 16]), :, at % 16] = float("nan")
    out, lse = p.run()
    hit = torch.zeros(11, dtype=torch.bool)
    hit[4] = hit[5] = True
    assert torch.equal(out[~hit], clean[~hit]) and torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


def test_queries_that_are_not_numbers_stay_in_their_row(qlin_gpu):
    p = Problem(qlin_gpu, [(45, 6)], 8, 2, 128, 16, "int8", torch.bfloat16, "tree", 4)
    clean = p.run()[0].clone()
    p.q[2, 3, 7] = float("nan")
    out, _ = p.run()
    same = torch.ones(6, 8, dtype=torch.bool)
    same[2, 3] = False
    assert torch.equal(out[same], clean[same]) and torch.isnan(out[2, 3]).all()


def test_large_and_small_queries(qlin_gpu):
    """Rows of q whose size is far from 1, down to where fp16 would lose them and up to bf16's range."""
    p = Problem(qlin_gpu, [(200, 5)], 8, 2, 128, 32, "int8", torch.bfloat16, "tree", 4)
    p.q[0] *= 2.0 ** -40
    p.q[1] *= 2.0 ** -20
    p.q[2] = 0
    p.q[3] *= 16
    p.q[4] *= 2.0 ** -130
    p.run()
    p.check()


def test_strides_streams_and_repeats(qlin_gpu):
    """q inside joint rows, out with heads outermost, another stream: the same bits, every time."""
    p = Problem(qlin_gpu, [(900, 4), (30, 9), (2000, 1)], 8, 2, 128, 64, "u4", torch.bfloat16, "tree", 6)
    first = p.run()[0].clone()
    p.check()
    joint = torch.randn(p.q.shape[0], 12, 128, device="cuda").bfloat16()
    joint[:, :8] = p.q.cuda()
    out = torch.empty(8, p.q.shape[0], 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    side = torch.cuda.Stream()
    p.run(joint[:, :8], out, side, lse=False)
    assert torch.equal(out, first)
    for _ in range(3):
        p.call.run()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_graph_replay_reads_lengths_on_the_device(qlin_gpu):
    """A captured call replayed with other lengths, pages and queries gives what a direct call gives."""
    q = qlin_gpu
    a = Problem(q, [(100, 4), (900, 4), (0, 4)], 8, 2, 128, 64, "int8", torch.float16, "tree", 6)
    b = Problem(q, [(901, 4), (3, 1), (200, 2)], 8, 2, 128, 64, "int8", torch.float16, "tree", 7, max_nodes=4)
    width = max(a.table.shape[1], b.table.shape[1])
    tq = 12
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    qs = torch.zeros(tq, 8, 128, dtype=torch.float16, device="cuda")
    mask = torch.zeros(tq, 1, dtype=torch.int64, device="cuda")
    indptr, ctx = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    pages = max(a.t[0].shape[0], b.t[0].shape[0])
    ten = [torch.zeros(pages, *t.shape[1:], dtype=t.dtype, device="cuda") for t in a.t]
    cache = q.qlin_kv_cache(*ten, q.QLIN_KV_INT8)
    out, lse = torch.empty_like(qs), torch.empty(tq, 8, device="cuda")
    ws = torch.empty(q.qlin_tree_attention_workspace_bytes(cache, 8, 4, 3), dtype=torch.uint8, device="cuda")
    call = q.qlin_tree_attention_prepare(qs, cache, table, indptr, ctx, mask, out, ws, 4, lse=lse)

    def load(p):
        n = p.q.shape[0]
        table[:, :p.table.shape[1]] = p.table.cuda()
        qs[:n] = p.q.cuda()
        mask[:n] = p.mask
        indptr.copy_(p.indptr)
        ctx.copy_(p.ctx)
        for x, y in zip(ten, p.t):
            x[:y.shape[0]] = y

    load(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.run()
    for p in (a, b, a):
        load(p)
        graph.replay()
        torch.cuda.synchronize()
        n = p.q.shape[0]
        p.out, p.lse = out[:n].clone(), lse[:n].clone()
        p.check()


def test_cache_beyond_32_bits(qlin_gpu):
    """Pages more than 2^32 bytes apart."""
    q = qlin_gpu
    p = Problem(q, [(60, 4)], 8, 2, 128, 16, "int8", torch.float16, "tree", 6, spare=1)
    pages = p.t[0].shape[0]
    gap = (1 << 30) + 4096
    if torch.cuda.mem_get_info()[0] < (2 * pages + 4) * gap:
        pytest.skip("not enough free memory")
    near = p.run()[0].clone()
    p.check()
    far = []
    for t in p.t[:2]:
        n = t[0].numel()
        buf = torch.empty((pages - 1) * gap + n, dtype=t.dtype, device="cuda")
        far.append(buf.as_strided(t.shape, (gap, *t.stride()[1:])))
        far[-1].copy_(t)
    p.cache = q.qlin_kv_cache(*far, *p.t[2:], q.QLIN_KV_INT8)
    out, _ = p.run()
    p.check()
    assert torch.equal(out, near)


def test_bad_pages_are_recorded(qlin_gpu):
    """A page number outside the cache, and lengths beyond the table: no access, an error word, the other
    sequences' outputs as before."""
    q = qlin_gpu
    p = Problem(q, [(100, 2), (50, 1), (300, 3)], 4, 2, 128, 32, "e4m3", torch.float16, "tree", 6)
    clean = p.run()[0].clone()
    p.check()
    keep = p.table.clone()
    for bad in (p.t[0].shape[0], -1, 1 << 30):
        p.table = keep.clone()
        p.table[2, 4] = bad
        out, _ = p.run()
        assert q.qlin_get_device_error() == 0x2000
        assert torch.equal(out[:3], clean[:3])
    p.table = keep
    p.ctx = torch.tensor([100, 50, 1 << 20], dtype=torch.int32)
    out, _ = p.run()
    assert q.qlin_get_device_error() == 0x2000
    assert torch.equal(out[:3], clean[:3])
