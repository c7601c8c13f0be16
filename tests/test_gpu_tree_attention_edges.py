"""Attention over the quantized cache at the edges of its arguments, for both
kernels: few rows of queries per key head (warp-level tensor cores) and many
(tcgen05).  Tolerances are those of test_gpu_tree_attention."""

import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_gpu_tree_attention import Problem

pytestmark = pytest.mark.gpu

LONGEST = (1 << 31) - 65536  # tokens of a sequence


def _bits(mask_rows):
    """bool [Tq][64 n] as the mask words of the call."""
    return torch.from_numpy(np.packbits(mask_rows, axis=1, bitorder="little").view(np.int64).copy()).cuda()


@pytest.mark.parametrize("nodes", [1, 20])
@pytest.mark.parametrize("over", [0, 1, 64, 60000])
def test_longest_sequences(qlin_gpu, nodes, over):
    """A sequence of the most tokens there may be: all pages but the first and the last two are one page whose
    tokens weigh nothing, so the result is that of the others.  A longer one is recorded and left out."""
    q, d, page = qlin_gpu, 64, 256
    total = LONGEST + over
    gen = torch.Generator().manual_seed(nodes)
    x = torch.randn(2, 4, 1, page, d, generator=gen)
    x[0, 3] = -1.0                               # with the scale below a score of -250 beside scores around 0
    codes, scales = ref.kv_quantize(x.numpy(), "int8")
    scales[0, 3] *= 31.25
    t = [torch.from_numpy(v.copy()).cuda() for v in (*codes, *scales)]
    cache = q.qlin_kv_cache(*t, q.QLIN_KV_INT8)
    pages = -(-total // page)
    table = torch.full((1, pages), 3, dtype=torch.int32)
    table[0, 0], table[0, -2], table[0, -1] = 0, 1, 2
    qs = (1 + 0.1 * torch.randn(nodes, 1, d, generator=gen)).half()
    out, lse = torch.full(qs.shape, 3.0, dtype=torch.float16, device="cuda"), torch.full((nodes, 1), 3.0, device="cuda")
    ws = torch.empty(q.qlin_tree_attention_workspace_bytes(cache, 1, nodes, 1), dtype=torch.uint8, device="cuda")
    q.qlin_tree_attention(qs.cuda(), cache, table.cuda(), torch.tensor([0, nodes], dtype=torch.int32, device="cuda"),
                          torch.tensor([total - nodes], dtype=torch.int32, device="cuda"), None, out, ws, nodes, scale=0.125, lse=lse)
    torch.cuda.synchronize()
    if over:
        assert q.qlin_get_device_error() == 0x2000
        assert (out == 3).all() and (lse == 3).all()
        return
    assert q.qlin_get_device_error() == 0
    k, v = (ref.kv_values(codes[i], scales[i], "int8").transpose(0, 2, 1, 3)[:3].reshape(-1, 1, d) for i in range(2))
    last = (total - 1) % page + 1
    at = np.r_[0:2 * page, 2 * page:2 * page + last]
    seen = np.ones((nodes, at.size), bool)
    seen[:, -nodes:] = np.tril(np.ones((nodes, nodes), bool))
    o, l, w, spread = ref.tree_attention(qs.double().numpy(), k[at], v[at], seen, 0.125)
    e, s = d * 2.0 ** -24 * spread, (at.size + 64) * 2.0 ** -24
    assert (np.abs(out.double().cpu().numpy() - o) <= (2.0 ** -11 + 2 * e + s)[..., None] * w + 2.0 ** -11 * np.abs(o) + 2.0 ** -24).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= e + s + 2.0 ** -22 * np.abs(l)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
def test_heads_of_256_over_long_contexts(qlin_gpu, fmt):
    """Each warp takes its turns at the ring for thousands of rounds, the codes from HBM: the same bits every time."""
    q, d = qlin_gpu, 256
    p = Problem(q, [(60000, 1), (30011, 3), (9000, 2)], 4, 2, d, 64, fmt, torch.bfloat16, "tree", 3)
    first, lse = (x.clone() for x in p.run())
    p.check()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        flush.fill_(i)                                # larger than L2
        p.call.run()
        torch.cuda.synchronize()
        assert q.qlin_get_device_error() == 0
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)


# One shape for each kernel and head size: few rows of queries per key head, and many.
SIZES = [(64, 1), (128, 3), (256, 2), (64, 7), (128, 9)]
FMTS = ["int8", "e4m3", "u4"]


def _leave_behind(q, fmt, d):
    """Fills the shared memory of every block with codes 0x80 (E4M3's -0) and scales of -0 before the next call."""
    kind = torch.int8 if fmt == "int8" else torch.uint8
    width = d // 2 if fmt == "u4" else d
    codes = torch.full((64, 1, 256, width), 128, dtype=torch.uint8, device="cuda").view(kind)
    scales = torch.full((64, 1, 256, 2) if fmt == "u4" else (64, 1, 256), -0.0, dtype=torch.float16 if fmt == "u4" else torch.float32,
                        device="cuda")
    cache = q.qlin_kv_cache(codes, codes, scales, scales, {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[fmt])
    for rows in (1, 20):
        x = torch.zeros(4 * rows, 1, d, dtype=torch.float16, device="cuda")
        ws = torch.empty(q.qlin_tree_attention_workspace_bytes(cache, 1, rows, 4), dtype=torch.uint8, device="cuda")
        q.qlin_tree_attention(x, cache, torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64).repeat(4, 16),
                              rows * torch.arange(5, dtype=torch.int32, device="cuda"),
                              torch.full((4,), 64 * 256 * 15, dtype=torch.int32, device="cuda"), None, torch.empty_like(x), ws, rows)


def _put(p, where, words, which=(2, 3)):
    """Scale words (numbers, or for "u4" pairs) of the given tensors at the places `where` (bool [pages][page])."""
    for i in which:
        dtype = p.t[i].dtype
        at = where[:, None, :].expand(p.t[i].shape[:3]).cuda()
        p.t[i][at] = torch.tensor(words, dtype=torch.float64).to(dtype).cuda()


def _live(p):
    where = torch.zeros(p.t[0].shape[0], p.page, dtype=torch.bool)
    for b, (c, n) in enumerate(p.seqs):
        j = torch.arange(c + n)
        where[p.table[b, j // p.page].long(), j % p.page] = True
    return where


def _place(p, b, j):
    where = torch.zeros(p.t[0].shape[0], p.page, dtype=torch.bool)
    where[int(p.table[b, j // p.page]), j % p.page] = True
    return where


def _hide(p, node):
    """No row of the first sequence sees node `node` of it."""
    p.bits[:p.seqs[0][1], node] = False
    p.mask = _bits(p.bits)


FAR = 2.0 ** -149
WORDS = [0.0, -0.0, -FAR, FAR, float("inf"), -float("inf"), -1.5, 3e38, float("nan")]
PAIRS = [(0.0, 0.0), (-0.0, 3.0), (-2.0 ** -24, 15.0), (float("inf"), 0.0), (-1.0, -0.0), (65504.0, 7.5), (0.01, float("nan")),
         (0.01, -300.0), (float("nan"), float("inf"))]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,nodes", SIZES)
@pytest.mark.parametrize("ctx", [37, 160])
def test_scales_that_nobody_sees(qlin_gpu, fmt, d, nodes, ctx):
    """Whatever the scale words of places behind a sequence's end and of a node that no row sees hold, and whatever
    lies in shared memory where a tile has no page: the same bits."""
    q = qlin_gpu
    p = Problem(q, [(ctx, nodes), (10, 2)], 8, 2, d, 16, fmt, torch.float16, "tree", nodes)
    if nodes > 1:
        _hide(p, 1)
    gone = ~_live(p) | (_place(p, 0, ctx + 1) if nodes > 1 else False)
    _put(p, gone, (1.0, 3.0) if fmt == "u4" else 1.0)
    clean, lse = p.run()
    p.check()
    clean = clean.clone()
    for word in PAIRS if fmt == "u4" else WORDS:
        _put(p, gone, word)
        _leave_behind(q, fmt, d)
        out, l2 = p.run()
        p.check()
        assert torch.equal(out, clean) and torch.equal(l2, lse), word


def _scale(p, i, b, j, word):
    """The scale of the keys (i = 0) or values (i = 1) of token j of sequence b, on the host and the device."""
    page, off = int(p.table[b, j // p.page]), j % p.page
    if p.fmt == "u4":
        p.scales[i][page, :, off, 0] = word
        p.t[2 + i][page, :, off, 0] = float(np.float16(word))
    else:
        p.scales[i][page, :, off] = word
        p.t[2 + i][page, :, off] = float(np.float32(word))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,nodes", SIZES)
def test_scales_of_zero_and_below_and_close_to_it(qlin_gpu, fmt, dtype, d, nodes):
    """Rows of zeros by their scale, negative scales and subnormal ones count in the sum as they are, at any place of
    a context and among the nodes."""
    p = Problem(qlin_gpu, [(300, nodes), (40, nodes)], 8, 2, d, 32, fmt, dtype, "tree", nodes)
    words = [0.0, -0.0, -0.01, 2.0 ** -24, -2.0 ** -20] if fmt == "u4" else [0.0, -0.0, -0.01, FAR, -2.0 ** -130, 2.0 ** -100, -2.0 ** -70]
    r = np.random.default_rng(d)
    for b, (c, n) in enumerate(p.seqs):
        for i in range(2):
            for j in r.permutation(c + n)[:(c + n) // 3]:
                _scale(p, i, b, int(j), words[int(r.integers(len(words)))])
    p.run()
    p.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,nodes", SIZES)
def test_one_scale_for_all_values(qlin_gpu, fmt, dtype, d, nodes):
    """All values zero; all near the smallest and the largest numbers of bf16; the lse is that of the keys throughout."""
    p = Problem(qlin_gpu, [(300, nodes), (40, nodes)], 8, 2, d, 32, fmt, dtype, "tree", nodes, wide=0.0)
    small = [0.0, -2.0 ** -24, 2.0 ** -16] if fmt == "u4" else [0.0, -0.0, 2.0 ** -126, -2.0 ** -131, 2.0 ** -92, -2.0 ** -64]
    for word in small + ([] if fmt == "u4" or dtype == torch.float16 else [2.0 ** 100, -2.0 ** 110]):
        for b, (c, n) in enumerate(p.seqs):
            for j in range(c + n):
                _scale(p, 1, b, j, word)
        p.run()
        p.check()
        if word == 0:
            assert not (p.out != 0).any()


def _lse_bound(p):
    """How far an lse may be off, [rows][heads]."""
    out, row = [], 0
    for b, (c, n) in enumerate(p.seqs):
        j = np.arange(c + n)
        pg = p.table[b, j // p.page].numpy()
        k = ref.kv_values(p.codes[0][pg, :, j % p.page], p.scales[0][pg, :, j % p.page], p.fmt)
        seen = np.ones((n, c + n), bool)
        seen[:, c:] = np.tril(np.ones((n, n), bool)) if p.bits is None else p.bits[row:row + n, :n]
        _, l, _, spread = ref.tree_attention(p.q[row:row + n].double().numpy(), k, k, seen, p.scale)
        out.append(p.q.shape[2] * 2.0 ** -24 * spread + (c + n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l))
        row += n
    return np.concatenate(out)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,nodes", SIZES)
def test_values_that_are_not_numbers(qlin_gpu, fmt, d, nodes):
    """A value row whose scale is NaN or infinite makes every row that sees it not a number, and no other; lse is of
    the keys alone."""
    p = Problem(qlin_gpu, [(100, nodes), (40, nodes)], 8, 2, d, 32, fmt, torch.bfloat16, "chain", nodes)
    clean, lse = (x.clone() for x in p.run())
    p.check()
    keep = [x.clone() for x in p.t]
    bound = torch.from_numpy(_lse_bound(p))
    for word in (float("nan"), float("inf"), -float("inf")):
        for j in (3, 100 + nodes - 1):
            for x, y in zip(p.t, keep):
                x.copy_(y)
            _put(p, _place(p, 0, j), (word, 3.0) if fmt == "u4" else word, (3,))
            out, l2 = p.run()
            hit = torch.zeros(2 * nodes, dtype=torch.bool)
            hit[0 if j < 100 else nodes - 1:nodes] = True
            assert torch.equal(out[~hit], clean[~hit]) and not torch.isfinite(out[hit]).any()
            assert ((l2 - lse).abs().double().cpu() <= 2 * bound).all()


@pytest.mark.parametrize("d,nodes", SIZES)
@pytest.mark.parametrize("word", [7.5, -1.0, 16.0, 15.25, 1024.0, float("nan"), float("inf"), -float("inf")])
def test_zero_points_that_are_none(qlin_gpu, d, nodes, word):
    """A zero-point that is not a whole number from 0 to 15 makes its token not a number: for the rows that see it,
    and no other."""
    p = Problem(qlin_gpu, [(100, nodes), (40, nodes)], 8, 2, d, 32, "u4", torch.float16, "chain", nodes)
    clean, lse = (x.clone() for x in p.run())
    p.check()
    keep = [x.clone() for x in p.t]
    for which in ((2,), (3,)):
        for j in (3, 100 + nodes - 1):
            for x, y in zip(p.t, keep):
                x.copy_(y)
            at = _place(p, 0, j)
            for i in which:
                p.t[i].view(-1, 2, p.page, 2)[int(p.table[0, j // p.page]), :, j % p.page, 1] = word
            assert at.any()
            out, l2 = p.run()
            hit = torch.zeros(2 * nodes, dtype=torch.bool)
            hit[0 if j < 100 else nodes - 1:nodes] = True
            assert torch.equal(out[~hit], clean[~hit]) and torch.isnan(out[hit]).all()
            assert torch.equal(l2[~hit], lse[~hit])
            assert torch.isnan(l2[hit]).all() if which == (2,) else torch.equal(l2, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,nodes", SIZES)
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_read_as_zeros(qlin_gpu, fmt, d, nodes, page):
    """Tokens on a page whose number is out of range are keys and values of zeros, as the read gives them: nothing of
    other sequences or of earlier calls reaches the result."""
    q = qlin_gpu
    p = Problem(q, [(300, nodes), (150, nodes)], 8, 2, d, page, fmt, torch.float16, "tree", nodes)
    p.run()
    p.check()
    keep, bad = p.table.clone(), (p.t[0].shape[0], -1, -(1 << 31))
    # the oracle's view: one more page, of zeros
    p.codes, p.scales = (np.concatenate([x, np.zeros_like(x[:, :1])], axis=1) for x in (p.codes, p.scales))
    first = None
    for number, at in zip(bad, (1, 150 // page, 300 // page)):
        for other in range(2):
            host = keep.clone()
            host[0, at] = host[0, 0] = p.codes.shape[1] - 1
            p.table = keep.clone()
            p.table[0, at] = p.table[0, 0] = number
            _leave_behind(q, fmt, d)
            out, _ = p.run()
            if other == 0:
                p.table = host
                p.check(0x2000)
                first = out.clone()
                for x in p.t[:2]:    # what the other sequence and the unused pages hold
                    gone = torch.ones(x.shape[0], dtype=torch.bool)
                    gone[keep[0, :-(-(300 + nodes) // page)].long()] = False
                    x[gone] = 0
            else:
                assert q.qlin_get_device_error() == 0x2000
                assert torch.equal(out[:nodes], first[:nodes])
                for x, y in zip(p.t, p.codes_dev):
                    x.copy_(torch.from_numpy(y.copy()))


@pytest.mark.parametrize("d,nodes", SIZES)
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_codes_that_nobody_sees(qlin_gpu, d, nodes, code):
    """E4M3 codes that are NaN (never written by the library) behind a sequence's end and in a node that no row sees:
    the same bits.  A row that sees such a node is not a number."""
    p = Problem(qlin_gpu, [(45, nodes), (10, 2)], 8, 2, d, 16, "e4m3", torch.float16, "tree", nodes)
    if nodes > 1:
        _hide(p, 1)
    gone = ~_live(p) | (_place(p, 0, 46) if nodes > 1 else False)
    clean, lse = (x.clone() for x in p.run())
    p.check()
    for i in range(2):
        p.t[i][gone[:, None, :].expand(p.t[i].shape[:3]).cuda()] = code
    out, l2 = p.run()
    p.check()
    assert torch.equal(out, clean) and torch.equal(l2, lse)
    page, off = int(p.table[0, 45 // 16]), 45 % 16
    p.t[1][page, 0, off, d - 1] = code              # one code of node 0, of the first key head
    out, l2 = p.run()
    hit = torch.from_numpy(p.bits[:, 0].copy())
    hit[nodes:] = False
    assert torch.isnan(out[hit][:, :4, d - 1]).all() and torch.equal(out[~hit], clean[~hit]) and torch.equal(out[:, 4:], clean[:, 4:])
    assert torch.equal(l2, lse)


# What the tests of test_gpu_tree_attention reach through one kernel only, through both.
BOTH = pytest.mark.parametrize("nodes", [3, 9])


@BOTH
def test_a_query_that_is_not_a_number(qlin_gpu, nodes):
    p = Problem(qlin_gpu, [(45, nodes)], 8, 2, 128, 16, "e4m3", torch.float16, "tree", 4)
    clean = p.run()[0].clone()
    for word in (float("nan"), float("inf")):
        x = p.q.clone()
        x[1, 5, 77] = word
        out, lse = p.run(x.cuda())
        same = torch.ones(nodes, 8, dtype=torch.bool)
        same[1, 5] = False
        assert torch.equal(out[same], clean[same]) and torch.isnan(out[1, 5]).all()
        assert torch.isnan(lse[1, 5]) and torch.isfinite(lse[same]).all()


@BOTH
@pytest.mark.parametrize("d,fmt", [(64, "u4"), (128, "int8"), (128, "e4m3")])
def test_queries_far_below_one(qlin_gpu, nodes, d, fmt):
    p = Problem(qlin_gpu, [(200, nodes)], 8, 2, d, 32, fmt, torch.bfloat16, "tree", 4)
    for i, by in enumerate((2.0 ** -40, 2.0 ** -130, 2.0 ** -20, 0.0, 2.0 ** -8)[:nodes]):
        p.q[i] *= by
    p.run()
    p.check()


@BOTH
def test_strides_and_another_stream(qlin_gpu, nodes):
    p = Problem(qlin_gpu, [(900, nodes), (30, nodes - 1), (2000, 1)], 8, 2, 128, 64, "e4m3", torch.float16, "tree", 6)
    first = p.run()[0].clone()
    p.check()
    n = p.q.shape[0]
    joint = torch.randn(n, 14, 128, device="cuda").half()
    joint[:, 3:11] = p.q.cuda()
    out = torch.empty(8, n, 128, dtype=torch.float16, device="cuda").transpose(0, 1)
    side = torch.cuda.Stream()
    p.run(joint[:, 3:11], out, side, lse=False)
    assert torch.equal(out, first)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        p.call.run(side)
        torch.cuda.synchronize()
        assert torch.equal(out, first)


@BOTH
def test_replay_with_other_lengths(qlin_gpu, nodes):
    """A captured call replayed while lengths, pages, masks and queries change on the device."""
    q = qlin_gpu
    a = Problem(q, [(100, nodes), (900, nodes), (0, nodes)], 8, 2, 128, 16, "u4", torch.float16, "tree", 6)
    b = Problem(q, [(1301, nodes), (3, 1), (0, 0)], 8, 2, 128, 16, "u4", torch.float16, "random", 7, max_nodes=nodes)
    tq, pages = 3 * nodes, max(a.t[0].shape[0], b.t[0].shape[0])
    table = torch.full((3, max(a.table.shape[1], b.table.shape[1])), -1, dtype=torch.int32, device="cuda")
    x, mask = torch.zeros(tq, 8, 128, dtype=torch.float16, device="cuda"), torch.zeros(tq, 1, dtype=torch.int64, device="cuda")
    indptr, ctx = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    ten = [torch.zeros(pages, *t.shape[1:], dtype=t.dtype, device="cuda") for t in a.t]
    cache = q.qlin_kv_cache(*ten, q.QLIN_KV_U4)
    out, lse = torch.empty_like(x), torch.empty(tq, 8, device="cuda")
    ws = torch.empty(q.qlin_tree_attention_workspace_bytes(cache, 8, nodes, 3), dtype=torch.uint8, device="cuda")
    call = q.qlin_tree_attention_prepare(x, cache, table, indptr, ctx, mask, out, ws, nodes, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call.run()
    for p in (a, b, a):
        n = p.q.shape[0]
        table[:, :p.table.shape[1]] = p.table.cuda()
        x[:n], mask[:n] = p.q.cuda(), p.mask
        indptr.copy_(p.indptr)
        ctx.copy_(p.ctx)
        for to, y in zip(ten, p.t):
            to[:y.shape[0]] = y
        graph.replay()
        torch.cuda.synchronize()
        p.out, p.lse = out[:n].clone(), lse[:n].clone()
        p.check()


@BOTH
def test_pages_beyond_32_bits(qlin_gpu, nodes):
    q = qlin_gpu
    p = Problem(q, [(60, nodes)], 8, 2, 128, 16, "e4m3", torch.float16, "tree", 6, spare=0)
    pages, gap = p.t[0].shape[0], (1 << 30) + 4096
    if torch.cuda.mem_get_info()[0] < (2 * pages + 4) * gap:
        pytest.skip("not enough free memory")
    near = p.run()[0].clone()
    p.check()
    far = []
    for t in p.t[:2]:
        buf = torch.empty((pages - 1) * gap + t[0].numel(), dtype=t.dtype, device="cuda")
        far.append(buf.as_strided(t.shape, (gap, *t.stride()[1:])))
        far[-1].copy_(t)
    p.cache = q.qlin_kv_cache(*far, *p.t[2:], q.QLIN_KV_E4M3)
    out, _ = p.run()
    p.check()
    assert torch.equal(out, near)


@BOTH
def test_bounds_that_do_not_fit(qlin_gpu, nodes):
    """A sequence whose length, rows or nodes are out of range is recorded and left out, its rows as they were."""
    q = qlin_gpu
    p = Problem(q, [(100, nodes), (50, nodes), (70, nodes)], 8, 2, 128, 32, "int8", torch.float16, "tree", 6)
    clean = p.run()[0].clone()
    p.check()
    ctx, indptr = p.ctx.clone(), p.indptr.clone()
    rows = slice(nodes, 2 * nodes)
    others = torch.ones(3 * nodes, dtype=torch.bool)
    others[rows] = False
    for bad in (1 << 20, -1, 0x7fffffff, -(1 << 31)):
        p.ctx = ctx.clone()
        p.ctx[1] = bad
        out, lse = p.run()
        assert q.qlin_get_device_error() == 0x2000
        assert torch.equal(out[others], clean[others]) and (out[rows] == 3).all() and (lse[rows] == 3).all()
    p.ctx = ctx
    for at, bad in ((3, 3 * nodes + 1), (0, -1), (3, -(1 << 31))):
        p.indptr = indptr.clone()
        p.indptr[at] = bad
        out, _ = p.run()
        assert q.qlin_get_device_error() == 0x2000
        assert torch.equal(out[rows], clean[rows])
