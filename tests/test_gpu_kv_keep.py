"""Accepted paths moved to the end of their sequences: codes and scales of every
head equal the ones at the path's places before, and nothing else changes."""

import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def _cache(q, fmt, pages, heads, page, d, seed=0, gap=False):
    g = torch.Generator().manual_seed(seed)
    width = d // 2 if fmt == "u4" else d
    code = {"int8": torch.int8, "e4m3": torch.uint8, "u4": torch.uint8}[fmt]
    many = pages * (2 if gap else 1)
    t = [torch.randint(0, 256, (many, heads, page, width), generator=g, dtype=torch.int32).to(code) for _ in range(2)]
    if fmt == "u4":
        t += [torch.randn(many, heads, page, 2, generator=g).half() for _ in range(2)]
    else:
        t += [torch.randn(many, heads, page, generator=g) for _ in range(2)]
    t = [x.cuda()[::2] if gap else x.cuda() for x in t]
    return t, q.qlin_kv_cache(*t, {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[fmt])


def _moved(tensors, table, page, ctx, paths):
    """What the cache should hold: each path's tokens read before any is written."""
    want = [t.cpu().clone() for t in tensors]
    for b, path in enumerate(paths):
        src, dst = ([(int(table[b, (ctx[b] + j) // page]), (ctx[b] + j) % page) for j in js] for js in (path, range(len(path))))
        for t, w in zip(tensors, want):
            rows = [t[p, :, o].cpu() for p, o in src]
            for (p, o), r in zip(dst, rows):
                w[p, :, o] = r
    return want


def _same(tensors, want):
    return all(torch.equal(t.cpu().view(torch.uint8) if t.dtype != torch.int8 else t.cpu(), w.view(torch.uint8) if w.dtype != torch.int8 else w)
               for t, w in zip([t.contiguous() for t in tensors], want))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
@pytest.mark.parametrize("heads,page,d,nodes", [(1, 16, 64, 5), (3, 32, 128, 26), (8, 64, 256, 64), (2, 16, 128, 256)])
def test_paths(qlin_gpu, fmt, heads, page, d, nodes):
    """Any ascending path: chains (nothing moves), dense ones whose places overlap, lone nodes, none."""
    q, r = qlin_gpu, random.Random(nodes)
    kept = [list(range(nodes)), [], [nodes - 1], list(range(1, nodes)), [0] + sorted(r.sample(range(1, nodes), nodes // 2)),
            sorted(r.sample(range(nodes), min(nodes, 3)))]
    ctx = [0, 5, page - 1, 3 * page + 2, 100, 2 * page]
    per = -(-(max(ctx) + nodes) // page) + 1
    t, cache = _cache(q, fmt, per * len(ctx), heads, page, d)
    table = torch.randperm(per * len(ctx), generator=torch.Generator().manual_seed(3)).int().view(len(ctx), per)
    path = torch.full((len(ctx), nodes), -1, dtype=torch.int32)
    for b, p in enumerate(kept):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = _moved(t, table, page, ctx, kept)
    lens = torch.full((len(ctx),), 9, dtype=torch.int32, device="cuda")
    q.qlin_kv_cache_keep(cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), path.cuda(),
                         torch.tensor([len(p) for p in kept], dtype=torch.int32, device="cuda"), lens)
    assert _same(t, want) and lens.tolist() == [c + len(p) for c, p in zip(ctx, kept)]
    assert q.qlin_get_device_error() == 0


@pytest.mark.parametrize("bad", [[1, 1], [2, 1], [-1, 3], [0, 200], "count", "ctx", "page"])
def test_refused_on_the_device(qlin_gpu, bad):
    """Paths that do not ascend or leave the table, counts and lengths out of range: recorded, the sequence stays, others move."""
    q, page = qlin_gpu, 16
    t, cache = _cache(q, "int8", 8, 2, page, 64)
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    path = torch.tensor([[0, 3], [0, 2]], dtype=torch.int32)
    count, ctx = [2, 2], [10, 20]
    if bad == "count":
        count[0] = 3
    elif bad == "ctx":
        ctx[0] = -1
    elif bad == "page":
        table[0, 0] = 8
    else:
        path[0] = torch.tensor(bad, dtype=torch.int32)
    want = _moved(t, torch.arange(8).view(2, 4), page, [0, 20], [[], [0, 2]])
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q.qlin_kv_cache_keep(cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), path.cuda(),
                         torch.tensor(count, dtype=torch.int32, device="cuda"), lens)
    assert q.qlin_get_device_error() == 0x2000 and _same(t, want)
    assert lens.tolist() == [12 if bad == "page" else ctx[0], 22]


def test_lengths_that_pass_31_bits(qlin_gpu):
    """A length that an int32 does not hold is recorded and its sequence left; the longest that it holds is not."""
    q, page = qlin_gpu, 256
    t, cache = _cache(q, "e4m3", 3, 2, page, 64)
    table = (torch.arange(2 ** 31 // page, dtype=torch.int32) % 3)[None].repeat(2, 1)
    top = 2 ** 31 - 1
    ctx, paths = [top - 1, top - 6], [[0, 1], [0, 2, 3]]
    want = _moved(t, table, page, ctx, [[], paths[1]])
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q.qlin_kv_cache_keep(cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                         torch.tensor([[0, 1, 0], paths[1]], dtype=torch.int32, device="cuda"),
                         torch.tensor([2, 3], dtype=torch.int32, device="cuda"), lens)
    assert q.qlin_get_device_error() == 0x2000 and lens.tolist() == [top - 1, top - 3] and _same(t, want)


def test_pages_apart_streams_and_replays(qlin_gpu):
    """Pages with others between them; a prepared call on another stream and replayed with other paths."""
    q, page = qlin_gpu, 32
    t, cache = _cache(q, "u4", 6, 3, page, 64, gap=True)
    table = torch.tensor([[4, 0, 2], [5, 1, 3]], dtype=torch.int32)
    ctx = torch.tensor([30, 64], dtype=torch.int32, device="cuda")
    path, count = torch.tensor([[0, 2, 9], [1, 5, 6]], dtype=torch.int32, device="cuda"), torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    call = q.qlin_kv_cache_keep_prepare(cache, table.cuda(), ctx, path, count)
    want = _moved(t, table, page, [30, 64], [[0, 2, 9], [1, 5]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert _same(t, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    path.copy_(torch.tensor([[3, 4, 5], [7, 8, 9]], dtype=torch.int32))
    ctx.copy_(torch.tensor([0, 33], dtype=torch.int32))
    want = _moved(t, table, page, [0, 33], [[3, 4, 5], [7, 8]])
    graph.replay()
    assert _same(t, want) and q.qlin_get_device_error() == 0
