"""Calls under way while other memory is mapped and given back, as in a
process's first calls: the same bits every time, and no error recorded."""

import pytest
import torch

from test_gpu_tree_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes,ctx,fmt", [(1, 6000, "e4m3"), (1, 6000, "int8"), (16, 6000, "int8"), (40, 3000, "u4")])
def test_attention(qlin_gpu, nodes, ctx, fmt):
    p = Problem(qlin_gpu, [(ctx // (1 + b % 3), nodes) for b in range(4 if nodes > 1 else 12)], 32, 8, 128, 64, fmt,
                torch.bfloat16, "tree", 3)
    first = p.run()[0].clone()
    lse = p.lse.clone()
    for i in range(12):
        torch.cuda.empty_cache()
        for _ in range(8):
            p.call.run()
        x = torch.empty((1 + i % 3) << 30, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del x
        assert qlin_gpu.qlin_get_device_error() == 0
        assert torch.equal(p.out, first) and torch.equal(p.lse, lse)
    torch.cuda.empty_cache()


def test_rotation_and_cache(qlin_gpu):
    q, t, d = qlin_gpu, 3000, 128
    x = torch.randn(t, 48, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    kv = [torch.zeros(t // 16 + 1, 8, 16, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    tens = (*kv, *[torch.zeros(t // 16 + 1, 8, 16, device="cuda") for _ in range(2)])
    at = torch.arange(t, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    out, k, v = (torch.zeros(t, h, d, dtype=torch.float16, device="cuda") for h in (32, 8, 8))
    cache = q.qlin_kv_cache(*tens, q.QLIN_KV_INT8)
    table = torch.arange(t // 16 + 1, dtype=torch.int32, device="cuda").view(1, -1)
    calls = [q.qlin_qk_norm_rope_cache_prepare(x[:, :32], x[:, 32:40], x[:, 40:], out, at, freq, at, cache),
             q.qlin_kv_cache_read_prepare(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                          torch.tensor([0, t], dtype=torch.int32, device="cuda"), k, v)]
    want = None
    for i in range(12):
        torch.cuda.empty_cache()
        for _ in range(5):
            for c in calls:
                c.run()
        y = torch.empty((1 + i % 3) << 30, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del y
        got = [z.clone() for z in (*tens, out, k, v)]
        want = want or got
        assert q.qlin_get_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.empty_cache()
