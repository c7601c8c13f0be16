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
