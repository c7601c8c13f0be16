"""The operators run together, as examples/tree_decoding.py does: a prompt in
chunks, a tree of drafts, an accepted path, one more token; prepared calls; and
rotations of part of a head whose other channels are not numbers.

Tolerances.  Attention: as in test_gpu_tree_attention.py, for the q and the
codes that the pass itself wrote: (2^-11 + 2 e + (L + 64) 2^-24) sum p |v| with
e = D 2^-24 spread, and the rounding of the output.  Linear layers: the parity
bar of the other tests."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from conftest import ROOT, assert_within_tolerance
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("tree_decoding", os.path.join(ROOT, "examples", "tree_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rows(cache, fmt, seq, n):
    at = torch.arange(n, device="cuda")
    s = cache.slots(torch.full((n,), seq, device="cuda"), at)
    k, v, ks, vs = (t[s // cache.page, :, s % cache.page].cpu().numpy() for t in cache.tensors)
    return ref.kv_values(k, ks, fmt), ref.kv_values(v, vs, fmt)


def _check_attention(block, cache, fmt, lengths, nodes, seen):
    """block.att against the oracle on block.q and the cache's codes; sequence b: lengths[b] cached, seen [nodes][nodes]."""
    q, got = block.q.double().cpu().numpy(), block.att.double().cpu().numpy()
    for b, c in enumerate(lengths):
        k, v = _rows(cache, fmt, b, c + nodes)
        bits = np.ones((nodes, c + nodes), bool)
        bits[:, c:] = seen
        at = slice(b * nodes, (b + 1) * nodes)
        o, _, w, spread = ref.tree_attention(q[at], k, v, bits, q.shape[2] ** -0.5)
        tol = (2.0 ** -11 + 2 * q.shape[2] * 2.0 ** -24 * spread + (c + nodes + 64) * 2.0 ** -24)[..., None] * w
        tol = tol + 2.0 ** -11 * np.abs(o) + 2.0 ** -24
        assert (np.abs(got[at] - o) <= tol).all(), np.nanmax(np.abs(got[at] - o) / tol)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
def test_block_with_drafts(qlin_gpu, fmt):
    ex = _example()
    seqs, hidden, heads, kv, d, prompt = 2, 256, 8, 2, 64, 70
    cache = ex.PagedCache(seqs, 120, kv, d, fmt, page=16)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.arange(seqs, device="cuda")

    def run(block, lengths, words, depth, n):
        ctx = torch.tensor(lengths, device="cuda")
        place = ctx.repeat_interleave(n) + torch.arange(n, device="cuda").repeat(seqs)
        block.load(torch.randn(seqs * n, hidden, generator=gen, device="cuda").half(),
                   ctx.repeat_interleave(n) + depth.repeat(seqs).cuda(), cache.slots(ids.repeat_interleave(n), place),
                   n * torch.arange(seqs + 1, device="cuda"), ctx, words.repeat(seqs, 1).cuda())
        block.run()
        torch.cuda.synchronize()
        assert qlin_gpu.qlin_get_device_error() == 0

    prefill = ex.TreeAttentionBlock(hidden, heads, kv, d, cache, seqs * prompt, seqs, prompt)
    run(prefill, [0] * seqs, ex.chain_words(prompt, 2), torch.arange(prompt), prompt)
    _check_attention(prefill, cache, fmt, [0] * seqs, prompt, np.tril(np.ones((prompt, prompt), bool)))

    parents = [-1, 0, 0, 1, 1, 2, 4, 4, 6]
    n = len(parents)
    words, depth = ex.tree_words(parents, 1)
    seen = ((words.numpy()[:, :1] >> np.arange(n)) & 1).astype(bool)
    tree = ex.TreeAttentionBlock(hidden, heads, kv, d, cache, seqs * n, seqs, n)
    run(tree, [prompt] * seqs, words, depth, n)
    _check_attention(tree, cache, fmt, [prompt] * seqs, n, seen)
    # the linear layers around it, against the oracle's on the same codes
    wq, ws, wz = (t.cpu().numpy() for t in tree.w_o)
    codes, zeros = oracle.unpack_u4(wq, wq.shape[1] * 2), oracle.unpack_u4(wz, ws.shape[1])
    want = oracle.w4a16_reference(tree.att.view(seqs * n, -1).cpu().numpy(), codes, ws, zeros)
    assert_within_tolerance(tree.y.float().cpu().numpy(), want, "o")

    # the path 0 1 4 6 8 of the first, 0 2 of the second: their codes move, the next pass sees them
    before = [_rows(cache, fmt, b, prompt + n) for b in range(seqs)]
    paths = [[0, 1, 4, 6, 8], [0, 2]]
    lengths = [ex.accept(cache, b, prompt, paths[b]) for b in range(seqs)]
    for b in range(seqs):
        for old, new in zip(before[b], _rows(cache, fmt, b, lengths[b])):
            assert np.array_equal(new[:prompt], old[:prompt]) and np.array_equal(new[prompt:], old[prompt:][paths[b]])
    one = ex.TreeAttentionBlock(hidden, heads, kv, d, cache, seqs, seqs, 1)
    run(one, lengths, ex.chain_words(1, 1), torch.zeros(1, dtype=torch.int64), 1)
    _check_attention(one, cache, fmt, lengths, 1, np.ones((1, 1), bool))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_channels_that_do_not_turn(qlin_gpu, dtype, inter):
    """Channels behind the rotated ones go out bit for bit (a NaN as a NaN): infinities and signed zeros
    stay, and reach no other channel."""
    q, t, d, rot = qlin_gpu, 9, 128, 64
    x = torch.randn(t, 3, d, generator=torch.Generator().manual_seed(2)).to(dtype)
    x[0, :, rot + 3], x[1, :, rot + 7], x[2, :, d - 1] = float("inf"), -float("inf"), float("nan")
    x[3, :, rot:] = -0.0
    dev = x.cuda()
    out = torch.empty_like(dev)
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).cuda()
    q.qlin_qk_norm_rope(dev, None, out, None, torch.arange(t, device="cuda"), freq, interleaved=inter)
    torch.cuda.synchronize()
    got, want = out.cpu()[..., rot:].contiguous(), x[..., rot:].contiguous()
    nan = torch.isnan(want)   # a NaN stays one; its bits mean nothing
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    assert torch.isfinite(out[..., :rot]).all()


def test_prepared_calls(qlin_gpu):
    """A prepared call run again, and on another stream, gives what the plain call gives, reading places anew."""
    q, t, hk, d, page = qlin_gpu, 21, 2, 128, 16
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(t, 8 + 2 * hk, d, generator=gen).half().cuda()
    pos = torch.arange(t, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    slots = torch.randperm(4 * page, generator=gen)[:t].cuda()

    def fresh():
        kv = [torch.zeros(4, hk, page, d, dtype=torch.int8, device="cuda") for _ in range(2)]
        return (*kv, *[torch.zeros(4, hk, page, device="cuda") for _ in range(2)])

    first, second = fresh(), fresh()
    a, b = q.qlin_kv_cache(*first, q.QLIN_KV_INT8), q.qlin_kv_cache(*second, q.QLIN_KV_INT8)
    args = (x[:, :8], x[:, 8:8 + hk], x[:, 8 + hk:])
    out, out2 = torch.zeros(t, 8, d, dtype=torch.float16, device="cuda"), torch.zeros(t, 8, d, dtype=torch.float16, device="cuda")
    q.qlin_qk_norm_rope_cache(*args, out, pos, freq, slots, a)
    where = torch.full_like(slots, -1)
    call = q.qlin_qk_norm_rope_cache_prepare(*args, out2, pos, freq, where, b)
    call.run()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and not any(s.any() for s in second)     # no place: nothing stored
    where.copy_(slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(m, n) for m, n in zip(first, second)) and first[0].any()
    assert q.qlin_get_device_error() == 0


def test_workspace_too_small(qlin_gpu):
    q = qlin_gpu
    kv = [torch.zeros(2, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    cache = q.qlin_kv_cache(*kv, *[torch.zeros(2, 2, 16, device="cuda") for _ in range(2)], q.QLIN_KV_INT8)
    x = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    table, indptr = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    size = q.qlin_tree_attention_workspace_bytes(cache, 4, 1, 1)
    args = (x, cache, table, indptr, torch.zeros(1, dtype=torch.int32, device="cuda"), None, torch.empty_like(x))
    with pytest.raises(q.QlinError, match="workspace"):
        q.qlin_tree_attention(*args, torch.empty(size - 1, dtype=torch.uint8, device="cuda"), 1)
    q.qlin_tree_attention(*args, torch.empty(size, dtype=torch.uint8, device="cuda"), 1)
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
