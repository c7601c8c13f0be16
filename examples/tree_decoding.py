"""One attention block that answers with drafts: W4A16 projections, head norms
and the position rotation with the cache write in one pass, attention of a tree
of drafted tokens over the paged, quantized cache.

    python examples/tree_decoding.py [--fmt int8|e4m3|u4] [--hidden 4096] [--prompt 4096] [--seqs 8]

A prompt goes in by chunks (a chain of up to 256 tokens each), then rounds of
drafts: every sequence proposes a tree, one pass answers for all its nodes, a
path of it is accepted and moved to the end of the sequence.  Weights and
hidden states are random; the time of each pass is printed.  The cache, the
page table and the lengths are the caller's tensors, as a serving loop keeps
them; the passes of one size are prepared once and captured as a CUDA graph,
which reads lengths, pages and places on the device at every replay.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import quantized_linear_layer_gb300 as qlin

FMT = {"int8": qlin.QLIN_KV_INT8, "e4m3": qlin.QLIN_KV_E4M3, "u4": qlin.QLIN_KV_U4}


def linear_w4(n, k, gen):
    """A random weight [n][k] in the W4A16 format."""
    w = torch.randn(n, k, generator=gen).mul_(k ** -0.5).to(torch.float16).cuda()
    wq = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, k // 128, dtype=torch.float16, device="cuda")
    zeros = torch.empty(n, (k // 128 + 1) // 2, dtype=torch.uint8, device="cuda")
    qlin.qlin_quant_w4_g128(w, wq, scales, zeros)
    return wq, scales, zeros


class PagedCache:
    """Pages for `seqs` sequences of up to `room` tokens, and the places of their tokens."""

    def __init__(self, seqs, room, heads, head_dim, fmt, page=64):
        self.page, per = page, -(-room // page)
        pages, width = seqs * per, head_dim // 2 if fmt == "u4" else head_dim
        code = torch.int8 if fmt == "int8" else torch.uint8
        kv = [torch.zeros(pages, heads, page, width, dtype=code, device="cuda") for _ in range(2)]
        if fmt == "u4":
            scales = [torch.zeros(pages, heads, page, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
        else:
            scales = [torch.zeros(pages, heads, page, device="cuda") for _ in range(2)]
        self.tensors = (*kv, *scales)
        self.handle = qlin.qlin_kv_cache(*self.tensors, FMT[fmt])
        self.table = torch.arange(pages, dtype=torch.int32).view(per, seqs).t().contiguous().cuda()

    def slots(self, seq, at):
        """The places of tokens `at` of sequences `seq` (int64 tensors)."""
        return self.table[seq, at // self.page].long() * self.page + at % self.page

    def move(self, src, dst):
        """Codes and scales from places src to dst: accepted drafts close the gaps that the others leave."""
        for t in self.tensors:
            t[dst // self.page, :, dst % self.page] = t[src // self.page, :, src % self.page]


class TreeAttentionBlock:
    """The attention half of a decoder layer for up to `tokens` new tokens a pass."""

    def __init__(self, hidden, heads, kv_heads, head_dim, cache, tokens, seqs, max_nodes, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.cache, self.max_nodes, f16 = cache, max_nodes, dict(dtype=torch.float16, device="cuda")
        self.w_qkv = [linear_w4(n * head_dim, hidden, gen) for n in (heads, kv_heads, kv_heads)]
        self.w_o = linear_w4(hidden, heads * head_dim, gen)
        self.q_gamma = (1 + 0.1 * torch.randn(head_dim, generator=gen)).to(**f16)
        self.k_gamma = (1 + 0.1 * torch.randn(head_dim, generator=gen)).to(**f16)
        self.inv_freq = (10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).cuda()
        self.x = torch.zeros(tokens, hidden, **f16)
        self.y = torch.zeros(tokens, hidden, **f16)
        self.qkv = [torch.zeros(tokens, n, head_dim, **f16) for n in (heads, kv_heads, kv_heads)]
        self.q = torch.zeros(tokens, heads, head_dim, **f16)
        self.att = torch.zeros(tokens, heads, head_dim, **f16)
        self.positions = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        self.slots = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")  # negative: not stored
        self.indptr = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.mask = torch.zeros(tokens, (max_nodes + 63) // 64, dtype=torch.int64, device="cuda")
        size = qlin.qlin_tree_attention_workspace_bytes(cache.handle, heads, max_nodes, seqs)
        workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.rotate = qlin.qlin_qk_norm_rope_cache_prepare(*self.qkv, self.q, self.positions, self.inv_freq, self.slots,
                                                           cache.handle, self.q_gamma, self.k_gamma)
        self.attend = qlin.qlin_tree_attention_prepare(self.q, cache.handle, cache.table, self.indptr, self.ctx, self.mask,
                                                       self.att, workspace, max_nodes)
        self.graph = None

    def load(self, x, positions, slots, indptr, ctx, mask):
        """A pass's inputs; rows behind the given ones belong to no sequence and are not stored."""
        n = x.shape[0]
        self.x[:n] = x
        self.positions[:n] = positions
        self.slots.fill_(-1)
        self.slots[:n] = slots
        self.indptr.copy_(indptr)
        self.ctx.copy_(ctx)
        self.mask[:n] = mask

    def launch(self):
        flat = [t.view(t.shape[0], -1) for t in self.qkv]
        qlin.qlin_w4a16_gemm_grouped(self.x, *map(list, zip(*self.w_qkv)), flat)
        self.rotate.run()
        self.attend.run()
        qlin.qlin_w4a16_gemm(self.att.view(self.att.shape[0], -1), *self.w_o, self.y)

    def run(self):
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.launch()
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.launch()
        self.graph.replay()
        return self.y


def tree_words(parents, words):
    """Mask words [nodes][words] of a tree: node i sees its ancestors and itself; and the nodes' depths."""
    seen, depth = [], []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    low = (1 << 64) - 1
    signed = [[((s >> 64 * w & low) ^ 1 << 63) - (1 << 63) for w in range(words)] for s in seen]
    return torch.tensor(signed, dtype=torch.int64), torch.tensor(depth)


def chain_words(n, words):
    return tree_words(range(-1, n - 1), words)[0]


def accept(cache, seq, ctx, path):
    """The nodes of `path` (ascending) become the tokens ctx .. of sequence `seq`; returns the new length."""
    s = torch.full((len(path),), seq, device="cuda")
    src = cache.slots(s, ctx + torch.tensor(path, device="cuda"))
    cache.move(src, cache.slots(s, ctx + torch.arange(len(path), device="cuda")))
    return ctx + len(path)


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--fmt", choices=FMT, default="int8")
    a.add_argument("--hidden", type=int, default=4096)
    a.add_argument("--heads", type=int, default=32)
    a.add_argument("--kv-heads", type=int, default=8)
    a.add_argument("--seqs", type=int, default=8)
    a.add_argument("--prompt", type=int, default=4096)
    a.add_argument("--rounds", type=int, default=4)
    a = a.parse_args()
    qlin.build()
    head_dim, chunk = 128, 256
    parents = [-1, 0, 0, 0, 1, 1, 2, 3, 4, 4, 5, 6, 8, 8, 10, 12]
    nodes = len(parents)
    cache = PagedCache(a.seqs, a.prompt + (a.rounds + 1) * nodes, a.kv_heads, head_dim, a.fmt)
    gen = torch.Generator(device="cuda").manual_seed(1)
    shape = (a.hidden, a.heads, a.kv_heads, head_dim, cache)
    seqs = torch.arange(a.seqs, device="cuda")

    def timed(block, what):
        block.run()  # the first run captures; a replay writes the same codes to the same places
        begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
        begin.record()
        block.run()
        end.record()
        torch.cuda.synchronize()
        if qlin.qlin_get_device_error() != 0:
            raise RuntimeError("device error")
        print("%-46s %8.1f us" % (what, 1e3 * begin.elapsed_time(end)))

    prefill = TreeAttentionBlock(*shape, tokens=a.seqs * chunk, seqs=a.seqs, max_nodes=chunk)
    words = chain_words(chunk, chunk // 64).repeat(a.seqs, 1).cuda()
    for at in range(0, a.prompt, chunk):
        n = min(chunk, a.prompt - at)
        pos = (at + torch.arange(n, device="cuda")).repeat(a.seqs)
        x = torch.randn(a.seqs * n, a.hidden, generator=gen, device="cuda").half()
        prefill.load(x, pos, cache.slots(seqs.repeat_interleave(n), pos), n * torch.arange(a.seqs + 1, device="cuda"),
                     torch.full((a.seqs,), at, device="cuda"), words.view(a.seqs, chunk, -1)[:, :n].reshape(a.seqs * n, -1))
        timed(prefill, "prompt, %d tokens behind %d, %d sequences" % (n, at, a.seqs))

    block = TreeAttentionBlock(*shape, tokens=a.seqs * nodes, seqs=a.seqs, max_nodes=nodes)
    words, depth = tree_words(parents, 1)
    words, depth = words.repeat(a.seqs, 1).cuda(), depth.repeat(a.seqs).cuda()
    lengths = [a.prompt] * a.seqs
    for r in range(a.rounds):
        ctx = torch.tensor(lengths, device="cuda")
        place = ctx.repeat_interleave(nodes) + torch.arange(nodes, device="cuda").repeat(a.seqs)
        x = torch.randn(a.seqs * nodes, a.hidden, generator=gen, device="cuda").half()
        block.load(x, ctx.repeat_interleave(nodes) + depth, cache.slots(seqs.repeat_interleave(nodes), place),
                   nodes * torch.arange(a.seqs + 1, device="cuda"), ctx, words)
        timed(block, "trees of %d drafts, %d tokens cached" % (nodes, min(lengths)))
        # a verifier would choose; here each sequence keeps another path of its tree
        paths = [[0, 1, 4, 8, 12, 15], [0, 2, 6, 11], [0, 3], [0, 1, 5, 10, 14]]
        lengths = [accept(cache, s, lengths[s], paths[(r + s) % len(paths)]) for s in range(a.seqs)]


if __name__ == "__main__":
    main()
