"""A serving loop around one attention block: prompts in long chunks, then steps
in which every sequence drafts a tree of tokens, one pass answers for all its
nodes, the target's probabilities verify it and the kept path stays in the cache.

    python examples/speculative_serving.py [--fmt int8|e4m3|u4] [--hidden 4096] [--prompt 4096] [--chunk 2048] [--seqs 8]

Lengths, pages, places, masks and tokens stay on the device: a step is one CUDA
graph with no read by the host,

    pages and slots from lengths -> W4A16 projections -> head norms, rotation,
    cache write -> tree attention -> W4A16 projections -> verification -> kept
    paths moved together -> lengths

Weights are random (the block's output is added to the token's embedding, and
the draft is what the head makes of the embedding alone); the time of each
pass and the tokens a step kept are printed.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch

import quantized_linear_layer_gb300 as qlin
from tree_decoding import FMT, linear_w4, tree_words

I32 = dict(dtype=torch.int32, device="cuda")
I64 = dict(dtype=torch.int64, device="cuda")


class Cache:
    """`pages` pages for `seqs` sequences of up to `room` tokens, none of them handed out yet."""

    def __init__(self, seqs, room, pages, heads, head_dim, fmt, page=64):
        width = head_dim // 2 if fmt == "u4" else head_dim
        kv = [torch.zeros(pages, heads, page, width, dtype=torch.int8 if fmt == "int8" else torch.uint8, device="cuda") for _ in range(2)]
        if fmt == "u4":
            scales = [torch.zeros(pages, heads, page, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
        else:
            scales = [torch.zeros(pages, heads, page, device="cuda") for _ in range(2)]
        self.fmt, self.page, self.tensors = fmt, page, (*kv, *scales)
        self.handle = qlin.qlin_kv_cache(*self.tensors, FMT[fmt])
        self.table = torch.zeros(seqs, -(-room // page), **I32)
        self.held = torch.zeros(seqs, **I32)
        self.free = torch.arange(pages, **I32)
        self.count = torch.full((1,), pages, **I32)
        self.pages = qlin.qlin_kv_pages(self.table, self.held, self.free, self.count, page)
        self.ctx = torch.zeros(seqs, **I32)    # tokens that stay
        self.last = torch.zeros(seqs, **I64)   # the token behind them, drawn but not in the cache yet


class Model:
    """Embedding, one attention block and a head."""

    def __init__(self, vocab, hidden, heads, kv_heads, head_dim, seed=0):
        gen = torch.Generator().manual_seed(seed)
        f16 = dict(dtype=torch.float16, device="cuda")
        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.embedding = torch.randn(vocab, hidden, generator=gen).to(**f16)
        self.w_qkv = [linear_w4(n * head_dim, hidden, gen) for n in (heads, kv_heads, kv_heads)]
        self.w_o = linear_w4(hidden, heads * head_dim, gen)
        self.w_head = linear_w4(vocab, hidden, gen)
        self.q_gamma = (1 + 0.1 * torch.randn(head_dim, generator=gen)).to(**f16)
        self.k_gamma = (1 + 0.1 * torch.randn(head_dim, generator=gen)).to(**f16)
        self.inv_freq = (10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)).cuda()

    def logits(self, h):
        out = torch.empty(h.shape[0], self.vocab, dtype=torch.float16, device="cuda")
        qlin.qlin_w4a16_gemm(h, *self.w_head, out)
        return out

    def probabilities(self, h):
        return torch.softmax(self.logits(h).float() * 8, -1)  # (of random weights the logits lie close together)


class Pass:
    """The block for `rows` rows of new tokens: buffers, and the calls that read lengths and pages on the device."""

    def __init__(self, model, cache, rows, depths=None):
        f16, m, seqs = dict(dtype=torch.float16, device="cuda"), model, cache.ctx.numel()
        self.model, self.cache = model, cache
        self.new = torch.zeros(seqs, **I32)
        self.indptr = torch.zeros(seqs + 1, **I32)
        self.positions, self.slots = torch.zeros(rows, **I64), torch.zeros(rows, **I64)
        self.tokens, self.at = torch.zeros(rows, **I64), torch.arange(rows, **I32)
        self.qkv = [torch.zeros(rows, n, m.head_dim, **f16) for n in (m.heads, m.kv_heads, m.kv_heads)]
        self.q, self.att = (torch.zeros(rows, m.heads, m.head_dim, **f16) for _ in range(2))
        self.y = torch.zeros(rows, m.embedding.shape[1], **f16)
        self.assign = qlin.qlin_kv_pages_assign_prepare(cache.pages, cache.ctx, self.new, self.indptr, self.positions, self.slots, depths)
        self.rotate = qlin.qlin_qk_norm_rope_cache_prepare(*self.qkv, self.q, self.positions, m.inv_freq, self.slots, cache.handle,
                                                           m.q_gamma, m.k_gamma)

    def rows(self):
        """The sequence of each row, and which of its new tokens it is: a sequence that pages or rows ran out for has no rows, and
        those behind it move up.  (Rows behind the last sequence's: of any.)"""
        seq = torch.searchsorted(self.indptr[1:], self.at, right=True).clamp(max=self.new.numel() - 1)
        return seq, self.at - self.indptr[seq]

    def hidden(self):
        """Pages, places and the block's output for the rows' tokens (rows behind the last sequence's mean nothing)."""
        self.assign.run()
        self.place()
        x = self.model.embedding[self.tokens]
        qlin.qlin_w4a16_gemm_grouped(x, *map(list, zip(*self.model.w_qkv)), [t.view(t.shape[0], -1) for t in self.qkv])
        self.rotate.run()
        self.attend.run()
        qlin.qlin_w4a16_gemm(self.att.view(self.att.shape[0], -1), *self.model.w_o, self.y)
        return x + self.y


class Prefill(Pass):
    """Prompts, up to `chunk` tokens of each sequence a pass."""

    def __init__(self, model, cache, chunk, **scores):
        seqs = cache.ctx.numel()
        super().__init__(model, cache, seqs * chunk)
        size = qlin.qlin_chunk_attention_workspace_bytes(cache.handle, model.heads, chunk, seqs)
        self.attend = qlin.qlin_chunk_attention_prepare(self.q, cache.handle, cache.table, self.indptr, cache.ctx, self.att,
                                                        torch.empty(size, dtype=torch.uint8, device="cuda"), chunk, **scores)
        self.given, self.starts = torch.zeros(seqs * chunk, **I64), torch.zeros(seqs, **I64)
        # the token behind a prompt: a tree of one node, from which nothing is kept
        self.none, self.nodes = torch.zeros(seqs, **I64), torch.zeros(seqs + 1, **I32)
        self.path, self.kept, self.next = torch.zeros(seqs, 1, **I32), torch.zeros(seqs, **I32), torch.zeros(seqs, **I64)

    def place(self):
        seq, i = self.rows()
        self.tokens.copy_(self.given[(self.starts[seq] + i).clamp(max=self.given.numel() - 1)])

    def run(self, tokens, sample):
        """`tokens`: a list of int64 tensors; the next token of each sequence that has any is drawn with `sample` [seqs].  Returns how
        many of them each sequence took, on the device: all, or none where pages or rows ran out (they can be given again)."""
        sizes = torch.tensor([t.numel() for t in tokens])
        self.new.copy_(sizes)
        self.starts.copy_(sizes.cumsum(0) - sizes)
        flat = torch.cat(tokens)
        self.given[:flat.numel()] = flat
        h = self.hidden()
        # a node for each sequence with rows, at the last of them; the others have none and keep the token that they have
        taken = self.indptr[1:] - self.indptr[:-1]
        some = taken > 0
        self.nodes[1:] = some.cumsum(0)
        ends = (self.indptr[1:].long() - 1).clamp(min=0)[(~some).long().argsort(stable=True)]
        probs = self.model.probabilities(h[ends])
        qlin.qlin_verify_drafts(probs, None, None, self.none, self.nodes, torch.zeros_like(sample), sample, self.path, self.kept, self.next)
        self.cache.last.copy_(torch.where(self.kept > 0, self.next, self.cache.last))
        self.cache.ctx += taken
        return taken


class Speculate(Pass):
    """One step: trees of drafts below each sequence's last token, verified; a captured graph."""

    def __init__(self, model, cache, parents):
        seqs, n = cache.ctx.numel(), len(parents)
        words, depth = tree_words(parents, (n + 63) // 64)
        super().__init__(model, cache, seqs * n, depth.repeat(seqs).to(**I32))
        self.seqs, self.n = seqs, n
        self.levels = [(p, torch.tensor([i for i, x in enumerate(parents) if x == p], **I64)) for p in sorted(set(parents[1:]))]
        self.new.fill_(n)
        # (a sequence with rows has n of them, so these are the same rows whoever has none)
        self.parent = torch.tensor([max(p, 0) for p in parents], **I32).repeat(seqs)
        self.mask = words.repeat(seqs, 1).cuda()
        self.tree = torch.zeros(seqs, n, **I64)
        self.accept, self.sample = torch.zeros(seqs * n, device="cuda"), torch.zeros(seqs, device="cuda")
        self.accept_rows = torch.zeros(seqs * n, device="cuda")
        self.path, self.kept = torch.zeros(seqs, n, **I32), torch.zeros(seqs, **I32)
        self.next, self.after = torch.zeros(seqs, **I64), torch.zeros(seqs, **I32)
        self.probs = torch.zeros(seqs * n, model.vocab, device="cuda")
        size = qlin.qlin_tree_attention_workspace_bytes(cache.handle, model.heads, n, seqs)
        self.attend = qlin.qlin_tree_attention_prepare(self.q, cache.handle, cache.table, self.indptr, cache.ctx, self.mask, self.att,
                                                       torch.empty(size, dtype=torch.uint8, device="cuda"), n)
        self.verify = qlin.qlin_verify_drafts_prepare(self.probs, None, self.parent, self.tokens, self.indptr, self.accept_rows, self.sample,
                                                      self.path, self.kept, self.next)
        self.keep = qlin.qlin_kv_cache_keep_prepare(cache.handle, cache.table, cache.ctx, self.path, self.kept, self.after)
        self.graph = None

    def draft(self):
        """Level by level, a node's children are the likeliest tokens behind it."""
        tree = self.tree
        tree[:, 0] = self.cache.last
        for p, children in self.levels:
            likely = self.model.logits(self.model.embedding[tree[:, p]]).topk(children.numel()).indices
            tree.index_copy_(1, children, likely)

    def place(self):
        seq, i = self.rows()
        i = i.clamp(max=self.n - 1)
        self.tokens.copy_(self.tree[seq, i])
        self.accept_rows.copy_(self.accept.view(self.seqs, self.n)[seq, i])

    def launch(self):
        self.draft()
        self.probs.copy_(self.model.probabilities(self.hidden()))
        self.verify.run()
        self.keep.run()
        self.cache.ctx.copy_(self.after)
        self.cache.last.copy_(torch.where(self.kept > 0, self.next, self.cache.last))  # (none kept: no pages, tried again)

    def capture(self):
        """Captures the step (on copies of the state, which a first run moves on)."""
        state = [self.cache.ctx, self.cache.last, self.cache.held, self.cache.free, self.cache.count, self.cache.table]
        saved = [t.clone() for t in state]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.launch()
        torch.cuda.current_stream().wait_stream(side)
        for t, s in zip(state, saved):
            t.copy_(s)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch()

    def run(self, accept, sample):
        """One step with these random numbers, [seqs][n] and [seqs]; returns the kept nodes and how many (none where pages ran out), as
        many, on the device."""
        self.accept.copy_(accept)
        self.sample.copy_(sample)
        if self.graph is None:
            self.capture()
        self.graph.replay()
        return self.path, self.kept


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--fmt", choices=FMT, default="int8")
    a.add_argument("--vocab", type=int, default=32000)
    a.add_argument("--hidden", type=int, default=4096)
    a.add_argument("--heads", type=int, default=32)
    a.add_argument("--kv-heads", type=int, default=8)
    a.add_argument("--seqs", type=int, default=8)
    a.add_argument("--prompt", type=int, default=4096)
    a.add_argument("--chunk", type=int, default=2048)
    a.add_argument("--steps", type=int, default=8)
    a = a.parse_args()
    qlin.build()
    parents = [-1, 0, 0, 0, 1, 1, 2, 3, 4, 4, 5, 6, 8, 8, 10, 12]
    room = a.prompt + (a.steps + 1) * len(parents)
    pages = a.seqs * -(-room // 64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda n: torch.rand(n, generator=gen, device="cuda")
    model = Model(a.vocab, a.hidden, a.heads, a.kv_heads, 128)
    cache = Cache(a.seqs, room, pages, a.kv_heads, 128, a.fmt)
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)

    def timed(what, run):
        begin.record()
        run()
        end.record()
        torch.cuda.synchronize()
        if qlin.qlin_get_device_error() != 0:
            raise RuntimeError("device error")
        print("%-46s %8.1f us" % (what, 1e3 * begin.elapsed_time(end)))

    prompts = torch.randint(a.vocab, (a.seqs, a.prompt), generator=gen, device="cuda")
    prefill = Prefill(model, cache, a.chunk)
    prefill.run(list(prompts[:, :a.chunk]), rand(a.seqs))  # (loads the kernels; the first timed pass writes the same again)
    cache.ctx.zero_()
    for at in range(0, a.prompt, a.chunk):
        part = prompts[:, at:at + a.chunk]
        timed("prompt, %d tokens behind %d, %d sequences" % (part.shape[1], at, a.seqs), lambda: prefill.run(list(part), rand(a.seqs)))
    if int(cache.ctx.min()) < a.prompt:
        raise RuntimeError("too few pages for the prompts")
    step = Speculate(model, cache, parents)
    step.capture()
    kept = 0
    for _ in range(a.steps):
        timed("trees of %d drafts" % len(parents), lambda: step.run(rand(a.seqs * len(parents)), rand(a.seqs)))
        kept += int(step.kept.sum())
    print("%.2f tokens a step and sequence; %d pages free" % (kept / (a.steps * a.seqs), int(cache.count)))


if __name__ == "__main__":
    main()
