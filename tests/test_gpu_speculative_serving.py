"""The serving operators run together, as examples/speculative_serving.py does: pages
and slots from lengths, prompts in chunks, trees of drafts, verification, kept paths;
each pass checked on what the passes before it left.

Tolerances.  Attention: as in test_gpu_chunk_attention.py (prompts) and
test_gpu_tree_attention.py (trees), for the q and the codes that the pass itself
wrote.  Pages, places, paths, tokens, moved codes: equal."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import attention as ref
from oracle import serving

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("speculative_serving", os.path.join(ROOT, "examples", "speculative_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rows(cache, b, n):
    """Codes and scales of a sequence's first n tokens, and what they stand for."""
    at = torch.arange(n, device="cuda")
    page, off = cache.table[b, at // cache.page].long(), at % cache.page
    raw = [t[page, :, off].cpu().numpy() for t in cache.tensors]
    return raw, [ref.kv_values(raw[i], raw[2 + i], cache.fmt) for i in range(2)]


def _state(cache):
    return serving.Pages(cache.table.tolist(), cache.held.tolist(), cache.free[:int(cache.count)].tolist(), cache.page, cache.table.shape[1])


def _check_pages(p, cache, state, ctx, new, depths=None):
    bounds, positions, slots = state.assign(ctx, new, p.slots.numel(), depths)
    assert p.indptr.tolist() == bounds and p.positions.tolist() == positions and p.slots.tolist() == slots
    assert cache.held.tolist() == state.held and cache.free[:int(cache.count)].tolist() == state.free
    for b, n in enumerate(state.held):
        assert cache.table[b, :n].tolist() == state.table[b][:n]


def _close(got, o, w, moved, err, length, top):
    s = (length + 64) * 2.0 ** -24
    tol = moved + (err[..., None] + 2.0 ** -11 + s) * w + length * 2.0 ** -34 * top
    tol = tol + 2.0 ** -11 * (np.abs(o) + tol) + 2.0 ** -25
    assert (np.abs(got - o) <= tol).all(), np.nanmax(np.abs(got - o) / tol)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "u4"])
def test_prompts_drafts_and_kept_paths(qlin_gpu, fmt):
    ex = _example()
    seqs, vocab, d, page, chunk = 3, 512, 64, 16, 90
    model = ex.Model(vocab, 256, 8, 2, d)
    cache = ex.Cache(seqs, 240, 40, 2, d, fmt, page)
    gen = torch.Generator().manual_seed(4)
    prefill = ex.Prefill(model, cache, chunk, window=50, prefix_lens=torch.tensor([4, 0, 100], **ex.I32))
    lens = [0] * seqs
    for new in ([90, 33, 1], [40, 0, 77]):  # prompts of different lengths, one of them done early
        state = _state(cache)
        tokens = [torch.randint(vocab, (n,), generator=gen).cuda() for n in new]
        prefill.run(tokens, torch.rand(seqs, generator=gen).cuda())
        torch.cuda.synchronize()
        assert qlin_gpu.qlin_get_device_error() == 0
        _check_pages(prefill, cache, state, lens, new)
        q, got = prefill.q.double().cpu().numpy(), prefill.att.double().cpu().numpy()
        a = 0
        for b, n in enumerate(new):
            if n > 0:
                _, (k, v) = _rows(cache, b, lens[b] + n)
                o, _, w, moved, err = serving.chunk_attention(q[a:a + n], k, v, lens[b], d ** -0.5, window=50,
                                                              prefix=min([4, 0, 100][b], lens[b] + n))
                _close(got[a:a + n], o, w, moved, err, lens[b] + n, np.abs(v).max())
            a += n
        lens = [x + n for x, n in zip(lens, new)]
        assert cache.ctx.tolist() == lens

    parents = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 6, 7]
    n, depth = len(parents), ex.tree_words(parents, 1)[1].tolist()
    seen = ((ex.tree_words(parents, 1)[0].numpy()[:, :1] >> np.arange(n)) & 1).astype(bool)
    step = ex.Speculate(model, cache, parents)
    longest = 0
    for turn in range(4):
        state, last = _state(cache), cache.last.tolist()
        accept, sample = torch.rand(seqs * n, generator=gen), torch.rand(seqs, generator=gen)
        if turn == 2:
            accept.zero_()  # every draft that the target gives any weight
        if step.graph is None:
            step.capture()
            assert cache.ctx.tolist() == lens and cache.last.tolist() == last
        # the step's state before the kept paths move: the same launches without the last three
        pages_before = [t.clone() for t in (cache.table, cache.held, cache.free, cache.count)]
        step.accept.copy_(accept)
        step.sample.copy_(sample)
        step.draft()
        probs = model.probabilities(step.hidden())
        torch.cuda.synchronize()
        before = [_rows(cache, b, lens[b] + n) for b in range(seqs)]
        for t, old in zip((cache.table, cache.held, cache.free, cache.count), pages_before):
            t.copy_(old)
        step.run(accept, sample)
        torch.cuda.synchronize()
        assert qlin_gpu.qlin_get_device_error() == 0
        _check_pages(step, cache, state, lens, [n] * seqs, depth * seqs)
        assert torch.equal(step.probs, probs)
        q, got = step.q.double().cpu().numpy(), step.att.double().cpu().numpy()
        for b in range(seqs):
            at = slice(b * n, (b + 1) * n)
            raw, (k, v) = before[b]
            bits = np.ones((n, lens[b] + n), bool)
            bits[:, lens[b]:] = seen
            o, _, w, spread = ref.tree_attention(q[at], k, v, bits, d ** -0.5)
            tol = (2.0 ** -11 + 2 * d * 2.0 ** -24 * spread + (lens[b] + n + 64) * 2.0 ** -24)[..., None] * w
            assert (np.abs(got[at] - o) <= tol + 2.0 ** -11 * np.abs(o) + 2.0 ** -24).all()
            toks = step.tokens[at].tolist()
            assert toks[0] == last[b]
            path, token = serving.verify(step.probs[at].cpu().numpy(), None, parents, toks, accept[at].numpy(), float(sample[b]))
            assert step.path[b].tolist() == path + [-1] * (n - len(path)) and int(step.kept[b]) == len(path)
            assert int(cache.last[b]) == token
            after, _ = _rows(cache, b, lens[b] + len(path))
            for x, y in zip(raw, after):
                assert np.array_equal(y[:lens[b]], x[:lens[b]]) and np.array_equal(y[lens[b]:], x[lens[b]:][path])
            longest = max(longest, len(path))
            lens[b] += len(path)
        assert cache.ctx.tolist() == lens
    assert longest > 1  # (accept of 0 takes a draft of any weight)

    # all pages go back
    cache.ctx.zero_()
    step.new.zero_()
    step.assign.run()
    torch.cuda.synchronize()
    assert int(cache.count) == 40 and sorted(cache.free.tolist()) == list(range(40)) and not cache.held.any()
    assert qlin_gpu.qlin_get_device_error() == 0


class _Spy:
    """A model's probabilities, and the rows that they were asked for."""

    def __init__(self, model):
        self.inner, self.calls = model.probabilities, []
        model.probabilities = self

    def __call__(self, h):
        probs = self.inner(h)
        self.calls.append((h.clone(), probs.clone()))
        return probs

    def of(self, row):
        """The last call's probabilities for a row equal to `row`."""
        h, probs = self.calls[-1]
        same = (h == row).all(1).nonzero()[:, 0]
        assert len(same)
        return probs[int(same[0])]


def _small(ex, seqs, pages, room=240, page=16):
    model = ex.Model(300, 256, 8, 2, 64)
    return model, ex.Cache(seqs, room, pages, 2, 64, "int8", page)


def test_prompts_of_some_sequences(qlin_gpu):
    """A sequence with tokens in a pass gets the one drawn behind its own; the others keep what they have."""
    ex = _example()
    model, cache = _small(ex, 4, 40)
    spy, gen = _Spy(model), torch.Generator().manual_seed(9)
    prefill = ex.Prefill(model, cache, 30)
    last, lens = [7, 8, 9, 10], [0] * 4
    cache.last.copy_(torch.tensor(last))
    for new in ([5, 0, 3, 0], [0, 30, 0, 1], [0, 0, 0, 2], [1, 1, 1, 1], [0, 0, 17, 0], [0, 0, 0, 0]):
        sample = torch.rand(4, generator=gen)
        prefill.run([torch.randint(300, (n,), generator=gen).cuda() for n in new], sample.cuda())
        torch.cuda.synchronize()
        h = model.embedding[prefill.tokens] + prefill.y
        for b, n in enumerate(new):
            if n > 0:
                probs = spy.of(h[int(prefill.indptr[b + 1]) - 1]).cpu().numpy()
                last[b] = serving.verify(probs[None], None, [-1], [0], [0.0], float(sample[b]))[1]
            lens[b] += n
        assert cache.last.tolist() == last and cache.ctx.tolist() == lens
    assert qlin_gpu.qlin_get_device_error() == 0


def test_prompts_that_pages_run_out_for(qlin_gpu):
    """A refused prompt changes nothing of its sequence and can be given again; one served behind it has its own tokens."""
    ex = _example()
    model, cache = _small(ex, 3, 4)
    spy, gen = _Spy(model), torch.Generator().manual_seed(3)
    prefill = ex.Prefill(model, cache, 60)
    last, lens = [7, 8, 9], [0] * 3
    cache.last.copy_(torch.tensor(last))
    for new, ended, want in (([30, 0, 3], None, [30, 0, 3]), ([0, 60, 5], None, [0, 0, 5]), ([0, 60, 0], None, [0, 0, 0]),
                             ([2, 60, 8], None, [2, 0, 8]), ([0, 60, 0], 0, [0, 0, 0]), ([0, 48, 0], None, [0, 48, 0]),
                             ([1, 0, 0], None, [0, 0, 0])):
        if ended is not None:
            cache.ctx[ended] = lens[ended] = 0
        sample = torch.rand(3, generator=gen)
        tokens = [torch.randint(300, (n,), generator=gen).cuda() for n in new]
        prefill.run(tokens, sample.cuda())
        torch.cuda.synchronize()
        assert (prefill.indptr[1:] - prefill.indptr[:-1]).tolist() == want
        h = model.embedding[prefill.tokens] + prefill.y
        for b, n in enumerate(want):
            if n > 0:
                a, e = int(prefill.indptr[b]), int(prefill.indptr[b + 1])
                assert torch.equal(prefill.tokens[a:e], tokens[b]) and prefill.positions[a:e].tolist() == list(range(lens[b], lens[b] + n))
                last[b] = serving.verify(spy.of(h[e - 1]).cpu().numpy()[None], None, [-1], [0], [0.0], float(sample[b]))[1]
            lens[b] += n
        assert cache.last.tolist() == last and cache.ctx.tolist() == lens
    assert qlin_gpu.qlin_get_device_error() == 0


def test_trees_that_pages_run_out_for(qlin_gpu):
    """A refused sequence keeps its length and its token, is taken up with them when pages come back, and the sequences behind it
    are verified with their own tokens and numbers."""
    ex = _example()
    model, cache = _small(ex, 3, 6)
    gen = torch.Generator().manual_seed(6)
    ex.Prefill(model, cache, 30).run([torch.randint(300, (n,), generator=gen).cuda() for n in (30, 16, 17)], torch.rand(3, generator=gen).cuda())
    parents = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 6, 7]
    n = len(parents)
    step = ex.Speculate(model, cache, parents)
    lens, last, refused = [30, 16, 17], cache.last.tolist(), 0
    for turn in range(6):
        if turn == 3:       # the first sequence ends
            cache.ctx[0] = step.new[0] = lens[0] = 0
        state = _state(cache)
        accept, sample = torch.rand(3 * n, generator=gen), torch.rand(3, generator=gen)
        if turn % 2:
            accept.zero_()
        step.run(accept, sample)
        torch.cuda.synchronize()
        bounds, _, _ = state.assign(lens, step.new.tolist(), 3 * n, ex.tree_words(parents, 1)[1].tolist() * 3)
        assert step.indptr.tolist() == bounds
        for b in range(3):
            a, e = bounds[b:b + 2]
            if a == e:
                assert int(step.kept[b]) == 0
                refused += turn < 3 and b == 1
                continue
            toks = step.tokens[a:e].tolist()
            assert toks[0] == last[b]
            path, last[b] = serving.verify(step.probs[a:e].cpu().numpy(), None, parents, toks, accept[b * n:b * n + n].numpy(), float(sample[b]))
            assert step.path[b].tolist() == path + [-1] * (n - len(path)) and int(step.kept[b]) == len(path)
            lens[b] += len(path)
        assert cache.ctx.tolist() == lens and cache.last.tolist() == last
    assert refused > 0 and lens[1] > 16 and qlin_gpu.qlin_get_device_error() == 0


def test_the_command_runs(qlin_gpu):
    import subprocess
    import sys
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "speculative_serving.py"), "--hidden", "512", "--heads", "8",
                        "--kv-heads", "2", "--vocab", "1024", "--seqs", "2", "--prompt", "300", "--chunk", "128", "--steps", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "pages free" in r.stdout, r.stdout + r.stderr
