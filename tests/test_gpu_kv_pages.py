"""Pages, row bounds, positions and slots from lengths: every output equals the
oracle's (whole numbers), and a random run of steps never loses a page."""

import random

import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class Pool:
    def __init__(self, q, seqs, pages, page, max_pages, seed=0):
        free = random.Random(seed).sample(range(pages), pages)
        self.q, self.table, self.held = q, torch.full((seqs, max_pages), -1, dtype=torch.int32, device="cuda"), _ints([0] * seqs)
        self.free, self.count = _ints(free), _ints([pages])
        self.pages = q.qlin_kv_pages(self.table, self.held, self.free, self.count, page)
        self.ref = ref.Pages(self.table.tolist(), [0] * seqs, free, page, max_pages)

    def step(self, ctx, new, rows, depths=None, stream=None):
        seqs = len(ctx)
        indptr, positions, slots = _ints([9] * (seqs + 1)), _ints([9] * rows, torch.int64), _ints([9] * rows, torch.int64)
        self.q.qlin_kv_pages_assign(self.pages, _ints(ctx), _ints(new), indptr, positions, slots,
                                    None if depths is None else _ints(depths), stream=stream)
        want = self.ref.assign(ctx, new, rows, depths)
        assert (indptr.tolist(), positions.tolist(), slots.tolist()) == want
        self.same()
        return indptr, positions, slots

    def same(self):
        held, count = self.held.tolist(), int(self.count)
        assert held == self.ref.held
        assert self.free.tolist()[:count] == self.ref.free
        for b, row in enumerate(self.table.tolist()):
            assert row[:held[b]] == self.ref.table[b][:held[b]]


@pytest.mark.parametrize("seqs,page,rows", [(1, 16, 1), (3, 32, 40), (70, 64, 300), (1024, 16, 2048), (1025, 16, 2049), (2500, 128, 9000)])
def test_random_steps(qlin_gpu, seqs, page, rows):
    """Sequences begin, grow, shrink and end; the pool and the rows run short now and then."""
    r = random.Random(seqs)
    most = 6
    pool = Pool(qlin_gpu, seqs, max(3, seqs * 3), page, most)
    ctx = [0] * seqs
    for step in range(12):
        new = [r.choice([0, 1, 1, r.randint(0, 2 * page)]) if r.random() < 0.8 else r.randint(0, max(1, rows // seqs)) for _ in ctx]
        new = [min(n, most * page - c) for n, c in zip(new, ctx)]
        depths = [r.randint(0, 9) for _ in range(rows)] if step % 3 == 0 else None
        indptr, _, _ = pool.step(ctx, new, rows, depths)
        served = (indptr[1:] - indptr[:-1]).tolist()
        for b in range(seqs):
            ctx[b] = 0 if r.random() < 0.15 else ctx[b] + r.randint(0, served[b])
        used = [x for b in range(seqs) for x in pool.ref.table[b][:pool.ref.held[b]]] + pool.ref.free
        assert sorted(used) == list(range(max(3, seqs * 3)))
    pool.step([0] * seqs, [0] * seqs, rows)
    assert int(pool.count) == max(3, seqs * 3)
    assert qlin_gpu.qlin_get_device_error() == 0


def test_a_step_taken_back(qlin_gpu):
    pool = Pool(qlin_gpu, 5, 64, 16, 12)
    pool.step([0] * 5, [33, 1, 160, 0, 16], 256)
    before = [t.clone() for t in (pool.free, pool.count, pool.held)]
    ctx = [33, 1, 160, 0, 16]
    for _ in range(3):
        first = [t.clone() for t in pool.step(ctx, [40, 16, 2, 70, 1], 256)]
        again = pool.step(ctx, [40, 16, 2, 70, 1], 256)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        pool.step(ctx, [0] * 5, 256)
        assert all(torch.equal(a, b) for a, b in zip(before, (pool.free, pool.count, pool.held)))


@pytest.mark.parametrize("seqs,rows", [(7, 40), (300, 1500), (1200, 5000)])
def test_depths_of_trees_that_differ(qlin_gpu, seqs, rows):
    """Sequences run out of pages or rows: depths packed by a first call's row bounds are those of their own sequences' nodes."""
    r = random.Random(rows)
    page = 16
    pool = Pool(qlin_gpu, seqs, seqs * 2, page, 5)
    refused = 0
    for turn in range(4):
        ctx = [r.randint(0, 3 * page) if turn else 0 for _ in range(seqs)]
        new = [r.randint(0, 2 * page - 4) if r.random() < 0.3 else r.randint(0, 4) for _ in range(seqs)]
        trees = [[r.randint(0, 9) for _ in range(n)] for n in new]
        indptr, _, slots = [t.clone() for t in pool.step(ctx, new, rows)]
        first = torch.tensor([0] + new).cumsum(0).cuda()
        flat = _ints([x for t in trees for x in t] + [0] * rows)
        at = torch.arange(rows, dtype=torch.int32, device="cuda")
        seq = torch.searchsorted(indptr[1:], at, right=True).clamp(max=seqs - 1)
        depths = flat[(first[seq] + at - indptr[seq]).clamp(max=flat.numel() - 1)]
        again, positions, slots2 = pool.step(ctx, new, rows, depths.tolist())
        assert torch.equal(indptr, again) and torch.equal(slots, slots2)
        bounds, positions = indptr.tolist(), positions.tolist()
        for b, (c, n) in enumerate(zip(ctx, new)):
            a, e = bounds[b:b + 2]
            assert positions[a:e] == [c + x for x in trees[b]][:e - a] and e - a in (0, n)
            refused += e - a < n
    assert refused > 0 and qlin_gpu.qlin_get_device_error() == 0


def test_long_prompt(qlin_gpu):
    """One sequence takes 8192 pages and gives them back."""
    pool = Pool(qlin_gpu, 2, 8200, 16, 8192)
    pool.step([0, 0], [131072, 128], 140000)
    pool.step([131072, 128], [0, 1], 1)
    pool.step([0, 128], [0, 0], 0)
    assert qlin_gpu.qlin_get_device_error() == 0


def test_no_sequences(qlin_gpu):
    slots = _ints([5, 5, 5], torch.int64)
    positions, indptr = slots.clone(), _ints([7])
    pages = qlin_gpu.qlin_kv_pages(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), _ints([]), _ints([0, 1]), _ints([2]), 16)
    qlin_gpu.qlin_kv_pages_assign(pages, _ints([]), _ints([]), indptr, positions, slots)
    assert slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3 and indptr.tolist() == [0]


@pytest.mark.parametrize("ctx,new", [([-1, 5], [3, 4]), ([5, 5], [-2, 4]), ([60, 5], [5, 4]), ([2 ** 31 - 1, 5], [2 ** 31 - 1, 4])])
def test_lengths_out_of_range(qlin_gpu, ctx, new):
    """Recorded; the sequence keeps what it has, the other one is served."""
    pool = Pool(qlin_gpu, 2, 8, 16, 4)
    pool.step([0, 0], [20, 0], 64)
    pool.step(ctx, new, 64)
    assert qlin_gpu.qlin_get_device_error() == 0x2000


def test_stack_out_of_range(qlin_gpu):
    """A count below 0 or above the pages, and pages given back beyond the stack's end: recorded, nothing is written past it."""
    q = qlin_gpu
    for count in (-3, 9):
        whole = torch.full((12,), 77, dtype=torch.int32, device="cuda")
        free = whole[2:10]
        pages = q.qlin_kv_pages(torch.zeros(1, 4, dtype=torch.int32, device="cuda"), _ints([2]), free, _ints([count]), 16)
        q.qlin_kv_pages_assign(pages, _ints([0]), _ints([0]), _ints([0, 0]), _ints([], torch.int64), _ints([], torch.int64))
        assert q.qlin_get_device_error() == 0x2000
        assert whole[:2].tolist() == [77, 77] and whole[10:].tolist() == [77, 77]


@pytest.mark.parametrize("seqs,rows", [(1, 0), (3, 40), (1500, 40), (3, 3000)])
@pytest.mark.parametrize("count", [-3, -2 ** 31, 0, 2 ** 31 - 1, "one too many", "one too many free"])
def test_a_stack_out_of_range_moves_nothing(qlin_gpu, seqs, rows, count):
    """Pages that would go back, be taken or be kept all stay where they are, and there are no rows."""
    q, most, pages = qlin_gpu, 4, seqs * 4
    gives = seqs * 2
    bad = {"one too many": pages - gives + 1, "one too many free": pages + 1}.get(count, count)
    held = [3] * seqs
    table = torch.arange(seqs * most, dtype=torch.int32, device="cuda").view(seqs, most)
    state = [table, _ints(held), _ints(list(range(pages))), _ints([bad])]
    before = [x.clone() for x in state]
    pool = q.qlin_kv_pages(*state, 16)
    indptr, positions, slots = _ints([9] * (seqs + 1)), _ints([9] * rows, torch.int64), _ints([9] * rows, torch.int64)
    ctx, new = [0 if b < gives // 2 else 40 for b in range(seqs)], [1] * seqs
    q.qlin_kv_pages_assign(pool, _ints(ctx), _ints(new), indptr, positions, slots)
    if count == 0:    # (an empty stack is one)
        assert q.qlin_get_device_error() == 0 and state[3].item() == gives and state[1].tolist() == [1] * seqs
        return
    assert q.qlin_get_device_error() == 0x2000
    assert all(torch.equal(x, y) for x, y in zip(state, before))
    assert not indptr.any() and not positions.any() and bool((slots == -1).all())


def test_page_numbers_out_of_range(qlin_gpu):
    """A table that holds a page that is none gives no slot there."""
    q = qlin_gpu
    table = _ints([[3, -1, 9, 0]])
    pages = q.qlin_kv_pages(table, _ints([4]), _ints([0] * 8), _ints([0]), 16)
    slots, positions, indptr = _ints([7] * 64, torch.int64), _ints([7] * 64, torch.int64), _ints([0, 0])
    q.qlin_kv_pages_assign(pages, _ints([0]), _ints([64]), indptr, positions, slots)
    assert q.qlin_get_device_error() == 0x2000
    assert slots.tolist() == list(range(48, 64)) + [-1] * 32 + list(range(16)) and positions.tolist() == list(range(64))


def test_replayed_and_on_another_stream(qlin_gpu):
    """A captured call follows the lengths it finds; calls on a side stream too."""
    q = qlin_gpu
    pool = Pool(q, 3, 40, 16, 10)
    ctx, new = _ints([0, 0, 0]), _ints([0, 0, 0])
    indptr, positions, slots = _ints([0] * 4), _ints([0] * 3000, torch.int64), _ints([0] * 3000, torch.int64)
    call = q.qlin_kv_pages_assign_prepare(pool.pages, ctx, new, indptr, positions, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.run(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for a, b in (([0, 0, 0], [5, 100, 16]), ([5, 100, 16], [1, 1, 1]), ([5, 0, 17], [12, 0, 1])):
        ctx.copy_(_ints(a))
        new.copy_(_ints(b))
        graph.replay()
        assert (indptr.tolist(), positions.tolist(), slots.tolist()) == pool.ref.assign(a, b, 3000)
        pool.same()
