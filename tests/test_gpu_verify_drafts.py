"""Drafted tokens verified from given random numbers: path, count and next token
equal the 64-bit oracle's.  (Its sums round at 2^-53, the library's weights are cut
at 2^-52: with fixed seeds no draw below lies that near to a border, as random ones
do with a probability of about V 2^-40.)"""

import numpy as np
import pytest
import torch

from oracle import serving as ref

pytestmark = pytest.mark.gpu


def _softmax(x):
    return torch.softmax(x, -1)


class Problem:
    def __init__(self, nodes, v, fan, drawn, agree=0.5, seed=0, offset=0, pad=0, max_nodes=None):
        g = torch.Generator().manual_seed(seed + 17 * v)
        self.nodes, tq = nodes, sum(nodes)
        base = 2.0 * torch.randn(tq, v, generator=g)

        def rows(x):
            whole = torch.full((tq, v + offset + pad), 7.0)
            whole[:, offset: offset + v] = _softmax(x)
            return whole.cuda()[:, offset: offset + v]
        self.target = rows(base + 3 * (1 - agree) * torch.randn(tq, v, generator=g))
        self.draft = rows(base) if drawn else None
        self.parents, up = [], []
        for n in nodes:
            first = len(up)
            for i in range(n):
                parent = -1 if i == 0 else (i - 1) // fan
                self.parents.append(parent)
                up.append(first + max(parent, 0))
        probs = _softmax(base)
        if drawn:
            self.tokens = torch.multinomial(probs[up], 1, generator=g)[:, 0] if tq else torch.zeros(0).long()
        else:
            which = torch.tensor([(i - 1) % fan if i else 0 for n in nodes for i in range(n)], dtype=torch.int64)
            self.tokens = probs[up].topk(min(v, fan), -1).indices[torch.arange(tq), which % min(v, fan)]
        self.accept, self.sample = torch.rand(tq, generator=g), torch.rand(len(nodes), generator=g)
        self.indptr = torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32)
        self.chain = fan == 1
        self.max_nodes = max_nodes or max(nodes + [1])

    def outputs(self):
        b = len(self.nodes)
        return (torch.full((b, self.max_nodes), 9, dtype=torch.int32, device="cuda"), torch.full((b,), 9, dtype=torch.int32, device="cuda"),
                torch.full((b,), 9, dtype=torch.int64, device="cuda"))

    def args(self):
        parents = None if self.chain else torch.tensor(self.parents, dtype=torch.int32).cuda()
        return (self.target, self.draft, parents, self.tokens.cuda(), self.indptr.cuda(), self.accept.cuda(), self.sample.cuda())

    def want(self):
        t, d = self.target.cpu().numpy(), None if self.draft is None else self.draft.cpu().numpy()
        got = []
        for b, n in enumerate(self.nodes):
            a = int(self.indptr[b])
            s = slice(a, a + n)
            got.append(ref.verify(t[s], None if d is None else d[s], self.parents[s], self.tokens[s].tolist(), self.accept[s].double().tolist(),
                                  float(self.sample[b])))
        return got

    def check(self, path, count, nxt, want=None):
        for b, (p, x) in enumerate(want or self.want()):
            assert path[b].tolist() == p + [-1] * (self.max_nodes - len(p)), b
            assert int(count[b]) == len(p) and int(nxt[b]) == x, b


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("fan", [1, 2, 4])
@pytest.mark.parametrize("v", [1, 5, 127, 1000, 32000, 50257])
def test_sizes(qlin_gpu, v, fan, drawn):
    for seed in range(4):
        p = Problem([1, 0, 7, 26, 3, 64], v, fan, drawn, agree=0.2 * seed, seed=seed)
        out = p.outputs()
        qlin_gpu.qlin_verify_drafts(*p.args(), *out)
        p.check(*out)
    assert qlin_gpu.qlin_get_device_error() == 0


@pytest.mark.parametrize("drawn", [True, False])
def test_large(qlin_gpu, drawn):
    """The largest vocabulary, the most nodes, many sequences."""
    p = Problem([3, 2], 1 << 20, 1, drawn)
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    p.check(*out)
    p = Problem([256, 1, 200], 3001, 6, drawn, agree=0.0)
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    p.check(*out)
    p = Problem([1 + i % 5 for i in range(700)], 515, 2, drawn)
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    p.check(*out)


@pytest.mark.parametrize("drawn,fan", [(True, 1), (True, 3), (False, 3)])
@pytest.mark.parametrize("seqs,v", [(19, 40001), (20, 40001), (76, 9000), (77, 9000), (90, 70003)])
def test_batches(qlin_gpu, seqs, v, drawn, fan):
    """Numbers of sequences around those at which fewer blocks take each of them."""
    p = Problem([1 + (b * 7) % 5 for b in range(seqs)], v, fan, drawn, agree=0.3)
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    p.check(*out)
    assert qlin_gpu.qlin_get_device_error() == 0


@pytest.mark.parametrize("offset,pad", [(1, 0), (2, 3), (4, 4), (0, 1), (3, 1)])
def test_strides_and_alignments(qlin_gpu, offset, pad):
    for v in (31, 4100):
        p = Problem([5, 9, 1], v, 2, True, seed=offset, offset=offset, pad=pad, max_nodes=20)
        out = p.outputs()
        qlin_gpu.qlin_verify_drafts(*p.args(), *out)
        p.check(*out)


def test_entries_that_are_no_probabilities(qlin_gpu):
    """NaN and what is below 0 counts as 0, above 1 as 1; random numbers outside [0, 1) as the nearest inside."""
    p = Problem([4, 4, 4, 4], 300, 3, True, agree=0.0)
    for t in (p.target, p.draft):
        t[:, ::7] = float("nan")
        t[:, 1::11] = -0.5
        t[3, 5] = float("inf")
    p.accept[5], p.accept[9] = -1.0, 1.0
    p.sample[0], p.sample[1], p.sample[2] = 1.5, -2.0, 0.0
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    below = float(np.nextafter(np.float32(1), np.float32(0)))
    p.accept[5], p.accept[9] = 0.0, below
    p.sample[0], p.sample[1] = below, 0.0
    p.check(*out)


def test_rows_without_weight(qlin_gpu):
    """Nothing left after a rejection: drawn from p; a row of zeros: no token."""
    q = qlin_gpu
    eye = torch.eye(8)
    p = Problem([2, 2, 1], 8, 1, True)
    p.target = torch.stack([eye[3], eye[1], eye[6], eye[0], 0 * eye[0]]).cuda()
    p.draft = p.target.clone()
    p.tokens = torch.tensor([0, 5, 0, 6, 0])             # 5 is impossible: rejected, and max(p - q, 0) is 0
    out = p.outputs()
    q.qlin_verify_drafts(*p.args(), *out)
    assert out[1].tolist() == [1, 2, 1] and out[2].tolist() == [3, 0, -1]
    p.draft = None
    p.tokens = torch.tensor([0, 3, 0, 6, 0])
    p.target[0, 3] = 0.5                                 # all of what there is, rejected
    p.accept = torch.tensor([0.0, 0.9, 0.0, 0.9, 0.0])
    q.qlin_verify_drafts(*p.args(), *out)
    p.check(*out)
    assert out[1].tolist() == [1, 2, 1] and out[2].tolist() == [3, 0, -1] and q.qlin_get_device_error() == 0


@pytest.mark.parametrize("v", [8, 4099])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("parents", [[-1, 0, 1], [-1, 0, 1, 2, 3, 4], [-1, 0, 0, 0], [-1, 0, 0, 1, 1, 2, 0], [-1, 0, 1, 1, 3], [-1, 0, 0, 2, 2, 1, 3]])
def test_nothing_left_before_the_last_node(qlin_gpu, parents, drawn, v):
    """A rejection after which nothing is left draws from p, whatever nodes follow: the rest of the chain, siblings, others' children."""
    n = len(parents)
    at = [(3 * i + 1) % v for i in range(n)]             # each row has one token
    for first in range(1, n):                            # the first node that cannot be, its drafts' row as the target's
        p = Problem([n, 1, n], v, 2, drawn)
        rows = torch.zeros(n, v)
        rows[torch.arange(n), at] = 1.0 if drawn else 0.5
        p.target = torch.cat([rows, rows[:1], rows]).cuda()
        p.draft = p.target.clone() if drawn else None
        up = [max(x, 0) for x in parents]
        own = torch.tensor([0] + [at[up[i]] if i < first or not drawn else (at[up[i]] + 1) % v for i in range(1, n)])
        p.tokens = torch.cat([own, own[:1], own])
        p.accept = torch.tensor([0.0 if i < first else 0.9 for i in range(n)]).repeat(3)[:2 * n + 1]
        p.accept[n:] = torch.cat([torch.zeros(1), p.accept[:n]])
        p.parents = parents + [-1] + parents
        out = p.outputs()
        qlin_gpu.qlin_verify_drafts(*p.args(), *out)
        p.check(*out)
        assert (out[2] >= 0).all() and qlin_gpu.qlin_get_device_error() == 0


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("v", [3, 6, 700])
def test_rows_of_eighths(qlin_gpu, v, drawn):
    """Rows of few whole eighths, alike more often than not, trees of any shape: everything is exact in the oracle too, and
    nothing left, ties and tokens twice among siblings are common."""
    r = np.random.default_rng(v)
    for turn in range(8):
        nodes = [int(x) for x in r.integers(0, 9, 60)]
        p = Problem(nodes, v, 2, drawn, seed=turn)
        rows = lambda: r.multinomial(8, np.r_[0.5, 0.3, 0.2, np.zeros(v - 3)], sum(nodes)) / 8
        target = rows()
        draft = np.where(r.random((sum(nodes), 1)) < 0.6, target, rows())
        p.target = torch.from_numpy(target).float().cuda()
        p.draft = torch.from_numpy(draft).float().cuda() if drawn else None
        p.parents = [-1 if i == 0 else int(r.integers(max(0, i - 4), i)) for n in nodes for i in range(n)]
        p.tokens = torch.from_numpy(r.integers(0, 3, sum(nodes)))
        p.accept = torch.from_numpy(r.integers(0, 8, sum(nodes)) / 8).float()
        out = p.outputs()
        qlin_gpu.qlin_verify_drafts(*p.args(), *out)
        p.check(*out)
    assert qlin_gpu.qlin_get_device_error() == 0


def test_bad_indexes(qlin_gpu):
    """A parent or a token out of range: the node is not accepted, and it is recorded; bounds out of range: no nodes."""
    q = qlin_gpu
    for what, value in (("parent", 4), ("parent", -1), ("parent", 100), ("token", 200), ("token", -1)):
        p = Problem([6], 200, 2, False, agree=1.0)
        p.accept[:] = 0.0
        if what == "parent":
            p.parents[2] = value
        else:
            p.tokens[2] = value
        out = p.outputs()
        q.qlin_verify_drafts(*p.args(), *out)
        assert q.qlin_get_device_error() == 0x2000
        p.parents[2] = p.parents[2] if what == "token" else -7
        p.check(*out)
    for bounds in ([0, 4, 2], [-1, 3, 6], [0, 5, 7]):
        p = Problem([3, 3], 200, 2, False)
        p.indptr = torch.tensor(bounds, dtype=torch.int32)
        out = p.outputs()
        q.qlin_verify_drafts(*p.args(), *out)
        assert q.qlin_get_device_error() == 0x2000
        assert 0 in out[1].tolist() and -1 in out[2].tolist()


def test_no_rows(qlin_gpu):
    p = Problem([0, 0], 10, 1, True)
    out = p.outputs()
    qlin_gpu.qlin_verify_drafts(*p.args(), *out)
    assert out[0].tolist() == [[-1]] * 2 and out[1].tolist() == [0, 0] and out[2].tolist() == [-1, -1]


def test_draws_follow_the_sums(qlin_gpu):
    """The token drawn moves with sample_u exactly where the sums of powers of two are."""
    q, v = qlin_gpu, 6000
    target = torch.zeros(1, v, device="cuda")
    at = [0, 17, 2047, 2048, 4095, 5999]
    for i, x in enumerate(at):
        target[0, x] = 2.0 ** -(i + 1) if i < 5 else 2.0 ** -5
    edge, u, want = 0.0, [], []
    for i, x in enumerate(at):
        u += [edge, float(np.nextafter(np.float32(edge + float(target[0, x])), np.float32(0)))]
        want += [x, x]
        edge += float(target[0, x])
    n = len(u)
    rows = target.expand(n, v).contiguous()
    out = (torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"),
           torch.zeros(n, dtype=torch.int64, device="cuda"))
    zeros = torch.zeros(n, device="cuda")
    q.qlin_verify_drafts(rows, None, None, torch.zeros(n, dtype=torch.int64, device="cuda"),
                         torch.arange(n + 1, dtype=torch.int32, device="cuda"), zeros, torch.tensor(u, device="cuda"), *out)
    assert out[2].tolist() == want


def test_replayed_and_on_another_stream(qlin_gpu):
    q = qlin_gpu
    a, b = Problem([5, 26, 1], 5000, 3, True, seed=1, max_nodes=30), Problem([12, 10, 10], 5000, 3, True, seed=2, max_nodes=30)
    args, out = a.args(), a.outputs()
    call = q.qlin_verify_drafts_prepare(*args, *out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.run(side)
    torch.cuda.current_stream().wait_stream(side)
    a.check(*out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for p in (b, a):
        for x, y in zip(args, p.args()):
            x.copy_(y)
        graph.replay()
        p.check(*out)
