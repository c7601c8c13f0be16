"""Pages and slots, chunk attention, verified drafts and kept paths: what is
refused on the host before the device is touched (no GPU here), empty problems,
and the oracle against closed forms and frequencies."""

import copy
import ctypes

import numpy as np
import pytest
import torch

import quantized_linear_layer_gb300 as q
from oracle import serving as ref
from test_kv_abi import ALIGN, INVALID, L, OK, P, UNSUPPORTED, cache, heads, ref as ptr  # noqa: F401


def changed(base, change):
    a = copy.copy(base)
    a.update(change)
    return a


def test_pages_refusals(L):
    def call(b=2, t=5, ctx=16, new=16, depths=None, indptr=16, positions=16, slots=16, null=False, **change):
        c = q._KvPages(16, 4, 16, 16, 16, 10, 32)
        for k, v in change.items():
            setattr(c, k, v)
        return L.qlin_kv_pages_assign(None if null else ptr(c), P(ctx), P(new), b, t, P(depths), P(indptr), P(positions), P(slots), None)
    assert call(null=True) == INVALID
    for change in ({"b": -1}, {"b": 65536}, {"t": -1}, {"t": 1 << 31}, {"pages": 0}, {"pages": 1 << 31}, {"max_pages": -1},
                   {"block_table": None}, {"held": None}, {"ctx": None}, {"new": None}, {"free_pages": None}, {"free_count": None},
                   {"indptr": None}, {"positions": None}, {"slots": None}):
        assert call(**change) == INVALID, change
    for size in (0, 8, 48, 512):
        assert call(page_size=size) == UNSUPPORTED
    for change in ({"block_table": 18}, {"held": 17}, {"free_pages": 18}, {"free_count": 18}, {"ctx": 18}, {"new": 18}, {"depths": 18},
                   {"indptr": 18}, {"positions": 20}, {"slots": 20}):
        assert call(**change) == ALIGN, change


def test_chunk_refusals(L):
    base = dict(qh=heads(8), out=heads(8), dtype=0, tq=3, c=cache(), table=16, pages=4, indptr=16, ctx=16, b=2, most=3, lse=16, ws=256,
                size=1 << 50, scale=0.1, cap=0.0, slopes=None, window=0, prefix=None)

    def call(**change):
        a = changed(base, change)
        how = q._Scores(a["scale"], a["cap"], a["slopes"], a["window"], a["prefix"])
        return L.qlin_chunk_attention(ptr(a["qh"]), ptr(a["out"]), a["dtype"], a["tq"], ptr(a["c"]), P(a["table"]), a["pages"],
                                      P(a["indptr"]), P(a["ctx"]), a["b"], a["most"], None if a.get("null") else ptr(how), P(a["lse"]),
                                      P(a["ws"]), a["size"], None)
    nan, inf = float("nan"), float("inf")
    for change in ({"dtype": 2}, {"tq": -1}, {"b": -1}, {"b": 65536}, {"pages": -1}, {"scale": nan}, {"scale": inf}, {"cap": nan},
                   {"cap": -1.0}, {"cap": inf}, {"cap": 1e-4}, {"window": -1}, {"window": 1 << 31}, {"most": 0}, {"most": 1 << 31},
                   {"c": None}, {"qh": None}, {"out": heads(4)}, {"qh": heads(3), "out": heads(3)}, {"table": None}, {"indptr": None},
                   {"ctx": None}, {"ws": None}, {"null": True}):
        assert call(**change) == INVALID, change
    assert call(c=cache(head_dim=96)) == UNSUPPORTED and call(c=cache(page_size=8)) == UNSUPPORTED
    for change in ({"table": 18}, {"indptr": 18}, {"ctx": 18}, {"lse": 18}, {"slopes": 18}, {"prefix": 18}, {"ws": 272},
                   {"qh": heads(8, data=24)}):
        assert call(**change) == ALIGN, change
    assert call(tq=0, table=None, ws=None) == OK and call(b=0, table=None, ws=None) == OK
    size = L.qlin_chunk_attention_workspace_bytes
    assert size(ptr(cache()), 8, 64, 4) > 0 and size(ptr(cache()), 8, 1 << 20, 4) > 0
    assert size(ptr(cache()), 7, 64, 4) == -1 and size(ptr(cache()), 8, 0, 4) == -1 and size(ptr(cache(fmt=7)), 8, 4, 4) == -1


def test_verify_and_keep_refusals(L):
    base = dict(target=16, ts=100, draft=16, ds=100, v=100, tq=3, parents=16, tokens=16, indptr=16, b=2, nodes=3, acc=16, smp=16,
                path=16, count=16, nxt=16)

    def verify(**change):
        a = changed(base, change)
        return L.qlin_verify_drafts(P(a["target"]), a["ts"], P(a["draft"]), a["ds"], a["v"], a["tq"], P(a["parents"]), P(a["tokens"]),
                                    P(a["indptr"]), a["b"], a["nodes"], P(a["acc"]), P(a["smp"]), P(a["path"]), P(a["count"]),
                                    P(a["nxt"]), None)
    for change in ({"tq": -1}, {"b": -1}, {"b": 65536}, {"ts": 99}, {"ds": 99}, {"ts": 1 << 41}, {"ts": -4, "tq": 1}, {"target": None},
                   {"tokens": None}, {"indptr": None}, {"acc": None}, {"smp": None}, {"path": None}, {"count": None}, {"nxt": None}):
        assert verify(**change) == INVALID, change
    for change in ({"v": 0}, {"v": (1 << 20) + 1}, {"nodes": 0}, {"nodes": 257}):
        assert verify(**change) == UNSUPPORTED, change
    for change in ({"target": 18}, {"draft": 18}, {"parents": 18}, {"tokens": 20}, {"acc": 18}, {"path": 18}, {"nxt": 20}):
        assert verify(**change) == ALIGN, change
    assert verify(b=0, path=None) == OK

    base2 = dict(c=cache(), table=16, pages=4, ctx=16, path=16, count=16, b=2, most=3, lens=32)

    def keep(**change):
        a = changed(base2, change)
        return L.qlin_kv_cache_keep(ptr(a["c"]), P(a["table"]), a["pages"], P(a["ctx"]), P(a["path"]), P(a["count"]), a["b"], a["most"],
                                    P(a["lens"]), None)
    for change in ({"c": None}, {"c": cache(fmt=9)}, {"b": -1}, {"b": 65536}, {"most": -1}, {"most": 65536}, {"pages": -1}, {"table": None},
                   {"ctx": None}, {"path": None}, {"count": None}, {"lens": 16}):
        assert keep(**change) == INVALID, change
    for change in ({"table": 18}, {"ctx": 18}, {"path": 18}, {"count": 18}, {"lens": 18}):
        assert keep(**change) == ALIGN, change
    assert keep(c=cache(page_size=48)) == UNSUPPORTED and keep(b=0, table=None) == OK


def test_keep_refuses_lengths_over_what_it_reads(L):
    """lens may share no byte with what the blocks of a sequence still read when one of them writes it."""
    call = ctypes.cast((ctypes.c_uint64 * 112)(), P)
    at = dict(table=1024, ctx=2048, path=4096, count=8192)          # 4 sequences: 48, 16, 80 and 16 bytes

    def keep(lens, **change):
        a = changed(at, change)
        return L.qlin_kv_cache_keep_prepare(ptr(cache()), P(a["table"]), 3, P(a["ctx"]), P(a["path"]), P(a["count"]), 4, 5,
                                            None if lens is None else P(lens), call)
    for name, size in (("table", 48), ("ctx", 16), ("path", 80), ("count", 16)):
        for lens in (at[name] - 12, at[name], at[name] + 4, at[name] + size - 4):
            assert keep(lens) == INVALID, (name, lens)
        for lens in (at[name] - 16, at[name] + size):
            assert keep(lens) != INVALID, (name, lens)
    assert keep(None) != INVALID


def test_prepared_refusals(L):
    c = (ctypes.c_uint64 * 112)()
    at = ctypes.cast(c, P)
    how = q._Scores(0.1, 0.0, None, 0, None)
    args = (ptr(heads(8)), ptr(heads(8)), 0, 0, ptr(cache()), None, 4, None, None, 2, 3, ptr(how), None, None, 0)
    assert L.qlin_chunk_attention_prepare(*args, None) == INVALID
    assert L.qlin_chunk_attention_prepare(*args, at) == OK and L.qlin_call_run(at, None) == OK
    assert L.qlin_kv_cache_keep_prepare(None, None, 4, None, None, None, 2, 3, None, at) == INVALID
    assert L.qlin_call_run(at, None) == INVALID
    assert L.qlin_verify_drafts_prepare(None, 9, None, 0, 9, 0, None, None, None, 0, 3, None, None, None, None, None, at) == OK
    assert L.qlin_call_run(at, None) == OK


def test_binding_refusals():
    """Wrong types, shapes and devices raise before a call is made (CPU tensors are refused, not computed)."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q.qlin_kv_pages(i(2, 4), i(2), i(8), i(1), 16)
    with pytest.raises(ValueError, match="max_pages"):
        q.qlin_kv_pages(i(8), i(2), i(8), i(1), 16)
    with pytest.raises(TypeError, match="dtype"):
        q.qlin_kv_pages(i(2, 4).long(), i(2), i(8), i(1), 16)
    probs = torch.zeros(3, 10)
    with pytest.raises(ValueError, match="CUDA"):
        q.qlin_verify_drafts(probs, None, None, torch.zeros(3).long(), i(2), probs[:, 0], probs[0, :1], i(1, 3), i(1), torch.zeros(1).long())
    with pytest.raises(ValueError, match="path"):
        q.qlin_verify_drafts(probs, None, None, None, None, None, None, i(3), None, None)
    with pytest.raises(TypeError, match="dtype"):
        q.qlin_verify_drafts(probs.half(), None, None, None, None, None, None, i(1, 3), None, None)


def test_oracle_pages():
    """Pages come from the top of the stack in the order of the sequences; a step that is taken back changes nothing."""
    s = ref.Pages([[7, -1, -1], [-1] * 3, [-1] * 3], [1, 0, 0], [1, 2, 3, 4], 16, 3)
    bounds, positions, slots = s.assign([15, 0, 0], [2, 33, 1], 40)
    assert s.table[0][:2] == [7, 4] and s.table[1] == [3, 2, 1] and s.held == [2, 3, 0] and s.free == []
    assert bounds == [0, 2, 35, 35]                      # nothing was left for the last
    assert slots[:3] == [7 * 16 + 15, 4 * 16, 3 * 16] and slots[34] == 16 and slots[35:] == [-1] * 5 and positions[:3] == [15, 16, 0]
    s.assign([15, 0, 0], [0, 0, 0], 40)
    assert s.free == [1, 2, 3, 4] and s.held == [1, 0, 0]


def test_oracle_chunk():
    """Equal keys average the values seen; a cap bounds the scores; a slope of ln 2 halves the weight a token further back."""
    r = np.random.default_rng(0)
    k, v, x = np.ones((6, 1, 4)), r.normal(size=(6, 1, 4)), r.normal(size=(3, 2, 4))
    out, lse, *_ = ref.chunk_attention(x, k, v, 3, 0.5, window=2, prefix=1)
    assert np.allclose(out[1, 0], v[[0, 3, 4], 0].mean(0)) and np.allclose(lse[:, 1], 0.5 * x[:, 1].sum(-1) + np.log(3))
    assert np.allclose(ref.chunk_attention(x, k, v, 3, 0.5, prefix=6)[0][0, 1], v[:, 0].mean(0))
    out, *_ = ref.chunk_attention(x, k, v, 3, 0.5, slopes=[np.log(2), 0.0])
    w = 2.0 ** np.arange(-3, 1)
    assert np.allclose(out[0, 0], w @ v[:4, 0] / w.sum()) and np.allclose(out[0, 1], v[:4, 0].mean(0))
    assert (ref.chunk_attention(100 * x, k, v, 3, 1.0, softcap=2.0)[1] <= 2 + np.log(6) + 1e-12).all()


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("fan", [1, 3])
def test_oracle_verify_keeps_the_distribution(drawn, fan):
    """The first token behind node 0 (a child that is accepted, or the next token) has the target's frequencies."""
    r = np.random.default_rng(5)
    v, n = 5, fan + 1
    p, d = r.dirichlet(np.ones(v), n), r.dirichlet(np.ones(v), n)
    parents = [-1] + [0] * fan
    likely = np.argsort(-d[0])[:fan]
    seen, trials = np.zeros(v), 20000
    for _ in range(trials):
        tokens = np.r_[0, r.choice(v, fan, p=d[0]) if drawn else likely]
        path, nxt = ref.verify(p, d if drawn else None, parents, tokens, r.random(n), r.random())
        seen[tokens[path[1]] if len(path) > 1 else nxt] += 1
    # a frequency's standard deviation is at most sqrt(1/4 / trials): five of them
    assert (np.abs(seen / trials - p[0]) < 2.5 / np.sqrt(trials)).all()


def test_oracle_verify_edges():
    one = np.eye(4)
    assert ref.verify(one[[2, 3, 1]], None, [-1, 0, 1], [0, 2, 3], [0.0, 0.99, 0.99], 0.5) == ([0, 1, 2], 1)   # sure drafts
    assert ref.verify(one[[2, 3]], one[[1, 1]], [-1, 0], [0, 1], [0.0, 0.0], 0.0) == ([0], 2)                  # impossible ones
    assert ref.verify(one[[2]], None, [-1], [0], [0.0], 0.0) == ([0], 2)
    assert ref.verify(0 * one[[2]], None, [-1], [0], [0.0], 0.5) == ([0], -1)
    p = np.full((2, 4), 0.25)
    assert ref.verify(p, p, [-1, 0], [0, 3], [0.0, 0.999], 0.5) == ([0, 1], 2)                                 # equal rows: always
