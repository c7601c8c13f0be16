"""Prepared calls on the host (no GPU needed): what is refused, and calls with
nothing to do; and the attention oracle against closed forms and differences."""

import ctypes

import numpy as np
import pytest

import quantized_linear_layer_gb300 as q
from oracle import attention as ref
from test_kv_abi import ALIGN, INVALID, L, OK, P, UNSUPPORTED, cache, heads, ref as ptr, rope  # noqa: F401


def _call():
    return (ctypes.c_uint64 * 112)()


def test_prepared_refusals(L):
    c = _call()
    at = ctypes.cast(c, P)
    assert L.qlin_call_run(None, None) == INVALID
    assert L.qlin_call_run(at, None) == INVALID                     # zeros: never prepared
    garbage = (ctypes.c_uint64 * 112)(*([0xABABABABABABABAB] * 112))
    assert L.qlin_call_run(ctypes.cast(garbage, P), None) == INVALID

    def prepare(out, t=3, d=128, qh=heads()):
        return L.qlin_qk_norm_rope_prepare(ptr(qh), ptr(heads(2)), ptr(heads()), ptr(heads(2)), 0, t, d, ptr(rope()), out)
    assert prepare(None) == INVALID and prepare(at, d=96) == UNSUPPORTED and prepare(at, qh=heads(data=24)) == ALIGN
    assert L.qlin_call_run(at, None) == INVALID                     # a refused preparation leaves no call
    assert prepare(at, t=0) == OK and L.qlin_call_run(at, None) == OK   # nothing to do: nothing is launched
    assert prepare(at, d=96) == UNSUPPORTED and L.qlin_call_run(at, None) == INVALID

    write = L.qlin_kv_cache_write_prepare
    assert write(ptr(heads(2)), ptr(heads(2)), 0, 3, P(12), ptr(cache()), at) == ALIGN
    assert write(ptr(heads(2)), ptr(heads(2)), 0, 0, None, ptr(cache()), at) == OK and L.qlin_call_run(at, None) == OK
    read = L.qlin_kv_cache_read_prepare
    assert read(ptr(cache(fmt=9)), P(16), 4, P(16), P(16), 2, 5, ptr(heads(2)), ptr(heads(2)), 0, at) == INVALID
    tree = L.qlin_tree_attention_prepare
    args = (ptr(heads(8)), ptr(heads(8)), 0, 3, ptr(cache()), P(16), 4, P(16), P(16), 2, P(16), 1, 3, 0.1, P(16), P(256))
    assert tree(*args, 1 << 40, None) == INVALID


def test_oracle_attention():
    """Equal keys average the seen values; one seen token gives its value; lse of equal scores is s + ln n."""
    r = np.random.default_rng(0)
    k, v = np.ones((7, 2, 4)), r.normal(size=(7, 2, 4))
    x = r.normal(size=(2, 4, 4))
    seen = np.zeros((2, 7), bool)
    seen[0, [1, 4, 6]] = True
    out, lse, weight, spread = ref.tree_attention(x, k, v, seen, 0.5)
    assert np.allclose(out[0, 3], v[[1, 4, 6], 1].mean(0)) and np.allclose(weight[0, 0], np.abs(v[[1, 4, 6], 0]).mean(0))
    assert np.allclose(lse[0], 0.5 * x[0].sum(-1) + np.log(3)) and np.isneginf(lse[1]).all() and not out[1].any()
    assert np.allclose(spread[0], 0.5 * np.abs(x[0]).sum(-1))
    # d lse / d q = scale sum p k, by differences
    k = r.normal(size=(7, 2, 4))
    seen[:] = True
    e = 1e-6 * np.eye(4)[2]
    up, down = (ref.tree_attention(x + s * e, k, v, seen, 0.5)[1] for s in (1, -1))
    mean_k = ref.tree_attention(x, k, k, seen, 0.5)[0]
    assert np.allclose((up - down) / 2e-6, 0.5 * mean_k[..., 2], atol=1e-7)


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_rotation(inter):
    """A rotation keeps each pair's length; scores of rotated rows depend on the distance of their places only."""
    r = np.random.default_rng(1)
    x, freq = r.normal(size=(1, 2, 16)), 100.0 ** -np.arange(4)
    at = lambda row, p: ref.norm_rope(x[:, row:row + 1], None, [p], freq, 0.0, inter)[0, 0]
    assert np.allclose(at(0, 11) @ at(1, 4), at(0, 1007) @ at(1, 1000))
    assert np.array_equal(at(0, 5)[8:], x[0, 0, 8:]) and np.allclose(np.linalg.norm(at(0, 5)), np.linalg.norm(x[0, 0]))
    y = ref.norm_rope(x, 2 * np.ones(16), [0], np.zeros(0), 0.0, inter)
    assert np.allclose((y ** 2).mean(-1), 4.0)


@pytest.mark.parametrize("fmt,step", [("int8", 1 / 127), ("e4m3", 1 / 14), ("u4", 2 / 15)])
def test_oracle_cache_formats(fmt, step):
    """Values come back within half a step of the row's largest (E4M3: half of 2^-3 relative); zeros as zeros."""
    x = np.random.default_rng(2).normal(size=(5, 64)).astype(np.float32)
    x[3] = 0
    got = ref.kv_values(*ref.kv_quantize(x, fmt), fmt)
    top = np.abs(x).max(-1, keepdims=True)
    slack = 2.0 ** -10 if fmt == "u4" else 2.0 ** -20      # fp16 scales
    assert (np.abs(got - x) <= top * (step / 2 + 15 * slack) + (0.0625 * np.abs(x) if fmt == "e4m3" else 0)).all()
    assert not got[3].any()
    x[1, 5], x[2, 6] = np.nan, np.inf
    bad = ref.kv_values(*ref.kv_quantize(x, fmt), fmt)
    assert np.isnan(bad[1:3]).all() and np.array_equal(bad[0], got[0])
