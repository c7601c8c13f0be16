"""The cache, rotation and attention entry points refuse bad arguments on the
host, before the device is touched (no GPU here), and take empty problems."""

import copy
import ctypes

import pytest
import torch

import quantized_linear_layer_gb300 as q

P = ctypes.c_void_p
OK, INVALID, ALIGN, UNSUPPORTED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def ref(s):
    return None if s is None else ctypes.cast(ctypes.pointer(s), P)


def heads(n=4, data=16, d=128, token=None, head=None):
    return q._Heads(data, n, n * d if token is None else token, d if head is None else head)


def cache(**change):
    c = q._KvCache(16, 16, 16, 16, 10, 2, 16, 128, 2 * 16 * 128, 2 * 16 * 4, 0)
    for k, v in change.items():
        setattr(c, k, v)
    return c


def rope(**change):
    r = q._Rope(16, 16, 128, 0, 16, 16, 1e-6)
    for k, v in change.items():
        setattr(r, k, v)
    return r


def test_norm_rope_refusals(L):
    def call(qh=heads(), kh=heads(2), qo=heads(), ko=heads(2), dtype=0, t=3, d=128, r=rope()):
        return L.qlin_qk_norm_rope(ref(qh), ref(kh), ref(qo), ref(ko), dtype, t, d, ref(r), None)
    assert call(dtype=2) == INVALID and call(t=-1) == INVALID and call(t=1 << 31) == INVALID
    assert call(d=96) == UNSUPPORTED
    assert call(qh=None) == INVALID and call(qo=None) == INVALID and call(r=None) == INVALID
    assert call(kh=None) == INVALID and call(ko=None) == INVALID
    assert call(qo=heads(8)) == INVALID and call(ko=heads(4)) == INVALID
    assert call(qh=heads(data=24)) == ALIGN and call(qh=heads(data=None)) == INVALID
    assert call(qh=heads(token=516)) == ALIGN and call(qh=heads(head=132)) == ALIGN
    assert call(qh=heads(head=64)) == INVALID and call(qh=heads(token=64)) == INVALID and call(qh=heads(0)) == INVALID
    for change in ({"rot": 8}, {"rot": 144}, {"rot": -16}, {"interleaved": 2}, {"positions": None}, {"inv_freq": None},
                   {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert call(r=rope(**change)) == INVALID, change
    for change in ({"positions": 12}, {"inv_freq": 12}, {"q_gamma": 24}, {"k_gamma": 24}):
        assert call(r=rope(**change)) == ALIGN, change
    assert call(t=0) == OK and call(t=0, kh=None, ko=None) == OK
    assert b"" == L.qlin_last_error_message()


def test_cache_refusals(L):
    def write(kh=heads(2), vh=heads(2), dtype=1, t=3, slots=16, c=cache()):
        return L.qlin_kv_cache_write(ref(kh), ref(vh), dtype, t, P(slots), ref(c), None)
    assert write(c=None) == INVALID and write(dtype=3) == INVALID and write(t=-1) == INVALID
    assert write(kh=None) == INVALID and write(vh=None) == INVALID
    assert write(kh=heads(4)) == INVALID and write(vh=heads(1)) == INVALID
    assert write(slots=None) == INVALID and write(slots=12) == ALIGN
    for change in ({"fmt": 3}, {"fmt": -1}, {"heads": 0}, {"pages": 0}, {"pages": 1 << 31}, {"k": None}, {"v_scale": None},
                   {"page_stride": 4080}, {"scale_page_stride": 112}, {"page_stride": 1 << 39}):
        assert write(c=cache(**change)) == INVALID, change
    for change in ({"k": 24}, {"v": 8}, {"k_scale": 20}, {"page_stride": 4104}, {"scale_page_stride": 132}):
        assert write(c=cache(**change)) == ALIGN, change
    for change in ({"head_dim": 80}, {"page_size": 8}, {"page_size": 48}, {"page_size": 512}):
        assert write(c=cache(**change)) == UNSUPPORTED, change
    assert write(t=0, slots=None) == OK

    def joint(qh=heads(), kh=heads(2), vh=heads(2), qo=heads(), ko=None, t=3, r=rope()):
        return L.qlin_qk_norm_rope_cache(ref(qh), ref(kh), ref(vh), ref(qo), ref(ko), 0, t, ref(r), P(16), ref(cache()), None)
    assert joint(qh=None) == INVALID and joint(qo=None) == INVALID and joint(r=rope(rot=8)) == INVALID
    assert joint(ko=heads(3)) == INVALID and joint(qo=heads(2)) == INVALID
    assert joint(t=0) == OK and joint(qh=None, qo=None, t=0) == OK

    def read(c=cache(), table=16, pages=4, starts=16, indptr=16, b=2, rows=5, ko=heads(2), vo=heads(2), dtype=0):
        return L.qlin_kv_cache_read(ref(c), P(table), pages, P(starts), P(indptr), b, rows, ref(ko), ref(vo), dtype, None)
    assert read(dtype=2) == INVALID and read(b=-1) == INVALID and read(rows=-1) == INVALID and read(pages=-1) == INVALID
    assert read(ko=heads(1)) == INVALID and read(vo=None) == INVALID and read(c=cache(fmt=9)) == INVALID
    assert read(table=None) == INVALID and read(starts=None) == INVALID and read(indptr=None) == INVALID
    assert read(table=18) == ALIGN and read(indptr=17) == ALIGN
    assert read(rows=0, table=None) == OK and read(b=0, table=None) == OK


def test_attention_refusals(L):
    base = dict(qh=heads(8), out=heads(8), dtype=0, tq=3, c=cache(), table=16, pages=4, indptr=16, ctx=16, b=2, mask=16, words=1,
                nodes=3, scale=0.1, lse=16, ws=256, size=1 << 40)

    def call(**change):
        a = copy.copy(base)
        a.update(change)
        return L.qlin_tree_attention(ref(a["qh"]), ref(a["out"]), a["dtype"], a["tq"], ref(a["c"]), P(a["table"]), a["pages"],
                                     P(a["indptr"]), P(a["ctx"]), a["b"], P(a["mask"]), a["words"], a["nodes"], a["scale"],
                                     P(a["lse"]), P(a["ws"]), a["size"], None)
    for change in ({"dtype": 2}, {"tq": -1}, {"b": -1}, {"b": 65536}, {"pages": -1}, {"scale": float("nan")},
                   {"scale": float("inf")}, {"c": None}, {"qh": None}, {"out": heads(4)}, {"qh": heads(3), "out": heads(3)},
                   {"words": 2}, {"nodes": 65}, {"table": None}, {"indptr": None}, {"ctx": None}, {"ws": None}):
        assert call(**change) == INVALID, change
    for change in ({"nodes": 0}, {"nodes": 257}, {"c": cache(head_dim=96)}):
        assert call(**change) == UNSUPPORTED, change
    for change in ({"table": 18}, {"indptr": 18}, {"ctx": 18}, {"lse": 18}, {"mask": 20}, {"ws": 272}, {"qh": heads(8, data=24)}):
        assert call(**change) == ALIGN, change
    assert call(tq=0, table=None, ws=None) == OK and call(b=0, table=None, ws=None) == OK
    size = L.qlin_tree_attention_workspace_bytes
    assert size(ref(cache()), 8, 64, 4) > 0
    assert size(ref(cache()), 7, 64, 4) == -1 and size(ref(cache()), 8, 257, 4) == -1 and size(ref(cache()), 8, 0, 4) == -1
    assert size(ref(cache(fmt=7)), 8, 4, 4) == -1 and size(ref(cache()), 8, 4, -1) == -1


def test_binding_refusals():
    """Wrong types, shapes and devices raise before a call is made (CPU tensors are refused, not computed)."""
    h = torch.zeros(3, 4, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        q.qlin_qk_norm_rope(h, None, h, None, torch.zeros(3, dtype=torch.int64), torch.ones(64, dtype=torch.float64))
    with pytest.raises(TypeError, match="dtype"):
        q.qlin_qk_norm_rope(h.float(), None, h, None, None, None)
    with pytest.raises(ValueError, match="go together|CUDA"):
        q.qlin_qk_norm_rope(h, h, h, None, None, None)
    codes, scales = torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 16)
    with pytest.raises(ValueError, match="unknown cache format"):
        q.qlin_kv_cache(codes, codes, scales, scales, 5)
    with pytest.raises(TypeError, match="dtype"):
        q.qlin_kv_cache(codes, codes, scales, scales, q.QLIN_KV_U4)
    with pytest.raises(ValueError, match="CUDA"):
        q.qlin_kv_cache(codes, codes, scales, scales, q.QLIN_KV_INT8)
