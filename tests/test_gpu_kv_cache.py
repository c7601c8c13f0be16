"""Head norms with the position rotation, and the quantized paged cache
written and read back, against the 64-bit oracle.

Tolerances.  A rounding to a 16-bit type is off by at most eps / 2 relative
(or half the smallest subnormal).  Before it, float32: the mean of squares and
the norm lose at most 16 roundings of 2^-24, the angle is within 2^-21 and the
sine and cosine within two units of theirs, so a rotated channel is within
(|a| + |b|) (2^-20 + 2^-19) of the exact one: 2^-18 of the row's largest
channel covers it.  Codes and scales written from 16-bit inputs are exact."""

import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

FMTS = ["int8", "e4m3", "u4"]
DTYPES = [torch.float16, torch.bfloat16]


def _fmt(q, fmt):
    return {"int8": q.QLIN_KV_INT8, "e4m3": q.QLIN_KV_E4M3, "u4": q.QLIN_KV_U4}[fmt]


def _np(t):
    return t.detach().double().cpu().numpy()


def _empty_cache(q, fmt, pages, heads, page, d, gap=0):
    """Caller-side tensors (every byte set to a pattern) and the handle; gap: extra bytes between pages."""
    width = d // 2 if fmt == "u4" else d
    kind = torch.int8 if fmt == "int8" else torch.uint8
    n = heads * page * width

    def paged(per, extra, dtype, shape):
        t = torch.full((pages, per + extra), 85, dtype=dtype, device="cuda")
        return t[:, :per].view(pages, *shape) if extra == 0 else t.as_strided((pages, *shape), (per + extra, *_dense(shape)))

    def _dense(shape):
        s, out = 1, []
        for v in reversed(shape):
            out.insert(0, s)
            s *= v
        return out

    codes = [paged(n, gap, kind, (heads, page, width)) for _ in range(2)]
    if fmt == "u4":
        scales = [paged(heads * page * 2, gap // 2, torch.float16, (heads, page, 2)) for _ in range(2)]
    else:
        scales = [paged(heads * page, gap // 4, torch.float32, (heads, page)) for _ in range(2)]
    t = (*codes, *scales)
    return t, q.qlin_kv_cache(*t, _fmt(q, fmt))


def _rows(gen, t, h, d, dtype, scale=1.0):
    x = torch.randn(t, h, d, generator=gen) * scale
    x[..., 3] *= 6
    return x.to(dtype)


def _close(y, want, dtype, what):
    y, want = _np(y), np.asarray(want)
    top = np.abs(want).max(axis=-1, keepdims=True)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -18 * top + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bad = ~(np.abs(y - want) <= tol)
    assert not bad.any(), "%s: %d of %d, worst %g" % (what, bad.sum(), bad.size, np.abs(y - want).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,hq,hk,d,rot,inter,norm", [
    (1, 32, 8, 128, 128, False, True), (1, 1, 1, 64, 64, True, False), (77, 5, 1, 64, 32, False, True),
    (33, 20, 4, 128, 64, True, True), (130, 8, 8, 256, 256, False, True), (19, 3, 1, 256, 16, False, False),
    (7, 40, 8, 128, 0, False, True), (259, 1, 1, 64, 64, False, True)])
def test_norm_rope(qlin_gpu, dtype, t, hq, hk, d, rot, inter, norm):
    q = qlin_gpu
    gen = torch.Generator().manual_seed(t * 7 + d)
    qkv = _rows(gen, t, hq + 2 * hk, d, dtype).cuda()          # q and k are views of the joint rows
    xq, xk = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos = torch.randint(0, 1 << 20, (t,), generator=gen)
    pos[0] = (1 << 31) - 5
    freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(1, rot)) if rot else None
    gq, gk = (((1 + 0.3 * torch.randn(d, generator=gen)).to(dtype).cuda()) if norm else None for _ in range(2))
    yq = torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda")
    yk = torch.full((hk, t, d), 7.0, dtype=dtype, device="cuda").transpose(0, 1)   # heads outermost
    q.qlin_qk_norm_rope(xq, xk, yq, yk, pos.cuda(), None if freq is None else freq.cuda(), gq, gk, 1e-6, inter)
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
    f = [] if freq is None else freq.numpy()
    for y, x, g, what in ((yq, xq, gq, "q"), (yk, xk, gk, "k")):
        _close(y, ref.norm_rope(_np(x), None if g is None else _np(g), pos.numpy(), f, 1e-6, inter), dtype, what)


def test_norm_rope_edges(qlin_gpu):
    """No tokens; q alone; in place; one gamma only; a zero head; a negative position; a NaN stays in its head."""
    q = qlin_gpu
    gen = torch.Generator().manual_seed(3)
    freq = 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)
    e = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    q.qlin_qk_norm_rope(e, e, e, e, torch.empty(0, dtype=torch.int64, device="cuda"), freq.cuda())
    x = _rows(gen, 5, 4, 64, torch.float16)
    x[1, 2] = 0
    x[2, 1, 9] = float("nan")
    x[3, 0, 5] = float("inf")
    pos = torch.tensor([0, -3, 17, 1 << 30, 5])
    g = torch.rand(64, generator=gen).half() + 0.5
    y = x.clone().cuda()
    q.qlin_qk_norm_rope(y, None, y, None, pos.cuda(), freq.cuda(), g.cuda(), None)
    clean = np.ones((5, 4), bool)
    clean[2, 1] = clean[3, 0] = False
    with np.errstate(invalid="ignore"):
        want = ref.norm_rope(_np(x), _np(g), pos.numpy(), freq.numpy(), 1e-6, False)
    _close(y.cpu()[torch.from_numpy(clean)], want[clean], torch.float16, "in place")
    assert torch.isnan(y[2, 1]).all() and torch.isnan(y[3, 0]).any()
    k, yk = _rows(gen, 5, 2, 64, torch.float16).cuda(), torch.empty(5, 2, 64, dtype=torch.float16, device="cuda")
    y2 = torch.empty_like(y)
    q.qlin_qk_norm_rope(x.cuda(), k, y2, yk, pos.cuda(), freq.cuda(), None, g.cuda())
    _close(yk, ref.norm_rope(_np(k), _np(g), pos.numpy(), freq.numpy(), 1e-6, False), torch.float16, "k normed, q not")
    want = ref.norm_rope(_np(x), None, pos.numpy(), freq.numpy(), 1e-6, False)
    _close(y2.cpu()[torch.from_numpy(clean)], want[clean], torch.float16, "q rotated only")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,hk,d,page,gap", [(1, 1, 64, 16, 0), (37, 3, 128, 16, 64), (70, 2, 256, 64, 0), (129, 8, 64, 256, 16)])
def test_write_is_exact(qlin_gpu, fmt, dtype, t, hk, d, page, gap):
    """Codes and scales bit for bit, at scattered places; every other byte of the cache stays."""
    q = qlin_gpu
    gen = torch.Generator().manual_seed(t + d)
    pages = -(-t // page) + 3
    tens, cache = _empty_cache(q, fmt, pages, hk, page, d, gap)
    before = [x.clone() for x in tens]
    kv = _rows(gen, t, 2 * hk, d, dtype)
    if t > 20:
        kv[0, 0] = 0
        kv[1, 0] = 1.0
        kv[2, 0] = -kv[2, 0].abs()                       # one sign only (U4: the range still holds 0)
        kv[3, 0] = torch.linspace(-127, 127, d).to(dtype)   # ties and the ends of the range
        kv[4, 0] *= 2.0 ** -20
        kv[5, 0, 1], kv[6, 1, 2], kv[7, 0, 0] = float("nan"), float("inf"), -float("inf")
        kv[8, 0] = 0
        kv[8, 0, 0] = torch.finfo(dtype).max
        kv[9, 0] = 0
        kv[9, 0, 1] = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        if dtype == torch.bfloat16:
            kv[10, 0] = torch.randn(d, generator=gen).to(dtype) * 2.0 ** -90   # below the scale floor
    slots = torch.randperm(pages * page, generator=gen)[:t]
    if t > 1:
        slots[t // 2] = -1                                # not stored
    dev = kv.cuda()
    q.qlin_kv_cache_write(dev[:, :hk], dev[:, hk:], slots.cuda(), cache)
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
    for part, codes, scales, c0, s0 in ((kv[:, :hk], tens[0], tens[2], before[0], before[2]),
                                        (kv[:, hk:], tens[1], tens[3], before[1], before[3])):
        wc, ws = ref.kv_quantize(part.float().numpy(), fmt)
        ec, es = c0.cpu().numpy().copy(), s0.cpu().numpy().copy()
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                ec[s // page, :, s % page], es[s // page, :, s % page] = wc[i], ws[i]
        assert np.array_equal(codes.cpu().numpy(), ec)
        assert np.array_equal(scales.cpu().numpy(), es, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,rot,inter,norm", [(64, 64, False, True), (128, 64, True, False), (256, 256, False, True)])
def test_norm_rope_cache(qlin_gpu, fmt, d, rot, inter, norm):
    """The joint pass: q as alone, v exact, and k's codes those of the rotated float32 row: within one step
    of the oracle's, at a scale within 2^-18 of its (fp16 scales: one unit)."""
    q, dtype, t, hq, hk, page = qlin_gpu, torch.bfloat16, 45, 6, 2, 32
    gen = torch.Generator().manual_seed(d)
    tens, cache = _empty_cache(q, fmt, 4, hk, page, d)
    x = _rows(gen, t, hq + 2 * hk, d, dtype)
    xd = x.cuda()
    pos = torch.randint(0, 1 << 18, (t,), generator=gen)
    freq = 500000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    gq, gk = ((1 + 0.3 * torch.randn(d, generator=gen)).to(dtype) if norm else None for _ in range(2))
    slots = torch.randperm(4 * page, generator=gen)[:t]
    yq, yk = torch.empty(t, hq, d, dtype=dtype, device="cuda"), torch.empty(t, hk, d, dtype=dtype, device="cuda")
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    args = (pos.cuda(), freq.cuda(), slots.cuda(), cache, dev(gq), dev(gk), 1e-6, inter)
    q.qlin_qk_norm_rope_cache(xd[:, :hq], xd[:, hq:hq + hk], xd[:, hq + hk:], yq, *args, k_out=yk)
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
    num = lambda v: None if v is None else _np(v)  # noqa: E731
    rq = ref.norm_rope(_np(x[:, :hq]), num(gq), pos.numpy(), freq.numpy(), 1e-6, inter)
    rk = ref.norm_rope(_np(x[:, hq:hq + hk]), num(gk), pos.numpy(), freq.numpy(), 1e-6, inter)
    _close(yq, rq, dtype, "q")
    _close(yk, rk, dtype, "k")
    at = (slots // page, slice(None), slots % page)
    got = [v.cpu()[at].numpy() for v in tens]
    wc, ws = ref.kv_quantize(x[:, hq + hk:].float().numpy(), fmt)
    assert np.array_equal(got[1], wc) and np.array_equal(got[3], ws)
    # k: reading back is within half a step of its scale (E4M3: 2^-4 relative), plus the float32 error
    back = ref.kv_values(got[0], got[2], fmt)
    top = np.abs(rk).max(axis=-1, keepdims=True)
    if fmt == "u4":
        step = got[2][..., :1].astype(np.float64)
        want = np.maximum(rk.max(-1), 0) - np.minimum(rk.min(-1), 0)
        assert np.all(np.abs(step[..., 0] - want / 15) <= 2.0 ** -10 * want / 15 + 2.0 ** -24)
        # fp16 rounding of the scale can cut the range's ends by 15 half units of it
        assert np.all(np.abs(back - rk) <= step * (0.5 + 16 * 2.0 ** -11) + 2.0 ** -16 * top)
    else:
        assert np.all(np.abs(got[2][..., None] - top / (127 if fmt == "int8" else 448)) <= 2.0 ** -17 * top / 127)
        half = got[2][..., None] / 2 if fmt == "int8" else np.maximum(np.abs(rk) * 2.0 ** -4, got[2][..., None] * 2.0 ** -10)
        assert np.all(np.abs(back - rk) <= half * (1 + 2.0 ** -10) + 2.0 ** -16 * top)
    # the same pass without q stores the same bytes
    other, cache2 = _empty_cache(q, fmt, 4, hk, page, d)
    args2 = args[:3] + (cache2,) + args[4:]
    q.qlin_qk_norm_rope_cache(None, xd[:, hq:hq + hk], xd[:, hq + hk:], None, *args2)
    # a shorter grid of rows moves no row to other arithmetic
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tens, other))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,starts,hk,d,page", [
    ([1], [0], 1, 64, 16), ([0, 5, 0, 100, 33], [3, 15, 0, 60, 1], 3, 128, 32), ([257, 1], [0, 511], 2, 256, 128),
    ([64], [64], 32, 64, 64)])
def test_read(qlin_gpu, fmt, dtype, lens, starts, hk, d, page):
    """One float32 product rounded once: exactly the oracle's product rounded to float32 and then to the type."""
    q = qlin_gpu
    gen = torch.Generator().manual_seed(sum(lens) + d)
    per = [-(-(s + n) // page) for s, n in zip(starts, lens)]
    pages = sum(per) + 2
    tens, cache = _empty_cache(q, fmt, pages, hk, page, d, 32)
    codes, scales = ref.kv_quantize(torch.randn(2, pages, hk, page, d, generator=gen).numpy(), fmt)
    for i in range(2):
        tens[i].copy_(torch.from_numpy(codes[i]))
        tens[2 + i].copy_(torch.from_numpy(scales[i]))
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((len(lens), max(per) + 1), -7, dtype=torch.int32)     # entries past the end are not read
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    rows = sum(lens)
    ko = torch.full((rows, hk, d), 9.0, dtype=dtype, device="cuda")
    vo = torch.full((hk, rows, d), 9.0, dtype=dtype, device="cuda").transpose(0, 1)
    indptr = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    q.qlin_kv_cache_read(cache, table.cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), indptr.cuda(), ko, vo)
    torch.cuda.synchronize()
    assert q.qlin_get_device_error() == 0
    for i, y in enumerate((ko, vo)):
        want = np.concatenate([ref.kv_values(codes[i], scales[i], fmt)[table[b, (p := np.arange(s, s + n)) // page].numpy(), :, p % page]
                               for b, (s, n) in enumerate(zip(starts, lens))])
        assert torch.equal(y.cpu(), torch.from_numpy(want).float().to(dtype))


def test_bad_places_are_skipped_and_recorded(qlin_gpu):
    """A place beyond the cache, a page number out of range, a sequence past its table: no access, an error word."""
    q = qlin_gpu
    tens, cache = _empty_cache(q, "int8", 3, 2, 16, 64)
    before = [x.clone() for x in tens]
    x = torch.randn(2, 2, 64, device="cuda").half()
    q.qlin_kv_cache_write(x, x, torch.tensor([48, 1 << 40], device="cuda"), cache)
    assert q.qlin_get_device_error() == 0x2000
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tens, before))
    q.qlin_kv_cache_write(x, x, torch.tensor([47, -5], device="cuda"), cache)
    assert q.qlin_get_device_error() == 0
    ko, vo = (torch.full((4, 2, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 3], [-1, 0]], dtype=torch.int32, device="cuda")
    q.qlin_kv_cache_read(cache, table, torch.tensor([15, 31], dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"), ko, vo)
    assert q.qlin_get_device_error() == 0x2000
    assert not torch.equal(ko[0], torch.zeros_like(ko[0])) and not (ko[1] != 0).any() and not (ko[3] != 0).any()


def test_write_and_read_beyond_32_bits(qlin_gpu):
    """Pages of a layer inside a buffer of many layers: byte offsets beyond 2^32."""
    q = qlin_gpu
    pages, hk, page, d = 5, 2, 16, 128
    gap = (1 << 30) + 4096
    if torch.cuda.mem_get_info()[0] < 14 * gap:
        pytest.skip("not enough free memory")
    far = [torch.empty(4 * gap + hk * page * d, dtype=torch.int8, device="cuda").as_strided((pages, hk, page, d), (gap, page * d, d, 1))
           for _ in range(2)]
    sc = [torch.empty(pages, hk, page, device="cuda") for _ in range(2)]
    cache = q.qlin_kv_cache(*far, *sc, q.QLIN_KV_INT8)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(pages * page, 2 * hk, d, generator=gen).half()
    slots = torch.randperm(pages * page, generator=gen)
    q.qlin_kv_cache_write(x[:, :hk].cuda(), x[:, hk:].cuda(), slots.cuda(), cache)
    ko, vo = (torch.empty(pages * page, hk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q.qlin_kv_cache_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         torch.tensor([0, pages * page], dtype=torch.int32, device="cuda"), ko, vo)
    assert q.qlin_get_device_error() == 0
    want = torch.empty(pages * page, 2 * hk, d, dtype=torch.float64)
    want[slots] = torch.from_numpy(ref.kv_values(*ref.kv_quantize(x.float().numpy(), "int8"), "int8"))
    want = want.float().half()
    assert torch.equal(ko.cpu(), want[:, :hk]) and torch.equal(vo.cpu(), want[:, hk:])
