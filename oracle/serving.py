"""A serving step around the paged, quantized cache (oracle side): pages and
slots from lengths, attention of a chunk of new tokens, verified drafts, kept
paths.

TEST INFRASTRUCTURE ONLY - see the package docstring.
"""

import math

import numpy as np


class Pages:
    """Block tables (lists), pages held and the stack of free pages (its top at the end)."""

    def __init__(self, table, held, free, page, max_pages):
        self.table, self.held, self.free = [list(r) for r in table], list(held), list(free)
        self.page, self.max_pages = page, max_pages

    def assign(self, ctx, new, rows, depths=None):
        """One step; returns (q_indptr, positions, slots)."""
        page = self.page
        good = [c >= 0 and n >= 0 and -(-(c + n) // page) <= self.max_pages and 0 <= h <= self.max_pages
                for c, n, h in zip(ctx, new, self.held)]
        need = [-(-(c + n) // page) if g else h for c, n, h, g in zip(ctx, new, self.held, good)]
        for b in reversed(range(len(ctx))):
            for j in reversed(range(need[b], self.held[b])):
                self.free.append(self.table[b][j])
        lack = [max(0, n - h) for n, h in zip(need, self.held)]
        self.held = [min(n, h) for n, h in zip(need, self.held)]
        room = len(self.free)
        bounds, positions, slots = [0], [], []
        for b, (c, n) in enumerate(zip(ctx, new)):
            n = n if good[b] else 0
            before = sum(x for x, g in zip(new[:b + 1], good) if g)
            if (lack[b] == 0 or sum(lack[:b + 1]) <= room) and (n == 0 or before <= rows):
                for _ in range(lack[b]):
                    self.table[b][self.held[b]] = self.free.pop()
                    self.held[b] += 1
                for i in range(n):
                    positions.append(c + (i if depths is None else depths[len(slots)]))
                    slots.append(self.table[b][(c + i) // page] * page + (c + i) % page)
            bounds.append(len(slots))
        pad = rows - len(slots)
        return bounds, positions + [0] * pad, slots + [-1] * pad


def chunk_attention(q, k, v, ctx, scale, softcap=0.0, slopes=None, window=0, prefix=0):
    """One sequence.  q [n][Hq][D], k, v [ctx + n][Hk][D] float64.

    Returns out, lse, and three bounds' parts: weight = sum p |v|; and with e_ij the error that float32 may make in a
    score (D roundings of its products' magnitudes, 2^-20 of the cap, of caps above 256 at most 2^-18 of the capped score, 2^-22 of the score and of the bias),
    sum p e |v| and sum p e."""
    n, hq, d = q.shape
    group, length = hq // k.shape[1], k.shape[0]
    at, j = ctx + np.arange(n)[:, None], np.arange(length)
    seen = j <= at
    if window:
        seen &= at - j < window
    seen |= j < prefix
    out, weight, moved = (np.zeros((n, hq, d)) for _ in range(3))
    lse, err = np.zeros((n, hq)), np.zeros((n, hq))
    for h in range(hq):
        kk, vv = k[:, h // group], v[:, h // group]
        s = q[:, h] @ kk.T * scale
        e = d * 2.0 ** -24 * (np.abs(q[:, h]) @ np.abs(kk).T) * abs(scale) + 2.0 ** -22 * np.abs(s)
        if softcap:
            s = softcap * np.tanh(s / softcap)
            e = e + (2.0 ** -20 * softcap if softcap <= 256 else np.minimum(2.0 ** -20 * softcap, 2.0 ** -18 * np.abs(s)))
        if slopes is not None:
            bias = slopes[h] * np.abs(at - j)
            s, e = s - bias, e + 2.0 ** -22 * np.abs(bias)
        s = np.where(seen, s, -np.inf)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        total = p.sum(-1, keepdims=True)
        p /= total
        lse[:, h] = (m + np.log(total))[:, 0]
        out[:, h], weight[:, h], moved[:, h] = p @ vv, p @ np.abs(vv), (p * e) @ np.abs(vv)
        err[:, h] = (p * e).sum(-1)
    return out, lse, weight, moved, err


def verify(target, draft, parents, tokens, accept_u, sample_u):
    """One sequence of n nodes: target, draft [n][V] (draft None: not drawn), parents and tokens [n].
    Returns (path, next token)."""
    clean = lambda x: np.clip(np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=1.0), 0.0, 1.0)
    n, v = len(tokens), target.shape[1]
    if n == 0:
        return [], -1
    path = [0]
    while True:
        here = path[-1]
        p = clean(target[here])
        q = None if draft is None else clean(draft[here])
        rest, total, drawn, moved = p, 1.0, 0.0, False
        for i in range(here + 1, n):
            x = tokens[i]
            if parents[i] != here or not 0 <= x < v:
                continue
            share = total if q is None else total * q[x]
            if accept_u[i] * share < rest[x]:
                path.append(i)
                moved = True
                break
            if q is None:
                total, rest = max(total - rest[x], 0.0), np.where(np.arange(v) == x, 0.0, rest)
            else:
                drawn += total
                rest = np.maximum(p - drawn * q, 0.0)
                total = math.fsum(rest)
        if not moved:
            break
    if not rest.any():
        rest = p
    if not rest.any():
        return path, -1
    sums = np.cumsum(rest)
    return path, int(np.searchsorted(sums, sample_u * sums[-1], side="right"))
