"""f64 oracle of the rotary and paged-cache calls (numpy, test infrastructure).

Plain restatements of the definitions in ``include/wq.h``, one loop per index, sharing no
code with the CUDA library.  Pools are numpy arrays seen as [page][head][row][dim].
"""
from __future__ import annotations

import math

import numpy as np

PLAIN, LINEAR, NTK, YARN, BANDS = range(5)
INTERLEAVED, TRANSPOSE = 1, 2


def frequencies(rot, base, kind=PLAIN, factor=1.0, low=1.0, high=32.0, original=0):
    """f_i, i < rot / 2."""
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == NTK:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == LINEAR:
        return f / factor
    if kind == YARN:
        def dim(turns):
            return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
        a, b = max(0.0, math.floor(dim(high))), min(rot - 1.0, math.ceil(dim(low)))
        t = np.clip((i - a) / max(b - a, 0.001), 0.0, 1.0)
        return f * (1 - t) + f / factor * t
    if kind == BANDS:
        turns = original * f / (2 * math.pi)
        s = (turns - low) / (high - low)
        mid = (1 - s) * f / factor + s * f
        return np.where(turns > high, f, np.where(turns < low, f / factor, mid))
    return f


def table(rows, rot, base, magnitude=None, kind=PLAIN, factor=1.0, **scaling):
    """[rows][rot/2][2] of m cos, m sin."""
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if kind == YARN and factor > 1 else 1.0
    a = np.arange(rows, dtype=np.float64)[:, None] * frequencies(rot, base, kind, factor, **scaling)
    return magnitude * np.stack([np.cos(a), np.sin(a)], -1)


def rotate(x, cs, rot, flags=0):
    """x [n][heads][d] by cs [n][rot/2][2]; also the bound sum of the terms' magnitudes."""
    x = np.asarray(x, np.float64)
    y, mag = x.copy(), np.abs(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if flags & INTERLEAVED else (i, i + rot // 2)
        c, s = cs[:, i, 0][:, None], cs[:, i, 1][:, None]
        if flags & TRANSPOSE:
            s = -s
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
        mag[:, :, a] = np.abs(x[:, :, a] * c) + np.abs(x[:, :, b] * s)
        mag[:, :, b] = np.abs(x[:, :, a] * s) + np.abs(x[:, :, b] * c)
    return y, mag


def attention(q, k, v, pages, lens, scale, window=0, mask=None, acc_in=None):
    """q [n][hq][d], pools k and v, pages [n][max_pages].  A dict of out [n][hq][d], lse
    [n][hq], acc [n][hkv][slots] (nan where not written), and the magnitudes that
    tolerances need: pv = sum p |v|, sx = max scale sum |q k|, mx = max |x|, p = sum of p."""
    n, hq, d = q.shape
    hkv, page = k.shape[1], k.shape[2]
    slots = pages.shape[1] * page
    group = hq // hkv
    r = dict(out=np.zeros((n, hq, d)), lse=np.full((n, hq), -np.inf),
             acc=np.full((n, hkv, slots), np.nan), pv=np.zeros((n, hq, d)),
             sx=np.zeros((n, hq)), mx=np.zeros((n, hq)), p=np.zeros((n, hkv, slots)))
    for s in range(n):
        size = min(int(lens[s]), slots)
        for g in range(hkv):
            if size > 0:
                r["acc"][s, g, :size] = 0.0 if acc_in is None else acc_in[s, g, :size]
            part = [j for j in range(max(0, size))
                    if not (window and j < size - window)
                    and not (mask is not None and mask[s, j] == -np.inf)
                    and 0 <= pages[s, j // page] < k.shape[0]]
            if not part:
                continue
            at = [(pages[s, j // page], j % page) for j in part]
            kk = np.array([k[p, g, i] for p, i in at], np.float64)
            vv = np.array([v[p, g, i] for p, i in at], np.float64)
            for h in range(g * group, (g + 1) * group):
                qq = q[s, h].astype(np.float64)
                x = scale * (kk @ qq)
                if mask is not None:
                    x = x + mask[s, part].astype(np.float64)
                top = x.max()
                e = np.exp(x - top)
                p = e / e.sum()
                r["out"][s, h] = p @ vv
                r["lse"][s, h] = top + math.log(e.sum())
                r["pv"][s, h] = p @ np.abs(vv)
                r["sx"][s, h] = abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
                r["mx"][s, h] = np.abs(x).max()
                r["p"][s, g, part] += p
                r["acc"][s, g, part] += p
    return r


def evict(k, v, pages, lens, seen, keep, sinks, recent, acc, pos):
    """Copies of k, v, acc, pos after the eviction, and the new lengths."""
    k, v, acc, pos = k.copy(), v.copy(), acc.copy(), pos.copy()
    page, hkv = k.shape[2], k.shape[1]
    new = np.minimum(np.maximum(lens, 0), keep).astype(np.int32)
    for s in range(len(lens)):
        size = int(lens[s])
        if size <= keep:
            continue
        for h in range(hkv):
            def rank(j):
                held = pos[s, h, j] < sinks or pos[s, h, j] >= seen[s] - recent
                w = acc[s, h, j]
                if held:
                    return (0, 0.0, j)
                return (2, 0.0, j) if np.isnan(w) else (1, -float(w), j)
            stay = set(sorted(range(size), key=rank)[:keep])
            holes = [j for j in range(keep) if j not in stay]
            moves = [j for j in range(keep, size) if j in stay]
            assert len(holes) == len(moves)
            for a, b in zip(moves, holes):
                pa, pb = pages[s, a // page], pages[s, b // page]
                k[pb, h, b % page] = k[pa, h, a % page]
                v[pb, h, b % page] = v[pa, h, a % page]
                acc[s, h, b], pos[s, h, b] = acc[s, h, a], pos[s, h, a]
    return k, v, acc, pos, new
