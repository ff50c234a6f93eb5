"""f64 oracle of the calls for several new tokens per sequence (numpy, test infrastructure).

Plain restatements of the definitions in ``include/wq.h``, sharing no code with the CUDA library.
Pools are numpy arrays seen as [page][head][row][dim].
"""
from __future__ import annotations

import math

import numpy as np

INTERLEAVED, DEALT, RESTART = 1, 4, 8
NONE, RMS, LAYER = 0, 1, 2


def pair_map(pairs, dealt=False, restart=False):
    """[(axis, column)] of each pair."""
    half, axes = sum(pairs), len(pairs)
    if dealt:
        axis = [i % axes if i // axes < pairs[i % axes] else 0 for i in range(half)]
    else:
        axis = [a for a in range(axes) for _ in range(pairs[a])]
    return [(a, axis[:i].count(a) if restart else i) for i, a in enumerate(axis)]


def cos_sin(pairs, pos, table, dealt=False, restart=False):
    """[n][rot/2][2] from pos [axes][n] and table [rows][columns][2]."""
    pos = np.atleast_2d(pos)
    m = pair_map(pairs, dealt, restart)
    return np.stack([table[pos[a], c] for a, c in m], 1) if m else np.zeros((pos.shape[1], 0, 2))


def hat(x, kind, eps):
    """(x - mu) r and r."""
    x = np.asarray(x, np.float64)
    if kind == LAYER:
        x = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def norm(x, kind, eps=0.0, weight=None, bias=None):
    """y and the magnitude of its terms."""
    x = np.asarray(x, np.float64)
    if kind == NONE:
        return x, np.abs(x)
    h, r = hat(x, kind, eps)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(x.shape[-1]) if bias is None else np.asarray(bias, np.float64)
    mag = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * r * np.abs(w) + np.abs(b)
    return h * w + b, mag


def turn(x, cs, inter=False, back=False, mag=None):
    """Pairs of x [n][heads][d] turned by cs [n][pairs][2]; with mag also the terms' magnitudes."""
    y = np.array(x, np.float64)
    m = np.abs(y) if mag is None else np.array(mag, np.float64)
    m2 = m.copy()
    half = cs.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, s = cs[:, i, 0][:, None], cs[:, i, 1][:, None] * (-1 if back else 1)
        xa, xb = x[:, :, a], x[:, :, b]
        y[:, :, a], y[:, :, b] = xa * c - xb * s, xa * s + xb * c
        m2[:, :, a] = m[:, :, a] * np.abs(c) + m[:, :, b] * np.abs(s)
        m2[:, :, b] = m[:, :, a] * np.abs(s) + m[:, :, b] * np.abs(c)
    return y, m2


def norm_grad(x, g, kind, eps, weight=None):
    """dx, dw, db of norm() for the gradient g of y."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    if kind == NONE:
        return g, None, None
    h, r = hat(x, kind, eps)
    u = g if weight is None else g * np.asarray(weight, np.float64)
    dx = u - h * (u * h).mean(-1, keepdims=True)
    if kind == LAYER:
        dx = dx - u.mean(-1, keepdims=True)
    return dx * r, (g * h).sum((0, 1)), g.sum((0, 1))


def sees(j, slot, base, count, length, first=0, prefix=0, window=0, bits=None, pos=None):
    """Does token j of a sequence see the slot?  bits: its row of the tree as a set of nodes; pos:
    the new tokens' positions."""
    if slot < 0 or slot >= length or slot < first:
        return False
    if bits is not None:
        if not (slot < base or (slot - base) in bits):
            return False
    elif not slot < max(base + j + 1, min(prefix, length)):
        return False
    if window:
        mine = pos[j] if pos is not None else base + j
        its = pos[slot - base] if pos is not None and slot >= base else slot
        return mine - its < window
    return True


def attention(q, k, v, pages, starts, lens, scale, softcap=0.0, window=0, slopes=None, first=None,
              prefix=None, tree=None, pos=None):
    """q [tokens][hq][d]; tree: a list of sets of nodes, one for each token.  out, lse, and the
    magnitudes for tolerances: pv = sum p |v|, sx = max scale sum |q k|, mx = max |x|, n = slots."""
    m, hq, d = q.shape
    hkv, page = k.shape[1], k.shape[2]
    group = hq // hkv
    r = dict(out=np.zeros((m, hq, d)), lse=np.full((m, hq), -np.inf), pv=np.zeros((m, hq, d)),
             sx=np.zeros((m, hq)), mx=np.zeros((m, hq)), n=np.zeros(m, int))
    for s in range(len(lens)):
        t0, t1 = starts[s], starts[s + 1]
        count = t1 - t0
        length = min(max(int(lens[s]), 0), pages.shape[1] * page)
        base = length - count
        own_pos = None if pos is None else pos[t0:t1]
        slots = [j for j in range(length) if 0 <= pages[s, j // page] < k.shape[0]]
        if not slots:
            continue
        rows = [(pages[s, j // page], j % page) for j in slots]
        kk = np.array([k[p, :, i] for p, i in rows], np.float64)  # [slots][hkv][d]
        vv = np.array([v[p, :, i] for p, i in rows], np.float64)
        for t in range(t0, t1):
            j = t - t0
            see = [sees(j, x, base, count, length, 0 if first is None else first[t],
                        0 if prefix is None else prefix[s], window,
                        None if tree is None else tree[t], own_pos) for x in slots]
            see = np.array(see, bool)
            r["n"][t] = see.sum()
            if not see.any():
                continue
            mine = own_pos[j] if own_pos is not None else base + j
            its = np.array([own_pos[x - base] if own_pos is not None and x >= base else x
                            for x in slots], np.float64)[see]
            for h in range(hq):
                g = h // group
                with np.errstate(all="ignore"):
                    qk = kk[see][:, g] @ q[t, h].astype(np.float64)
                    x = scale * qk
                    if softcap:
                        x = softcap * np.tanh(x / softcap)
                    if slopes is not None:
                        x = x + float(slopes[h]) * (its - mine)
                    top = x.max()
                    e = np.exp(x - top)
                    p = e / e.sum()
                    r["out"][t, h] = p @ vv[see][:, g]
                    r["lse"][t, h] = top + math.log(e.sum()) if e.sum() > 0 else np.nan
                    r["pv"][t, h] = p @ np.abs(vv[see][:, g])
                    r["sx"][t, h] = abs(scale) * (np.abs(kk[see][:, g]) @ np.abs(q[t, h])).max()
                    r["mx"][t, h] = np.abs(x).max()
    return r


def accept(starts, parent, tokens, choice, lens):
    """path (-1 beyond it), accepted, next, new lengths, and each sequence's nodes."""
    n = len(lens)
    path = np.full(len(parent), -1, np.int64)
    count, nxt, out, nodes = np.zeros(n, int), np.full(n, -1), np.array(lens).copy(), []
    for s in range(n):
        t0, t1 = starts[s], starts[s + 1]
        chain = []
        if t1 > t0:
            chain = [0]
            while True:
                tip = chain[-1]
                kids = [c for c in range(1, t1 - t0)
                        if parent[t0 + c] == tip and tokens[t0 + c] == choice[t0 + tip]]
                if not kids:
                    break
                chain.append(min(kids))
            path[t0:t0 + len(chain)] = chain
            count[s], nxt[s] = len(chain), choice[t0 + chain[-1]]
            out[s] = lens[s] - (t1 - t0) + len(chain)
        nodes.append(chain)
    return path, count, nxt, out, nodes
