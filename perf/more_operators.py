"""Operators of a step of several new tokens per sequence over a paged key-value cache: cases, plain forms
and the library's calls.

A prompt, a piece of one, or a tree of drafted tokens goes through a layer at once:

  heads   norm of each head and rotary positions on one to three axes in one pass, and its gradient
  append  the same for the new tokens' q and k, then k and v into their cache pages
  attn    attention of the new tokens over their sequences' pages: causal, a drafted tree, a
          prefix, packed documents, a window, a distance bias, scores capped by a tanh
  accept  the drafted path that the model agrees with, its k and v moved together in every layer

``run`` computes the plain form with elementary torch operations in 32 bits, or, where ``own``
is true, calls the library.  ``exact`` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------- cases

def listed():
    base = dict(op="attn", hq=32, hkv=8, d=128, type="bf16", qtype="bf16", page=16, major="head",
                tree=False, cap=0.0, window=0, slopes=False, docs=0, prefix=0)
    return [
        # One user's drafted tree over a short context: latency is all.
        dict(base, name="tree_one", n=1, tlo=16, thi=16, clo=900, chi=900, tree=True),
        # A serving batch that verifies trees over ragged contexts.
        dict(base, name="tree_batch", n=32, tlo=8, thi=32, clo=100, chi=8192, tree=True),
        # The same with f32 queries (the projection's own) and capped scores.
        dict(base, name="tree_f32", n=12, tlo=5, thi=16, clo=1, chi=6000, tree=True, qtype="f32",
             cap=50.0),
        # A long prompt into an empty cache.
        dict(base, name="prompt", n=1, tlo=8192, thi=8192, clo=0, chi=0, page=64),
        # A batch of pieces of prompts over what is cached, heads of 64 in f16, a window on
        # every token.
        dict(base, name="pieces", n=5, tlo=1, thi=1531, clo=37, chi=6001, hq=16, hkv=4, d=64,
             type="f16", qtype="f16", page=32, major="token", window=1024),
        # Packed documents, the first slots (an image) seen both ways, odd pages, a distance bias, an
        # f32 cache.
        dict(base, name="documents", n=3, tlo=100, thi=701, clo=0, chi=300, hq=12, hkv=6, d=96,
             type="f32", qtype="f32", page=7, slopes=True, docs=256, prefix=130),
        # Drafted tokens of a batch: norms, rotation, into the pages.
        dict(name="append_drafts", op="append", n=32, each=8, hi=2048, hq=32, hkv=8, d=128, rot=128,
             inter=False, type="bf16", qtype="bf16", page=16, major="head", kind="rms", axes=1,
             dealt=False),
        # A prompt with images: positions by time, height and width.
        dict(name="append_prompt", op="append", n=2, each=4001, hi=4096, hq=28, hkv=4, d=128,
             rot=128, inter=False, type="bf16", qtype="bf16", page=64, major="token", kind="rms",
             axes=3, dealt=True),
        # An image encoder's queries and keys: LayerNorm, rows and columns.
        dict(name="heads_image", op="heads", n=4900, h=32, d=80, rot=80, inter=False, kind="layer",
             axes=2, dealt=False, otype="bf16", back=False),
        # The gradient of a training step through norm and rotation.
        dict(name="heads_back", op="heads", n=4096, h=40, d=128, rot=128, inter=True, kind="rms",
             axes=1, dealt=False, otype="f32", back=True),
        # One user's tree verified in a deep model.
        dict(name="accept_one", op="accept", n=1, t=16, ctx=900, hkv=8, d=128, type="bf16", page=16,
             major="head", layers=32),
        # A batch's.
        dict(name="accept_batch", op="accept", n=64, t=32, ctx=500, hkv=8, d=128, type="bf16",
             page=16, major="head", layers=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "heads", "append", "accept"])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 128, 192, 256])
    kind = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    page = rng.choice([1, 7, 16, 16, 32, 64, 100])
    major = rng.choice(["head", "token"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = min(64, hkv * rng.choice([1, 2, 4, 4, 5, 8, 16]))
    hq = max(hkv, hq - hq % hkv)
    inter = rng.random() < 0.5
    rot = rng.choice([d, d, d // 2])
    axes = rng.choice([1, 1, 2, 3])
    norm = rng.choice(["rms", "rms", "layer"])
    if op == "heads":
        n, h = _log(rng, 1, 8192), _log(rng, 1, 64)
        n = max(1, min(n, 4096 * 40 * 128 // (h * d)))
        return dict(op=op, n=n, h=h, d=d, rot=rot, inter=inter, kind=norm, axes=axes,
                    dealt=rng.random() < 0.5, otype=rng.choice(["f32", "bf16", "f16"]),
                    back=rng.random() < 0.5)
    if op == "append":
        tokens = min(_log(rng, 1, 8192), 8002 * 36 * 128 // ((hq + 2 * hkv) * d))
        n = max(1, min(tokens, _log(rng, 1, 128)))
        each = max(1, tokens // n)
        n = max(1, min(n, (1 << 28) // ((each + 1024) * hkv * d * _BYTES[kind])))
        return dict(op=op, n=n, each=each, hi=each + rng.randrange(0, 1024), hq=hq, hkv=hkv, d=d,
                    rot=rot, inter=inter, type=kind, qtype=rng.choice([kind, "f32"]), page=page,
                    major=major, kind=norm, axes=axes, dealt=rng.random() < 0.5)
    if op == "accept":
        layers = _log(rng, 1, 48)
        t = _log(rng, 2, 128)
        ctx = rng.randrange(0, 1024)
        slots = (1 << 31) // (2 * layers * hkv * d * _BYTES[kind])
        n = max(1, min(_log(rng, 1, 64), slots // (ctx + t + page)))
        return dict(op=op, n=n, t=t, ctx=ctx, hkv=hkv, d=d, type=kind, page=page, major=major,
                    layers=layers)
    tree = rng.random() < 0.5
    # Scores of all heads in 32 bits: at most those of the longest prompt.
    most = 8192 * 8192 * 32 // hq
    if tree:
        thi = _log(rng, 2, 96)
        chi = min(_log(rng, 16, 65536), (1 << 30) // (4 * hkv * d))
    else:
        thi = _log(rng, 1, 6000)
        chi = rng.choice([0, _log(rng, 1, 16384)])
        chi = max(0, min(chi, most // thi - thi))
    n = max(1, min(_log(rng, 1, 48), most // 4 // (thi * (thi + chi)),
                   (1 << 30) // (4 * hkv * d * (thi + chi))))
    same = rng.random() < 0.3
    docs = 0 if tree else rng.choice([0, 0, 0, max(8, thi // 3)])
    return dict(op=op, n=n, tlo=thi if same else rng.randrange(0, thi + 1), thi=thi,
                clo=chi if same else rng.randrange(0, chi + 1), chi=chi, hq=hq, hkv=hkv, d=d,
                type=kind, qtype=rng.choice([kind, kind, "f32"]), page=page, major=major, tree=tree,
                cap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.choice([0, 0, 0, max(1, (thi + chi) // 3)]),
                slopes=rng.random() < 0.2, docs=docs,
                prefix=0 if tree else rng.choice([0, 0, max(1, thi // 4)]))


def _spread(n, lo, hi):
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _extents(case):
    """Each sequence's (new tokens, context before them): both spread over their ranges, the long
    contexts not with the long pieces (their order goes by the seed)."""
    n = case["n"]
    t, c = _spread(n, case["tlo"], case["thi"]), _spread(n, case["clo"], case["chi"])
    return [(t[i], c[i * 7 % n if n % 7 else n - 1 - i]) for i in range(n)]


# ----------------------------------------------------------------------------- inputs

def _cache(case, lens, g, layers=0):
    """K and V pools seen as [page][head][slot][dim] (or [layer][page]...), filled, and a table of
    scattered pages."""
    ps, h, d = case["page"], case["hkv"], case["d"]
    need = [-(-x // ps) for x in lens]
    wide = max(1, max(need))
    count = sum(need) + 3
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    col = torch.arange(wide, device="cuda")
    live = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(live, order[(first[:, None] + col).clamp(max=count - 1)], -1)
    pools = []
    for _ in range(2):
        shape = (count, h, ps, d) if case["major"] == "head" else (count, ps, h, d)
        shape = ((layers,) if layers else ()) + shape
        pool = torch.randn(shape, generator=g, device="cuda",
                           dtype=torch.float32).to(_TYPES[case["type"]])
        pools.append(pool if case["major"] == "head" else pool.transpose(-3, -2))
    return pools[0], pools[1], table.to(torch.int32).contiguous()


def _angles(rows, rot):
    """cos and sin of position times frequency, [rows][rot/2][2], as a program keeps them."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _pairs(case):
    """How many pairs each axis has."""
    half, axes = case["rot"] // 2, case["axes"]
    rest = half // (axes + 1) if axes > 1 else 0
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def _tree(counts, wide, g):
    """Random trees: a node's parent is one of the four before it; the root is node 0.  Parents
    [n][wide], and whether b is a or above it, [n][wide][wide]."""
    n = len(counts)
    back = torch.randint(1, 5, (n, wide), generator=g, device="cuda")
    node = torch.arange(wide, device="cuda")
    parent = (node - back).clamp(min=0)
    parent[:, 0] = -1
    above = torch.zeros(n, wide, wide, dtype=torch.bool, device="cuda")
    row = torch.arange(n, device="cuda")
    for j in range(wide):
        if j:
            above[:, j] = above[row, parent[:, j]]
        above[:, j, j] = True
    return parent, above


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = dict(case=case)
    op, n, d = case["op"], case["n"], case["d"]
    if op in ("heads", "append"):
        m = n if op == "heads" else n * case["each"]
        s["rows"] = 4096 if op == "heads" else max(case["hi"], 64)
        s["table"] = _angles(s["rows"], case["rot"])
        s["weight"] = 1.0 + 0.2 * normal(2, d)
        s["bias"] = 0.1 * normal(2, d)
        s["pos"] = ints(0, s["rows"], case["axes"], m)
    if op == "heads":
        h = case["h"]
        s["x"] = 3.0 * normal(n, h * d)
        if case["back"]:
            s["grad"] = normal(n, h * d)
            s["grad_x"] = torch.zeros_like(s["x"])
            s["grad_w"], s["grad_b"] = torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
        else:
            s["out"] = torch.zeros(n, h * d, device="cuda", dtype=_TYPES[case["otype"]])
        return s
    hkv = case["hkv"]
    if op == "append":
        each, hi = case["each"], case["hi"]
        s["k"], s["v"], s["pages"] = _cache(case, [hi] * n, g)
        base = torch.randint(0, hi - each + 1, (n, 1), generator=g, device="cuda")
        slot = base + torch.arange(each, device="cuda")
        s["slot"] = slot.reshape(-1).to(torch.int32)
        s["seq"] = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(each)
        s["pos"][0] = s["slot"]
        # One fused projection's rows: q, then k, then v.
        s["qkv"] = 2.0 * normal(n * each, (case["hq"] + 2 * hkv) * d)
        s["q_out"] = torch.zeros(n * each, case["hq"] * d, device="cuda",
                                 dtype=_TYPES[case["qtype"]])
        return s
    if op == "accept":
        t, ctx, layers = case["t"], case["ctx"], case["layers"]
        s["k"], s["v"], s["pages"] = _cache(case, [ctx + t] * n, g, layers)
        parent, s["above"] = _tree([t] * n, t, g)
        s["parent"] = parent.to(torch.int32).reshape(-1).contiguous()
        # The model agrees with about two of three drafted tokens (of few values, so that
        # siblings with the same token are met).
        tokens = ints(0, 6, n, t)
        choice = ints(0, 6, n, t)
        agree = torch.rand(n, t, generator=g, device="cuda") < 0.6
        child = torch.randint(1, 5, (n, t), generator=g, device="cuda")
        node = (torch.arange(t, device="cuda") + child).clamp(max=t - 1)
        choice = torch.where(agree, tokens.gather(1, node), choice)
        s["tokens"], s["choice"] = tokens.reshape(-1).contiguous(), choice.reshape(-1).contiguous()
        s["starts"] = torch.arange(n + 1, device="cuda", dtype=torch.int32) * t
        s["lens"] = torch.full((n,), ctx + t, device="cuda", dtype=torch.int32)
        s["path"] = torch.zeros(n * t, device="cuda", dtype=torch.int32)
        s["count"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["next"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["lens_out"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        return s
    ext = _extents(case)
    mix = torch.randperm(n, generator=g, device="cuda").tolist()
    ext = [ext[i] for i in mix]
    counts, lens = [t for t, _ in ext], [t + c for t, c in ext]
    s["k"], s["v"], s["pages"] = _cache(case, lens, g)
    m, wide = sum(counts), max(counts)
    s["m"], s["wide"] = m, wide
    s["starts"] = torch.tensor([sum(counts[:i]) for i in range(n + 1)], device="cuda",
                               dtype=torch.int32)
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    kind = _TYPES[case["qtype"]]
    s["q"] = (1.5 * normal(max(m, 1), case["hq"] * d)).to(kind)
    s["out"] = torch.zeros(max(m, 1), case["hq"] * d, device="cuda", dtype=kind)
    s["lse"] = torch.zeros(max(m, 1), case["hq"], device="cuda")
    node = torch.arange(wide, device="cuda")
    held = node < torch.tensor(counts, device="cuda")[:, None]
    base = torch.tensor([c for _, c in ext], device="cuda")[:, None]
    if case["tree"]:
        parent, above = _tree(counts, wide, g)
        words = -(-wide // 32)
        bit = torch.zeros(n, wide, words * 32, dtype=torch.int64, device="cuda")
        bit[:, :, :wide] = above
        bit = (bit.view(n, wide, words, 32) << torch.arange(32, device="cuda")).sum(-1)
        bit = torch.where(bit >= 1 << 31, bit - (1 << 32), bit).to(torch.int32)
        s["tree"] = bit[held].contiguous()
        depth = above.sum(-1) - 1
        s["pos"] = (base + depth)[held].to(torch.int32).contiguous()
    if case["docs"]:
        # A document begins every `docs` slots.
        slot = base + node
        s["first"] = (slot - slot % case["docs"])[held].to(torch.int32).contiguous()
    if case["prefix"]:
        s["prefix"] = torch.full((n,), case["prefix"], device="cuda", dtype=torch.int32)
    if case["slopes"]:
        h = torch.arange(1, case["hq"] + 1, device="cuda", dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * h / case["hq"]).contiguous()
    return s


# -------------------------------------------------------------------------- plain forms

def _axis_of(case, device):
    """The axis of each pair: runs of pairs, or dealt in turn with the rest on axis 0."""
    half, axes, pairs = case["rot"] // 2, case["axes"], _pairs(case)
    i = torch.arange(half, device=device)
    if case["dealt"]:
        size = torch.tensor(pairs, device=device)
        axis = i % axes
        return torch.where(i < axes * size[axis], axis, 0)
    return torch.repeat_interleave(torch.arange(axes, device=device),
                                   torch.tensor(pairs, device=device))


def _cos_sin(s):
    """[tokens][pairs] cos and sin, each pair by the position on its axis."""
    axis = _axis_of(s["case"], "cuda")
    pos = s["pos"].long()[axis]                                     # [pairs][tokens]
    pair = torch.arange(axis.numel(), device="cuda")
    cs = s["table"][pos, pair[:, None]]                             # [pairs][tokens][2]
    return cs[..., 0].T[:, None], cs[..., 1].T[:, None]


def _turn(x, c, t, rot, inter):
    """x [tokens][heads][d] turned."""
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * t, a * t + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * t, a * t + b * c
    return y


_EPS = 1e-6


def _hat(x, kind):
    """x without its mean (LayerNorm) over its root mean square, and one over that root."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * r, r


def _norm(x, kind, w, b):
    y = _hat(x, kind)[0] * w
    return y + b if kind == "layer" else y


def _plain_heads(s):
    c = s["case"]
    x = s["x"].view(c["n"], c["h"], c["d"])
    cos, sin = _cos_sin(s)
    w, b = s["weight"][0], s["bias"][0]
    if not c["back"]:
        y = _turn(_norm(x, c["kind"], w, b), cos, sin, c["rot"], c["inter"])
        return y.view_as(s["x"]).to(_TYPES[c["otype"]])
    g = _turn(s["grad"].view_as(x), cos, -sin, c["rot"], c["inter"])
    hat, r = _hat(x, c["kind"])
    u = g * w
    dx = u - hat * (u * hat).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - u.mean(-1, keepdim=True)
    out = dict(x=(dx * r).view_as(s["x"]), w=(g * hat).sum((0, 1)))
    if c["kind"] == "layer":
        out["b"] = g.sum((0, 1))
    return out


def _plain_append(s):
    c = s["case"]
    hq, hkv, d, ps = c["hq"], c["hkv"], c["d"], c["page"]
    m = s["qkv"].shape[0]
    q, k, v = s["qkv"].view(m, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    cos, sin = _cos_sin(s)
    q = _turn(_norm(q, c["kind"], s["weight"][0], s["bias"][0]), cos, sin, c["rot"], c["inter"])
    k = _turn(_norm(k, c["kind"], s["weight"][1], s["bias"][1]), cos, sin, c["rot"], c["inter"])
    seq, slot = s["seq"].long(), s["slot"].long()
    page, row = s["pages"].long()[seq, slot // ps], slot % ps
    s["k"][page, :, row] = k.to(s["k"].dtype)
    s["v"][page, :, row] = v.to(s["v"].dtype)
    return dict(q=q.reshape(m, hq * d).to(_TYPES[c["qtype"]]), k=s["k"], v=s["v"])


def _plain_attn(s):
    c = s["case"]
    n, hq, hkv, d, ps, wide, m = c["n"], c["hq"], c["hkv"], c["d"], c["page"], s["wide"], s["m"]
    cap = s["pages"].shape[1] * ps
    col = torch.arange(cap, device="cuda")
    page = s["pages"].long().clamp(min=0)[:, col // ps]
    k = s["k"][page, :, col % ps].float()            # [n][cap][hkv][d]
    v = s["v"][page, :, col % ps].float()
    starts, lens = s["starts"].long(), s["lens"].long()[:, None]
    count = (starts[1:] - starts[:-1])[:, None]
    node = torch.arange(wide, device="cuda")
    held = node < count                              # [n][wide]: the ragged tokens, padded
    at = (starts[:-1, None] + node).clamp(max=max(m, 1) - 1)
    base = lens - count
    slot = base + node                               # [n][wide]
    # [n][hkv][group][wide][d] . [n][hkv][d][cap]
    q = s["q"].float()[at].view(n, wide, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(n, hkv, -1, d), k.permute(0, 2, 3, 1)) * d ** -0.5
    x = x.view(n, hkv, hq // hkv, wide, cap)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = slot
    col_pos = col.expand(n, cap)
    if c["tree"]:
        pos = s["pos"].long()[at]
        own_pos = pos.gather(1, (col - base).clamp(0, wide - 1))
        col_pos = torch.where(col >= base, own_pos, col_pos)
        word = (col - base).clamp(0, wide - 1)       # [n][cap]
        bits = s["tree"][at].long()                  # [n][wide][words]
        bit = bits.gather(2, (word // 32)[:, None].expand(n, wide, cap))
        bit = (bit >> (word % 32)[:, None]) & 1
        seen = (col < base)[:, None] | ((bit == 1) & (col < lens)[:, None])
    else:
        last = slot + 1
        if c["prefix"]:
            last = torch.maximum(last, torch.minimum(s["prefix"].long()[:, None], lens))
        seen = col < last[..., None]                 # [n][wide][cap]
    if c["docs"]:
        seen = seen & (col >= s["first"].long()[at][..., None])
    far = (pos[..., None] - col_pos[:, None])        # [n][wide][cap]
    if c["window"]:
        seen = seen & (far < c["window"])
    if c["slopes"]:
        x = x - s["slopes"].view(hkv, -1)[:, :, None, None] * far[:, None, None].float()
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.matmul(p.view(n, hkv, -1, cap), v.permute(0, 2, 1, 3))
    out = out.view(n, hkv, hq // hkv, wide, d).permute(0, 3, 1, 2, 4)[held]
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)[held]
    return dict(out=out.reshape(m, hq * d).to(_TYPES[c["qtype"]]), lse=lse.reshape(m, hq))


def _plain_accept(s):
    c = s["case"]
    n, t, ps, layers = c["n"], c["t"], c["page"], c["layers"]
    token, choice = s["tokens"].view(n, t), s["choice"].view(n, t)
    parent = s["parent"].view(n, t).long()
    node = torch.arange(t, device="cuda")
    agrees = (token == choice.gather(1, parent.clamp(min=0))) & (node > 0)
    # Of siblings that agree the lowest counts.
    twin = (parent[:, :, None] == parent[:, None]) & agrees[:, None] & (node < node[:, None])
    agrees = (agrees & ~twin.any(-1)) | (node == 0)
    taken = ~(s["above"] & ~agrees[:, None]).any(-1)          # every node above it too
    count = taken.sum(-1)
    order = torch.where(taken, node, t).sort(-1).values
    live = node < count[:, None]
    path = torch.where(live, order, -1)
    last = path.gather(1, count[:, None] - 1)
    lens = s["lens"].long()[:, None]
    base = lens - t
    seq, to = live.nonzero(as_tuple=True)
    src, dst = (base[seq, 0] + path[seq, to]), (base[seq, 0] + to)
    pages = s["pages"].long()
    a, b = pages[seq, src // ps], pages[seq, dst // ps]
    for pool in (s["k"], s["v"]):
        pool[:, b, :, dst % ps] = pool[:, a, :, src % ps]
    return dict(path=path.to(torch.int32).reshape(-1), count=count.to(torch.int32),
                next=choice.gather(1, last).squeeze(1),
                lens=(base[:, 0] + count).to(torch.int32), k=s["k"], v=s["v"])


# ---------------------------------------------------------------------- library's calls

def _wq_type(wq, name):
    return {"bf16": wq.WQ_BF16, "f16": wq.WQ_F16, "f32": wq.WQ_F32}[name]


def _own_axes(wq, s):
    c = s["case"]
    flags = wq.WQ_ROPE_INTERLEAVED if c["inter"] else 0
    flags |= wq.WQ_AXES_DEALT if c["dealt"] else 0
    return wq.rope_axes(c["rot"], flags, _pairs(c), s["pos"], s["table"])


def _own_norm(wq, s, i):
    layer = s["case"]["kind"] == "layer"
    return wq.head_norm(wq.WQ_HEAD_LAYER if layer else wq.WQ_HEAD_RMS, _EPS, s["weight"][i],
                        s["bias"][i] if layer else None)


def _own(s):
    import gemv_transformer_gb300 as wq
    c = s["case"]
    op, n, d = c["op"], c["n"], c["d"]
    if op == "heads":
        if "axes" not in s:  # descriptors that a program keeps beside its buffers
            s["axes"], s["norm"] = _own_axes(wq, s), _own_norm(wq, s, 0)
        h, row = c["h"], c["h"] * d
        if not c["back"]:
            wq.check(wq.wq_norm_rope(n, h, d, s["norm"], s["axes"], s["x"], row,
                                     _wq_type(wq, c["otype"]), s["out"], row))
            return s["out"]
        layer = c["kind"] == "layer"
        if "room" not in s:
            s["size"] = wq.wq_norm_rope_grad_workspace_bytes(n, h, d)
            s["room"] = torch.empty(max(s["size"], 256), dtype=torch.uint8, device="cuda")
        wq.check(wq.wq_norm_rope_grad(n, h, d, s["norm"], s["axes"], s["x"], row, s["grad"], row,
                                      s["grad_x"], row, s["grad_w"],
                                      s["grad_b"] if layer else None, s["room"], s["size"]))
        out = dict(x=s["grad_x"], w=s["grad_w"])
        if layer:
            out["b"] = s["grad_b"]
        return out
    hkv, wide = c["hkv"], s["pages"].shape[1]
    if op == "append":
        if "cache" not in s:
            s["cache"] = wq.kv_cache(s["k"], s["v"])
            s["axes"] = _own_axes(wq, s)
            s["norms"] = _own_norm(wq, s, 0), _own_norm(wq, s, 1)
        m, hq, row = n * c["each"], c["hq"], (c["hq"] + 2 * hkv) * d
        q = s["qkv"].data_ptr()
        wq.check(wq.wq_kv_append_norm(
            s["cache"], m, hq, s["norms"][0], s["norms"][1], s["axes"], q, row, q + 4 * hq * d, row,
            q + 4 * (hq + hkv) * d, row, n, s["seq"], s["slot"], s["pages"], wide,
            _wq_type(wq, c["qtype"]), s["q_out"], hq * d))
        return dict(q=s["q_out"], k=s["k"], v=s["v"])
    if op == "accept":
        if "caches" not in s:
            s["caches"] = wq.kv_caches(list(s["k"].unbind()), list(s["v"].unbind()))
        wq.check(wq.wq_kv_accept(s["caches"], n, n * c["t"], s["pages"], wide, s["starts"],
                                 s["parent"], s["tokens"], s["choice"], s["lens"], s["path"],
                                 s["count"], s["next"], s["lens_out"]))
        return dict(path=s["path"], count=s["count"], next=s["next"], lens=s["lens_out"], k=s["k"],
                    v=s["v"])
    hq, m, kind = c["hq"], s["m"], _wq_type(wq, c["qtype"])
    if m == 0:
        return dict(out=s["out"][:0], lse=s["lse"][:0])
    if "room" not in s:
        s["cache"] = wq.kv_cache(s["k"], s["v"])
        s["form"] = wq.attn_form(softcap=c["cap"], window=c["window"], slopes=s.get("slopes"),
                                 first=s.get("first"), prefix=s.get("prefix"), tree=s.get("tree"),
                                 pos=s.get("pos"))
        s["size"] = wq.wq_attn_tokens_workspace_bytes(s["cache"], n, m, hq, kind)
        s["room"] = torch.empty(max(s["size"], 256), dtype=torch.uint8, device="cuda")
    wq.check(wq.wq_attn_tokens(s["cache"], n, m, hq, d ** -0.5, s["form"], kind, s["q"], hq * d,
                               s["starts"], s["pages"], wide, s["lens"], kind, s["out"], hq * d,
                               s["lse"], s["room"], s["size"]))
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"heads": _plain_heads, "append": _plain_append, "attn": _plain_attn,
            "accept": _plain_accept}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work

def work(case):
    op, n, d = case["op"], case["n"], case["d"]
    if op == "heads":
        x = n * case["h"] * d
        each = 12 if case["back"] else 4 + _BYTES[case["otype"]]
        table = 4 * min(n, 4096) * case["rot"]
        return dict(bytes=each * x + 4 * n * case["axes"] + table, flops=(16 if case["back"] else 8) * x)
    hkv, b = case["hkv"], _BYTES[case["type"]]
    if op == "append":
        m, hq = n * case["each"], case["hq"]
        x = m * (hq + 2 * hkv) * d
        return dict(bytes=4 * x + m * d * (_BYTES[case["qtype"]] * hq + 2 * b * hkv)
                    + 4 * m * (2 + case["axes"]) + 4 * min(m, case["hi"]) * case["rot"],
                    flops=8 * m * (hq + hkv) * d)
    if op == "accept":
        # About two accepted tokens beyond the root, each moved in every layer.
        return dict(bytes=n * case["t"] * 16 + n * 2 * 4 * case["layers"] * hkv * d * b,
                    flops=n * case["t"])
    flops, kv = 0, 0
    hq, m = case["hq"], 0
    for t, c in _extents(case):
        m += t
        window, docs, prefix = case["window"] or 1 << 30, case["docs"], min(case["prefix"], c + t)
        low = c
        for j in range(t):
            at = c + j
            lo = max(at - window + 1, at - at % docs if docs else 0, 0)
            hi = at + 1 if not case["tree"] else c + 1
            hi = max(hi, prefix)
            low = min(low, lo)
            flops += 4 * d * hq * max(0, hi - lo)
        kv += max(0, c + t - low) if t else 0
    io = 2 * m * hq * d * _BYTES[case["qtype"]] + 4 * m * hq
    return dict(bytes=io + 2 * kv * hkv * d * b, flops=flops)


# ---------------------------------------------------------------------- definition, 64 bits

def _turn64(x, table, pos, axis, inter, back):
    """Each pair as a complex number times e^(i angle); x [tokens][heads][d] in 64 bits."""
    half = axis.numel()
    rot = 2 * half
    e = torch.view_as_complex(table.double())                       # [rows][pairs]
    pair = torch.arange(half, device=x.device)
    e = e[pos.long()[axis].T, pair]                                 # [tokens][pairs]
    if back:
        e = e.conj()
    y = x.clone()
    if inter:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], half, 2).contiguous())
        z = torch.view_as_real(z * e[:, None])
        y[..., :rot] = z.reshape(*x.shape[:-1], rot)
    else:
        z = torch.complex(x[..., :half], x[..., half:rot]) * e[:, None]
        y[..., :half], y[..., half:rot] = z.real, z.imag
    return y


def _axis_list(case):
    half, axes, left = case["rot"] // 2, case["axes"], _pairs(case)
    if not case["dealt"]:
        return [a for a in range(axes) for _ in range(left[a])]
    return [i % axes if i // axes < left[i % axes] else 0 for i in range(half)]


def _norm64(x, kind, w, b):
    if kind == "rms":
        return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt() * w
    mu = x.sum(-1, keepdim=True) / x.shape[-1]
    var = (x - mu).square().sum(-1, keepdim=True) / x.shape[-1]
    return (x - mu) / (var + _EPS).sqrt() * w + b


def exact(case, seed):
    op, n, d = case["op"], case["n"], case["d"]
    s = prepare(case, seed)
    if op in ("heads", "append"):
        axis = torch.tensor(_axis_list(case), device="cuda")
        w, b = s["weight"].double(), s["bias"].double()
    if op == "heads":
        x = s["x"].double().view(n, case["h"], d)
        if not case["back"]:
            y = _turn64(_norm64(x, case["kind"], w[0], b[0]), s["table"], s["pos"], axis,
                        case["inter"], False)
            return y.reshape(n, -1)
        # The gradient by torch's own differentiation of the definition.
        x.requires_grad_(True)
        w0, b0 = w[0].clone().requires_grad_(True), b[0].clone().requires_grad_(True)
        y = _norm64(x, case["kind"], w0, b0)
        g = _turn64(s["grad"].double().view(n, case["h"], d), s["table"], s["pos"], axis,
                    case["inter"], True)
        y.backward(g)
        out = dict(x=x.grad.reshape(n, -1), w=w0.grad)
        if case["kind"] == "layer":
            out["b"] = b0.grad
        return out
    hkv, ps = case["hkv"], case["page"]
    if op == "append":
        hq, m = case["hq"], n * case["each"]
        x = s["qkv"].double().view(m, hq + 2 * hkv, d)
        q = _turn64(_norm64(x[:, :hq], case["kind"], w[0], b[0]), s["table"], s["pos"], axis,
                    case["inter"], False)
        new = [_turn64(_norm64(x[:, hq:hq + hkv], case["kind"], w[1], b[1]), s["table"], s["pos"],
                       axis, case["inter"], False), x[:, hq + hkv:]]
        out = dict(q=q.reshape(m, -1))
        slot = s["slot"].long()
        page = s["pages"][s["seq"].long(), slot // ps].long()
        for name, rows in zip("kv", new):
            pool = s[name].double()
            # [page][slot][head][dim], so that a token is one row
            pool.transpose(1, 2)[page, slot % ps] = rows
            out[name] = pool
        return out
    if op == "accept":
        return None  # whole numbers, and rows that are moved as they are
    hq, group = case["hq"], case["hq"] // hkv
    m = s["m"]
    out = torch.zeros(m, hq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((m, hq), -math.inf, device="cuda", dtype=torch.float64)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    q = s["q"].view(-1, hq, d)
    for i in range(n):
        t0, t1, size = starts[i], starts[i + 1], lens[i]
        t = t1 - t0
        if not t:
            continue
        base = size - t
        j = torch.arange(size, device="cuda")
        pages = s["pages"][i, j // ps].long()
        pos_q = base + torch.arange(t, device="cuda")
        pos_k = j.clone()
        if case["tree"]:
            pos_q = s["pos"][t0:t1].long()
            pos_k[base:] = pos_q
        for g in range(hkv):
            k, v = (s[x][pages, g, j % ps].double() for x in "kv")
            step = max(1, (1 << 28) // max(1, group * size))
            for a in range(0, t, step):
                e = min(t, a + step)
                rows = base + torch.arange(a, e, device="cuda")[:, None]
                if case["tree"]:
                    word = s["tree"][t0 + a:t0 + e].long() & 0xFFFFFFFF
                    bits = (word[:, :, None] >> torch.arange(32, device="cuda")) & 1
                    bits = bits.reshape(e - a, -1)[:, :t]
                    hide = torch.cat([torch.zeros(e - a, base, device="cuda", dtype=torch.bool),
                                      bits == 0], 1)
                else:
                    hide = (j > rows)
                    if case["prefix"]:
                        hide = hide & (j >= s["prefix"][i])
                if case["docs"]:
                    hide = hide | (j < s["first"][t0 + a:t0 + e, None])
                away = pos_q[a:e, None] - pos_k
                if case["window"]:
                    hide = hide | (away >= case["window"])
                qq = q[t0 + a:t0 + e, g * group:(g + 1) * group].double()
                x = torch.einsum("thd,jd->htj", qq, k) / math.sqrt(d)
                if case["cap"]:
                    x = (x / case["cap"]).tanh() * case["cap"]
                if case["slopes"]:
                    x = x - s["slopes"][g * group:(g + 1) * group, None, None].double() * away
                x = x.masked_fill(hide, -math.inf)
                total = torch.logsumexp(x, -1)
                p = torch.where(total[..., None] > -math.inf, (x - total[..., None]).exp(), 0.0)
                out[t0 + a:t0 + e, g * group:(g + 1) * group] = torch.einsum("htj,jd->thd", p, v)
                lse[t0 + a:t0 + e, g * group:(g + 1) * group] = total.T
                del x, p
    return dict(out=out.view(m, hq * d), lse=lse)
