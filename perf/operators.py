"""The operators of a decode step over a paged key-value cache: cases, plain forms and the library's calls.

Four operators, each measured as one call of a serving program makes it:

  rope    rotary positions on packed rows of heads, forward and transposed (the gradient)
  append  rotate q and k of new tokens, write k and v into their cache pages
  attn    attention of one new token per sequence over its pages (optionally a mask, a
          window, and the slots' accumulated attention weight)
  evict   keep a budget of slots per sequence and kv head, by accumulated weight

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
    return [
        # One user's first decode steps: a few hundred slots, latency is all.
        dict(name="attn_one_short", op="attn", n=1, lo=391, hi=391, hq=32, hkv=8, d=128, type="bf16",
             page=16, major="head", window=0, mask="", acc=False),
        # One user with a very long context: the cache's length has to be split over the GPU.
        dict(name="attn_one_long", op="attn", n=1, lo=131072, hi=131072, hq=32, hkv=8, d=128,
             type="bf16", page=64, major="head", window=0, mask="", acc=False),
        # A serving batch of ragged lengths, eight query heads to a kv head.
        dict(name="attn_batch", op="attn", n=64, lo=1, hi=8192, hq=64, hkv=8, d=128, type="bf16",
             page=16, major="head", window=0, mask="", acc=False),
        # An encoder-decoder's sixteen plain heads on an f16 cache, odd pages, padding masked out
        # (one sequence has nothing left).
        dict(name="attn_mask_f16", op="attn", n=9, lo=0, hi=1500, hq=16, hkv=16, d=64, type="f16",
             page=7, major="token", window=0, mask="padding", acc=False),
        # Wide heads in f32, sixteen query heads to a kv head, a sliding window.
        dict(name="attn_window_f32", op="attn", n=5, lo=700, hi=6001, hq=32, hkv=2, d=256,
             type="f32", page=32, major="head", window=1024, mask="", acc=False),
        # The same step where the cache is bounded by eviction: the slots' weights are summed.
        dict(name="attn_weights", op="attn", n=16, lo=2049, hi=4096, hq=32, hkv=8, d=128,
             type="bf16", page=32, major="token", window=0, mask="", acc=True),
        # Rotation of a prompt's queries and keys (40 heads), half layout.
        dict(name="rope_prompt", op="rope", n=8192, h=40, d=128, rot=128, inter=False, back=False,
             rows=8192),
        # Its gradient in the interleaved layout, 80 of 96 dims, odd count of tokens.
        dict(name="rope_back", op="rope", n=1237, h=12, d=96, rot=80, inter=True, back=True,
             rows=2048),
        # One decode step of a batch: one token of each sequence.
        dict(name="append_step", op="append", n=64, each=1, hi=2048, hq=32, hkv=8, d=128, rot=128,
             inter=False, type="bf16", page=16, major="head", acc=True),
        # A prompt written into fresh pages.
        dict(name="append_prompt", op="append", n=4, each=2047, hi=4096, hq=32, hkv=8, d=128,
             rot=64, inter=False, type="f16", page=64, major="token", acc=False),
        # The steady state of a bounded cache: each step one slot over the budget.
        dict(name="evict_step", op="evict", n=64, len=2049, keep=2048, sinks=4, recent=256, hkv=8,
             d=128, type="bf16", page=16, major="head", mixed=True),
        # A long prompt cut down to its budget.
        dict(name="evict_prompt", op="evict", n=4, len=65536, keep=4096, sinks=4, recent=512, hkv=8,
             d=128, type="bf16", page=64, major="head", mixed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rope", "append", "evict"])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    page = rng.choice([1, 7, 16, 16, 32, 64, 100])
    major = rng.choice(["head", "token"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 4, 5, 8, 16])
    inter = rng.random() < 0.5
    rot = rng.choice([d, d, d // 2])
    if op == "rope":
        n, h = _log(rng, 1, 8192), _log(rng, 1, 64)
        n = min(n, 8192 * 40 * 128 // (h * d))
        rows = _log(rng, max(16, n), 32768)
        return dict(op=op, n=n, h=h, d=d, rot=rot, inter=inter, back=rng.random() < 0.5, rows=rows)
    if op == "append":
        tokens = min(_log(rng, 1, 8192), 8192 * 48 * 128 // ((hq + 2 * hkv) * d))
        n = max(1, min(tokens, _log(rng, 1, 128)))
        each = 1 if rng.random() < 0.4 else max(1, tokens // n)
        n = max(1, min(n, (1 << 28) // ((each + 1024) * hkv * d * _BYTES[kind])))
        return dict(op=op, n=n, each=each, hi=each + rng.randrange(0, 1024), hq=hq, hkv=hkv, d=d,
                    rot=rot, inter=inter, type=kind, page=page, major=major,
                    acc=rng.random() < 0.5)
    if op == "evict":
        slots = _log(rng, 64, min(262144, (1 << 30) // (2 * _BYTES[kind] * hkv * d)))
        n = max(1, min(_log(rng, 1, 64), slots // 64))
        length = slots // n
        keep = length - 1 if rng.random() < 0.4 else rng.randrange(length // 8, length)
        keep = max(keep, 8)
        recent = rng.randrange(1, max(2, keep // 4))
        return dict(op=op, n=n, len=length, keep=keep, sinks=rng.choice([0, 4]), recent=recent,
                    hkv=hkv, d=d, type=kind, page=page, major=major, mixed=rng.random() < 0.5)
    hq = min(hq, 64)
    hkv = min(hkv, hq)
    slots = _log(rng, 64, min(262144, (1 << 30) // (2 * _BYTES[kind] * hkv * d),
                              (1 << 28) // (hq * 4)))
    n = max(1, min(_log(rng, 1, 128), slots // 32))
    hi = slots // n
    lo = hi if rng.random() < 0.3 else rng.randrange(0, hi)
    return dict(op=op, n=n, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, type=kind, page=page, major=major,
                window=rng.choice([0, 0, 0, max(1, hi // 3)]),
                mask=rng.choice(["", "", "padding", "bias"]), acc=rng.random() < 0.3)


def _lengths(case):
    """The sequences' lengths, evenly spread from lo to hi (their order goes by the seed)."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


# ----------------------------------------------------------------------------- inputs

def _cache(case, lens, g):
    """K and V pools seen as [page][head][slot][dim], filled, and a table of scattered pages."""
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
        pool = torch.randn(shape, generator=g, device="cuda",
                           dtype=torch.float32).to(_TYPES[case["type"]])
        pools.append(pool if case["major"] == "head" else pool.permute(0, 2, 1, 3))
    return pools[0], pools[1], table.to(torch.int32).contiguous()


def _angles(rows, rot):
    """cos and sin of position times frequency, [rows][rot/2][2], as a program keeps them."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    op, n, d = case["op"], case["n"], case["d"]
    if op == "rope":
        s["table"] = _angles(case["rows"], case["rot"])
        s["x"] = normal(n, case["h"] * d)
        s["pos"] = torch.randint(0, case["rows"], (n,), generator=g, device="cuda",
                                 dtype=torch.int32)
        s["out"] = torch.zeros_like(s["x"])
        return s
    hkv = case["hkv"]
    if op == "append":
        each, hi = case["each"], case["hi"]
        s["k"], s["v"], s["pages"] = _cache(case, [hi] * n, g)
        base = torch.randint(0, hi - each + 1, (n, 1), generator=g, device="cuda")
        slot = base + torch.arange(each, device="cuda")
        s["slot"] = slot.reshape(-1).to(torch.int32)
        s["seq"] = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(each)
        s["pos"] = s["slot"].clone()
        s["table"] = _angles(hi, case["rot"])
        # One fused projection's rows: q, then k, then v.
        s["qkv"] = normal(n * each, (case["hq"] + 2 * hkv) * d)
        s["q_out"] = torch.zeros(n * each, case["hq"] * d, device="cuda")
        if case["acc"]:
            s["acc"] = normal(n, hkv, hi).abs()
            s["slot_pos"] = torch.zeros(n, hkv, hi, device="cuda", dtype=torch.int32)
        return s
    if op == "evict":
        length = case["len"]
        s["k"], s["v"], s["pages"] = _cache(case, [length] * n, g)
        s["lens"] = torch.full((n,), length, device="cuda", dtype=torch.int32)
        # Sums of softmax weights are positive and heavy-tailed.
        s["acc"] = torch.exp(2.0 * normal(n, hkv, length))
        seen = length + (1000 if case["mixed"] else 0)
        s["seen"] = torch.full((n,), seen, device="cuda", dtype=torch.int32)
        if case["mixed"]:
            # Slots in the order that earlier evictions left them; the newest came in last.
            pos = torch.rand(n, hkv, length - 1, generator=g, device="cuda").argsort(-1)
            pos = torch.where(pos < case["sinks"], pos, pos + 1000)
            new = torch.full((n, hkv, 1), seen - 1, device="cuda")
            s["slot_pos"] = torch.cat([pos, new], -1).to(torch.int32)
        else:
            s["slot_pos"] = torch.arange(length, device="cuda", dtype=torch.int32).expand(
                n, hkv, length).contiguous()
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["pos_out"] = torch.zeros_like(s["slot_pos"])
        s["lens_out"] = torch.zeros_like(s["lens"])
        return s
    lens = _lengths(case)
    mix = torch.randperm(n, generator=g, device="cuda").tolist()
    lens = [lens[i] for i in mix]
    s["k"], s["v"], s["pages"] = _cache(case, lens, g)
    s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    cap = s["pages"].shape[1] * case["page"]
    s["q"] = normal(n, case["hq"] * d)
    s["out"] = torch.zeros(n, case["hq"] * d, device="cuda")
    s["lse"] = torch.zeros(n, case["hq"], device="cuda")
    if case["mask"] == "padding":
        # Left padding of a share of each sequence; the last sequence is all padding.
        share = torch.rand(n, 1, generator=g, device="cuda") * 0.5
        share[-1] = 1.0
        col = torch.arange(cap, device="cuda")
        s["mask"] = torch.where(col < (share * cap).long(), -math.inf, 0.0).float().contiguous()
    elif case["mask"] == "bias":
        # A linear distance bias.
        col = torch.arange(cap, device="cuda", dtype=torch.float32)
        s["mask"] = (0.01 * (col - s["lens"][:, None])).contiguous()
    if case["acc"]:
        s["acc"] = normal(n, hkv, cap).abs()
        s["acc_out"] = torch.zeros_like(s["acc"])
    return s


# -------------------------------------------------------------------------- plain forms

def _turn(x, cs, rot, inter, back):
    """x [n][heads][d] turned by the angles cs [n][rot/2][2]."""
    c, t = cs[:, None, :, 0], cs[:, None, :, 1]
    if back:
        t = -t
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * t, a * t + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * t, a * t + b * c
    return y


def _plain_rope(s):
    c = s["case"]
    x = s["x"].view(c["n"], c["h"], c["d"])
    return _turn(x, s["table"][s["pos"].long()], c["rot"], c["inter"], c["back"]).view_as(s["x"])


def _plain_append(s):
    c = s["case"]
    hq, hkv, d, ps = c["hq"], c["hkv"], c["d"], c["page"]
    m = s["qkv"].shape[0]
    q, k, v = s["qkv"].view(m, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    cs = s["table"][s["pos"].long()]
    q, k = _turn(q, cs, c["rot"], c["inter"], False), _turn(k, cs, c["rot"], c["inter"], False)
    seq, slot = s["seq"].long(), s["slot"].long()
    page, row = s["pages"].long()[seq, slot // ps], slot % ps
    s["k"][page, :, row] = k.to(s["k"].dtype)
    s["v"][page, :, row] = v.to(s["v"].dtype)
    out = dict(q=q.reshape(m, hq * d), k=s["k"], v=s["v"])
    if c["acc"]:
        s["acc"][seq, :, slot] = 0.0
        s["slot_pos"][seq, :, slot] = s["pos"][:, None]
        out.update(acc=s["acc"], slot_pos=s["slot_pos"])
    return out


def _plain_attn(s):
    c = s["case"]
    n, hq, hkv, d, ps = c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    cap = s["pages"].shape[1] * ps
    col = torch.arange(cap, device="cuda")
    page = s["pages"].long().clamp(min=0)[:, col // ps]
    k = s["k"][page, :, col % ps].float()            # [n][cap][hkv][d]
    v = s["v"][page, :, col % ps].float()
    q = s["q"].view(n, hkv, hq // hkv, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5
    lens = s["lens"][:, None]
    live = col < lens
    if c["mask"]:
        x = x + s["mask"][:, None, None, :]
    seen = live & (col >= lens - c["window"]) if c["window"] else live
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, 0.0)
    out = dict(out=torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(n, hq * d),
               lse=(m + torch.log(l)).reshape(n, hq))
    if c["acc"]:
        out["acc"] = torch.where(live[:, None, :], s["acc"] + p.sum(2), 0.0)
    return out


def _plain_evict(s):
    c = s["case"]
    n, hkv, ps, keep = c["n"], c["hkv"], c["page"], c["keep"]
    length = s["acc"].shape[-1]
    col = torch.arange(length, device="cuda")
    pos, seen = s["slot_pos"], s["seen"][:, None, None]
    held = (pos < c["sinks"]) | (pos >= seen - c["recent"])
    key = torch.where(held, math.inf, s["acc"])
    order = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, col.expand_as(order).contiguous())
    kept = rank < keep
    new = s["lens"].clamp(max=keep)
    below = col < new[:, None, None]
    # Row by row, the i-th survivor beyond the budget goes to the i-th hole below it.
    si, hi, dst = (below & ~kept).nonzero(as_tuple=True)
    _, _, src = (kept & ~below).nonzero(as_tuple=True)
    pages = s["pages"].long()
    a, b = pages[si, src // ps], pages[si, dst // ps]
    s["k"][b, hi, dst % ps] = s["k"][a, hi, src % ps]
    s["v"][b, hi, dst % ps] = s["v"][a, hi, src % ps]
    acc, at = torch.where(below, s["acc"], 0.0), torch.where(below, pos, 0)
    acc[si, hi, dst] = s["acc"][si, hi, src]
    at[si, hi, dst] = pos[si, hi, src]
    return dict(k=s["k"], v=s["v"], acc=acc, slot_pos=at, lens=new)


# ---------------------------------------------------------------------- library's calls

def _room(wq, s, size):
    """The workspace that a program keeps beside its cache."""
    if "room" not in s:
        s["cache"] = wq.kv_cache(s["k"], s["v"])
        s["room_bytes"] = size(s["cache"])
        s["room"] = torch.empty(max(s["room_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s["cache"], s["room"], s["room_bytes"]


def _own(s):
    import gemv_transformer_gb300 as wq
    c = s["case"]
    op, n, d = c["op"], c["n"], c["d"]
    turn = (wq.WQ_ROPE_INTERLEAVED if c.get("inter") else 0)
    if op == "rope":
        turn |= wq.WQ_ROPE_TRANSPOSE if c["back"] else 0
        wq.check(wq.wq_rope(n, c["h"], d, c["rot"], turn, s["x"], c["h"] * d, s["pos"], s["table"],
                            c["rows"], s["out"], c["h"] * d))
        return s["out"]
    hkv, wide = c["hkv"], s["pages"].shape[1]
    if op == "append":
        if "cache" not in s:
            s["cache"] = wq.kv_cache(s["k"], s["v"])
        m, hq, row = n * c["each"], c["hq"], (c["hq"] + 2 * hkv) * d
        q = s["qkv"].data_ptr()
        wq.check(wq.wq_kv_append(
            s["cache"], m, hq, c["rot"], turn, q, row, q + 4 * hq * d, row,
            q + 4 * (hq + hkv) * d, row, s["pos"], s["table"], c["hi"], n, s["seq"], s["slot"],
            s["pages"], wide, s["q_out"], hq * d, s.get("acc"), s.get("slot_pos"), c["hi"]))
        out = dict(q=s["q_out"], k=s["k"], v=s["v"])
        if c["acc"]:
            out.update(acc=s["acc"], slot_pos=s["slot_pos"])
        return out
    if op == "evict":
        cache, room, size = _room(wq, s, lambda cache: wq.wq_kv_evict_workspace_bytes(
            cache, n, wide, c["keep"]))
        wq.check(wq.wq_kv_evict(
            cache, n, s["pages"], wide, s["lens"], s["seen"], c["keep"], c["sinks"], c["recent"],
            s["acc"], s["slot_pos"], s["acc_out"], s["pos_out"], c["len"], s["lens_out"], room,
            size))
        return dict(k=s["k"], v=s["v"], acc=s["acc_out"], slot_pos=s["pos_out"],
                    lens=s["lens_out"])
    hq = c["hq"]
    cache, room, size = _room(wq, s, lambda cache: wq.wq_attn_paged_workspace_bytes(
        cache, n, hq, wide, c["acc"]))
    wq.check(wq.wq_attn_paged(
        cache, n, hq, d ** -0.5, c["window"], s["q"], hq * d, s["pages"], wide, s["lens"],
        s.get("mask"), wide * c["page"], s["out"], hq * d, s["lse"], s.get("acc"),
        s.get("acc_out"), wide * c["page"], room, size))
    out = dict(out=s["out"], lse=s["lse"])
    if c["acc"]:
        out["acc"] = s["acc_out"]
    return out


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work

def work(case):
    op, n, d = case["op"], case["n"], case["d"]
    if op == "rope":
        x = n * case["h"] * d
        return dict(bytes=8 * x + 4 * n + 4 * min(n, case["rows"]) * case["rot"],
                    flops=3 * n * case["h"] * case["rot"])
    hkv, b = case["hkv"], _BYTES[case["type"]]
    if op == "append":
        m, hq = n * case["each"], case["hq"]
        return dict(bytes=4 * m * (2 * hq + 2 * hkv) * d + 2 * b * m * hkv * d + 16 * m
                    + 4 * min(m, case["hi"]) * case["rot"] + (8 * m * hkv if case["acc"] else 0),
                    flops=3 * m * (hq + hkv) * case["rot"])
    if op == "evict":
        length, keep = case["len"], case["keep"]
        over = length - keep
        if case["mixed"]:
            # The newest slot, and its even share of the other slots beyond the budget.
            moved = 1 + (over - 1) * keep / length
        else:
            # The recent ones that lie beyond the budget, and the others' even share.
            late = min(case["recent"], over)
            rest = max(1, length - case["sinks"] - case["recent"])
            moved = late + (keep - case["sinks"] - case["recent"]) * (over - late) / rest
        rows = n * hkv
        return dict(bytes=rows * (8 * length + 8 * keep + 4 * b * d * moved) + 12 * n,
                    flops=rows * length)
    hq = case["hq"]
    lens = _lengths(case)
    read = [min(x, case["window"]) if case["window"] else x for x in lens]
    size = 2 * b * d * hkv * sum(read) + 8 * n * hq * d + 4 * n * hq
    size += 4 * sum(-(-x // case["page"]) for x in read)
    size += 4 * sum(read) if case["mask"] else 0
    size += 8 * hkv * sum(lens) if case["acc"] else 0
    return dict(bytes=size, flops=4 * hq * d * sum(read))


# ------------------------------------------------------------- the definition in 64 bits

def _exact_turn(x, table, pos, rot, inter, back):
    """Pairs as complex numbers times exp(i angle)."""
    z = torch.view_as_complex(table.double())[pos.long()][:, None, :]
    z = z.conj() if back else z
    x = x.double()
    lead, tail = x[..., :rot], x[..., rot:]
    if inter:
        pair = torch.view_as_complex(lead.reshape(*lead.shape[:-1], rot // 2, 2).contiguous())
        return torch.cat([torch.view_as_real(pair * z).flatten(-2), tail], -1)
    pair = torch.complex(lead[..., :rot // 2].contiguous(), lead[..., rot // 2:].contiguous()) * z
    return torch.cat([pair.real, pair.imag, tail], -1)


def _slots(pages, page, count):
    """Pool page and row in it of the first `count` slots of one sequence."""
    whole = pages[:-(-count // page)].long().repeat_interleave(page)[:count]
    return whole, torch.arange(count, device=pages.device) - torch.arange(
        count, device=pages.device).div(page, rounding_mode="floor") * page


def exact(case, seed):
    s = prepare(case, seed)
    op, n, d = case["op"], case["n"], case["d"]
    if op == "rope":
        y = _exact_turn(s["x"].view(n, case["h"], d), s["table"], s["pos"], case["rot"],
                        case["inter"], case["back"])
        return y.reshape(n, -1)
    hkv = case["hkv"]
    if op == "append":
        hq, each = case["hq"], case["each"]
        x = s["qkv"].view(n * each, -1, d)
        turned = _exact_turn(x[:, :hq + hkv], s["table"], s["pos"], case["rot"], case["inter"],
                             False)
        k, v = s["k"].double(), s["v"].double()
        for i in range(n):
            page, row = _slots(s["pages"][i], case["page"], case["hi"])
            t = slice(i * each, (i + 1) * each)
            at = s["slot"][t].long()
            k[page[at], :, row[at]] = turned[t, hq:]
            v[page[at], :, row[at]] = x[t, hq + hkv:].double()
        out = dict(q=turned[:, :hq].reshape(n * each, -1), k=k, v=v)
        if case["acc"]:
            # Sums start at zero and positions are copied: nothing is computed.
            out.update(acc=None, slot_pos=None)
        return out
    if op == "evict":
        k, v = s["k"].double(), s["v"].double()
        acc = torch.zeros(n, hkv, case["len"], dtype=torch.float64, device="cuda")
        for i in range(n):
            page, row = _slots(s["pages"][i], case["page"], case["len"])
            size, pos = int(s["lens"][i]), s["slot_pos"][i]
            new = min(size, case["keep"])
            for h in range(hkv):
                w = s["acc"][i, h].double().clone()
                w[(pos[h] < case["sinks"]) | (pos[h] >= int(s["seen"][i]) - case["recent"])] = \
                    math.inf
                # The new-th largest bounds the survivors; of its equals the first few stay.
                bound = w.topk(new).values[-1]
                stay = w > bound
                same = (w == bound).nonzero()[:, 0]
                stay[same[:new - int(stay.sum())]] = True
                src, dst = stay[new:].nonzero()[:, 0] + new, (~stay[:new]).nonzero()[:, 0]
                k[page[dst], h, row[dst]] = k[page[src], h, row[src]]
                v[page[dst], h, row[dst]] = v[page[src], h, row[src]]
                acc[i, h, :new] = s["acc"][i, h, :new].double()
                acc[i, h, dst] = s["acc"][i, h, src].double()
        return dict(k=k, v=v, acc=acc, slot_pos=None, lens=None)
    hq = case["hq"]
    out = torch.zeros(n, hkv, hq // hkv, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hkv, hq // hkv), -math.inf, dtype=torch.float64, device="cuda")
    acc = torch.zeros(n, hkv, s["pages"].shape[1] * case["page"], dtype=torch.float64,
                      device="cuda")
    for i in range(n):
        size = int(s["lens"][i])
        if case["acc"]:
            acc[i, :, :size] = s["acc"][i, :, :size].double()
        if not size:
            continue
        page, row = _slots(s["pages"][i], case["page"], size)
        q = s["q"][i].double().view(hkv, -1, d)
        x = torch.einsum("hgd,lhd->hgl", q, s["k"][page, :, row].double()) / math.sqrt(d)
        if case["mask"]:
            x = x + s["mask"][i, :size].double()
        if case["window"]:
            x[..., :max(0, size - case["window"])] = -math.inf
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - z.clamp(min=-1e300)[..., None])
        out[i] = torch.einsum("hgl,lhd->hgd", p, s["v"][page, :, row].double())
        lse[i] = z
        if case["acc"]:
            acc[i, :, :size] += p.sum(1)
    result = dict(out=out.reshape(n, -1), lse=lse.reshape(n, -1))
    if case["acc"]:
        result["acc"] = acc
    return result
