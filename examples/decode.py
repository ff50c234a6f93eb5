"""Decode steps of a small random decoder over a paged, bounded key-value cache.

    python examples/decode.py [--tokens 200] [--sequences 4] [--budget 96]

One layer of a step, each line one call of the library:

    wq_gemm_ln_ws   qkv = LayerNorm(x) Wqkv^T            (Q8_0 weights)
    wq_kv_append    rotate q and k, write k and v into the sequences' pages
    wq_attn_paged   attention over the pages, the slots' weights summed
    wq_gemm         x += attention Wo^T
    wq_gemm_ln_ws   h = GELU(LayerNorm(x) W1^T + b1)
    wq_gemm         x += h W2^T + b2
    wq_kv_evict     a cache over its budget gives up the slots of least weight

The cache of a sequence never holds more than its budget and a few slots, so its pages are
allotted once, whatever the number of tokens.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_transformer_gb300 as wq  # noqa: E402


def quantise_q8_0(w: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """The Q8_0 byte image of w [m][k] (blocks of 32: f16 d, 32 int8) and its values."""
    m, k = w.shape
    blocks = w.reshape(m, k // 32, 32)
    d = (np.abs(blocks).max(-1) / 127).astype(np.float16)
    d = np.where(d == 0, np.float16(1), d)
    q = np.clip(np.rint(blocks / d.astype(np.float32)[..., None]), -127, 127).astype(np.int8)
    image = np.concatenate([d[..., None].view(np.uint8).reshape(m, k // 32, 2),
                            q.view(np.uint8)], -1)
    return image.reshape(-1), (q * d.astype(np.float32)[..., None]).reshape(m, k)


class Model:
    """Random weights of a decoder; `host` keeps their values in numpy for a check."""

    def __init__(self, layers=2, dim=256, heads=8, kv_heads=2, head_dim=64, rot=32, inner=512,
                 vocab=512, seed=0):
        self.layers, self.dim, self.heads, self.kv_heads = layers, dim, heads, kv_heads
        self.head_dim, self.rot, self.inner, self.vocab = head_dim, rot, inner, vocab
        self.qkv = (heads + 2 * kv_heads) * head_dim
        g = np.random.default_rng(seed)
        self.host, self.device = {}, {}
        for i in range(layers):
            self.matrix(g, f"{i}.qkv", self.qkv, dim)
            self.matrix(g, f"{i}.out", dim, heads * head_dim)
            self.matrix(g, f"{i}.up", inner, dim)
            self.matrix(g, f"{i}.down", dim, inner)
            for name, size in (("ln1", dim), ("ln2", dim)):
                self.vector(f"{i}.{name}", np.concatenate([1 + 0.1 * g.standard_normal(size),
                                                           0.1 * g.standard_normal(size)]))
            self.vector(f"{i}.b1", 0.1 * g.standard_normal(inner))
            self.vector(f"{i}.b2", 0.1 * g.standard_normal(dim))
        self.matrix(g, "embed", vocab, dim, 1.0)
        self.matrix(g, "head", vocab, dim)
        self.vector("ln", np.concatenate([np.ones(dim), np.zeros(dim)]))

    def matrix(self, g, name, m, k, scale=None):
        image, self.host[name] = quantise_q8_0(
            (g.standard_normal((m, k)) * (scale or k ** -0.5)).astype(np.float32))
        room = np.zeros(wq.wq_weight_bytes(wq.WQ_Q8_0, m, k), np.uint8)
        room[:image.size] = image
        self.device[name] = torch.from_numpy(room).cuda()

    def vector(self, name, x):
        self.host[name] = x.astype(np.float32)
        self.device[name] = torch.from_numpy(self.host[name]).cuda()


class Decoder:
    """Caches and buffers of `n` sequences that decode in step."""

    def __init__(self, model: Model, n: int, budget: int, slack: int = 8, sinks: int = 2,
                 recent: int = 16, page: int = 16, context: int = 4096):
        m, self.model, self.n = model, model, n
        self.budget, self.slack, self.sinks, self.recent = budget, slack, sinks, recent
        self.context = context
        # A sequence holds at most budget + slack slots before it is cut.
        self.wide = -(-(budget + slack) // page)
        self.slots = self.wide * page
        pages = torch.randperm(n * self.wide).to(torch.int32).view(n, self.wide)
        self.pages = pages.cuda()
        shape = (n * self.wide, m.kv_heads, page, m.head_dim)
        self.layers = []
        for _ in range(m.layers):
            k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.layers.append(dict(
                k=k, v=v, cache=wq.kv_cache(k, v),
                acc=torch.zeros(n, m.kv_heads, self.slots, device="cuda"),
                pos=torch.zeros(n, m.kv_heads, self.slots, dtype=torch.int32, device="cuda")))
        self.table = torch.empty(context, m.rot, device="cuda")
        wq.check(wq.wq_rope_table(context, m.rot, 10000.0, None, self.table), "wq_rope_table")
        f = dict(device="cuda")
        self.x = torch.empty(n, m.dim, **f)
        self.qkv = torch.empty(n, m.qkv, **f)
        self.q = torch.empty(n, m.heads * m.head_dim, **f)
        self.mix = torch.empty(n, m.heads * m.head_dim, **f)
        self.hidden = torch.empty(n, m.inner, **f)
        self.logits = torch.empty(n, m.vocab, **f)
        self.lens = torch.zeros(n, dtype=torch.int32, **f)   # live slots, this step's included
        self.seen = torch.zeros(n, dtype=torch.int32, **f)   # tokens so far
        self.cut_lens = torch.zeros(n, dtype=torch.int32, **f)
        cache = self.layers[0]["cache"]
        sizes = [wq.wq_attn_paged_workspace_bytes(cache, n, m.heads, self.wide, True),
                 wq.wq_kv_evict_workspace_bytes(cache, n, self.wide, budget),
                 wq.wq_gemm_ln_workspace_bytes(n, m.qkv, m.dim, wq.WQ_Q8_0, 0)]
        self.size = max(sizes)
        self.room = torch.empty(self.size, dtype=torch.uint8, device="cuda")
        self.held = 0  # live slots per sequence: all decode in step

    def ln_gemm(self, x, ln, w, out, m, flags=0, bias=None):
        k = x.shape[1]
        wq.check(wq.wq_gemm_ln_ws(self.n, m, k, wq.WQ_Q8_0, flags, x, ln, w, bias, None, out,
                                  self.room, self.size), "wq_gemm_ln_ws")

    def add_gemm(self, x, w, out, flags=0, bias=None):
        m, k = out.shape[1], x.shape[1]
        wq.check(wq.wq_gemm(self.n, m, k, wq.WQ_Q8_0, flags | wq.WQ_RESIDUAL, x, w, bias, out,
                            out), "wq_gemm")

    def step(self, tokens: torch.Tensor) -> torch.Tensor:
        """Append one token (int32 [n], on the device) to each sequence; the next logits."""
        m, n, d = self.model, self.n, self.model.head_dim
        w = m.device
        wq.check(wq.wq_embed(n, m.vocab, m.dim, wq.WQ_Q8_0, w["embed"], tokens, None, None,
                             self.x), "wq_embed")
        slot, pos = self.lens.clone(), self.seen.clone()
        self.lens += 1
        self.seen += 1
        self.held += 1
        cut = self.held > self.budget + self.slack - 1
        for i, layer in enumerate(self.layers):
            cache, acc, at = layer["cache"], layer["acc"], layer["pos"]
            self.ln_gemm(self.x, w[f"{i}.ln1"], w[f"{i}.qkv"], self.qkv, m.qkv)
            k = self.qkv[:, m.heads * d:]
            v = self.qkv[:, (m.heads + m.kv_heads) * d:]
            wq.check(wq.wq_kv_append(
                cache, n, m.heads, m.rot, 0, self.qkv, m.qkv, k, m.qkv, v, m.qkv, pos, self.table,
                self.context, n, None, slot, self.pages, self.wide, self.q, m.heads * d, acc, at,
                self.slots), "wq_kv_append")
            wq.check(wq.wq_attn_paged(
                cache, n, m.heads, d ** -0.5, 0, self.q, m.heads * d, self.pages, self.wide,
                self.lens, None, 0, self.mix, m.heads * d, None, acc, acc, self.slots, self.room,
                self.size), "wq_attn_paged")
            self.add_gemm(self.mix, w[f"{i}.out"], self.x)
            self.ln_gemm(self.x, w[f"{i}.ln2"], w[f"{i}.up"], self.hidden, m.inner,
                         wq.WQ_BIAS | wq.WQ_GELU, w[f"{i}.b1"])
            self.add_gemm(self.hidden, w[f"{i}.down"], self.x, wq.WQ_BIAS, w[f"{i}.b2"])
            if cut:
                # Every layer cuts by the lengths of this step; the new ones are for the next.
                wq.check(wq.wq_kv_evict(
                    cache, n, self.pages, self.wide, self.lens, self.seen, self.budget, self.sinks,
                    self.recent, acc, at, acc, at, self.slots, self.cut_lens, self.room,
                    self.size), "wq_kv_evict")
        if cut:
            self.lens.copy_(self.cut_lens)
            self.held = self.budget
        self.ln_gemm(self.x, w["ln"], w["head"], self.logits, m.vocab)
        return self.logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--budget", type=int, default=96)
    a = ap.parse_args()
    model = Model()
    run = Decoder(model, a.sequences, a.budget)
    tokens = torch.arange(1, a.sequences + 1, dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    out = []
    for t in range(a.tokens):
        if t == 10:
            start.record()
        tokens = run.step(tokens).argmax(-1).to(torch.int32)
        out.append(tokens)
    end.record()
    status = wq.wq_get_device_status()
    wq.check(status, "device status")
    text = torch.stack(out, 1).tolist()
    for s in range(a.sequences):
        print(f"sequence {s}: {' '.join(map(str, text[s][:16]))} ...")
    print(f"{run.held} slots held of {a.tokens} tokens seen")
    if a.tokens > 20:
        print(f"{start.elapsed_time(end) / (a.tokens - 10) * 1e3:.0f} us per step")


if __name__ == "__main__":
    main()
