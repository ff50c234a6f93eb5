"""Shared by the tests of the rotary and paged-cache calls."""
from __future__ import annotations

import numpy as np
import torch

import gemv_transformer_gb300 as wq

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Cache:
    """Two pools on the device, filled with NaN outside the live slots, and a table of
    scattered pages; `k64`, `v64` are the host's f64 copies as [page][head][row][dim]."""

    def __init__(self, g, lens, hkv, d, kind="bf16", page=16, major="head", max_pages=None,
                 scale=1.0, fill=np.nan):
        self.hkv, self.d, self.page, self.kind = hkv, d, page, kind
        need = [-(-max(0, x) // page) for x in lens]
        self.max_pages = max_pages or max(1, max(need))
        count = sum(need) + 2
        order = g.permutation(count).astype(np.int32)
        self.pages = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for s, m in enumerate(need):
            self.pages[s, :m] = order[at:at + m]
            at += m
        host = []
        for _ in range(2):
            x = np.full((count, hkv, page, d), fill, np.float32)
            for s, size in enumerate(lens):
                for j in range(max(0, size)):
                    x[self.pages[s, j // page], :, j % page] = \
                        scale * g.standard_normal((hkv, d)).astype(np.float32)
            host.append(torch.from_numpy(x).to(TYPES[kind]))
        self.pools = [self.place(x, major) for x in host]
        self.pages_dev = torch.from_numpy(self.pages).cuda()
        self.desc = wq.kv_cache(*self.pools)

    @staticmethod
    def place(x, major):
        if major == "head":
            return x.contiguous().cuda()
        if major == "token":
            return x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
        # "gap": both pools' rows padded, pages far apart
        p, h, r, d = x.shape
        room = torch.full((p, h + 1, r + 2, d + 8), float("nan"), dtype=x.dtype, device="cuda")
        room[:, :h, 1:r + 1, :d] = x.cuda()
        return room[:, :h, 1:r + 1, :d]

    def host(self):
        return [p.cpu().double().numpy() for p in self.pools]


def bits(t):
    """The tensor's bytes, for bit-exact comparisons."""
    return t.contiguous().cpu().view(torch.uint8).numpy()


def workspace(size):
    return torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device="cuda")
