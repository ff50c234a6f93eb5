"""The decode example, step by step against the same decoder in f64: projections, rotary
positions, appended pages, attention with weight sums, eviction.

Tolerance: weights are Q8_0 in both (exact); the device rounds k and v to bf16, and so does
the check.  Of the rest, each of the 2 layers' ~10 chained f32 operations is within 1e-5 of
its terms (the GEMV's tau), so logits within 2^-12 of their largest.  A key or value that
lies within f32's error of a rounding boundary may round the other way: one unit of 2^-8
of one of >= 20 slots' values, 2^-8 / 20 of a head's output, inside the same 2^-12 after
the sums over heads and dims that dilute it.  Sums of weights carry the same error, so an
eviction is right if no victim's f64 sum is over a survivor's by more than 2^-12 of the
largest; the check then goes on with the device's choice."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import gemv_transformer_gb300 as wq
from helpers import status_ok
from oracle import kv as okv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from gemv_transformer_gb300 import build
    build.build()
    wq.load()
    spec = importlib.util.spec_from_file_location("decode", os.path.join(ROOT, "examples",
                                                                         "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def bf16(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


class Plain:
    """The decoder in f64, its caches as lists of slots."""

    def __init__(self, run):
        self.run, self.m = run, run.model
        n, h = run.n, self.m.kv_heads
        self.slots = [[[[] for _ in range(h)] for _ in range(n)] for _ in range(self.m.layers)]
        self.seen = 0

    def ln(self, x, gb):
        k = x.shape[1]
        y = (x - x.mean(1, keepdims=True)) / np.sqrt(x.var(1, keepdims=True) + 1e-5)
        return y * gb[:k] + gb[k:]

    def step(self, tokens):
        m, run = self.m, self.run
        w = {name: v.astype(np.float64) for name, v in m.host.items()}
        d, group = m.head_dim, m.heads // m.kv_heads
        x = w["embed"][tokens]
        cs = okv.table(self.seen + 1, m.rot, 10000.0)[[self.seen] * run.n]
        for i in range(m.layers):
            y = (self.ln(x, w[f"{i}.ln1"]) @ w[f"{i}.qkv"].T).reshape(run.n, -1, d)
            q = okv.rotate(y[:, :m.heads], cs, m.rot)[0]
            k = okv.rotate(y[:, m.heads:m.heads + m.kv_heads], cs, m.rot)[0]
            v = y[:, m.heads + m.kv_heads:]
            mix = np.zeros((run.n, m.heads, d))
            for s in range(run.n):
                for h in range(m.kv_heads):
                    row = self.slots[i][s][h]
                    row.append([bf16(k[s, h]), bf16(v[s, h]), 0.0, self.seen])
                    kk, vv = np.array([r[0] for r in row]), np.array([r[1] for r in row])
                    for u in range(group):
                        z = kk @ q[s, h * group + u] / np.sqrt(d)
                        p = np.exp(z - z.max())
                        p /= p.sum()
                        mix[s, h * group + u] = p @ vv
                        for r, e in zip(row, p):
                            r[2] += e
            x = x + mix.reshape(run.n, -1) @ w[f"{i}.out"].T
            z = self.ln(x, w[f"{i}.ln2"]) @ w[f"{i}.up"].T + w[f"{i}.b1"]
            erf = torch.erf(torch.from_numpy(z / np.sqrt(2))).numpy()
            x = x + (0.5 * z * (1 + erf)) @ w[f"{i}.down"].T + w[f"{i}.b2"]
        self.seen += 1
        return self.ln(x, w["ln"]) @ w["head"].T

    def follow(self, i, s, h, kept):
        """Check the device's choice of positions, then hold what it holds."""
        run, row = self.run, self.slots[i][s][h]
        if len(row) <= run.budget + run.slack - 1:
            assert sorted(kept) == [r[3] for r in row]
            return
        assert len(set(kept)) == run.budget and set(kept) <= {r[3] for r in row}
        victims = [r for r in row if r[3] not in kept]
        assert all(run.sinks <= r[3] < self.seen - run.recent for r in victims)
        free = [r[2] for r in row
                if r[3] in kept and run.sinks <= r[3] < self.seen - run.recent]
        slip = 2.0 ** -12 * max(r[2] for r in row)
        assert max(r[2] for r in victims) <= min(free) + slip
        row[:] = [r for r in row if r[3] in kept]


@pytest.mark.parametrize("n,budget,steps", [(1, 20, 40), (3, 32, 75)])
def test_steps_against_f64(example, n, budget, steps):
    model = example.Model(dim=128, heads=4, kv_heads=2, head_dim=32, rot=16, inner=256, vocab=96,
                          seed=3)
    run = example.Decoder(model, n, budget, slack=8, sinks=1, recent=8)
    plain = Plain(run)
    g = np.random.default_rng(5)
    for t in range(steps):
        tokens = g.integers(0, 96, n)
        got = run.step(torch.from_numpy(tokens.astype(np.int32)).cuda()).cpu().numpy()
        want = plain.step(tokens)
        assert np.abs(got - want).max() <= 2.0 ** -12 * np.abs(want).max(), t
        lens = run.lens.tolist()
        for i in range(model.layers):
            pos = run.layers[i]["pos"].cpu().numpy()
            for s in range(n):
                for h in range(model.kv_heads):
                    plain.follow(i, s, h, pos[s, h, :lens[s]].tolist())
        assert lens == [len(plain.slots[0][0][0])] * n
    assert run.held <= budget + 8
    status_ok()


def test_the_command_runs(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["decode.py", "--tokens", "40", "--sequences", "2",
                                     "--budget", "24"])
    example.main()
    assert "slots held of 40 tokens seen" in capsys.readouterr().out
