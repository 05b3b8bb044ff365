"""Paged caches for the attention tests: random rows in scattered pages, everything that no query
row may see filled with NaN, and the oracle's result for every query row."""
from __future__ import annotations

import numpy as np
import torch

import kda_gated_delta_gate_b200 as kda
import oracle


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Case:
    """Slots of lengths `lens`; the last rows[i] tokens of slot i are its query rows. kinds of hidden rows: past the
    length, and before every query row's window (their pages' table entries hold `evicted` where the whole page is hidden)."""

    def __init__(self, lens, rows, heads, kv_heads, dim, page, window=0, sinks=0, layers=1, layer=0, seed=0, spread=2.0,
                 evicted=-1, order=None, device="cuda"):
        self.lens, self.rows, self.heads, self.kv_heads, self.dim = list(lens), list(rows), heads, kv_heads, dim
        self.window, self.sinks, self.layer, self.scale = window, sinks, layer, dim ** -0.5
        gen = torch.Generator().manual_seed(seed)
        max_pages = max(1, max(-(-n // page) for n in lens)) + 1
        pages = sum(-(-n // page) for n in lens) + 3
        perm = torch.randperm(pages, generator=gen).tolist()
        self.k, self.v = [], []  # per slot [len, kv_heads, dim], as the oracle reads them
        pk = torch.full((pages, kv_heads, page, dim), float("nan"), dtype=torch.bfloat16)
        pv = pk.clone()
        table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
        for s, n in enumerate(lens):
            k = torch.randn((n, kv_heads, dim), generator=gen).bfloat16()
            v = torch.randn((n, kv_heads, dim), generator=gen).bfloat16()
            self.k.append(k)
            self.v.append(v)
            first = n - rows[s] - window + 1 if window else 0  # no query row sees rows in [sinks, first)
            for j in range(-(-n // page)):
                lo, hi = j * page, min(n, (j + 1) * page)
                seen = [x for x in range(lo, hi) if x >= first or x < sinks]
                if not seen:
                    table[s, j] = evicted
                    continue
                p = perm.pop()
                table[s, j] = p
                for x in seen:
                    pk[p, :, x - lo], pv[p, :, x - lo] = k[x], v[x]
        self.total = sum(rows)
        self.q = (torch.randn((max(self.total, 1), heads, dim), generator=gen) * spread).bfloat16()
        k5 = torch.full((layers, *pk.shape), float("nan"), dtype=torch.bfloat16)
        v5 = k5.clone()
        k5[layer], v5[layer] = pk, pv
        ref = torch.zeros(pages, dtype=torch.int32)
        self.cache = kda.KVCache(k5.to(device), v5.to(device), table.to(device),
                                 torch.tensor(lens, dtype=torch.int32).to(device), ref.to(device))
        self.d = kda.dims(heads, dim, scale=self.scale)
        self.order = list(range(len(lens))) if order is None else list(order)  # the slots, as the call lists them
        self.qd = torch.cat([self.q[self._rows(s)] for s in self.order]).to(device) if self.total else self.q.to(device)
        self.cu = [0]
        for s in self.order:
            self.cu.append(self.cu[-1] + self.rows[s])

    def _rows(self, s):
        a = sum(self.rows[:s])
        return slice(a, a + self.rows[s])

    def expected(self):
        """(o, lse, spread) of the listed slots' rows in order, FP64."""
        g, out = self.heads // self.kv_heads, []
        for s in self.order:
            n, r = self.lens[s], self.rows[s]
            q = self.q[self._rows(s)].double().numpy()
            o, lse, sp = np.zeros((r, self.heads, self.dim)), np.zeros((r, self.heads)), np.zeros((r, self.heads, self.dim))
            for h in range(self.heads):
                o[:, h], lse[:, h], sp[:, h] = oracle.attention(
                    q[:, h], self.k[s][:, h // g].double().numpy(), self.v[s][:, h // g].double().numpy(),
                    np.arange(n - r, n), self.scale, self.window, self.sinks)
            out.append((o, lse, sp))
        return tuple(np.concatenate([x[i] for x in out]) for i in range(3))


def check(out, lse, expected):
    """Element by element: the BF16 output's own rounding (2^-8 of it) and the weights': each is
    rounded to BF16 before the second product (2^-8 of sum a |v|), and its FP32 score is off by at most (D + 2) 2^-24
    scale sum |q k| < 2^-13 at these inputs (sum |q k| scale < 16, D <= 128), above and below the line: 2^-12; 2^-11 with
    the exponential's and the sums' own errors. lse: the score's error and FP32 rounding of its value."""
    o, l, sp = expected
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(l))
    fin = np.isfinite(l)
    assert np.all(np.abs(gl[fin] - l[fin]) <= 2.0 ** -12 + 2.0 ** -22 * np.abs(l[fin]))
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11) * sp
    assert np.all(np.abs(got - o) <= bound), float(np.nanmax(np.abs(got - o) - bound))
