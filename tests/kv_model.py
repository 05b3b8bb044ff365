"""The page bookkeeping of the key-value cache written out one slot at a time on the host: the
semantics include/kda.h gives kda_kv_reserve, _fork, _truncate, _compact and _append. Page contents
are numpy arrays of 16-bit patterns, so copies can be compared bit for bit."""
from __future__ import annotations

import numpy as np


class KvModel:
    def __init__(self, k, v, table, seq_len, ref):
        self.k, self.v = k.copy(), v.copy()  # [layers, pages, heads, page_size, D] uint16
        self.table, self.seq_len, self.ref = table.copy(), seq_len.copy(), ref.copy()
        self.page = k.shape[3]
        self.status = 0

    def _free(self):
        return [p for p in range(len(self.ref)) if self.ref[p] == 0]

    def _ok(self, s, seen):
        ok = 0 <= s < len(self.seq_len) and s not in seen
        seen.add(s)
        return ok

    def _pages(self, n):
        return -(-n // self.page)

    def _copy(self, src, dst, rows):
        for pool in (self.k, self.v):
            pool[:, dst, :, :rows] = pool[:, src, :, :rows]

    def reserve(self, slots, add):
        seen, plan, free, at, ref0 = set(), [], self._free(), 0, self.ref.copy()
        for s, a in zip(slots, add):
            good = self._ok(s, seen) and a >= 0 and self.seq_len[s] + a <= self.table.shape[1] * self.page
            if not good:
                self.status = 1
                continue
            n = int(self.seq_len[s])
            cow = a > 0 and n % self.page > 0 and ref0[self.table[s, n // self.page]] > 1
            need = self._pages(n + a) - self._pages(n) + cow
            plan.append((s, a, n, cow, need, at))
            at += need
        copies = []
        for s, a, n, cow, need, at in plan:
            if need and at + need > len(free):
                self.status = 3
                continue
            got = free[at:at + need]
            if cow:
                src = self.table[s, n // self.page]
                copies.append((src, got[0], n % self.page))
                self.ref[src] -= 1
                self.ref[got[0]] = 1
                self.table[s, n // self.page] = got[0]
                got = got[1:]
            for j, p in enumerate(got):
                self.table[s, self._pages(n) + j] = p
                self.ref[p] = 1
            self.seq_len[s] = n + a
        for c in copies:
            self._copy(*c)

    def fork(self, parent, child):
        seen, plan, free, at, len0 = set(), [], self._free(), 0, self.seq_len.copy()
        for p, c in zip(parent, child):
            if not (self._ok(c, seen) and 0 <= p < len(len0) and p != c and len0[c] == 0):
                self.status = 1
                continue
            need = int(len0[p] % self.page > 0)
            plan.append((p, c, int(len0[p]), need, at))
            at += need
        copies = []
        for p, c, n, need, at in plan:
            if need and at + need > len(free):
                self.status = 3
                continue
            full = n // self.page
            for j in range(full):
                self.table[c, j] = self.table[p, j]
                self.ref[self.table[p, j]] += 1
            if need:
                self.table[c, full] = free[at]
                self.ref[free[at]] = 1
                copies.append((self.table[p, full], free[at], n % self.page))
            self.seq_len[c] = n
        for c in copies:
            self._copy(*c)

    def truncate(self, slots, new_len):
        seen = set()
        for s, n in zip(slots, new_len):
            if not (self._ok(s, seen) and 0 <= n <= self.seq_len[s]):
                self.status = 1
                continue
            for j in range(self._pages(n), self._pages(int(self.seq_len[s]))):
                self.ref[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.seq_len[s] = n

    def compact(self):
        live = int((self.ref > 0).sum())
        dst = [p for p in range(live) if self.ref[p] == 0]
        src = [p for p in range(live, len(self.ref)) if self.ref[p] > 0]
        for a, b in zip(src, dst):
            self._copy(a, b, self.page)
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.table[self.table == a] = b
        return live

    def append(self, layer, k_new, v_new, cu, slots):
        """k_new, v_new [rows, heads, D] uint16."""
        seen = set()
        for b, s in enumerate(slots):
            c0, c1 = cu[b], cu[b + 1]
            n = c1 - c0
            if not self._ok(s, seen) or n > self.seq_len[s]:
                self.status = 1 if n else self.status
                continue
            for t in range(n):
                at = int(self.seq_len[s]) - n + t
                p = self.table[s, at // self.page]
                if p < 0 or self.ref[p] != 1:
                    self.status = 1
                    continue
                self.k[layer, p, :, at % self.page] = k_new[c0 + t]
                self.v[layer, p, :, at % self.page] = v_new[c0 + t]
