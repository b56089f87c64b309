"""Page tables on host lists: what the strata_kv_pages calls leave, one sequence after another. Test infrastructure only."""
from __future__ import annotations

import numpy as np

BAD_SLOT, NO_PAGES = 0x10, 0x20


class Pages:
    def __init__(self, n_pages, n_seq, max_pages, P):
        self.n_pages, self.n_seq, self.E, self.P = n_pages, n_seq, max_pages, P
        self.table = np.full((n_seq, max_pages), -1, dtype=np.int64)
        self.length = np.zeros(n_seq, dtype=np.int64)
        self.refs = np.zeros(n_pages, dtype=np.int64)

    def extend(self, new, T_max):
        """Returns the rows (slots, positions, q_start), the copies and the status."""
        P, status = self.P, 0
        free = iter(np.nonzero(self.refs == 0)[0])
        n_free, refs = int((self.refs == 0).sum()), self.refs.copy()
        slots, positions, q_start, copies = np.full(T_max, -1), np.zeros(T_max, dtype=np.int64), [0], []
        rows = need = 0
        for s, n in enumerate(new):
            L, n = int(self.length[s]), int(n)
            bad = n < 0 or (n > 0 and (L < 0 or L + n > self.E * P))
            last = int(self.table[s, L // P]) if L % P and not bad and n else 0
            if L % P and n and not bad:
                bad = not 0 <= last < self.n_pages or refs[last] < 1
            if bad:
                status, n = status | BAD_SLOT, 0
            moved = bool(n and L % P and refs[last] > 1)
            rows += n
            need += -(-(L + n) // P) - -(-L // P) + moved if n else 0
            if rows > T_max or need > n_free:
                status |= NO_PAGES if n else 0
                n = 0
            if n and moved:
                page = int(next(free))
                copies.append((last, page))
                self.refs[last] -= 1
                self.table[s, L // P] = page
                self.refs[page] = 1
            for e in range(-(-L // P), -(-(L + n) // P) if n else 0):
                self.table[s, e] = next(free)
                self.refs[self.table[s, e]] = 1
            pos = np.arange(L, L + n)
            at = slice(q_start[-1], q_start[-1] + n)
            positions[at], slots[at] = pos, self.table[s, pos // P] * P + pos % P
            self.length[s] += n
            q_start.append(q_start[-1] + n)
        return slots, positions, np.array(q_start), copies, status

    def fork(self, parent):
        status = 0
        for s, of in enumerate(parent):
            if of < 0:
                continue
            if of >= self.n_seq or parent[of] >= 0 or self.length[s] != 0:
                status |= BAD_SLOT
                continue
            n = -(-self.length[of] // self.P)
            self.table[s, :n] = self.table[of, :n]
            np.add.at(self.refs, self.table[s, :n][self.table[s, :n] >= 0], 1)
            self.length[s] = self.length[of]
        return status

    def release(self, keep=None, window=0, sinks=0):
        P = self.P
        for s in range(self.n_seq):
            cut = keep is not None and keep[s] >= 0
            L = min(self.length[s], keep[s]) if cut else self.length[s]
            for e in np.nonzero(self.table[s] >= 0)[0]:
                behind = cut and e * P >= L
                between = window > 0 and e * P >= sinks and (e + 1) * P - 1 <= L - window
                if behind or between:
                    self.refs[self.table[s, e]] -= 1
                    self.table[s, e] = -1
            self.length[s] = L

    def compact(self, n_pages, max_pages):
        live = np.nonzero(self.refs > 0)[0]
        to = Pages(n_pages, self.n_seq, max_pages, self.P)
        if len(live) > n_pages:
            return to, [], NO_PAGES
        number = np.full(self.n_pages + 1, -1)
        number[live] = np.arange(len(live))
        to.table[:, :self.E] = number[self.table]  # (-1: the last one)
        to.length[:] = self.length
        to.refs[:len(live)] = self.refs[live]
        return to, [(int(p), i) for i, p in enumerate(live)], 0

    def check(self):
        """Every entry is counted, and no sequence has entries behind its tokens."""
        held = self.table[self.table >= 0]
        assert np.array_equal(np.bincount(held, minlength=self.n_pages), self.refs)
        for s in range(self.n_seq):
            assert (self.table[s, -(-self.length[s] // self.P):] == -1).all()
