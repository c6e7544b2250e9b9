"""A plain model of the paged cache's page ownership (numpy, one page at a time).

Written from the calls' definitions in include/mk_cache.h; the GPU tests hold the
library's tables, lengths, holders and pool contents to it, bit for bit."""
import numpy as np


class Refused(Exception):
    def __init__(self, code):
        self.code = code


INVALID_ARG, PAGE_OOB, NO_PAGES = 1, 3, 12


class KvModel:
    def __init__(self, pool, tables, lens, refs, page_size):
        self.pool, self.P = pool.copy(), page_size          # [pools][pages][bytes]
        self.tables, self.lens, self.refs = tables.copy(), lens.copy(), refs.copy()
        self.cap = tables.shape[1] * page_size

    def used(self, L):
        return -(-int(L) // self.P)

    def held(self, row, j):
        p = int(self.tables[row, j])
        if not 0 <= p < len(self.refs) or self.refs[p] < 1:
            raise Refused(PAGE_OOB)
        return p

    def lowest_free(self, refs, taken, n):
        free = [p for p in range(len(refs)) if refs[p] == 0 and p not in taken]
        if len(free) < n:
            raise Refused(NO_PAGES)
        return free[:n]

    def copy_pages(self, src, dst):
        N = len(self.refs)
        if any(not 0 <= p < N for p in list(src) + list(dst)):
            raise Refused(PAGE_OOB)
        pairs = [(int(s), int(d)) for s, d in zip(src, dst) if s != d]
        targets = [d for _, d in pairs]
        if len(set(targets)) < len(targets) or set(targets) & {s for s, _ in pairs}:
            raise Refused(INVALID_ARG)
        for s, d in pairs:
            self.pool[:, d] = self.pool[:, s]

    def fork(self, src, dst):
        S = len(self.lens)
        if any(not 0 <= i < S for i in list(src) + list(dst)):
            raise Refused(INVALID_ARG)
        if len(set(map(int, dst))) < len(dst):
            raise Refused(INVALID_ARG)
        refs, pairs = self.refs.copy(), [(int(s), int(d)) for s, d in zip(src, dst) if s != d]
        rows, sources = [], []
        for s, d in pairs:
            full = int(self.lens[s]) // self.P
            row = [self.held(s, j) for j in range(self.used(self.lens[s]))]
            for p in row[:full]:
                refs[p] += 1
            for j in range(self.used(self.lens[d])):
                refs[self.held(d, j)] -= 1
            rows.append(row)
            sources += row[full:]
        fresh = self.lowest_free(refs, set(sources), len(sources))
        before = self.pool.copy()
        lens = [int(self.lens[s]) for s, _ in pairs]
        at = 0
        for (s, d), row, L in zip(pairs, rows, lens):
            if len(row) > L // self.P:
                self.pool[:, fresh[at]] = before[:, row[-1]]
                row = row[:-1] + [fresh[at]]
                refs[fresh[at]] = 1
                at += 1
            old = self.used(self.lens[d])
            self.tables[d, :max(old, len(row))] = -1
            self.tables[d, :len(row)] = row
        for (_, d), L in zip(pairs, lens):
            self.lens[d] = L
        self.refs = refs

    def resize(self, seqs, lens):
        if any(not 0 <= i < len(self.lens) for i in seqs):
            raise Refused(INVALID_ARG)
        if any(not 0 <= n <= self.cap for n in lens):
            raise Refused(PAGE_OOB)
        if len(set(map(int, seqs))) < len(seqs):
            raise Refused(INVALID_ARG)
        refs, wants = self.refs.copy(), []
        for i, n in zip(seqs, lens):
            L = int(self.lens[i])
            u0, u1 = self.used(L), self.used(n)
            for j in range(u1, u0):
                refs[self.held(i, j)] -= 1
            cow = None
            if n > L and L % self.P:
                p = self.held(i, u0 - 1)
                if self.refs[p] > 1:
                    cow = p
                    refs[p] -= 1
            wants.append((int(i), int(n), u0, u1, cow))
        need = sum((c is not None) + max(0, u1 - u0) for _, _, u0, u1, c in wants)
        fresh = self.lowest_free(refs, {c for *_, c in wants if c is not None}, need)
        before, at = self.pool.copy(), 0
        for i, n, u0, u1, cow in wants:
            if cow is not None:
                self.pool[:, fresh[at]] = before[:, cow]
                self.tables[i, u0 - 1] = fresh[at]
                at += 1
            for j in range(u0, u1):
                self.tables[i, j] = fresh[at]
                at += 1
            self.tables[i, u1:u0] = -1
            self.lens[i] = n
        for p in fresh:
            refs[p] = 1
        self.refs = refs

    def compact(self):
        N = len(self.refs)
        for i, L in enumerate(self.lens):
            for j in range(self.used(L)):
                self.held(i, j)
        live = [p for p in range(N) if self.refs[p] > 0]
        H = len(live)
        holes = [p for p in range(H) if self.refs[p] == 0]
        movers = [p for p in live if p >= H]
        page_map = np.where(self.refs > 0, np.arange(N), -1).astype(np.int32)
        for s, d in zip(movers, holes):
            self.pool[:, d] = self.pool[:, s]
            self.refs[d], self.refs[s] = self.refs[s], 0
            page_map[s] = d
        for i, L in enumerate(self.lens):
            for j in range(self.used(L)):
                self.tables[i, j] = page_map[self.tables[i, j]]
        return page_map
