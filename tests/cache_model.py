"""The paged cache's calls one entry after the other, on host lists and tensors:
what each call has to leave behind, to the bit."""

import torch


class CacheModel:
    def __init__(self, cache):
        self.k, self.v = cache.k.cpu().clone(), cache.v.cpu().clone()
        self.table, self.lengths = cache.table.tolist(), cache.lengths.tolist()
        self.refs = cache.refs.tolist()
        self.P, self.M, self.S = cache.page_size, cache.max_pages, cache.slots

    def check(self, cache):
        torch.cuda.synchronize()
        assert cache.table.tolist() == self.table
        assert cache.lengths.tolist() == self.lengths
        assert cache.refs.tolist() == self.refs
        bits = lambda t: t.cpu().contiguous().view(torch.int16)  # noqa: E731  NaN compares by its bits
        assert torch.equal(bits(cache.k), bits(self.k)) and torch.equal(bits(cache.v), bits(self.v))

    def consistent(self):
        """refs are what the tables hold, every table begins with its pages."""
        held = [0] * len(self.refs)
        for row, n in zip(self.table, self.lengths):
            used = -(-n // self.P)
            assert all(p >= 0 for p in row[:used]) and all(p == -1 for p in row[used:])
            for p in row[:used]:
                held[p] += 1
        assert held == self.refs

    def extend(self, slots, tokens):
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        shared = [r > 1 for r in self.refs]
        start, asked, seen = [], 0, set()
        grants = []
        for s, t in zip(slots, tokens):
            start.append(-1)
            if not 0 <= s < self.S or s in seen:
                continue
            seen.add(s)
            n = self.lengths[s]
            have, want = -(-n // self.P), -(-(n + t) // self.P)
            if t < 0 or want > self.M:
                continue
            own = t > 0 and n % self.P != 0 and shared[self.table[s][have - 1]]
            need = want - have + own
            asked += need
            if need and asked > len(free):
                continue
            start[-1] = n
            grants.append((s, n, t, have, want, own, free[asked - need:asked] if need else []))
        for s, n, t, have, want, own, pages in grants:
            if own:
                old, new = self.table[s][have - 1], pages.pop(0)
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s][have - 1] = new
                for x in (self.k, self.v):
                    x[:, new, :, :n % self.P] = x[:, old, :, :n % self.P]
            for c in range(have, want):
                self.table[s][c] = pages.pop(0)
                self.refs[self.table[s][c]] = 1
            self.lengths[s] = n + t
        return start

    def write(self, layer, k, v, slots, start, cu=None):
        for i, (s, first) in enumerate(zip(slots, start)):
            rows = range(i, i + 1) if cu is None else range(cu[i], cu[i + 1])
            if first < 0 or not 0 <= s < self.S:
                continue
            for pos, r in enumerate(rows, first):
                if pos // self.P < self.M and self.table[s][pos // self.P] >= 0:
                    page = self.table[s][pos // self.P]
                    self.k[layer, page, :, pos % self.P] = k[r].cpu()
                    self.v[layer, page, :, pos % self.P] = v[r].cpu()

    def fork(self, src, dst):
        before = [list(row) for row in self.table], list(self.lengths)
        seen = set()
        for s, d in zip(src, dst):
            again = d in seen
            seen.add(d)
            if again or s == d or not (0 <= s < self.S and 0 <= d < self.S):
                continue
            for p in before[0][s]:
                if p >= 0:
                    self.refs[p] += 1
            for p in before[0][d]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[d], self.lengths[d] = list(before[0][s]), before[1][s]

    def free(self, slots):
        for s in slots:
            if 0 <= s < self.S:
                for p in self.table[s]:
                    if p >= 0:
                        self.refs[p] -= 1
                self.table[s], self.lengths[s] = [-1] * self.M, 0

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] <= 0]
        now = {}
        for p in range(used, len(self.refs)):
            if self.refs[p] > 0:
                to = now[p] = holes.pop(0)
                self.k[:, to], self.v[:, to] = self.k[:, p].clone(), self.v[:, p].clone()
                self.refs[to], self.refs[p] = self.refs[p], 0
        self.table = [[now.get(p, p) for p in row] for row in self.table]
        return used

    def copy_pages(self, src, dst, source=None):
        of = source or self
        pairs = []
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < len(of.refs) and 0 <= d < len(self.refs)):
                continue
            if d in dst[:i] or (source is None and d in src):
                continue
            pairs.append((s, d))
        for s, d in pairs:
            self.k[:, d], self.v[:, d] = of.k[:, s], of.v[:, s]
