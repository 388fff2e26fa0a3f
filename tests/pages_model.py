"""The pool of qsa_pages_* sequence by sequence, in whole numbers on the host
(test infrastructure)."""

from __future__ import annotations


class Model:
    """refs, table (lists), lengths and planes (CPU uint8 tensors [pages,
    segments, units, bytes]); `errors` counts what the calls count."""

    def __init__(self, refs, table, lengths, page, planes):
        self.refs, self.table, self.lengths = refs.tolist(), table.tolist(), lengths.tolist()
        self.page, self.planes, self.errors = page, planes, 0
        self.stride = len(self.table[0])
        self.capacity = self.stride * page

    def pages(self, tokens):
        return -(-tokens // self.page)

    def inside(self, p):
        return 0 <= p < len(self.refs)

    def copy_tokens(self, src, dst, used):
        for t in self.planes:
            per = self.page // t.shape[2]
            n = -(-used // per)
            t[dst, :, :n] = t[src, :, :n].clone()

    def fork(self, parents, children):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        old, tails, given, named = list(self.lengths), [], 0, set()
        copies, shared = [], []
        for a, c in zip(parents, children):
            if a < 0 or c < 0:
                tails.append(-1)
                continue
            bad = a >= len(self.table) or c >= len(self.table) or c in named or old[c] != 0
            bad = bad or not 0 <= old[a] <= self.capacity
            named.add(c)
            tail = not bad and old[a] % self.page and self.inside(self.table[a][old[a] // self.page])
            if tail:
                bad = given >= len(free)
                given += 1
            if bad:
                tails.append(-2)
                self.errors += 1
                continue
            full, used = divmod(old[a], self.page)
            row = [-1] * self.stride
            for k in range(full):
                p = self.table[a][k]
                if self.inside(p):
                    row[k] = p
                    shared.append(p)
                else:
                    self.errors += 1
            tails.append(-1)
            if tail:
                tails[-1] = row[full] = free[given - 1]
                copies.append((self.table[a][full], tails[-1], used))
            elif used:
                self.errors += 1
            self.lengths[c] = old[a]
            self.table[c] = row
        for p in shared:
            self.refs[p] += 1
        for t in tails:
            if t >= 0:
                self.refs[t] = 1
        for c in copies:
            self.copy_tokens(*c)
        return tails

    def extend(self, qsl, t2r):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        rows, given, ok = len(t2r), 0, []
        old = list(self.lengths)
        for r in range(len(self.table)):
            n, l = qsl[r + 1] - qsl[r], old[r]
            good = qsl[r] >= 0 and n >= 0 and qsl[r + 1] <= rows and l >= 0 and l + n <= self.capacity
            if good:
                need = self.pages(l + n) - self.pages(l)
                first, given = given, given + need
                good = need == 0 or given <= len(free)
                if good:
                    for k in range(need):
                        p = free[first + k]
                        self.table[r][self.pages(l) + k] = p
                        self.refs[p] = 1
                    self.lengths[r] = l + n
            if not good:
                self.errors += 1
            ok.append(good)
        pos, slots = [], []
        for i, r in enumerate(t2r):
            pos.append(-1)
            slots.append(-1)
            if 0 <= r < len(self.table) and ok[r] and qsl[r] <= i < qsl[r + 1]:
                pos[-1] = old[r] + i - qsl[r]
                p = self.table[r][pos[-1] // self.page]
                if self.inside(p):
                    slots[-1] = p * self.page + pos[-1] % self.page
                else:
                    self.errors += 1
        return pos, slots

    def free(self, requests):
        for r in requests:
            if r < 0:
                continue
            if r >= len(self.table):
                self.errors += 1
                continue
            l, self.lengths[r] = self.lengths[r], 0
            if not 0 <= l <= self.capacity:
                self.errors += 1
                continue
            for k in range(self.pages(l)):
                p, self.table[r][k] = self.table[r][k], -1
                if self.inside(p) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.errors += 1

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        used = {p for p, r in enumerate(self.refs) if r > 0}
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.copy_tokens(a, b, self.page)
            self.refs[b], self.refs[a] = self.refs[a], 0
        for r, l in enumerate(self.lengths):
            if not 0 <= l <= self.capacity:
                self.errors += 1
                continue
            for k in range(self.pages(l)):
                p = self.table[r][k]
                if p in used:
                    self.table[r][k] = to.get(p, p)
                else:
                    self.errors += 1
        return live

    def copy(self, src, dst, num_pages):
        pairs = [(s, d) for s, d in zip(src, dst)]
        before = [t.clone() for t in self.planes]
        for i, (s, d) in enumerate(pairs):
            if s < 0 or d < 0:
                continue
            bad = s >= num_pages or d >= num_pages
            for j, (sj, dj) in enumerate(pairs):
                if j != i and sj >= 0 and dj >= 0 and (sj == d or (j < i and dj == d)):
                    bad = True
            if bad:
                self.errors += 1
                continue
            for t, b in zip(self.planes, before):
                t[d] = b[s]
