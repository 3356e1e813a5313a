"""The paged KV cache by its definition: Python lists for the tables, rows moved one by one on the CPU.  Test infrastructure:
shares no code with the library."""
import torch

D = 128


class Pages:
    """k, v [layers][pages][page][h_kv][128] on the CPU.  Every call returns the status bits it sets."""

    def __init__(self, k, v, batch, max_pages):
        self.k, self.v, self.batch, self.max_pages = k, v, batch, max_pages
        self.pages, self.page = k.shape[1], k.shape[2]
        self.table, self.length = [[] for _ in range(batch)], [0] * batch

    def refs(self):
        n = [0] * self.pages
        for row in self.table:
            for p in row:
                n[p] += 1
        return n

    def _up(self, n):
        return -(-n // self.page)

    def reserve(self, new):
        refs, copies, need = self.refs(), {}, []
        for b in range(self.batch):
            if new[b] < 0 or self._up(self.length[b] + new[b]) > self.max_pages:
                return 8
        tails = {b: self.table[b][self.length[b] // self.page] for b in range(self.batch)
                 if new[b] > 0 and self.length[b] % self.page}
        for b, p in tails.items():
            holders = [x for x in tails if tails[x] == p]
            if refs[p] > 1 and (len(holders) < refs[p] or holders[0] != b):
                copies[b] = p
        for b in range(self.batch):
            add = max(0, self._up(self.length[b] + new[b]) - len(self.table[b])) if new[b] > 0 else 0
            need.append(add)
        free = [p for p in range(self.pages) if refs[p] == 0]
        if sum(need) + len(copies) > len(free):
            return 2
        free = iter(free)
        for b in range(self.batch):
            if b in copies:
                a, z, rows = copies[b], next(free), self.length[b] % self.page
                self.table[b][self.length[b] // self.page] = z
                for x in (self.k, self.v):
                    x[:, z, :rows] = x[:, a, :rows]
            for _ in range(need[b]):
                self.table[b].append(next(free))
        return 0

    def _place(self, b, t):
        """(page, row) of token t, None where there is no page or a shared one."""
        if t >= len(self.table[b]) * self.page or t < 0:
            return None
        return self.table[b][t // self.page], t % self.page

    def append(self, k, v, layers, n):
        """k, v [layers][batch][n][h_kv][128] of the listed layers."""
        refs, bits = self.refs(), 0
        for b in range(self.batch):
            m = min(max(n[b], 0), k.shape[2])
            if m != n[b]:
                bits = 8
            for i in range(m):
                at = self._place(b, self.length[b] + i)
                if at is None or refs[at[0]] != 1:
                    bits = 8
                    continue
                for x, l in enumerate(layers):
                    self.k[l, at[0], at[1]], self.v[l, at[0], at[1]] = k[x, b, i], v[x, b, i]
        return bits

    def accept(self, count, path=None):
        refs, bits = self.refs(), 0
        for b in range(self.batch):
            n, t = count[b], self.length[b]
            ok = 0 <= n and t + n <= len(self.table[b]) * self.page and (path is None or n <= len(path[b]))
            if ok:
                dst = [self._place(b, t + j) for j in range(n)]
                ok = all(refs[d[0]] == 1 for d in dst)
            if ok and path is not None:
                line = list(path[b][:n])
                src = [self._place(b, t + p) if p >= 0 else None for p in line]
                ok = all(s is not None for s in src) and all(x < y for x, y in zip(line, line[1:]))
                if ok:
                    for x in (self.k, self.v):
                        rows = [x[:, s[0], s[1]].clone() for s in src]
                        for d, row in zip(dst, rows):
                            x[:, d[0], d[1]] = row
            if ok:
                self.length[b] += n
            else:
                bits = 8
        return bits

    def select(self, src):
        table, length, bits = [list(r) for r in self.table], list(self.length), 0
        for b, s in enumerate(src):
            if s == -1:
                table[b], length[b] = [], 0
            elif not 0 <= s < self.batch:
                bits = 8
            elif s != b:
                length[b] = self.length[s]
                table[b] = self.table[s][:self._up(length[b])]
        self.table, self.length = table, length
        return bits

    def trim(self, length):
        for b, n in enumerate(length):
            if n >= 0:
                self.length[b] = min(self.length[b], n)
                self.table[b] = self.table[b][:self._up(self.length[b])]
        return 0

    def compact(self):
        refs = self.refs()
        used = [p for p in range(self.pages) if refs[p]]
        n = len(used)
        moves = dict(zip([p for p in used if p >= n], [p for p in range(n) if not refs[p]]))
        for a, z in moves.items():
            for x in (self.k, self.v):
                x[:, z] = x[:, a]
        self.table = [[moves.get(p, p) for p in row] for row in self.table]
        return 0

    def arrays(self):
        """length, held, table, refs, n_free as the library keeps them."""
        refs = self.refs()
        table = [row + [-1] * (self.max_pages - len(row)) for row in self.table]
        i32 = torch.int32
        return (torch.tensor(self.length, dtype=i32), torch.tensor([len(r) for r in self.table], dtype=i32),
                torch.tensor(table, dtype=i32).view(self.batch, self.max_pages), torch.tensor(refs, dtype=i32),
                sum(x == 0 for x in refs))
