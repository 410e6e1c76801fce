"""Plain references of the shared-page operators, in Python integers, row by row:
the plan with holder counts, forks and compaction.  They share no code with the library."""
import copy

BAD_ROW, NO_PAGES, BAD_INDEX, BAD_LEN = 4, 8, 16, 32


class State:
    """Tables, counts and the free stack of a cache that rows may share."""

    def __init__(self, B, page, max_pages, n_pages, order=None):
        self.B, self.P, self.M, self.n = B, page, max_pages, n_pages
        self.held, self.table = [0] * B, [[-1] * max_pages for _ in range(B)]
        self.free = list(range(n_pages) if order is None else order)
        self.count, self.refs = n_pages, [0] * n_pages

    def check(self):
        """Every page is held as often as its count says, or free once."""
        seen = [0] * self.n
        for b in range(self.B):
            for c in range(self.held[b]):
                seen[self.table[b][c]] += 1
        assert seen == self.refs
        assert sorted(self.free[: self.count]) == [i for i in range(self.n) if not seen[i]]

    def plan(self, T, N, lens, add, active):
        """A cycle's plan; returns its outputs and status."""
        B, P, status = self.B, self.P, 0
        a = [max(int(x), 0) if f else 0 for x, f in zip(add, active)]
        want = []
        for b in range(B):
            w = -(-(int(lens[b]) + a[b]) // P)
            if lens[b] < 0 or w > self.M or (T > 0 and a[b] > T) or not 0 <= self.held[b] <= self.M:
                status, w, a[b] = status | BAD_LEN, self.held[b], 0
            want.append(w)
        releases = [(b, c) for b in range(B) for c in range(want[b], self.held[b])]
        last = {}
        for b, c in releases:
            page = self.table[b][c]
            if not 0 <= page < self.n or self.refs[page] <= 0:
                status |= BAD_INDEX
                continue
            self.refs[page] -= 1
            last[page] = (b, c)
        for b, c in releases:
            page = self.table[b][c]
            if last.get(page) == (b, c) and self.refs[page] == 0:
                self.free[self.count] = page
                self.count += 1
            self.table[b][c] = -1
        need_sum = token_sum = 0
        avail = self.count
        for b in range(B):
            need = max(want[b] - self.held[b], 0)
            need_sum, token_sum = need_sum + need, token_sum + a[b]
            fits = need_sum <= avail and (T > 0 or token_sum <= N)
            if not fits and (need or a[b]):
                status |= NO_PAGES
            if not fits:
                need = a[b] = 0
            for c in range(need):
                self.count -= 1
                page = self.free[self.count]
                self.table[b][self.held[b] + c] = page
                self.refs[page] = 1
            self.held[b] = min(self.held[b], want[b]) + need
        q_start, at = [], 0
        slots, positions = [-1] * N, [-1] * N
        for b in range(B):
            q_start.append(b * T if T else at)
            at += a[b]
            for k in range(a[b]):
                pos = int(lens[b]) + k
                positions[q_start[b] + k] = pos
                slots[q_start[b] + k] = self.table[b][pos // P] * P + pos % P
        q_start.append(B * T if T else at)
        return dict(q_start=q_start, q_count=a, kv_len=[max(int(x), 0) + y for x, y in zip(lens, a)], slots=slots, positions=positions), status

    def fork(self, src, dst, lens):
        """Returns copy_src, copy_dst, status."""
        before, status, out, short = copy.deepcopy(self.held), 0, [], False
        taken = set()
        for s, d, n in zip(src, dst, lens):
            want = -(-n // self.P)
            rows = 0 <= s < self.B and 0 <= d < self.B and s != d
            if n < 0 or want > self.M or (rows and before[s] < want):
                status |= BAD_LEN
                out.append((-2, -2))
            elif not rows or before[d] or (n and d in taken):
                status |= BAD_ROW
                out.append((-2, -2))
            elif n == 0:
                out.append((-1, -1))
            else:
                taken.add(d)
                whole, need = n // self.P, n % self.P > 0
                if need and (short or self.count == 0):
                    short, status = True, status | NO_PAGES
                    out.append((-2, -2))
                    continue
                for c in range(whole):
                    self.table[d][c] = self.table[s][c]
                    self.refs[self.table[s][c]] += 1
                pair = (-1, -1)
                if need:
                    self.count -= 1
                    pair = (self.table[s][whole], self.free[self.count])
                    self.table[d][whole] = pair[1]
                    self.refs[pair[1]] = 1
                self.held[d] = want
                out.append(pair)
        return [a for a, _ in out], [b for _, b in out], status

    def compact(self):
        """Returns the state afterwards, the map and the moves."""
        used = [i for i in range(self.n) if self.refs[i] > 0]
        U = len(used)
        src = [i for i in used if i >= U]
        dst = [i for i in range(U) if self.refs[i] <= 0]
        page_map = [-1] * self.n
        for i in used:
            page_map[i] = i
        for a, b in zip(src, dst):
            page_map[a] = b
        new = State(self.B, self.P, self.M, self.n)
        new.held = list(self.held)
        new.table = [[page_map[x] if c < self.held[b] else x for c, x in enumerate(r)] for b, r in enumerate(self.table)]
        new.refs = [0] * self.n
        for i in used:
            new.refs[page_map[i]] = self.refs[i]
        new.count = self.n - U
        new.free = [self.n - 1 - i if i < new.count else -1 for i in range(self.n)]
        return new, page_map, src, dst
