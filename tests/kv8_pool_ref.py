"""The page pool of the 8-bit cache, entry by entry in plain Python. Shares no code with the library."""

PAGE = 64
CAPACITY, INDEX = 1, 32  # bits of the error word


class Pool:
    """table [b][h][p], refs [page], len [b]; tails [b][h] and summaries [b][h][p] as tokens that stand for the rows there."""

    def __init__(self, table, refs, tails=None, summaries=None):
        self.table, self.refs, self.tails, self.summaries = table, refs, tails, summaries
        self.error = 0
        self.max_pages = len(table[0][0])

    def fits(self, past, new):
        return past >= 0 and 0 <= new and past + new <= PAGE * self.max_pages + PAGE - 1

    def reserve(self, past, new):
        """-> free pages"""
        wanted = []
        for b, (a, n) in enumerate(zip(past, new)):
            if not self.fits(a, n):
                self.error |= INDEX if a < 0 else CAPACITY
                continue
            wanted += [(b, h, p) for h in range(len(self.table[b])) for p in range(a // PAGE, (a + n) // PAGE)
                       if self.table[b][h][p] < 0]
        free = [i for i, r in enumerate(self.refs) if r == 0]
        if len(wanted) > len(free):
            self.error |= CAPACITY
            return len(free)
        for (b, h, p), i in zip(wanted, free):
            self.table[b][h][p], self.refs[i] = i, 1
        return len(free) - len(wanted)

    def fork(self, length, src):
        B = len(src)
        old = [[list(r) for r in head] for head in self.table]
        tails = [[list(r) for r in head] for head in self.tails] if self.tails else None
        sums = [[list(r) for r in head] for head in self.summaries] if self.summaries else None
        was = list(length)
        for b, a in enumerate(src):
            if a == b:
                continue
            if a < -1 or a >= B or (a >= 0 and was[a] < 0):
                self.error |= INDEX
                continue
            n = was[a] if a >= 0 else 0
            if n > PAGE * self.max_pages + PAGE - 1:
                self.error |= CAPACITY
                continue
            length[b] = n
            for h in range(len(self.table[b])):
                for p in range(self.max_pages):
                    mine, new = old[b][h][p], old[a][h][p] if a >= 0 and p < n // PAGE else -1
                    if mine >= 0:
                        self.refs[mine] -= 1
                    if new >= 0:
                        self.refs[new] += 1
                    self.table[b][h][p] = new
                    if sums and a >= 0 and p < n // PAGE:
                        self.summaries[b][h][p] = sums[a][h][p]
                if tails and a >= 0:
                    for half in (0, 1):
                        self.tails[b][h][half * PAGE: half * PAGE + n % PAGE] = tails[a][h][half * PAGE: half * PAGE + n % PAGE]

    def compact(self):
        """-> free pages, and where each page that goes goes"""
        used = sum(r != 0 for r in self.refs)
        holes = [i for i in range(used) if self.refs[i] == 0]
        go = dict(zip([i for i in range(used, len(self.refs)) if self.refs[i] != 0], holes))
        in_use = [r != 0 for r in self.refs]
        for head in self.table:
            for row in head:
                for p, x in enumerate(row):
                    if x >= len(in_use) or (x >= 0 and not in_use[x]):
                        self.error |= INDEX
                    else:
                        row[p] = go.get(x, x)
        for a, z in go.items():
            self.refs[z], self.refs[a] = self.refs[a], 0
        return len(self.refs) - used, go
