"""64-bit references of the calls on a cache in 8 bits and of its pages, from
their definitions (numpy, on the CPU)."""
import numpy as np

MOST = 448.0


def e4m3(x):
    """The nearest e4m3 values (ties to even) of |x| <= 448; infinities and NaN give NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        step = np.exp2(np.maximum(np.floor(np.log2(np.abs(x))), -6) - 3)
        y = np.rint(x / step) * step
    return np.where(np.isfinite(x), np.where(x == 0, 0.0, y), np.nan)


def need(most):
    """The least power of two s in 2^-64 .. 2^64 with most <= 448 s."""
    s = 2.0 ** -64
    while s < 2.0 ** 64 and most > MOST * s:
        s *= 2
    return s


def write(cache, scale, block, table, ctx, rows):
    """One request's tokens [count, heads, D] (64 bits) into payload values cache [pages, page, heads, D] and scale
    [pages, blocks, heads], in place, token by token of each block."""
    page = cache.shape[1]
    for b0 in range(ctx // block * block, ctx + len(rows), block):
        lo, hi = max(ctx, b0), min(ctx + len(rows), b0 + block)
        if lo >= hi:
            continue
        pg, at = table[b0 // page], b0 % page
        for h in range(cache.shape[2]):
            x = rows[lo - ctx:hi - ctx, h]
            s = need(np.abs(x[np.isfinite(x)]).max(initial=0.0))
            if lo > b0:
                was = scale[pg, at // block, h]
                s = max(was, s)
                if s > was:
                    old = cache[pg, at:at + lo - b0, h]
                    cache[pg, at:at + lo - b0, h] = e4m3(old * (was / s))
            scale[pg, at // block, h] = s
            cache[pg, at + lo - b0:at + hi - b0, h] = e4m3(x / s)


class Pool:
    """The pages of a pool, call by call.  cache: what a page holds (any object), copied by fork and compaction."""

    def __init__(self, pages, page, max_pages, rows):
        self.page, self.max_pages, self.pages = page, max_pages, pages
        self.table = [[] for _ in range(rows)]
        self.lens, self.refs = [0] * rows, [0] * pages
        self.cache = [None] * pages

    def _free(self):
        return [p for p in range(self.pages) if self.refs[p] == 0]

    def reserve(self, rows, tokens):
        done, named, short = [], set(), False
        for r, t in zip(rows, tokens):
            ok = 0 <= r < len(self.table) and r not in named and 0 <= t <= self.max_pages * self.page
            if 0 <= r < len(self.table):
                named.add(r)
            if ok:
                lack = max(0, -(-t // self.page) - len(self.table[r]))
                free = self._free()
                if lack > 0 and (short or lack > len(free)):
                    ok, short = False, True
                elif lack > 0:
                    for p in free[:lack]:
                        self.refs[p] = 1
                        self.table[r].append(p)
            done.append(int(ok))
        return done

    def fork(self, src, dst):
        n = len(self.table)
        targets = {d for d in dst if 0 <= d < n}
        done, named, plan = [], set(), []
        free = self._free()
        for a, b in zip(src, dst):
            ok = 0 <= a < n and 0 <= b < n and b not in named and a not in targets and not self.table[b]
            if 0 <= b < n:
                named.add(b)
            if ok and self.lens[a] % self.page:
                ok = bool(free)
                if ok:
                    plan.append((a, b, free.pop(0)))
            elif ok:
                plan.append((a, b, None))
            done.append(int(ok))
        for a, b, fresh in plan:
            full = self.lens[a] // self.page
            self.table[b] = self.table[a][:full]
            for p in self.table[b]:
                self.refs[p] += 1
            if fresh is not None:
                self.cache[fresh] = self.cache[self.table[a][full]]
                self.refs[fresh] = 1
                self.table[b].append(fresh)
            self.lens[b] = self.lens[a]
        return done

    def free(self, rows):
        for r in rows:
            for p in self.table[r]:
                self.refs[p] -= 1
            self.table[r], self.lens[r] = [], 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        for to, p in zip(holes, [p for p in range(live, self.pages) if self.refs[p] > 0]):
            self.cache[to], self.refs[to], self.refs[p] = self.cache[p], self.refs[p], 0
            self.table = [[to if x == p else x for x in row] for row in self.table]
        return live
