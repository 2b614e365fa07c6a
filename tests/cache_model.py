"""The paged 8-bit cache in plain numpy, written from the definitions in include/tbik.h: what a page holds after
tokens were written, and the bookkeeping of the page operations."""
import numpy as np

E_MIN = -100


def bf16_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_table():
    """The value of each e4m3 byte."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e.astype(float) - 7), m * 2.0 ** -9)
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


E4M3 = e4m3_table()


def round4(x):
    """To 4 significant bits, nearest, ties to even."""
    f, e = np.frexp(x)
    return np.ldexp(np.rint(f * 16), e - 4)


def need(amax):
    """The smallest E >= E_MIN with amax <= 448 * 2^E (amax already of 4 significant bits)."""
    E = E_MIN
    if amax > 0:
        E = max(E_MIN, int(np.ceil(np.log2(amax / 448))))  # amax / 448 is 8/7 times a power of two at the nearest: no border case
        while amax > 448 * 2.0 ** E:
            E += 1
        while E > E_MIN and amax <= 448 * 2.0 ** (E - 1):
            E -= 1
    return E


def cut(y):
    """Truncation to e4m3's grid (its spacing is 2^-9 below 2^-6)."""
    return np.where(np.abs(y) < 2.0 ** -6, np.trunc(y * 512) / 512, y)


def page_values(x):
    """(stored values [tokens, D] in units of the scale, E) of one page and head whose tokens are x (float64)."""
    fin = np.where(np.isfinite(x), x, 0.0)
    r = round4(fin)
    E = need(np.abs(r).max(initial=0.0))
    y = cut(r * 2.0 ** -E)
    y = np.where(np.isinf(x), np.sign(x) * 448.0, y)
    return np.where(np.isnan(x), 0.0, y), E


def unpack(raw):
    """uint8 [..., page/8, D/16, 8, 16] -> values [..., page, D]."""
    v = E4M3[raw]
    v = np.swapaxes(v, -3, -2)
    return v.reshape(v.shape[:-4] + (v.shape[-4] * 8, v.shape[-2] * 16))


class Book:
    """table, lens and refs, with the page operations (each all or nothing)."""

    def __init__(self, slots, max_pages, num_pages, page):
        self.table = np.full((slots, max_pages), -1, np.int32)
        self.lens, self.refs, self.page = np.zeros(slots, np.int32), np.zeros(num_pages, np.int32), page

    def pages_of(self, n):
        return -(-int(n) // self.page)

    def extend(self, rows, n_new):
        S, P = self.table.shape
        refused = [-1] * len(rows)
        if len(set(rows)) < len(rows) or any(r < 0 or r >= S or n < 0 for r, n in zip(rows, n_new)):
            return refused
        want = [self.pages_of(self.lens[r] + n) - self.pages_of(self.lens[r]) for r, n in zip(rows, n_new)]
        free = list(np.flatnonzero(self.refs == 0))
        if any(self.pages_of(self.lens[r] + n) > P for r, n in zip(rows, n_new)) or sum(want) > len(free):
            return refused
        start = []
        for r, n, w in zip(rows, n_new, want):
            have = self.pages_of(self.lens[r])
            for j in range(w):
                p = free.pop(0)
                self.table[r, have + j], self.refs[p] = p, 1
            start.append(int(self.lens[r]))
            self.lens[r] += n
        return start

    def fork(self, parents, children):
        """The page copies [(from, to)], or None when refused."""
        S = self.table.shape[0]
        if any(not 0 <= x < S for x in list(parents) + list(children)) or len(set(children)) < len(children):
            return None
        if any(self.lens[c] for c in children) or set(parents) & set(children):
            return None
        free = list(np.flatnonzero(self.refs == 0))
        if sum(self.lens[p] % self.page != 0 for p in parents) > len(free):
            return None
        moves = []
        for p, c in zip(parents, children):
            n = int(self.lens[p])
            full = n // self.page
            self.table[c, :full] = self.table[p, :full]
            for j in range(full):
                self.refs[self.table[p, j]] += 1
            if n % self.page:
                new = free.pop(0)
                moves.append((int(self.table[p, full]), int(new)))
                self.table[c, full], self.refs[new] = new, 1
            self.lens[c] = n
        return moves

    def free(self, rows):
        for r in rows:
            for j in range(self.pages_of(self.lens[r])):
                self.refs[self.table[r, j]] -= 1
                self.table[r, j] = -1
            self.lens[r] = 0

    def compact(self):
        """(live pages, moves)."""
        n = int((self.refs > 0).sum())
        holes = [p for p in range(n) if self.refs[p] == 0]
        high = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(high, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for r in range(self.table.shape[0]):
            for j in range(self.pages_of(self.lens[r])):
                self.table[r, j] = to.get(int(self.table[r, j]), self.table[r, j])
        return n, list(to.items())
