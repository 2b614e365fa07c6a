"""The paged 8-bit cache on the device: writes and page operations bit for bit against tests/cache_model.py,
attention against binary64, its bitwise independence of the batch and the split, and the refusals."""
import numpy as np
import pytest

from tests import cache_model as cm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import invariant_tree_ordered_b200 as tbik  # noqa: E402

DEV = "cuda"
NAN_BYTE = 0x7F


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def cu_of(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


def raw(pages):
    return pages.view(torch.uint8)


class Cache:
    """Device state and its numpy model side by side."""

    def __init__(self, slots, max_pages, num_pages, H, D, page, layers=1, fill=NAN_BYTE):
        self.pages, self.scales, self.refs = tbik.cache_pages(num_pages, H, D, page, layers)
        raw(self.pages).fill_(fill)  # what no token has reached is garbage
        self.table, self.lens = tbik.cache_table(slots, max_pages)
        self.book = cm.Book(slots, max_pages, num_pages, page)
        self.page, self.H, self.D = page, H, D

    def check(self):
        for a, b in ((self.table, self.book.table), (self.lens, self.book.lens), (self.refs, self.book.refs)):
            assert np.array_equal(a.cpu().numpy(), b)

    def extend(self, rows, n):
        start = tbik.cache_extend(self.table, self.lens, self.refs, i32(n), page=self.page, rows=i32(rows))
        ref = self.book.extend(rows, n)
        assert start.tolist() == ref
        self.check()
        return start

    def append(self, k, v, start, n, rows, layer=0, packed=True):
        tbik.cache_append(k, v, self.pages[layer], self.scales[layer], self.table, self.refs, start,
                          cu=cu_of(n) if packed else None, rows=i32(rows))

    def attend(self, q, start, n, rows, layer=0, packed=True, **kw):
        return tbik.cache_attention(q, self.pages[layer], self.scales[layer], self.table, start,
                                    cu=cu_of(n) if packed else None, rows=i32(rows), **kw)

    def stored(self, row, n, layer=0):
        """float64 [2, H, n, D]: what the device holds of a sequence's first n positions."""
        ids = self.book.table[row, :self.book.pages_of(n)]
        v = cm.unpack(raw(self.pages)[layer][:, ids].cpu().numpy())          # [2, pages, H, page, D]
        v = v * self.scales[layer][:, ids].double().cpu().numpy()[..., None, None]
        return np.swapaxes(v, 1, 2).reshape(2, self.H, -1, self.D)[:, :, :n]


def tokens(seed, n, H, D, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, H, D, device=DEV, generator=g)
    if spread:  # magnitudes over many binades, zeros and tiny values among them
        x = x * torch.exp2(torch.randint(-24, 6, (n, H, 1), device=DEV, generator=g).float())
        x = x * torch.exp2(torch.randint(-12, 1, (n, H, D), device=DEV, generator=g).float())
        x = x * (torch.rand(n, H, 1, device=DEV, generator=g) > 0.1)
    return x.to(torch.bfloat16)


def model_pages(x, page):
    """[(values [tokens, D] in units, E)] per page and head of one sequence's tokens x float64 [n, H, D]."""
    return [[cm.page_values(x[a:a + page, h]) for h in range(x.shape[1])] for a in range(0, x.shape[0], page)]


def check_written(c, row, k, v, layer=0):
    n = k.shape[0]
    ids = c.book.table[row, :c.book.pages_of(n)]
    for kv, x in ((0, k), (1, v)):
        x = x.double().cpu().numpy()
        got = cm.unpack(raw(c.pages)[layer][kv, ids].cpu().numpy())
        byt = raw(c.pages)[layer][kv, ids].cpu().numpy().swapaxes(-3, -2).reshape(len(ids), c.H, c.page, c.D)
        sc = c.scales[layer][kv, ids].cpu().numpy()
        for i, per_head in enumerate(model_pages(x, c.page)):
            for h, (val, E) in enumerate(per_head):
                assert sc[i, h] == np.float32(2.0 ** E), (i, h)
                assert np.array_equal(got[i, h, :len(val)], val), (i, h)
                assert (byt[i, h, len(val):] == NAN_BYTE).all()  # not reached by any token: untouched


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
def test_append_matches_the_definition_for_every_split(page, D, H):
    lens = [1, page - 1, page, page + 1, 3 * page + 5]
    parts = {r: (tokens(10 * page + r, n, H, D), tokens(10 * page + r + 5, n, H, D)) for r, n in enumerate(lens)}
    states = []
    for cuts in ("whole", "single", "odd"):
        c = Cache(len(lens), 5, 24, H, D, page)
        at = [0] * len(lens)
        step = 0
        while any(a < n for a, n in zip(at, lens)):
            take = [n - a if cuts == "whole" else min(n - a, 1 if cuts == "single" else 1 + (7 * step + 3 * r) % (page + 9))
                    for r, (a, n) in enumerate(zip(at, lens))]
            rows = [r for r in reversed(range(len(lens))) if take[r]]
            n = [take[r] for r in rows]
            start = c.extend(rows, n)
            k = torch.cat([parts[r][0][at[r]:at[r] + take[r]] for r in rows])
            v = torch.cat([parts[r][1][at[r]:at[r] + take[r]] for r in rows])
            c.append(k, v, start, n, rows, packed=cuts != "single")
            at = [a + t for a, t in zip(at, take)]
            step += 1
        assert tbik.get_error() == tbik.TBIK_OK
        for r in range(len(lens)):
            check_written(c, r, *parts[r])
        states.append(c)


def test_append_takes_values_that_are_not_finite():
    c = Cache(1, 2, 3, 2, 64, 16)
    k, v = tokens(1, 3, 2, 64, False), tokens(2, 3, 2, 64, False)
    k[0, 0, 3], k[1, 1, 5], v[2, 0, 0], v[2, 1, 7] = float("inf"), float("-inf"), float("nan"), float("inf")
    c.append(k, v, c.extend([0], [3]), [3], [0])
    assert tbik.get_error() == tbik.TBIK_ERR_VALUE
    check_written(c, 0, k, v)
    k2 = torch.full_like(k[:1], float("inf"))  # nothing finite: the smallest scale
    c2 = Cache(1, 2, 3, 2, 64, 16)
    c2.append(k2, v[:1], c2.extend([0], [1]), [1], [0])
    check_written(c2, 0, k2, v[:1])
    assert tbik.get_error() == tbik.TBIK_ERR_VALUE
    big = torch.full((1, 2, 64), float(torch.finfo(torch.bfloat16).max), device=DEV).to(torch.bfloat16)
    c3 = Cache(1, 2, 3, 2, 64, 16)
    c3.append(big, -big, c3.extend([0], [1]), [1], [0])
    check_written(c3, 0, big, -big)
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("packed", [True, False])
def test_append_refuses_pages_it_must_not_write(packed):
    H, D, page = 2, 64, 16
    c = Cache(4, 2, 8, H, D, page)
    start = c.extend([0, 1, 2, 3], [1, 1, 1, 1])
    before, sc = raw(c.pages).clone(), c.scales.clone()
    k, v = tokens(1, 4, H, D), tokens(2, 4, H, D)

    def attempt(rows, start, code):
        c.append(k[:len(rows)], v[:len(rows)], start, [1] * len(rows), rows, packed=packed)
        assert tbik.get_error() == code
        same = torch.equal(raw(c.pages), before) and torch.equal(c.scales, sc)
        return same

    assert attempt([0], i32([-1]), tbik.TBIK_OK)                 # not granted: nothing to do
    assert attempt([4], i32([0]), tbik.TBIK_ERR_PAGE)            # no such slot
    assert attempt([-1], i32([0]), tbik.TBIK_ERR_PAGE)
    assert attempt([0], i32([2 * page]), tbik.TBIK_ERR_PAGE)     # behind the table's row
    assert attempt([0], i32([page]), tbik.TBIK_ERR_PAGE)         # a page that the sequence does not have
    assert attempt([1, 1], i32([0, 0]), tbik.TBIK_ERR_PAGE)      # the same slot twice
    c.refs[c.table[2, 0].long()] = 2
    assert attempt([2], i32([0]), tbik.TBIK_ERR_PAGE)            # a shared page
    c.table[3, 0] = 8
    assert attempt([3], i32([0]), tbik.TBIK_ERR_PAGE)            # outside the pool
    assert not attempt([0], start[:1].contiguous(), tbik.TBIK_OK)


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128)])
def test_rejected_drafts_are_written_over(page, D):
    """Drafts are written, some rejected and other tokens written over them from there, at places inside a page and at its
    first position, with sizes over many binades: the new tokens are held, and a scale that a rejected one raised stays
    until the page begins anew.  lens is lowered, and pages behind it given up, as the header says."""
    H, r = 2, np.random.RandomState(page)
    c = Cache(1, 8, 8, H, D, page)
    vals = np.full((2, 8 * page, H, D), np.nan)  # in units of the page's scale; nan: not reached
    E = np.zeros((2, 8, H), int)
    n = 0
    for step in range(30):
        m = int(r.choice([1, 3, 5, page - 1, page + 2]))
        if n + m > 8 * page:
            break
        start = c.extend([0], [m])
        x = [tokens(2 * step + kv, m, H, D) for kv in (0, 1)]
        c.append(*x, start, [m], [0])
        for kv in (0, 1):
            xs = x[kv].double().cpu().numpy()
            for pg in range(n // page, (n + m - 1) // page + 1):
                o0, o1 = max(n - pg * page, 0), min(n + m - pg * page, page)
                for h in range(H):
                    new = cm.round4(xs[pg * page + o0 - n:pg * page + o1 - n, h])
                    e = cm.need(np.abs(new).max())
                    v = vals[kv, pg * page:(pg + 1) * page, h]
                    if o0:
                        e = max(e, E[kv, pg, h])
                        v[:o0] = cm.cut(v[:o0] * 2.0 ** (E[kv, pg, h] - e))
                    v[o0:o1] = cm.cut(new * 2.0 ** -e)
                    E[kv, pg, h] = e
        n += m
        held = c.book.table[0, :c.book.pages_of(n)]
        got = cm.unpack(raw(c.pages)[0][:, held].cpu().numpy())  # [2, pages, H, page, D]
        sc = c.scales[0][:, held].cpu().numpy()
        assert np.array_equal(sc, np.exp2(E[:, :len(held)]).astype(np.float32))
        got = got.transpose(0, 1, 3, 2, 4).reshape(2, -1, H, D)[:, :n]
        assert np.array_equal(got, vals[:, :n])
        # some of the step's tokens are rejected
        n -= int(r.randint(0, m + 1))
        keep = c.book.pages_of(n)
        for j in range(keep, 8):
            if c.book.table[0, j] >= 0:
                c.book.refs[c.book.table[0, j]] -= 1
                c.book.table[0, j] = -1
        c.book.lens[0] = n
        c.table.copy_(torch.from_numpy(c.book.table).to(DEV))
        c.refs.copy_(torch.from_numpy(c.book.refs).to(DEV))
        c.lens.fill_(n)
    assert step > 8 and tbik.get_error() == tbik.TBIK_OK


def test_append_passes_over_offsets_that_cannot_be():
    H, D, page = 2, 64, 16
    for cu in ([0, 5, 10], [0, 5, 4], [-1, 5, 9]):  # beyond the tokens, descending, before the first
        c = Cache(2, 2, 6, H, D, page)
        start = c.extend([0, 1], [5, 4])
        k, v = tokens(1, 9, H, D), tokens(2, 9, H, D)
        untouched = raw(c.pages).clone()
        tbik.cache_append(k, v, c.pages[0], c.scales[0], c.table, c.refs, start, cu=i32(cu))
        assert tbik.get_error() == tbik.TBIK_ERR_POSITION
        good, a, b = (0, 0, 5) if cu[0] == 0 else (1, 5, 9)
        check_written(c, good, k[a:b], v[a:b])
        assert torch.equal(raw(c.pages)[0][:, int(c.table[1 - good, 0])], untouched[0][:, int(c.table[1 - good, 0])])


@pytest.mark.parametrize("batch,slots,lens", [(300, 65536, 1), (8192, 8192, 1), (8192, 9000, 40), (129, 140, 200), (1000, 1000, 7)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_append_of_many_sequences_in_any_slots(batch, slots, lens, D, page):
    """What a call with `rows` and `cu` writes, against the same tokens written without them into slots 0, 1, ...; slots
    named twice, wherever in the call, are not written."""
    if batch * lens * D > 2 ** 25:
        lens = 10
    H = 1
    r = np.random.RandomState(batch + lens)
    n = np.maximum(0, r.randint(0, lens + 1, batch)) if lens > 1 else np.ones(batch, int)
    at = r.randint(0, 2 * page, batch)
    most = 3 + lens // page
    pool = int(sum(-(-int(a + m) // page) for a, m in zip(at, n))) + 5
    pages, scales, refs = tbik.cache_pages(pool, H, D, page)
    table, lensd = tbik.cache_table(slots, most)
    tbik.cache_extend(table, lensd, refs, i32(at + n), page=page, rows=i32(range(batch)))
    g = torch.Generator(device=DEV).manual_seed(1)
    raw(pages).copy_(torch.randint(0, 127, pages.shape, dtype=torch.uint8, device=DEV, generator=g))
    scales.copy_(torch.exp2(torch.randint(-9, 3, scales.shape, device=DEV, generator=g).float()))
    k, v = tokens(1, int(n.sum()), H, D), tokens(2, int(n.sum()), H, D)
    start = i32(at)
    assert tbik.get_error() == tbik.TBIK_OK

    def wrote(table, rows, packed):
        pg, sc = pages.clone(), scales.clone()
        tbik.cache_append(k, v, pg[0], sc[0], table, refs, start, cu=cu_of(n) if packed else None, rows=None if rows is None else i32(rows))
        return raw(pg), sc

    for packed in ([True, False] if lens == 1 else [True]):
        ref = wrote(table, None, packed)
        assert tbik.get_error() == tbik.TBIK_OK
        assert not torch.equal(ref[0], raw(pages))
        rows = r.permutation(slots)[:batch]
        moved = torch.full_like(table, -1)
        moved[torch.from_numpy(rows).to(DEV)] = table[:batch]
        got = wrote(moved, rows, packed)
        assert tbik.get_error() == tbik.TBIK_OK
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        # the first, the last and a few others name the slot of another sequence; both of a pair stay unwritten
        twice = rows.copy()
        pairs = [(0, batch - 1), (batch // 2, batch // 2 + 1), (17, batch - 30)]
        for a, b in pairs:
            twice[b] = twice[a]
        got = wrote(moved, twice, packed)
        assert tbik.get_error() == tbik.TBIK_ERR_PAGE
        want = [x.clone() for x in ref]
        for b in [x for p in pairs for x in p]:
            ids = table[b][table[b] >= 0].long()
            want[0][0][:, ids] = raw(pages)[0][:, ids]
            want[1][0][:, ids] = scales[0][:, ids]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("with_rows", [True, False])
def test_the_time_of_a_write_grows_with_the_call(packed, with_rows):
    """8 times the sequences take about 8 times as long, not 8 times 8 (a search over the whole call in every block): less
    than twice that, in a captured graph."""
    H, D, page = 8, 128, 16
    times = []
    for B in (1024, 8192):
        pages, scales, refs = tbik.cache_pages(B, H, D, page)
        table, lens = tbik.cache_table(B, 2)
        start = tbik.cache_extend(table, lens, refs, i32([1] * B), page=page)
        k = torch.randn(B, H, D, device=DEV).to(torch.bfloat16)
        kw = dict(cu=cu_of([1] * B) if packed else None, rows=i32(range(B)) if with_rows else None)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                for _ in range(10):
                    tbik.cache_append(k, k, pages[0], scales[0], table, refs, start, **kw)
        torch.cuda.current_stream().wait_stream(side)
        best = 1e9
        for _ in range(5):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            ev[0].record()
            g.replay()
            ev[1].record()
            torch.cuda.synchronize()
            best = min(best, ev[0].elapsed_time(ev[1]))
        times.append(best)
    assert tbik.get_error() == tbik.TBIK_OK
    assert times[1] < 16 * times[0], times


# ---------------------------------------------------------------- attention

def filled(ctx, H, D, page, seed, slots=None, spare=3):
    """A cache whose sequences hold ctx tokens each, written in one call, rows in a mixed order."""
    rows = list(np.random.RandomState(seed).permutation(slots or len(ctx))[:len(ctx)])
    rows = [int(r) for r in rows]
    used = sum(-(-n // page) for n in ctx)
    c = Cache(slots or len(ctx), max(-(-n // page) for n in ctx) + 1, used + spare, H, D, page)
    # the pool's pages in a mixed order: one page each in turn
    left = list(ctx)
    while any(left):
        live = [i for i in range(len(ctx)) if left[i]]
        n = [min(left[i], page) for i in live]
        c.extend([rows[i] for i in live], n)
        for i, m in zip(live, n):
            left[i] -= m
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = (torch.randn(sum(ctx), H, D, device=DEV, generator=g) * (1 + 3 * (torch.rand(H, D, device=DEV, generator=g) < .05))).to(torch.bfloat16)
    v = torch.randn(sum(ctx), H, D, device=DEV, generator=g).to(torch.bfloat16)
    c.append(k, v, i32([0] * len(ctx)), ctx, rows)
    assert tbik.get_error() == tbik.TBIK_OK
    return c, rows


def reference(c, q, rows, start, n):
    """float64 attention over what the device holds, and the largest |v| that each query could see."""
    q = q.double().cpu().numpy()
    T, NH, D = q.shape
    G = NH // c.H
    out, top, at = np.zeros(q.shape), np.zeros((T, NH)), 0
    for r, s, m in zip(rows, start, n):
        if m == 0:
            continue
        kv = c.stored(r, s + m)
        for h in range(NH):
            k, v = kv[0, h // G], kv[1, h // G]
            a = q[at:at + m, h] @ k.T / np.sqrt(D)
            a[np.arange(s + m)[None] > s + np.arange(m)[:, None]] = -np.inf
            a = np.exp(a - a.max(1, keepdims=True))
            out[at:at + m, h] = (a @ v) / a.sum(1, keepdims=True)
            top[at:at + m, h] = np.abs(v).max()
        at += m
    return out, top


def bound(ref, top):
    """The weights are rounded to about 8 significant bits (2^-8 each, in the weights and in their sum: 2^-7 of the
    largest value) with a floor of 2^-18 of the leaf's largest weight (128 keys of it: 2^-11), the scores are off by
    less than 2^-13 (fp32 sums and hardware exponential at |s| < 100), and the output is rounded once (2^-8)."""
    return (2.0 ** -7 + 2.0 ** -11 + 2.0 ** -12) * top[..., None] + 2.0 ** -8 * np.abs(ref)


CASES = [
    # H, heads, D, page, contexts before the call, new tokens
    (1, 1, 128, 16, [0], [1]),
    (1, 1, 64, 16, [0, 1, 126, 127, 128], [1, 1, 1, 1, 1]),
    (2, 8, 128, 64, [0, 15, 63, 64, 127, 128, 129, 1000], [1] * 8),
    (2, 10, 64, 32, [300, 5, 2000], [1, 1, 1]),
    (3, 3, 128, 128, [255, 256, 4100], [1, 1, 1]),
    (2, 8, 128, 16, [0, 100, 120, 500], [5, 1, 30, 0]),
    (1, 16, 128, 32, [10, 0], [3, 140]),
    (2, 2, 64, 64, [0, 700, 1], [300, 17, 129]),
    (1, 64, 128, 64, [130], [2]),
    (2, 12, 64, 128, [1, 3000, 250], [9, 8, 10]),
    (4, 32, 128, 64, [900, 77], [64, 200]),
]


@pytest.mark.parametrize("H,heads,D,page,before,n", CASES)
def test_attention_matches_binary64(H, heads, D, page, before, n):
    c, rows = filled([b + m for b, m in zip(before, n)], H, D, page, seed=len(before) + page + D, slots=len(before) + 2)
    T = sum(n)
    g = torch.Generator(device=DEV).manual_seed(5)
    q = (torch.randn(T + 2, heads, D, device=DEV, generator=g) * 2).to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    # two rows behind the last sequence stay as they are
    got = tbik.cache_attention(q, c.pages[0], c.scales[0], c.table, i32(before), cu=cu_of(n), rows=i32(rows), out=out,
                               max_q=max(n), max_keys=max(b + m for b, m in zip(before, n)))
    assert tbik.get_error() == tbik.TBIK_OK
    assert (got[T:] == 7.0).all()
    ref, top = reference(c, q[:T], rows, before, n)
    err = np.abs(got[:T].double().cpu().numpy() - ref)
    assert (err <= bound(ref, top)).all(), float((err / bound(ref, top)).max())
    if all(m == 1 for m in n):  # the form without cu, bounds left to their defaults, in place
        one = q[:T].clone()
        tbik.cache_attention(one, c.pages[0], c.scales[0], c.table, i32(before), rows=i32(rows), out=one)
        assert torch.equal(one, got[:T])


def weighted_reference(c, q, rows, start, n):
    """float64 attention, the sums of |weight x value|, the square sums of them, and what the weights' floor can take: 2^-18 of
    the leaf's largest weight for each of its keys, in units of the largest value that the leaf's pages can hold."""
    q = q.double().cpu().numpy()
    T, NH, D = q.shape
    G = NH // c.H
    out, av, sq, floor, at = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, NH)), 0
    for r, s, m in zip(rows, start, n):
        if m == 0:
            continue
        kv = c.stored(r, s + m)
        ids = c.book.table[r, :c.book.pages_of(s + m)]
        vs = 448 * c.scales[0][1, ids].double().cpu().numpy()
        for h in range(NH):
            k, v = kv[0, h // G], kv[1, h // G]
            a = q[at:at + m, h] @ k.T / np.sqrt(D)
            a[np.arange(s + m)[None] > s + np.arange(m)[:, None]] = -np.inf
            a = np.exp(a - a.max(1, keepdims=True))
            a /= a.sum(1, keepdims=True)
            out[at:at + m, h], av[at:at + m, h], sq[at:at + m, h] = a @ v, a @ np.abs(v), (a * a) @ (v * v)
            big = np.repeat(vs[:, h // G], c.page)[:s + m]
            for l in range(0, s + m, 128):
                floor[at:at + m, h] += 2.0 ** -18 * a[:, l:l + 128].max(1) * big[l:l + 128].max() * min(128, s + m - l)
        at += m
    return out, av, sq, floor


@pytest.mark.parametrize("H,heads,D,page,before,n", [
    (2, 8, 128, 64, [4100, 15, 1000], [1, 1, 1]), (1, 16, 128, 32, [10, 2000], [3, 140]), (2, 2, 64, 16, [0, 9000], [300, 2]),
    (4, 16, 64, 128, [20000], [5]), (2, 16, 128, 16, [700, 127, 128], [1, 2, 1])])
def test_attention_is_as_close_as_its_weights(H, heads, D, page, before, n):
    """Each output within the bound of its own weights, and all of them together as close as roundings that do not know of
    one another.

    A weight p is two e4m3 terms: off by 2^-9 p at most, or by the floor.  Scores are off by less than 2^-13 (fp32 sums and the
    hardware's exponential at |s| < 100), which moves a weight and the sum of the weights by 2^-13 each, and with them the
    output by 2^-12 sum(p |v|); fp32 sums of values add less than 2^-14 of it.  The output is rounded to bf16: 2^-8.
    The errors of the roundings are spread evenly, a third of their largest square each: over n outputs the mean square is
    sum((2^-9 p v)^2) / 3 + (2^-8 out)^2 / 3, whose estimate strays by less than a quarter for the 768 and more outputs here."""
    c, rows = filled([b + m for b, m in zip(before, n)], H, D, page, seed=page + D, slots=len(before) + 1)
    g = torch.Generator(device=DEV).manual_seed(3)
    q = (torch.randn(sum(n), heads, D, device=DEV, generator=g) * 2).to(torch.bfloat16)
    got = c.attend(q, i32(before), n, rows).double().cpu().numpy()
    assert tbik.get_error() == tbik.TBIK_OK
    ref, av, sq, floor = weighted_reference(c, q, rows, before, n)
    err = np.abs(got - ref)
    lim = (2.0 ** -9 + 2.0 ** -12 + 2.0 ** -14) * av + floor[..., None] + 2.0 ** -8 * np.abs(ref)
    assert (err <= lim).all(), float((err / lim).max())
    rms, want = (err ** 2).mean(), (sq * 2.0 ** -18 / 3 + ref ** 2 * 2.0 ** -16 / 3).mean()
    assert rms <= 1.25 * want, rms / want


def test_queries_that_are_not_finite():
    """A row whose query holds an infinity or a NaN anywhere is NaN; every other row keeps its bits, in tiles of every
    size, in cut and uncut trees."""
    H, D, page = 2, 64, 16
    for heads, before, n in ((8, [5, 3000, 90], [1, 1, 1]), (8, [5, 2000], [3, 40]), (32, [700], [1])):
        c, rows = filled([b + m for b, m in zip(before, n)], H, D, page, seed=7)
        q = torch.randn(sum(n), heads, D, device=DEV).to(torch.bfloat16)
        good = c.attend(q, i32(before), n, rows)
        bad = torch.zeros(sum(n), heads, dtype=torch.bool, device=DEV)
        x = q.clone()
        for i, value in enumerate((float("nan"), float("inf"), float("-inf"), float("nan"))):
            t, h, d = (5 * i) % sum(n), (3 * i + 1) % heads, (17 * i) % D
            x[t, h, d] = value
            bad[t, h] = True
        got = c.attend(x, i32(before), n, rows)
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], good[~bad])
        assert tbik.get_error() == tbik.TBIK_OK


def test_attention_bits_do_not_depend_on_batch_split_or_pages():
    H, heads, D = 2, 8, 128
    before, n = [0, 60, 127, 500, 2600, 1023, 9000], [1, 80, 2, 33, 40, 1, 5]
    outs = []
    g = torch.Generator(device=DEV).manual_seed(11)
    q = torch.randn(sum(n), heads, D, device=DEV, generator=g).to(torch.bfloat16)
    for page in (16, 64):
        # equal contents need equal scales: one scale for all pages
        c, rows = filled([b + m for b, m in zip(before, n)], H, D, page, seed=3)
        gen = torch.Generator().manual_seed(1)
        vals = torch.randn(2, H, max(b + m for b, m in zip(before, n)) + 128, D, generator=gen).mul(60).clamp(-448, 448)
        byts = vals.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
        for r, b, m in zip(rows, before, n):
            for j in range(-(-(b + m) // page)):
                x = byts[:, :, j * page:(j + 1) * page].reshape(2, H, page // 8, 8, D // 16, 16).transpose(3, 4)
                raw(c.pages)[0][:, int(c.book.table[r, j])] = x
        c.scales.fill_(2.0 ** -6)
        whole = c.attend(q, i32(before), n, rows)
        outs.append(whole)
        # one query at a time, one sequence at a time
        at = 0
        for r, b, m in zip(rows, before, n):
            part = q[at:at + m].contiguous()
            assert torch.equal(c.attend(part, i32([b]), [m], [r]), whole[at:at + m])
            pick = sorted({0, m // 2, m - 1})
            single = c.attend(part[pick].contiguous(), i32([b + t for t in pick]), [1] * len(pick), [r] * len(pick), packed=False)
            assert torch.equal(single, whole[at:at + m][pick])
            at += m
        # a large batch of the same sequence: another split of the work
        many = 40
        qq = q[-1:].repeat(many, 1, 1).contiguous()
        res = c.attend(qq, i32([before[-1] + n[-1] - 1] * many), [1] * many, [rows[-1]] * many, packed=False)
        assert torch.equal(res, whole[-1:].expand_as(res))
        # heads by themselves: the same bits for any split of the heads
        for h in range(H):
            one = tbik.cache_attention(q[:, h * 4:h * 4 + 4].contiguous(), c.pages[0][:, :, h:h + 1].contiguous(),
                                       c.scales[0][:, :, h:h + 1].contiguous(), c.table, i32(before), cu=cu_of(n), rows=i32(rows))
            assert torch.equal(one, whole[:, h * 4:h * 4 + 4])
    assert torch.equal(outs[0], outs[1])
    assert tbik.get_error() == tbik.TBIK_OK


def test_attention_with_page_scales_far_apart():
    """Neighbouring pages whose scales differ by many binades, and keys so large that one weight takes all."""
    H, D, page = 1, 128, 16
    c = Cache(1, 20, 24, H, D, page)
    n = 300
    start = c.extend([0], [n])
    g = torch.Generator(device=DEV).manual_seed(2)
    size = torch.exp2(torch.randint(-14, 4, (n // page + 1,), device=DEV, generator=g).float()).repeat_interleave(page)[:n, None, None]
    k = (torch.randn(n, H, D, device=DEV, generator=g) * size).to(torch.bfloat16)
    v = (torch.randn(n, H, D, device=DEV, generator=g) * size.flip(0)).to(torch.bfloat16)
    c.append(k, v, start, [n], [0])
    q = (torch.randn(3, 4, D, device=DEV, generator=g)).to(torch.bfloat16)
    q[1] *= 2.0 ** -20
    got = c.attend(q, i32([n - 3]), [3], [0]).double().cpu().numpy()
    ref, top = reference(c, q, [0], [n - 3], [3])
    # |s| reaches a few thousand here: an fp32 score is off by up to 2^-22 |s| < 2^-9, and so is its weight
    assert (np.abs(got - ref) <= bound(ref, top) + 2.0 ** -8 * top[..., None]).all()


def test_attention_refuses_or_marks_what_cannot_be():
    H, D, page = 2, 64, 32
    c, rows = filled([40, 200, 70], H, D, page, seed=1)
    q = torch.randn(3, 4, D, device=DEV).to(torch.bfloat16)
    good = c.attend(q, i32([39, 199, 69]), [1, 1, 1], rows, packed=False)

    def bad(start, rws, code, which, **kw):
        got = c.attend(q, i32(start), [1, 1, 1], rws, packed=False, **kw)
        assert tbik.get_error() == code
        nan = torch.isnan(got).all(-1).all(-1).tolist()
        assert nan == [b in which for b in range(3)]
        for b in range(3):
            assert b in which or torch.equal(got[b], good[b])

    bad([39, -1, 69], rows, tbik.TBIK_OK, {1})                                  # not granted
    bad([39, 199, 69], [rows[0], 3, -1], tbik.TBIK_ERR_PAGE, {1, 2})            # no such slots
    bad([39, 199, 69], rows, tbik.TBIK_ERR_PAGE, {1}, max_keys=199)             # beyond the bound
    bad([39, c.table.shape[1] * page, 69], rows, tbik.TBIK_ERR_PAGE, {1})       # beyond the table
    saved = c.table.clone()
    c.table[rows[1], 2] = c.refs.numel()                                        # a page outside the pool
    bad([39, 199, 69], rows, tbik.TBIK_ERR_PAGE, {1})
    c.table[rows[1], 2] = -1
    bad([39, 199, 69], rows, tbik.TBIK_ERR_PAGE, {1})
    c.table.copy_(saved)
    with pytest.raises(ValueError):
        c.attend(q[:2].contiguous(), i32([39, 199, 69]), [1, 1, 1], rows, packed=False)
    with pytest.raises(ValueError):
        c.attend(q[:, :, :32].contiguous(), i32([39, 199, 69]), [1, 1, 1], rows, packed=False)
    with pytest.raises(ValueError):
        c.attend(q[:, ::2], i32([39, 199, 69]), [1, 1, 1], rows, packed=False)
    with pytest.raises(tbik.TbikError):
        c.attend(torch.zeros(3, 3, D, dtype=torch.bfloat16, device=DEV), i32([39, 199, 69]), [1, 1, 1], rows, packed=False)
    with pytest.raises(tbik.TbikError):  # a workspace that is too small
        need = tbik.cache_attention_workspace(3, 3, 1, 224, 4, H, D, page)
        if need == 0:
            raise tbik.TbikError(tbik.TBIK_ERR_WORKSPACE, "none needed")
        c.attend(q, i32([39, 199, 69]), [1, 1, 1], rows, packed=False, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert c.attend(q[:0].contiguous(), i32([]), [], [], packed=False).shape == (0, 4, D)


def test_attention_on_other_streams_and_in_graphs():
    """Two captured graphs that share a workspace, replayed in turn, a call on a side stream, and the eager call give
    the same bits."""
    H, heads, D, page = 2, 8, 128, 16
    c, rows = filled([3000, 40, 700], H, D, page, seed=9)
    q = [torch.randn(3, heads, D, device=DEV).to(torch.bfloat16) for _ in range(2)]
    start = i32([2999, 39, 699])
    args = (c.pages[0], c.scales[0], c.table, start)
    kw = dict(rows=i32(rows), max_keys=3000)
    need = tbik.cache_attention_workspace(3, 3, 1, 3000, heads, H, D, page)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    eager = [tbik.cache_attention(x, *args, **kw) for x in q]
    outs = [torch.zeros_like(x) for x in q]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        res = tbik.cache_attention(q[0], *args, **kw)
        for x, o in zip(q, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                tbik.cache_attention(x, *args, out=o, workspace=ws, **kw)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    ws.fill_(255)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, eager[0]) and all(torch.equal(a, b) for a, b in zip(outs, eager))
    assert tbik.get_error() == tbik.TBIK_OK


# ---------------------------------------------------------- page operations

def stamp(c):
    """Every page's bytes name it."""
    L, _, N = c.pages.shape[:3]
    g = torch.Generator(device=DEV).manual_seed(4)
    raw(c.pages).copy_(torch.randint(0, 127, c.pages.shape, dtype=torch.uint8, device=DEV, generator=g))
    c.scales.copy_(torch.exp2(torch.randint(-9, 9, c.scales.shape, device=DEV, generator=g).float()))
    return raw(c.pages).clone(), c.scales.clone()


def check_moves(c, before, moves):
    ref, sc = before
    for a, b in moves:
        ref[:, :, b], sc[:, :, b] = ref[:, :, a].clone(), sc[:, :, a].clone()
    assert torch.equal(raw(c.pages), ref) and torch.equal(c.scales, sc)


@pytest.mark.parametrize("seed,slots,max_pages,num_pages,page,H,D,layers", [
    (0, 6, 5, 17, 16, 1, 64, 1), (1, 40, 9, 203, 32, 3, 128, 2), (2, 5, 3, 7, 128, 2, 64, 3),
    (3, 300, 4, 4500, 16, 1, 64, 1)])
def test_random_life_of_pages(seed, slots, max_pages, num_pages, page, H, D, layers):
    r = np.random.RandomState(seed)
    c = Cache(slots, max_pages, num_pages, H, D, page, layers)
    refused = 0
    for step in range(40):
        before = stamp(c)
        op = r.choice(["extend", "extend", "fork", "free", "compact"])
        moves = []
        if op == "extend":
            rows = r.permutation(slots)[:r.randint(1, min(slots, 40) + 1)].tolist()
            n = r.randint(0, 2 * page, len(rows)).tolist()
            refused += c.extend(rows, n)[0].item() == -1
        elif op == "fork":
            empty = np.flatnonzero(c.book.lens == 0)
            children = r.permutation(empty)[:r.randint(0, 6)].tolist()
            parents = r.choice([x for x in range(slots) if x not in children], len(children)).tolist()
            tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(parents), i32(children))
            moves = c.book.fork(parents, children)
            refused += moves is None
            moves = moves or []
        elif op == "free":
            rows = r.randint(0, slots, r.randint(0, 5)).tolist()  # a slot may come twice
            tbik.cache_free(c.table, c.lens, c.refs, i32(rows), page=page)
            c.book.free(rows)
        else:
            live = tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs)
            n, moves = c.book.compact()
            assert live.item() == n
        c.check()
        check_moves(c, before, moves)
        tbik.get_error()
    assert refused or seed in (1, 3)


def test_page_operations_refuse_without_a_trace():
    c = Cache(4, 3, 6, 2, 64, 16)
    c.extend([0, 1], [20, 16])
    before = stamp(c)

    def refused(f):
        f()
        assert tbik.get_error() == tbik.TBIK_ERR_PAGE
        c.check()
        check_moves(c, before, [])

    ext = lambda rows, n: (lambda: c.extend(rows, n))  # noqa: E731
    fork = lambda p, ch: (lambda: tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(p), i32(ch)))  # noqa: E731
    copy = lambda a, b: (lambda: tbik.cache_copy(c.pages, c.scales, i32(a), i32(b)))  # noqa: E731
    for f in (ext([0, 4], [1, 1]), ext([-1], [1]), ext([2, 2], [1, 1]), ext([2], [-1]), ext([2], [49]),
              ext([0, 1, 2], [28, 32, 1]),  # one page more than there are
              fork([0], [1]), fork([0, 0], [2, 2]), fork([4], [2]), fork([0], [4]), fork([2], [2]), fork([0, 2], [2, 3]),
              copy([0], [6]), copy([-1], [1]), copy([0, 1], [2, 2]), copy([0, 1], [1, 3])):
        refused(f)
    refused(lambda: tbik.cache_free(c.table, c.lens, c.refs, i32([9]), page=16))
    tbik.cache_copy(c.pages, c.scales, i32([0, 0, 1]), i32([5, 3, 4]))
    check_moves(c, before, [(0, 5), (0, 3), (1, 4)])
    c.extend([0, 1, 2], [28, 16, 0])  # exactly what is left
    assert tbik.get_error() == tbik.TBIK_OK
    for f in (lambda: tbik.cache_extend(c.table, c.lens, c.refs, i32([1, 1]), page=16, rows=i32([0])),
              lambda: tbik.cache_extend(c.table, c.lens, c.refs[:5].float(), i32([1]), page=16),
              lambda: tbik.cache_fork(c.pages[0], c.scales[0], c.table, c.lens, c.refs, i32([0]), i32([3])),
              lambda: tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs[:4].clone())):
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: tbik.cache_extend(c.table, c.lens, c.refs, i32([1]), page=24),
              lambda: tbik.cache_copy(c.pages, c.scales, i32([0]), i32([1]), workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
              lambda: tbik.cache_extend(c.table, c.lens, c.refs, i32([1] * 5), page=16)):
        with pytest.raises(tbik.TbikError):
            f()


def test_free_with_one_slot_out_of_range_changes_nothing():
    c = Cache(300, 3, 900, 1, 64, 16)
    assert c.extend(range(300), [17 + i % 30 for i in range(300)])[0] == 0
    for rows in ([0, 300], [300, 0], [5, 7, -1, 9], list(range(299)) + [300], [2 ** 31 - 1] + list(range(299))):
        tbik.cache_free(c.table, c.lens, c.refs, i32(rows), page=16)
        assert tbik.get_error() == tbik.TBIK_ERR_PAGE
        c.check()
    rows = [4, 5, 4, 5] + list(range(100, 300))  # slots named twice
    tbik.cache_free(c.table, c.lens, c.refs, i32(rows), page=16)
    c.book.free(rows)
    c.check()
    assert tbik.get_error() == tbik.TBIK_OK


def test_free_of_more_sequences_than_blocks():
    """8192 sequences of one or two pages, some slots empty: the grid takes several of them a block."""
    slots = 8192
    c = Cache(slots, 2, 2 * slots, 1, 64, 16, fill=0)
    n = [(7 * i) % 33 for i in range(slots)]
    start = tbik.cache_extend(c.table, c.lens, c.refs, i32(n), page=16)
    assert c.book.extend(list(range(slots)), n) == start.tolist() == [0] * slots
    c.check()
    rows = np.random.RandomState(0).permutation(slots)[:8000].tolist() + [3] * 100
    tbik.cache_free(c.table, c.lens, c.refs, i32(rows), page=16)
    c.book.free(rows)
    c.check()
    tbik.cache_free(c.table, c.lens, c.refs, i32([0] * slots), page=16)  # mostly nothing, no slot twice in effect
    c.book.free([0])
    c.check()
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("copies", [1, 50, 300])
def test_fork_of_a_row_that_names_no_page_changes_nothing(copies):
    """A bad entry anywhere among a parent's pages: outside the pool, none, or a free page."""
    page, parents = 16, 6
    c = Cache(parents + copies, 40, 700, 1, 64, page, layers=2)
    c.extend(range(parents), [16 * (3 + i) + i for i in range(parents)])
    before = stamp(c)
    par = [i % parents for i in range(copies)][::-1]
    children = list(range(parents, parents + copies))
    saved = c.table.clone()
    victim = par[-1]
    last = c.book.pages_of(c.book.lens[victim]) - 1
    for j in (0, 1, last):
        for value in (-1, 700, 2 ** 31 - 1, 699):  # 699 is free
            c.table[victim, j] = value
            c.book.table[victim, j] = value
            tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(par), i32(children))
            assert tbik.get_error() == tbik.TBIK_ERR_PAGE
            c.check()
            check_moves(c, before, [])
            c.table.copy_(saved)
            c.book.table[:] = saved.cpu().numpy()
    tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(par), i32(children))
    moves = c.book.fork(par, children)
    c.check()
    check_moves(c, before, moves)
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("slots", [5, 40, 700, 20000])
def test_compaction_of_a_table_that_names_no_page_changes_nothing(slots):
    """A row with a page outside the pool, none, or a free one, or a length that cannot be."""
    page, num = 16, 900
    c = Cache(slots, 9, num, 1, 64, page, layers=2)
    r = np.random.RandomState(slots)
    rows = r.permutation(slots)[:min(slots, 200)].tolist()
    c.extend(rows, r.randint(1, 5 * page if slots < 700 else page * 4, len(rows)).tolist())
    gone = rows[::3]
    tbik.cache_free(c.table, c.lens, c.refs, i32(gone), page=page)
    c.book.free(gone)
    live = [x for x in rows if x not in gone]
    before = stamp(c)
    free = int(np.flatnonzero(c.book.refs == 0)[0])  # below the front
    table, lens = c.table.clone(), c.lens.clone()

    def refused():
        c.book.table, c.book.lens = c.table.cpu().numpy(), c.lens.cpu().numpy()
        assert tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs).item() == -1
        assert tbik.get_error() == tbik.TBIK_ERR_PAGE
        c.check()
        check_moves(c, before, [])
        c.table.copy_(table)
        c.lens.copy_(lens)

    for x in (live[0], live[-1], max(live)):
        last = -(-int(lens[x]) // page) - 1
        for j, value in ((last, -1), (0, num), (last, 2 ** 31 - 1), (0, free), (last, num - 1), (0, -7)):
            c.table[x, j] = value
            refused()
        for value in (-1, 9 * page + 1, 2 ** 31 - 1):
            c.lens[x] = value
            refused()
    c.book.table, c.book.lens = table.cpu().numpy(), lens.cpu().numpy()
    n, moves = c.book.compact()
    assert tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs).item() == n
    c.check()
    check_moves(c, before, moves)
    assert tbik.get_error() == tbik.TBIK_OK


def test_a_large_pool():
    """Page numbers over many scan steps, and page bytes behind 2^32."""
    H, D, page, num = 8, 128, 128, 20000  # 5.2 GB
    c = Cache(3, 19990, num, H, D, page)
    c.extend([0], [19980 * page])
    start = c.extend([1], [page + 3])
    k, v = tokens(1, page + 3, H, D), tokens(2, page + 3, H, D)
    c.append(k, v, start, [page + 3], [1])
    check_written(c, 1, k, v)
    q = torch.randn(1, H, D, device=DEV).to(torch.bfloat16)
    got = c.attend(q, i32([page + 2]), [1], [1], packed=False, max_keys=page + 3).double().cpu().numpy()
    ref, top = reference(c, q, [1], [page + 2], [1])
    assert (np.abs(got - ref) <= bound(ref, top)).all()
    tbik.cache_free(c.table, c.lens, c.refs, i32([0]), page=page)
    c.book.free([0])
    live = tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs)
    assert c.book.compact()[0] == live.item() == 2
    c.check()
    check_written(c, 1, k, v)
    assert torch.equal(c.attend(q, i32([page + 2]), [1], [1], packed=False, max_keys=page + 3).double().cpu(), torch.from_numpy(got))
    assert tbik.get_error() == tbik.TBIK_OK


# ------------------------------------------------- calls at their edges

def test_nan_bytes_that_a_row_does_not_see():
    """Bytes behind a row's position (written by nobody, or NaN under a later query of the same tile) leave it alone."""
    H, D, page = 2, 64, 16
    c, rows = filled([300], H, D, page, seed=4)
    q = torch.randn(6, 8, D, device=DEV).to(torch.bfloat16)
    good = c.attend(q, i32([294]), [6], rows)
    at = 298  # the last two queries see it, the first four do not
    pg, o = int(c.book.table[rows[0], at // page]), at % page
    raw(c.pages)[0][:, pg, :, o // 8, :, o % 8] = NAN_BYTE
    raw(c.pages)[0][:, pg, :, (o + 2) // 8:, :, (o + 2) % 8:] = NAN_BYTE
    got = c.attend(q, i32([294]), [6], rows)
    assert torch.equal(got[:4], good[:4])
    assert tbik.get_error() == tbik.TBIK_OK


def test_attention_bounds_that_are_too_tight_and_offsets_that_cannot_be():
    H, D, page = 2, 128, 32
    c, rows = filled([300, 200], H, D, page, seed=7)
    q = torch.randn(9, 4, D, device=DEV).to(torch.bfloat16)
    good = c.attend(q, i32([295, 196]), [5, 4], rows)
    got = c.attend(q, i32([295, 196]), [5, 4], rows, max_q=4)      # one query more than announced
    assert tbik.get_error() == tbik.TBIK_ERR_PAGE
    assert torch.isnan(got[4]).all() and torch.equal(got[:4], good[:4]) and torch.equal(got[5:], good[5:])
    got = c.attend(q, i32([295, 196]), [5, 4], rows, max_keys=298)  # the last two queries see more keys
    assert tbik.get_error() == tbik.TBIK_ERR_PAGE
    assert torch.isnan(got[3:5]).all() and torch.equal(got[:3], good[:3]) and torch.equal(got[5:], good[5:])
    for cu in ([0, 5, 10], [0, 5, 4], [-1, 5, 9]):  # beyond the tokens, descending, before the first
        out = torch.full_like(q, 3.0)
        tbik.cache_attention(q, c.pages[0], c.scales[0], c.table, i32([295, 196]), cu=i32(cu), rows=i32(rows), out=out, max_q=5, max_keys=300)
        assert tbik.get_error() == tbik.TBIK_ERR_POSITION
        which = slice(0, 5) if cu[0] == 0 else slice(5, 9)  # the sequence whose range is sound
        rest = slice(5, 9) if cu[0] == 0 else slice(0, 5)
        assert torch.equal(out[which], good[which]) and (out[rest] == 3.0).all()


@pytest.mark.parametrize("cu", [[0, 9, 0, 9], [0, 6, 3, 9, 5, 9], [0, 9, 8, 9] + [0, 9] * 300])
def test_offsets_whose_ranges_overlap(cu):
    """More tokens than there are: nothing is computed."""
    H, D, page = 2, 64, 32
    c, rows = filled([400], H, D, page, seed=7)
    q = torch.randn(9, 4, D, device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    n = len(cu) - 1
    for kw in (dict(max_q=9, max_keys=400), {}):
        tbik.cache_attention(q, c.pages[0], c.scales[0], c.table, i32([300] * n), cu=i32(cu), rows=i32(rows * n), out=out, **kw)
        assert tbik.get_error() == tbik.TBIK_ERR_POSITION and (out == 3.0).all()
    # empty ranges at any place, and ranges that leave tokens out, are sound
    got = tbik.cache_attention(q, c.pages[0], c.scales[0], c.table, i32([390, 100, 391, 392]), cu=i32([0, 0, 5, 5, 8]), rows=i32(rows * 4))
    assert tbik.get_error() == tbik.TBIK_OK and (got[8] == 0).all() and not (got[:8] == 0).all(-1).any()


def captured_time(f, calls=5):
    """Device time of `calls` calls in a captured graph, the best of five replays."""
    f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(calls):
                f()
    torch.cuda.current_stream().wait_stream(side)
    best = 1e9
    for _ in range(5):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        g.replay()
        ev[1].record()
        torch.cuda.synchronize()
        best = min(best, ev[0].elapsed_time(ev[1]))
    return best


@pytest.mark.parametrize("batch,n,ctx", [(1024, 8, 100), (3000, 5, 60), (3, 700, 900), (1, 5000, 300), (191, 3, 500), (193, 130, 140)])
def test_bounds_left_at_their_defaults(batch, n, ctx):
    """max_q = all tokens: the same bits, in about the same time (the output's fill and a larger workspace come on top)."""
    H, heads, D, page = 1, 2, 64, 64
    r = np.random.RandomState(batch)
    new = r.randint(0, n + 1, batch)
    new[-1] = n
    before = r.randint(0, ctx + 1, batch)
    c, rows = filled((before + new).tolist(), H, D, page, seed=batch) if batch < 1000 else (None, None)
    if c is None:  # one page run for all
        c = Cache(batch, -(-(ctx + n) // page), 40, H, D, page)
        raw(c.pages).copy_(torch.randint(0, 120, c.pages.shape, dtype=torch.uint8, device=DEV))
        c.table.copy_(torch.from_numpy(r.randint(0, 40, c.table.shape)).to(DEV))
        rows = list(range(batch))
    T = int(new.sum())
    q = torch.randn(T, heads, D, device=DEV).to(torch.bfloat16)
    args = (q, c.pages[0], c.scales[0], c.table, i32(before))
    kw = dict(cu=cu_of(new), rows=i32(rows))
    tight = dict(max_q=int(new.max()), max_keys=int((before + new).max()))
    want = tbik.cache_attention(*args, **kw, **tight)
    assert torch.equal(tbik.cache_attention(*args, **kw), want) and not torch.isnan(want).any()
    assert tbik.get_error() == tbik.TBIK_OK
    out = torch.empty_like(q)
    times = [captured_time(lambda: tbik.cache_attention(*args, out=out, **kw, **b)) for b in (tight, {})]
    assert times[1] < 1.5 * times[0] + 0.05, times  # ms for five calls


def test_default_bounds_take_the_tiles_of_short_sequences():
    """24 sequences with a few drafted tokens each: with max_q = all tokens in the time of the tight bound."""
    H, D, page, batch = 16, 64, 32, 24
    new = [1 + i % 5 for i in range(batch)]
    before = [300 + 150 * i for i in range(batch)]
    c, rows = filled([a + b for a, b in zip(before, new)], H, D, page, seed=1)
    q = torch.randn(sum(new), H, D, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    args, kw = (q, c.pages[0], c.scales[0], c.table, i32(before)), dict(cu=cu_of(new), rows=i32(rows), max_keys=4096)
    want = tbik.cache_attention(*args, max_q=5, **kw)
    assert torch.equal(tbik.cache_attention(*args, **kw), want)
    times = [captured_time(lambda: tbik.cache_attention(*args, out=out, **b, **kw)) for b in (dict(max_q=5), {})]
    assert times[1] < 1.25 * times[0], times


def test_workspace_of_a_loose_bound():
    """64 sequences over a table of 131072 positions: 8 heads x 64 tiles of 1024 leaves in nodes of 32 to 64 make up to 2 x 16
    of them, of 8 rows and 128 dims in fp32 (67 MB) and a little more."""
    nodes = 8 * 64 * 32
    need = tbik.cache_attention_workspace(64, 64, 1, 131072, 32, 8, 128, 64)
    assert nodes * 8 * 128 * 4 <= need <= 1.03 * nodes * 8 * 128 * 4
    # a call that makes the most of it: every sequence a little above 64 or 128 leaves, so that nodes are small
    for batch, ctx in ((300, 64 * 128 + 1), (200, 128 * 128 + 1)):
        H, heads, D, page = 1, 8, 64, 128
        c = Cache(batch, -(-(ctx + 1) // page), 50, H, D, page)
        raw(c.pages).copy_(torch.randint(0, 120, c.pages.shape, dtype=torch.uint8, device=DEV))
        c.scales.fill_(2.0 ** -7)
        c.table.copy_(torch.from_numpy(np.random.RandomState(1).randint(0, 50, c.table.shape)).to(DEV))
        q = torch.randn(batch, heads, D, device=DEV).to(torch.bfloat16)
        got = tbik.cache_attention(q, c.pages[0], c.scales[0], c.table, i32([ctx] * batch), max_keys=ctx + 1)
        for b in (0, batch // 2, batch - 1):
            one = tbik.cache_attention(q[b:b + 1].contiguous(), c.pages[0], c.scales[0], c.table, i32([ctx]), rows=i32([b]), max_keys=ctx + 1)
            assert torch.equal(one[0], got[b])
        assert tbik.get_error() == tbik.TBIK_OK and torch.isfinite(got).all()


def test_the_same_slot_for_many_sequences_and_two_streams_at_once():
    """Reading needs no slot of its own: 300 queries over one sequence, in two calls that run side by side."""
    H, heads, D, page = 1, 4, 128, 64
    c, rows = filled([5000], H, D, page, seed=3)
    q = torch.randn(300, heads, D, device=DEV).to(torch.bfloat16)
    start = i32(np.arange(300) * 16 + 5)
    args = (c.pages[0], c.scales[0], c.table, start)
    ref = tbik.cache_attention(q, *args, rows=i32(rows * 300), max_keys=5000)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [tbik.cache_attention(q, *args, rows=i32(rows * 300), max_keys=5000, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("heads,H,ctx,n", [(8, 2, [3000, 700], [1, 1]), (16, 2, [1500, 130], [40, 3])])
def test_withheld_arrive_times_out_and_context_survives(heads, H, ctx, n):
    """The softmax warps are told to withhold their "weights written" arrive: the MMA issuer's bounded wait expires,
    every role leaves, and the next call gives the same bits as before."""
    c, rows = filled(ctx, H, 128, 64, seed=2)
    q = torch.randn(sum(n), heads, 128, device=DEV).to(torch.bfloat16)
    start = i32([a - b for a, b in zip(ctx, n)])
    good = c.attend(q, start, n, rows)
    assert tbik.get_error() == tbik.TBIK_OK
    try:
        tbik.debug_set(tbik.DEBUG_WITHHOLD_ACC_ARRIVE, 50_000_000)  # 50 ms per wait
        c.attend(q, start, n, rows)
        status = tbik.get_error()
    finally:
        tbik.debug_set(0, 0)
    assert status == tbik.TBIK_ERR_TIMEOUT
    assert torch.equal(c.attend(q, start, n, rows), good)
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("num_pages,H", [(201, 1), (67, 3)])
def test_a_layer_of_a_pool_with_an_odd_number_of_scales(num_pages, H):
    """One layer's scales then start 8 bytes behind a 16-byte boundary."""
    D, page, layers = 64, 16, 3
    c = Cache(2, 6, num_pages, H, D, page, layers)
    assert c.scales[1].data_ptr() % 16 == 8
    n = [40, 90]
    start = c.extend([0, 1], n)
    q = torch.randn(2, 4 * H, D, device=DEV).to(torch.bfloat16)
    for layer in range(layers):
        k, v = tokens(layer, 130, H, D), tokens(layer + 9, 130, H, D)
        c.append(k, v, start, n, [0, 1], layer=layer)
        check_written(c, 0, k[:40], v[:40], layer)
        check_written(c, 1, k[40:], v[40:], layer)
        alone = tbik.cache_attention(q, c.pages[layer].clone(), c.scales[layer].clone(), c.table, i32([39, 89]), rows=i32([0, 1]))
        assert torch.equal(c.attend(q, i32([39, 89]), [1, 1], [0, 1], layer=layer, packed=False), alone)
    assert tbik.get_error() == tbik.TBIK_OK


def test_pools_and_tables_of_the_largest_size():
    """2^20 pages, 65536 slots, 8192 sequences a call (the model's loops as array operations)."""
    num, slots, page, B = 1 << 20, 65536, 16, 8192
    c = Cache(slots, 140, num, 1, 64, page, fill=0)
    book, r = c.book, np.random.RandomState(0)
    order = r.permutation(slots)
    rows, more, children = order[:B], order[B:2 * B], order[2 * B:2 * B + 500]
    pages_of = lambda n: -(-n // page)  # noqa: E731

    def extend(rows, n):
        start = tbik.cache_extend(c.table, c.lens, c.refs, i32(n), page=page, rows=i32(rows))
        have = pages_of(book.lens[rows])
        want = pages_of(book.lens[rows] + n) - have
        free = np.flatnonzero(book.refs == 0)
        if want.sum() > len(free):
            assert (start == -1).all() and tbik.get_error() == tbik.TBIK_ERR_PAGE
        else:
            assert np.array_equal(start.cpu().numpy(), book.lens[rows])
            who = np.repeat(np.arange(len(rows)), want)
            ids = free[:len(who)]
            book.table[rows[who], have[who] + np.arange(len(who)) - (np.cumsum(want) - want)[who]] = ids
            book.refs[ids] = 1
            book.lens[rows] += n
        c.check()
        return want.sum() <= len(free)

    n = r.randint(0, 127 * page, B)
    assert extend(rows, n)
    raw(c.pages).copy_(torch.randint(0, 127, c.pages.shape, dtype=torch.uint8, device=DEV))
    assert not extend(more, np.full(B, 130 * page))  # more pages than are left
    assert extend(more, n[::-1].copy())
    before, sc = raw(c.pages).clone(), c.scales.clone()
    parents = rows[:500]
    tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(parents), i32(children))
    moves = book.fork(parents.tolist(), children.tolist())
    c.check()
    a, b = (torch.tensor(x, device=DEV) for x in zip(*moves))
    before[:, :, b] = before[:, :, a]
    sc[:, :, b] = sc[:, :, a]
    assert torch.equal(raw(c.pages), before) and torch.equal(c.scales, sc)
    tbik.cache_free(c.table, c.lens, c.refs, i32(rows), page=page)
    np.subtract.at(book.refs, book.table[rows][book.table[rows] >= 0], 1)
    book.table[rows], book.lens[rows] = -1, 0
    c.check()
    live = tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs)
    n_live = int((book.refs > 0).sum())
    assert live.item() == n_live
    hole, high = np.flatnonzero(book.refs[:n_live] == 0), n_live + np.flatnonzero(book.refs[n_live:] > 0)
    to = np.arange(num, dtype=np.int32)
    to[high] = hole
    book.refs[hole], book.refs[high] = book.refs[high], 0
    book.table = np.where(book.table >= 0, to[book.table], -1).astype(np.int32)
    c.check()
    before[:, :, torch.from_numpy(hole).to(DEV)] = before[:, :, torch.from_numpy(high).to(DEV)]
    assert len(hole) > 100000 and torch.equal(raw(c.pages), before)
    assert tbik.get_error() == tbik.TBIK_OK
    # copies between the two ends of the pool
    tbik.cache_copy(c.pages, c.scales, i32(range(100)), i32(range(num - 100, num)))
    before[:, :, num - 100:] = before[:, :, :100]
    assert torch.equal(raw(c.pages), before) and tbik.get_error() == tbik.TBIK_OK
    # one sequence with every page of a pool
    del before, a, b
    one = Cache(2, num, num, 1, 64, page, fill=0)
    assert one.pages.shape[2] == num
    start = tbik.cache_extend(one.table, one.lens, one.refs, i32([num * page - 3]), page=page, rows=i32([1]))
    assert start.item() == 0 and one.table[1].tolist() == list(range(num)) and (one.refs == 1).all()
    k = torch.randn(3, 1, 64, device=DEV).to(torch.bfloat16)
    start = tbik.cache_extend(one.table, one.lens, one.refs, i32([3]), page=page, rows=i32([1]))
    tbik.cache_append(k, k, one.pages[0], one.scales[0], one.table, one.refs, start, cu=i32([0, 3]), rows=i32([1]))
    q = torch.randn(1, 8, 64, device=DEV).to(torch.bfloat16)
    out = tbik.cache_attention(q, one.pages[0], one.scales[0], one.table, i32([num * page - 1]), rows=i32([1]))
    assert tbik.get_error() == tbik.TBIK_OK and torch.isfinite(out).all()
    v = one.pages[0][1, num - 1, 0].float().permute(0, 2, 1, 3).reshape(page, 64)[-3:] * one.scales[0][1, num - 1, 0]
    s = (q[0].float() @ (one.pages[0][0, num - 1, 0].float().permute(0, 2, 1, 3).reshape(page, 64)[-3:] * one.scales[0][0, num - 1, 0]).T) / 8
    w = torch.exp(s.double())  # every other score is 0, its value too
    want = (w @ v.double()) / (w.sum(1, keepdim=True) + num * page - 3)
    assert (out[0].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()


def test_a_decode_step_in_a_graph():
    """Room, write, attention with its default bounds, choice, captured once on a side stream and replayed, against the same
    steps called one by one: the same pages, tokens and bits, also where a page fills up and where the pool runs out."""
    H, heads, D, page, V, B = 2, 8, 64, 16, 3000, 5
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)  # noqa: E731
    kv, head, us = rnd(V, 2, H, D), rnd(heads * D, V) / 8, torch.rand(60, B, device=DEV, generator=g)
    qs = rnd(V, heads, D)
    rows, one = i32([6, 0, 3, 7, 1]), i32([1] * B)
    full = lambda x: torch.full((B,), x, device=DEV)  # noqa: E731
    temp, top_p = full(0.9), full(0.95)

    def fresh():
        c = Cache(8, 5, 16, H, D, page)
        return c, torch.arange(B, device=DEV, dtype=torch.int32), torch.zeros(B, device=DEV), torch.zeros(B, heads, D, device=DEV, dtype=torch.bfloat16)

    def step(c, tok, u, out):
        start = tbik.cache_extend(c.table, c.lens, c.refs, one, page=page, rows=rows)
        x = kv[tok.long()]
        tbik.cache_append(x[:, 0].contiguous(), x[:, 1].contiguous(), c.pages[0], c.scales[0], c.table, c.refs, start, rows=rows)
        tbik.cache_attention(qs[tok.long()], c.pages[0], c.scales[0], c.table, start, rows=rows, out=out)
        z = torch.nan_to_num(out.float().reshape(B, -1)) @ head.float()
        tbik.sample(z, u, temperature=temp, top_p=top_p, out=tok)

    c1, tok1, u1, out1 = fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*fresh())  # nothing is set up while the graph is captured
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(c1, tok1, u1, out1)
    torch.cuda.synchronize()
    c2, tok2, u2, out2 = fresh()
    refused = 0
    for s in range(60):  # 16 pages for 5 sequences: refused from position 48 on
        u1.copy_(us[s])
        u2.copy_(us[s])
        graph.replay()
        step(c2, tok2, u2, out2)
        torch.cuda.synchronize()
        assert torch.equal(tok1, tok2) and torch.equal(out1.view(torch.int16), out2.view(torch.int16))
        assert torch.equal(c1.table, c2.table) and torch.equal(c1.lens, c2.lens) and torch.equal(c1.refs, c2.refs)
        assert torch.equal(raw(c1.pages), raw(c2.pages)) and torch.equal(c1.scales, c2.scales)
        code = tbik.get_error()
        assert code == (tbik.TBIK_OK if s < 48 else tbik.TBIK_ERR_PAGE), (s, code)
        assert torch.isnan(out1).any().item() == (s >= 48)
        refused += code != tbik.TBIK_OK
    assert refused == 12


# ------------------------------------------------- together, as a rollout uses them

def test_a_rollout_and_its_replay():
    """Prompts written, forked into samples, generated token by token (room, write, attention, logits, choice), some
    freed and the pool compacted on the way.  Every sequence by itself gives the same pages, bits and tokens."""
    L, H, G, D, page, V, E = 2, 2, 4, 64, 16, 1000, 512
    heads = H * G
    g = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: (torch.randn(*s, device=DEV, generator=g) / s[0] ** 0.5).to(torch.bfloat16)  # noqa: E731
    emb = (torch.randn(V, E, device=DEV, generator=g)).to(torch.bfloat16)
    wq, wk, wv, wo = [[rnd(E, k * D) for _ in range(L)] for k in (heads, H, H)] + [[rnd(heads * D, E) for _ in range(L)]]
    head = rnd(E, V)

    def forward(c, tok, start, n, rows):
        """Hidden states of packed tokens; every GEMM in tree order, so a row's bits do not depend on the others."""
        h = emb[tok]
        for l in range(L):
            mm = lambda x, w: tbik.gemm(x, w, T=1, leaf=64, out_bf16=True)  # noqa: E731
            c.append(mm(h, wk[l]).view(-1, H, D), mm(h, wv[l]).view(-1, H, D), start, n, rows, layer=l)
            a = c.attend(mm(h, wq[l]).view(-1, heads, D), start, n, rows, layer=l)
            h = tbik.gemm(a.reshape(-1, heads * D).contiguous(), wo[l], T=1, leaf=64, residual=h.contiguous())
        return h

    def choose(h, u):
        B = h.shape[0]
        z = tbik.gemm(h.contiguous(), head, T=1, leaf=64)
        full = lambda x, dt: torch.full((B,), x, dtype=dt, device=DEV)  # noqa: E731
        return tbik.sample(z, u, temperature=full(0.8, torch.float32), top_k=full(200, torch.int32),
                           top_p=full(0.95, torch.float32), min_p=full(0.001, torch.float32))

    prompts = [torch.randint(0, V, (m,), device=DEV, generator=g) for m in (37, 16, 150)]
    slots, steps, per = 16, 20, 3
    c = Cache(slots, 20, 200, H, D, page, layers=L)
    n = [len(p) for p in prompts]
    h = forward(c, torch.cat(prompts), c.extend([0, 1, 2], n), n, [0, 1, 2])
    ends = (torch.tensor(n, device=DEV).cumsum(0) - 1)
    parents, children = [i for i in range(3) for _ in range(per)], list(range(3, 3 + 3 * per))
    tbik.cache_fork(c.pages, c.scales, c.table, c.lens, c.refs, i32(parents), i32(children))
    c.book.fork(parents, children)
    tbik.cache_free(c.table, c.lens, c.refs, i32([0, 1, 2]), page=page)
    c.book.free([0, 1, 2])
    c.check()
    us = torch.rand(steps + 1, len(children), device=DEV, generator=g)
    tok = choose(h[ends][torch.tensor(parents, device=DEV)], us[0])
    seqs = [[p.tolist() for p in prompts][i] + [t] for i, t in zip(parents, tok.tolist())]
    live, hidden = list(children), {}
    for s in range(steps):
        if s == 7:  # two sequences end
            for r in (live[1], live[5]):
                tbik.cache_free(c.table, c.lens, c.refs, i32([r]), page=page)
                c.book.free([r])
            live = [r for i, r in enumerate(live) if i not in (1, 5)]
            assert tbik.cache_compact(c.pages, c.scales, c.table, c.lens, c.refs).item() == c.book.compact()[0]
            c.check()
        start = c.extend(live, [1] * len(live))
        h = forward(c, torch.tensor([seqs[r - 3][-1] for r in live], device=DEV), start, [1] * len(live), live)
        tok = choose(h, us[s + 1][torch.tensor([r - 3 for r in live], device=DEV)].contiguous())
        for r, t, x in zip(live, tok.tolist(), h):
            seqs[r - 3].append(t)
            hidden[r, len(seqs[r - 3]) - 2] = x
    assert tbik.get_error() == tbik.TBIK_OK
    # the replay: every sequence by itself, never forked, in other slots and pages; its tokens in the same steps, since a
    # page's scale grows while it fills and a query sees the page as it is at its time
    for i, r in enumerate(live):
        one = Cache(3, 20, 40, H, D, page, layers=L)
        prompt = prompts[parents[r - 3]]
        m = len(prompt)
        h = forward(one, prompt, one.extend([2], [m]), [m], [2])
        u = us[:, r - 3]
        assert choose(h[-1:], u[:1].contiguous()).item() == seqs[r - 3][m]
        for pos in range(m, len(seqs[r - 3]) - 1):
            h = forward(one, torch.tensor([seqs[r - 3][pos]], device=DEV), one.extend([2], [1]), [1], [2])
            assert torch.equal(h[0], hidden[r, pos])
            assert choose(h, u[pos - m + 1:pos - m + 2].contiguous()).item() == seqs[r - 3][pos + 1]
        n_tok = len(seqs[r - 3]) - 1
        for l in range(L):
            assert np.array_equal(c.stored(r, n_tok, l), one.stored(2, n_tok, l))
    assert tbik.get_error() == tbik.TBIK_OK
