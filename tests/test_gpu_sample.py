"""Sampling against its definition in binary64: every filter and their combinations, odd vocabularies, masks, ties,
infinities and NaN, and the independence of a row's token from the batch."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import invariant_tree_ordered_b200 as tbik  # noqa: E402

DEV = "cuda"


def ref_row(z, u, temp, k, p, mp):
    """(token, kept [V], its slack): the definition in binary64; -1 when there is nothing to choose."""
    z = z.astype(np.float64)
    V = len(z)
    if np.isnan(z).any() or z.max() == -np.inf:
        return -1, np.zeros(V, bool), None
    m = z.max()
    order = np.lexsort((np.arange(V), -z))
    if not temp > 0 or k == 1:
        return int(order[0]), z == z[order[0]], None
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(z == m, 1.0, np.exp((z - m) / temp))
    w[z == -np.inf] = 0
    if np.isinf(m):
        w = (z == m).astype(float)
    keep = np.zeros(V, bool)
    keep[order[:k] if 0 < k < V else order] = True
    if p < 1:
        ws = (w * keep)[order]
        before = np.cumsum(ws) - ws
        sel = before < p * ws.sum()
        sel[0] = True
        keep[order] &= sel
    keep &= (w >= mp) | (z == m)
    c = np.cumsum(w * keep)
    tok = int(np.searchsorted(c, u * c[-1], side="right"))
    return min(tok, int(np.flatnonzero(w * keep)[-1])), keep, (w, c)


def check(logits, u, temp=None, k=None, p=None, mp=None):
    B, V = logits.shape
    f = lambda x, dt: None if x is None else torch.tensor(np.broadcast_to(x, B).copy(), dtype=dt, device=DEV)  # noqa: E731
    ut = torch.tensor(np.broadcast_to(u, B).copy(), dtype=torch.float32, device=DEV)
    args = dict(temperature=f(temp, torch.float32), top_k=f(k, torch.int32), top_p=f(p, torch.float32), min_p=f(mp, torch.float32))
    got = tbik.sample(logits, ut, **args)
    again = tbik.sample(logits, ut, **args)
    assert torch.equal(got, again)
    z = logits.float().cpu().numpy()
    val = lambda t, d, b: d if t is None else float(t[b])  # noqa: E731
    got = got.cpu().numpy()
    for b in range(B):
        tok, keep, more = ref_row(z[b], float(ut[b]), val(args["temperature"], 1.0, b), int(val(args["top_k"], 0, b)),
                                  val(args["top_p"], 1.0, b), val(args["min_p"], 0.0, b))
        if got[b] == tok:
            continue
        # a border between two tokens may move by the weights' own precision: fp32 weights and their units of 2^-32
        # (sums off by less than 2^-20 of the total), nothing else
        assert more is not None and 0 <= got[b] < V, (b, got[b], tok)
        w, c = more
        x, slack = float(ut[b]) * c[-1], 2.0 ** -20 * c[-1]
        assert c[got[b]] - w[got[b]] - slack <= x <= c[got[b]] + slack and w[got[b]] > 0, (b, got[b], tok)
    return got


def rows(seed, B, V, std=2.5, half=False, peaks=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(B, V, device=DEV, generator=g) * std
    if peaks and V > 20:
        x.scatter_add_(1, torch.randint(0, V, (B, 8), device=DEV, generator=g), torch.rand(B, 8, device=DEV, generator=g) * 9)
    return x.to(torch.bfloat16) if half else x


def uni(seed, B):
    return np.random.RandomState(seed).rand(B).astype(np.float32)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [1, 2, 15, 17, 511, 1000, 4097, 32000, 50257, 151936, 393216])
def test_every_filter(V, half):
    B = 12 if V < 100000 else 6
    z = rows(V, B, V, half=half)
    check(z, uni(1, B))
    check(z, uni(2, B), temp=np.linspace(0.2, 2.0, B))
    check(z, uni(3, B), k=np.resize([1, 2, 50, 1000, V, 0], B))
    check(z, uni(4, B), p=np.resize([0.9, 0.5, 0.999, 1.0, 0.01, 0.0], B))
    check(z, uni(5, B), mp=np.resize([0.0, 0.1, 0.5, 1.0], B))
    check(z, uni(6, B), temp=np.resize([0.0, 0.7, 1.0, 3.0], B), k=np.resize([0, 40, 3, 2000, 5], B),
          p=np.resize([0.95, 1.0, 0.6], B), mp=np.resize([0.0, 0.05], B))
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("V", [300, 40000, 151936])
def test_flat_rows_and_large_k(V):
    """Almost flat and exactly flat rows: a border with thousands of tokens."""
    B = 6
    check(rows(1, B, V, std=0.01, peaks=False), uni(1, B), p=np.resize([0.9, 0.3], B), k=np.resize([0, V // 2, V - 1], B))
    check(rows(2, B, V, std=0.01, peaks=False, half=True), uni(2, B), p=np.resize([0.9, 0.3], B), k=np.resize([0, V // 3, V - 1], B))
    flat = torch.full((B, V), -3.5, device=DEV)
    check(flat, uni(3, B), k=np.resize([0, 7, V // 2], B), p=np.resize([1.0, 0.25], B))
    lowest = torch.full((B, V), torch.finfo(torch.float32).min, device=DEV)
    check(lowest, uni(4, B), k=np.resize([0, 9], B), p=0.5)
    check(rows(5, B, V, std=1e-30, peaks=False), uni(5, B), k=np.resize([3, V // 2], B), p=0.7)
    check(rows(6, B, V, std=50), uni(6, B), temp=np.resize([1e-3, 100.0, 1e4], B), k=np.resize([0, V // 2, 5000], B), p=0.99)


def test_equal_logits_keep_the_lower_indices():
    V = 5000
    z = torch.zeros(4, V, device=DEV)
    z[:, 1000:] = 1.0
    z[:, 4321] = 2.0
    # the top 11: token 4321 and the ten lowest indices of the next level
    got = check(z, [0.0, 0.999999, 0.3, 0.9], k=11)
    assert got[0] == 1000 and got[1] == 4321
    # signed zeros are equal
    s = torch.zeros(1, 64, device=DEV)
    s[0, ::2] = -0.0
    assert check(s, [0.0], temp=0.0)[0] == 0
    assert check(s, [0.999999], k=3)[0] == 2


def test_masked_and_broken_rows():
    V = 3000
    z = rows(1, 8, V)
    z[0, :-1] = float("-inf")                       # one token left
    z[1, :] = float("-inf")                         # nothing left
    z[2, 5:] = torch.finfo(torch.float32).min       # a mask of the type's lowest value
    z[3, 17] = float("inf")
    z[4, 3], z[4, 9] = float("inf"), float("inf")
    z[5, 100:] = float("-inf")
    for kw in ({}, {"k": 50}, {"p": 0.9}, {"k": 20, "p": 0.5, "mp": 0.1}, {"temp": 0.0}, {"temp": 1e-40}, {"k": 200}):
        got = check(z, uni(3, 8), **kw)
        assert got[0] == V - 1 and got[1] == -1 and got[3] == 17 and got[4] in (3, 9) and got[5] < 100
    assert tbik.get_error() == tbik.TBIK_OK
    z[6, 2999] = float("nan")
    got = check(z, uni(4, 8), k=5)
    assert got[6] == -1 and got[7] >= 0
    assert tbik.get_error() == tbik.TBIK_ERR_VALUE


def test_the_ends_of_u():
    z = rows(5, 6, 777)
    check(z, [0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 0.5, 1e-10, 0.25], k=30)
    u = torch.tensor([1.0, -1.0, float("nan"), 7.0, 0.0, 0.5], device=DEV)  # outside [0, 1): the nearest token there is
    got = tbik.sample(z, u).cpu().numpy()
    order = [int(np.flatnonzero(np.isfinite(z[b].cpu().numpy()))[i]) for b, i in ((1, 0), (2, 0), (4, 0))]
    assert got[1] == order[0] and got[2] == order[1] and got[4] == order[2]
    assert (got >= 0).all() and (got < 777).all()


def test_a_row_does_not_depend_on_its_batch():
    V = 60001  # rows that start at odd addresses
    for half in (False, True):
        z = rows(7, 300, V, half=half)
        u = torch.from_numpy(uni(8, 300)).to(DEV)
        t = torch.from_numpy(np.resize([0.5, 1.0, 1.5], 300).astype(np.float32)).to(DEV)
        k = torch.from_numpy(np.resize([0, 40, 5000], 300).astype(np.int32)).to(DEV)
        p = torch.from_numpy(np.resize([0.9, 1.0], 300).astype(np.float32)).to(DEV)
        whole = tbik.sample(z, u, temperature=t, top_k=k, top_p=p)
        for a, b in ((0, 1), (1, 3), (17, 40), (299, 300)):
            part = tbik.sample(z[a:b].clone(), u[a:b].clone(), temperature=t[a:b].clone(), top_k=k[a:b].clone(), top_p=p[a:b].clone())
            assert torch.equal(part, whole[a:b])
        perm = torch.randperm(300, generator=torch.Generator().manual_seed(1)).to(DEV)
        assert torch.equal(tbik.sample(z[perm], u[perm], temperature=t[perm], top_k=k[perm], top_p=p[perm]), whole[perm])


def test_streams_graphs_and_refusals():
    z, u = rows(9, 5, 32000), torch.from_numpy(uni(9, 5)).to(DEV)
    eager = tbik.sample(z, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros(5, dtype=torch.int32, device=DEV)
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            tbik.sample(z, u, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    for f in (lambda: tbik.sample(z[:, ::2], u), lambda: tbik.sample(z, u[:4]), lambda: tbik.sample(z[0], u),
              lambda: tbik.sample(z, u, out=torch.zeros(4, dtype=torch.int32, device=DEV)),
              lambda: tbik.sample(z, u, temperature=u[:2])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: tbik.sample(z.half(), u), lambda: tbik.sample(z, u.double()), lambda: tbik.sample(z, u, top_k=u)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(tbik.TbikError):
        tbik.sample(torch.zeros(1, 393217, device=DEV), u[:1])
    with pytest.raises(tbik.TbikError):
        tbik.sample(torch.zeros(8 * 5 + 1, device=DEV)[1:].view(5, 8), u)
    assert tbik.sample(z[:0], u[:0]).shape == (0,)


@pytest.mark.parametrize("B,V,half", [(80, 50257, False), (150, 33001, False), (76, 151936, True)])
def test_more_rows_than_the_device_holds(B, V, half):
    """Rows that stay in global memory: every filter, masked tokens, low and high temperatures, flat rows among others,
    and the same tokens as in a small batch."""
    z = rows(B, B, V, half=half)
    z[1::7, : V // 2] = float("-inf")
    z[2::7] *= 0.001
    z[3] = -1.25
    z[4::9] += 40
    z[5::9] -= 300
    t = np.resize([1.0, 0.7, 0.2, 1.3, 0.0, 5.0, 0.05], B)
    k = np.resize([0, 50, 1000, 0, V // 2, 2, 0, 0], B)
    p = np.resize([0.95, 1.0, 0.9, 0.999, 0.3], B)
    mp = np.resize([0.0, 0.05, 0.0], B)
    got = check(z, uni(1, B), temp=t, k=k, p=p, mp=mp)
    check(z, uni(2, B))
    check(z, uni(3, B), p=p)
    f = lambda x, dt: torch.tensor(np.asarray(x), dtype=dt, device=DEV)  # noqa: E731
    for a in range(0, B, 40):
        r = slice(a, a + 5)
        few = tbik.sample(z[r].contiguous(), f(uni(1, B)[r], torch.float32), temperature=f(t[r], torch.float32),
                          top_k=f(k[r], torch.int32), top_p=f(p[r], torch.float32), min_p=f(mp[r], torch.float32))
        assert few.tolist() == got[r].tolist()
    z[6, V - 1] = float("nan")
    z[8] = float("-inf")
    z[9, 7] = float("inf")
    out = tbik.sample(z, f(uni(4, B), torch.float32), top_p=f(p, torch.float32))
    assert tbik.get_error() == tbik.TBIK_ERR_VALUE
    assert out[6].item() == -1 and out[8].item() == -1 and out[9].item() == 7


@pytest.mark.parametrize("temp,back", [(0.97, -6.051175), (0.98, -6.1135583), (1.11, -6.9245405), (1.94, -12.10235)])
@pytest.mark.parametrize("p", [None, 0.9])
def test_a_background_of_2_to_the_minus_9(temp, back, p):
    """Thousands of equal weights of 2^-9 - 2^-33 of the largest, which is 2^23 units: 512 of them are 2^32."""
    V = 151936
    z = torch.full((8, V), back, device=DEV)
    z[:, 123] = 0.0
    check(z, np.linspace(0.02, 0.98, 8), temp=temp, p=p)
    assert tbik.get_error() == tbik.TBIK_OK


# ------------------------------------------------- the kept set itself

SLACK = 2.0 ** -20  # of the row's mass: fp32 weights off by a few 2^-24 each, all one way at worst, and units of 2^-32


def strict(logits, u, temp=None, k=None, p=None, mp=None):
    """Every token is one that the filters keep.  Only a token whose mass before it (top-p) or whose weight (min-p) is within
    the slack of the limit may be kept or not; top-k and ties are exact.  Returns how many of the rows had no such token."""
    B, V = logits.shape
    f = lambda x, dt: None if x is None else torch.tensor(np.broadcast_to(x, B).copy(), dtype=dt, device=DEV)  # noqa: E731
    ut = f(u, torch.float32)
    t, kk, pp, mm = f(temp, torch.float32), f(k, torch.int32), f(p, torch.float32), f(mp, torch.float32)
    got = tbik.sample(logits, ut, temperature=t, top_k=kk, top_p=pp, min_p=mm).cpu().numpy()
    z = logits.float().cpu().numpy().astype(np.float64)
    sure = 0
    for b in range(B):
        T, K = (1.0 if t is None else float(t[b])), (0 if kk is None else int(kk[b]))
        P, M = (1.0 if pp is None else float(pp[b])), (0.0 if mm is None else float(mm[b]))
        order = np.lexsort((np.arange(V), -z[b]))
        if not T > 0 or K == 1:
            assert got[b] == order[0]
            continue
        with np.errstate(invalid="ignore"):
            w = np.exp((z[b] - z[b].max()) / T)
        w[(z[b] == -np.inf) | (w < 2.0 ** -33)] = 0
        keep = np.zeros(V, bool)
        keep[order[:K] if 0 < K < V else order] = True
        amb = np.zeros(V, bool)
        if P < 1:
            ws = (w * keep)[order]
            S, before = ws.sum(), np.cumsum(ws) - ws
            sel = before < P * S
            sel[0] = True
            near = (np.abs(before - P * S) <= SLACK * S) & keep[order] & (ws > 0)
            near[0] = False
            amb[order[near]] = True
            keep[order] &= sel
        if M > 0:
            # an exponent is off by a rounding of the difference, 2^-24 of |x|, and the hardware's 2^-22
            amb |= keep & (np.abs(w - M) <= M * (2.0 ** -21 + 2.0 ** -22 * np.abs(np.log(max(M, 1e-30))))) & (z[b] != z[b].max())
            keep &= (w >= M) | (z[b] == z[b].max())
        keep &= w > 0
        c = np.cumsum(w * (keep | amb))
        slack = SLACK * c[-1] + (w * amb).sum()
        assert keep[got[b]] or amb[got[b]], (b, int(got[b]))
        x = min(max(float(ut[b]), 0.0), 1.0) * c[-1]
        assert c[got[b]] - w[got[b]] - slack <= x <= c[got[b]] + slack, (b, int(got[b]))
        if not amb.any():
            sure += 1
            if float(ut[b]) >= 1:
                assert got[b] == np.flatnonzero(keep)[-1], (b, int(got[b]))
    return sure


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [700, 4097, 32000, 151936])
def test_every_token_is_one_that_the_filters_keep(V, half):
    """u = 1 takes the last kept token by index, u = 0 the first, and numbers between come near the borders."""
    B = 8
    ends = np.resize([1.0, 0.0, 0.999999, 0.5, 1.0], B)
    for seed, std in ((1, 2.5), (2, 0.3), (3, 6.0)):
        z = rows(seed + V, B, V, std=std, half=half)
        assert strict(z, ends, k=np.resize([2, 3, 50, 1000, V - 1, 2047, 2049, 5], B)) == B
        assert strict(z, ends, k=np.resize([50, V // 2], B), temp=np.linspace(0.3, 3, B)) == B
        sure = strict(z, ends, p=np.resize([0.9, 0.5, 0.999, 0.05], B))
        sure += strict(z, ends, p=np.resize([0.9, 0.5, 0.99], B), k=np.resize([40, 3000, 7], B), temp=np.linspace(0.5, 1.5, B))
        assert sure >= B // 2 or half or V > 10000
        strict(z, ends, mp=np.resize([0.01, 0.3, 0.001, 0.9], B))
        strict(z, ends, mp=0.02, p=0.97, k=2000, temp=np.linspace(0.5, 5, B))
    assert tbik.get_error() == tbik.TBIK_OK


def test_the_last_kept_token_for_u_of_one_and_more():
    z = rows(11, 4, 777)
    for u in (1.0, 7.0, float("inf")):
        assert strict(z, [u] * 4) == 4
        assert strict(z, [u] * 4, k=30) == 4
        got = tbik.sample(z, torch.full((4,), u, device=DEV), top_k=torch.full((4,), 30, dtype=torch.int32, device=DEV)).tolist()
        assert got == z.topk(30, dim=1).indices.max(1).values.tolist()  # no ties among the largest here


@pytest.mark.parametrize("B,V,half", [(400, 33001, False), (150, 151936, True)])
def test_rows_of_all_kinds_when_clusters_come_in_waves(B, V, half):
    """More clusters than the device holds at once: masked tokens, flat rows, hot and cold temperatures among others."""
    z = rows(B, B, V, half=half)
    z[1::7, : V // 2] = -1e30
    z[2::7] *= 0.001
    z[3] = -1.25
    z[5::9] -= 300
    strict(z, uni(1, B), temp=np.resize([1.0, 0.7, 0.2, 1.3, 0.0, 5.0, 0.05], B), k=np.resize([0, 50, 1000, 0, V // 2, 2, 0, 0], B),
           p=np.resize([0.95, 1.0, 0.9, 0.999, 0.3], B), mp=np.resize([0.0, 0.05, 0.0], B))
    assert tbik.get_error() == tbik.TBIK_OK


@pytest.mark.parametrize("V,std", [(3000, 2.5), (151936, 2.5), (40000, 0.0)])
def test_settings_that_are_not_numbers(V, std):
    """A NaN temperature takes the most likely token; NaN top_p and min_p (and a negative min_p) filter nothing."""
    B = 12
    z = rows(V, B, V, std=std, peaks=std > 0)
    u = torch.from_numpy(uni(1, B)).to(DEV)
    full = lambda x: torch.full((B,), x, device=DEV)  # noqa: E731
    nan = float("nan")
    for kw in ({}, dict(top_k=torch.full((B,), 300, dtype=torch.int32, device=DEV))):
        plain = tbik.sample(z, u, **kw)
        assert torch.equal(tbik.sample(z, u, min_p=full(nan), **kw), plain)
        assert torch.equal(tbik.sample(z, u, min_p=full(-1.0), **kw), plain)
        assert torch.equal(tbik.sample(z, u, top_p=full(nan), **kw), plain)
        half = tbik.sample(z, u, top_p=full(0.5), **kw)
        assert torch.equal(tbik.sample(z, u, top_p=full(0.5), min_p=full(nan), **kw), half)
        assert torch.equal(tbik.sample(z, u, temperature=full(nan), **kw), tbik.sample(z, u, temperature=full(0.0), **kw))
    assert tbik.get_error() == tbik.TBIK_OK
