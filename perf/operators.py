"""The serving operators beside the decoder, as cases to measure: attention over a paged key/value cache held in
8 bits, the writes into that cache, its page operations, and sampling from logits.

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is one pass (the plain torch form, or
with `own` the library's call), `exact` is the definition in 64 bits and `work` the bytes and operations that a pass
cannot do without.

The cache.  K and V are float8 e4m3 values times a power-of-two fp32 scale for each page and head:
    pages   [layers, 2, pages, kv_heads, page / 8, head_dim / 16, 8, 16]   (2: keys, values; token t, dim d of a page
            at [t // 8, d // 16, t % 8, d % 16])
    scales  [layers, 2, pages, kv_heads]
    table   [slots, max_pages] page numbers of each sequence, -1 behind the last; lens [slots]; refs [pages]
A sequence's tokens of one call sit at positions start[b] .. start[b] + n_b - 1.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E_MIN = -100  # the smallest exponent of a page's scale (also that of a page of zeros)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one user's sequence, one new token: the smallest attention call of a decode step
        dict(name="attend_one", op="attend", batch=1, q_lo=1, q_hi=1, ctx_lo=1999, ctx_hi=1999, heads=32, kv_heads=8,
             head_dim=128, page=64),
        # a serving batch in its decode step, contexts of all lengths, small pages
        dict(name="attend_batch", op="attend", batch=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=8192, heads=32, kv_heads=8,
             head_dim=128, page=16),
        # few sequences with very long contexts: the keys have to be split over the device
        dict(name="attend_long", op="attend", batch=4, q_lo=1, q_hi=1, ctx_lo=120000, ctx_hi=131071, heads=32,
             kv_heads=4, head_dim=128, page=128),
        # checking drafted tokens: a few queries for each sequence, a cache head for each query head, 64 dims
        dict(name="attend_verify", op="attend", batch=24, q_lo=1, q_hi=5, ctx_lo=300, ctx_hi=4096, heads=16,
             kv_heads=16, head_dim=64, page=32),
        # a chunk of each prompt over what the cache already holds of it
        dict(name="attend_chunk", op="attend", batch=4, q_lo=300, q_hi=512, ctx_lo=5000, ctx_hi=8192, heads=32,
             kv_heads=8, head_dim=128, page=64),
        # the decode step's write: one token for each sequence
        dict(name="append_step", op="append", batch=64, n_lo=1, n_hi=1, at_lo=0, at_hi=8191, kv_heads=8, head_dim=128,
             page=16),
        # prompts of all lengths written at once
        dict(name="append_prompt", op="append", batch=32, n_lo=100, n_hi=4096, at_lo=0, at_hi=500, kv_heads=8,
             head_dim=128, page=64),
        # several samples of each prompt: fork the sequences, make room for a token each, and free them
        dict(name="pages_branch", op="branch", parents=8, copies=16, ctx_lo=500, ctx_hi=2048, n_new=1, layers=4,
             kv_heads=8, head_dim=128, page=64),
        # after many sequences have come and gone: the live pages to the front of the pool
        dict(name="pages_compact", op="compact", pages=2048, live=0.6, slots=48, layers=4, kv_heads=8, head_dim=128,
             page=32),
        # one row of logits over the whole vocabulary
        dict(name="sample_one", op="sample", batch=1, vocab=151936, half=False, mix="nucleus"),
        # a serving batch, every row with its own settings
        dict(name="sample_batch", op="sample", batch=256, vocab=151936, half=False, mix="all"),
        # bf16 logits (many equal values) over a smaller vocabulary
        dict(name="sample_half", op="sample", batch=97, vocab=32000, half=True, mix="all"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) )))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "branch", "compact", "sample", "sample"])
    head_dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "attend":
        kv_heads, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        while kv_heads * group > 32:
            group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        q_hi = rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 512)])
        ctx_hi = _log(rng, 64, 65536)
        budget = 4 * 16384 if q_hi > 16 else 600_000  # keys over all sequences
        batch = max(1, min(_log(rng, 1, 256), budget // ctx_hi))
        if q_hi > 16:
            ctx_hi, batch = min(ctx_hi, 8192), min(batch, 4)
        return dict(op=op, batch=batch, q_lo=max(1, q_hi // 2), q_hi=q_hi, ctx_lo=max(1, ctx_hi // rng.choice([1, 2, 20])),
                    ctx_hi=ctx_hi, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
    if op == "append":
        n_hi = rng.choice([1, _log(rng, 1, 4096)])
        batch = max(1, min(_log(rng, 1, 256), 65536 // n_hi))
        return dict(op=op, batch=batch, n_lo=max(1, n_hi // 8), n_hi=n_hi, at_lo=0, at_hi=_log(rng, 1, 2000),
                    kv_heads=rng.choice([1, 2, 4, 8]), head_dim=head_dim, page=page)
    if op == "branch":
        ctx_hi = _log(rng, 20, 2048)
        return dict(op=op, parents=rng.randint(1, 8), copies=rng.randint(1, 16), ctx_lo=max(1, ctx_hi // 4),
                    ctx_hi=ctx_hi, n_new=_log(rng, 1, 200), layers=rng.randint(1, 4), kv_heads=rng.choice([1, 2, 4, 8]),
                    head_dim=head_dim, page=page)
    if op == "compact":
        return dict(op=op, pages=_log(rng, 64, 2048), live=round(rng.uniform(0.05, 0.95), 3), slots=rng.randint(3, 48),
                    layers=rng.randint(1, 3), kv_heads=rng.choice([1, 2, 4, 8]), head_dim=head_dim,
                    page=rng.choice([16, 32]))
    vocab = _log(rng, 500, 200_000)
    return dict(op=op, batch=max(1, min(_log(rng, 1, 256), 38_000_000 // vocab)), vocab=vocab,
                half=rng.random() < 0.5, mix=rng.choice(["plain", "top_k", "nucleus", "min_p", "all"]))


# --------------------------------------------- sizes that belong to the case

def _sizes(case):
    """Lengths and page numbers of a case: the same for every seed, so that `work` knows them."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    op = case["op"]
    if op == "attend":
        n = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
        ctx = [max(q, _log(r, case["ctx_lo"], case["ctx_hi"])) for q in n]
        ctx[-1] = max(n[-1], case["ctx_hi"])
        return {"n": n, "start": [c - q for c, q in zip(ctx, n)]}
    if op == "append":
        n = [_log(r, case["n_lo"], case["n_hi"]) for _ in range(case["batch"])]
        return {"n": n, "start": [r.randint(case["at_lo"], case["at_hi"]) for _ in n]}
    if op == "branch":
        return {"lens": [_log(r, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["parents"])]}
    if op == "compact":
        live = sorted(r.sample(range(case["pages"]), max(1, int(case["pages"] * case["live"]))))
        order = live[:]
        r.shuffle(order)
        cuts = sorted(r.sample(range(len(order) + 1), min(case["slots"] - 1, len(order) + 1)))
        rows = [order[a:b] for a, b in zip([0] + cuts, cuts + [len(order)])]
        rows += [[]] * (case["slots"] - len(rows))
        lens = [len(x) * case["page"] - (r.randint(0, case["page"] - 1) if x else 0) for x in rows]
        return {"rows": rows, "lens": lens, "moves": sum(p >= len(live) for p in live)}
    return {}


def _table(rng, used, pool):
    """Rows of distinct page numbers in a mixed order, and the page count of the pool."""
    order = list(range(pool))
    rng.shuffle(order)
    width, at, rows = max(max(used), 1), 0, []
    for u in used:
        rows.append(order[at:at + u] + [-1] * (width - u))
        at += u
    return rows


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return _i32(c)


def _values(shape, gen):
    """e4m3 values as a cache holds them: normal ones, scaled so that a page's largest is near 448's binade."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat, step = out.view(-1), 1 << 26
    for a in range(0, flat.numel(), step):
        m = min(step, flat.numel() - a)
        flat[a:a + m] = (torch.randn(m, device=DEV, generator=gen) * 72).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return out


def _scales(shape, gen):
    return torch.exp2(torch.randint(-8, -5, shape, device=DEV, generator=gen).float())


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng, z, op = random.Random(seed), _sizes(case), case["op"]
    if op == "sample":
        B, V = case["batch"], case["vocab"]
        logits = torch.randn(B, V, device=DEV, generator=gen) * 2.5
        # a few likely tokens in each row, as a model's next-token distribution has
        at = torch.randint(0, V, (B, 12), device=DEV, generator=gen)
        logits.scatter_add_(1, at, torch.rand(B, 12, device=DEV, generator=gen) * 9)
        if case["half"]:
            logits = logits.to(torch.bfloat16)
        u = torch.rand(B, device=DEV, generator=gen)
        pick = lambda values, dt: torch.tensor([values[i] for i in torch.randint(0, len(values), (B,), generator=torch.Generator().manual_seed(seed + 7)).tolist()], dtype=dt, device=DEV)  # noqa: E731
        mix = case["mix"]
        temp = pick([1.0, 0.7, 0.6, 1.3, 0.0] if mix == "all" else [1.0, 0.8], torch.float32)
        top_k = pick([0, 50, 20, 1000, 0], torch.int32) if mix in ("all", "top_k") else None
        top_p = pick([0.95, 0.9, 1.0, 0.8, 0.5], torch.float32) if mix in ("all", "nucleus") else None
        min_p = pick([0.0, 0.05, 0.1, 0.02], torch.float32) if mix in ("all", "min_p") else None
        return {"op": op, "logits": logits, "u": u, "temperature": temp, "top_k": top_k, "top_p": top_p, "min_p": min_p}
    H, D, page = case["kv_heads"], case["head_dim"], case["page"]
    inner = (H, page // 8, D // 16, 8, 16)
    if op in ("attend", "append"):
        n, start = z["n"], z["start"]
        used = [-(-(s + m) // page) for s, m in zip(start, n)]
        pool = sum(used) + 3
        s = {"op": op, "table": _i32(_table(rng, used, pool)), "start": _i32(start), "max_q": max(n),
             "max_keys": max(a + b for a, b in zip(start, n)), "cu": None if max(n) == 1 else _cu(n),
             "pages": _values((2, pool) + inner, gen), "scales": _scales((2, pool, H), gen)}
        if op == "attend":
            s["q"] = (torch.randn(sum(n), case["heads"], D, device=DEV, generator=gen) * 2).to(torch.bfloat16)
        else:
            s["refs"] = (torch.bincount(s["table"].flatten()[s["table"].flatten() >= 0].long(), minlength=pool)).to(torch.int32)
            # keys have a few large dims, values are even
            big = 1 + 7 * (torch.rand(H, D, device=DEV, generator=gen) < 0.04)
            s["k"] = (torch.randn(sum(n), H, D, device=DEV, generator=gen) * big).to(torch.bfloat16)
            s["v"] = torch.randn(sum(n), H, D, device=DEV, generator=gen).to(torch.bfloat16)
        return s
    L = case["layers"]
    if op == "branch":
        P, C = case["parents"], case["parents"] * case["copies"]
        used = [-(-x // page) for x in z["lens"]]
        pool = sum(used) + C * (2 + -(-case["n_new"] // page)) + 5
        rows = _table(rng, used, pool)
        width = max(-(-(x + case["n_new"]) // page) for x in z["lens"])
        table = torch.full((P + C, width), -1, dtype=torch.int32, device=DEV)
        table[:P, :len(rows[0])] = _i32(rows)
        refs = torch.bincount(table.flatten()[table.flatten() >= 0].long(), minlength=pool).to(torch.int32)
        lens = _i32(z["lens"] + [0] * C)
        children = list(range(P, P + C))
        rng.shuffle(children)
        return {"op": op, "table": table, "lens": lens, "refs": refs, "pages": _values((L, 2, pool) + inner, gen),
                "scales": _scales((L, 2, pool, H), gen), "parents": _i32([i // case["copies"] for i in range(C)]),
                "children": _i32(children), "n_new": _i32([case["n_new"]] * C), "max_new": case["n_new"]}
    width = max(1, max(len(x) for x in z["rows"]))
    table = _i32([x + [-1] * (width - len(x)) for x in z["rows"]])
    refs = torch.bincount(table.flatten()[table.flatten() >= 0].long(), minlength=case["pages"]).to(torch.int32)
    return {"op": op, "table": table, "lens": _i32(z["lens"]), "refs": refs,
            "pages": _values((L, 2, case["pages"]) + inner, gen), "scales": _scales((L, 2, case["pages"], H), gen)}


def work(case):
    z, op = _sizes(case), case["op"]
    if op == "sample":
        # one pass over the logits: each read once, a subtraction, a product, an exponential and a sum
        b = case["batch"] * case["vocab"] * (2 if case["half"] else 4)
        return {"bytes": b + 24 * case["batch"], "flops": 4 * case["batch"] * case["vocab"]}
    H, D, page = case["kv_heads"], case["head_dim"], case["page"]
    if op == "attend":
        keys = sum(s + n for s, n in zip(z["start"], z["n"]))
        pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(z["start"], z["n"]))
        tok = sum(z["n"])
        # K and V of every key that a query sees (a byte a value, a scale a page and head), q read, out written
        return {"bytes": 2 * keys * H * (D + 4 / page) + 4 * tok * case["heads"] * D + 4 * sum(-(-(s + n) // page) for s, n in zip(z["start"], z["n"])),
                "flops": 4 * pairs * case["heads"] * D}
    if op == "append":
        tok = sum(z["n"])
        # bf16 in, a byte out
        return {"bytes": 2 * tok * H * D * 3, "flops": 4 * tok * H * D}
    L = case["layers"]
    one = 2 * L * H * (page * D + 4)  # a page of every layer, keys and values, and their scales
    if op == "branch":
        moved = case["copies"] * sum(x % page != 0 for x in z["lens"])
        rows = case["copies"] * sum(-(-x // page) for x in z["lens"])
        return {"bytes": 2 * moved * one + 12 * rows, "flops": rows}
    return {"bytes": 2 * z["moves"] * one + 8 * sum(len(x) for x in z["rows"]), "flops": 2 * case["pages"]}


# ------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["op"]
    if own:
        import invariant_tree_ordered_b200 as tbik
        if op == "attend":
            return tbik.cache_attention(s["q"], s["pages"], s["scales"], s["table"], s["start"], cu=s["cu"],
                                        max_q=s["max_q"], max_keys=s["max_keys"])
        if op == "append":
            tbik.cache_append(s["k"], s["v"], s["pages"], s["scales"], s["table"], s["refs"], s["start"], cu=s["cu"])
            return {"pages": s["pages"], "scales": s["scales"]}
        if op == "branch":
            tbik.cache_fork(s["pages"], s["scales"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
            start = tbik.cache_extend(s["table"], s["lens"], s["refs"], s["n_new"], page=s["pages"].shape[4] * 8,
                                      rows=s["children"])
            tbik.cache_free(s["table"], s["lens"], s["refs"], s["children"], page=s["pages"].shape[4] * 8)
            return {"start": start, "pages": s["pages"], "scales": s["scales"], "table": s["table"], "lens": s["lens"],
                    "refs": s["refs"]}
        if op == "compact":
            table, refs = s["table"].clone(), s["refs"].clone()
            live = tbik.cache_compact(s["pages"], s["scales"], table, s["lens"], refs)
            return {"live": live, "table": table, "refs": refs, "pages": s["pages"], "scales": s["scales"]}
        return tbik.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"])
    if op == "attend":
        return _attend(s)
    if op == "append":
        return _append(s)
    if op == "branch":
        _fork(s)
        start = _extend(s)
        _free(s)
        return {"start": start, "pages": s["pages"], "scales": s["scales"], "table": s["table"], "lens": s["lens"],
                "refs": s["refs"]}
    if op == "compact":
        return _compact(s)
    return _sample(s)


def _tokens_of(s, tokens):
    """(sequence, place in the sequence's new tokens) of each packed token."""
    t = torch.arange(tokens, device=DEV)
    if s["cu"] is None:
        return t, torch.zeros_like(t)
    cu = s["cu"].long()
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return b, t - cu[b]


def _attend(s):
    q, table = s["q"], s["table"].long()
    T, NH, D = q.shape
    _, _, H, p8, d16 = s["pages"].shape[:5]
    page, B, G = p8 * 8, table.shape[0], NH // H
    W = -(-s["max_keys"] // page)
    ids = table[:, :W].clamp(min=0)
    # [2, B, W, H, page, D] fp32 -> [2, B, H, keys, D]
    kv = s["pages"].view(torch.uint8)[:, ids].view(torch.float8_e4m3fn).float()
    kv = kv.permute(0, 1, 3, 2, 4, 6, 5, 7).reshape(2, B, H, W, page, D)
    kv = (kv * s["scales"][:, ids].permute(0, 1, 3, 2)[..., None, None]).reshape(2, B, H, W * page, D)
    b, t = _tokens_of(s, T)
    M = s["max_q"]
    qp = torch.zeros(B, M, NH, D, device=DEV)
    qp[b, t] = q.float()
    qp = qp.view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    sc = torch.matmul(qp, kv[0].transpose(2, 3)) * (1.0 / math.sqrt(D))
    pos = s["start"].long()[:, None] + torch.arange(M, device=DEV)[None]
    see = torch.arange(W * page, device=DEV)[None, None] <= pos[:, :, None]
    sc = sc.view(B, H, M, G, -1).masked_fill_(~see[:, None, :, None], float("-inf")).view(B, H, M * G, -1)
    sc = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.matmul(sc, kv[1]) / sc.sum(-1, keepdim=True)
    o = o.view(B, H, M, G, D).permute(0, 2, 1, 3, 4).reshape(B, M, NH, D)
    return o[b, t].to(torch.bfloat16)


def _round4(x):
    """fp32 values that bf16 holds, rounded to 4 significant bits (nearest, ties to even), as integers of their bits."""
    i = x.contiguous().view(torch.int32)
    i = (i + 0x7FFFF + ((i >> 20) & 1)) & -0x100000
    return i.view(torch.float32)


def _need(amax):
    """The smallest exponent E with round4(amax) <= 448 * 2^E."""
    i = _round4(amax).view(torch.int32)
    e, m = (i >> 23) - 127, (i >> 20) & 7
    return torch.where(i == 0, E_MIN, torch.where(m <= 6, e - 8, e - 7)).clamp(min=E_MIN)


def _grid(y):
    """Values of 4 significant bits on e4m3's grid: below 2^-6 its spacing is 2^-9, and what is finer is cut off."""
    return torch.where(y.abs() < 2.0 ** -6, torch.trunc(y * 512) / 512, y).to(torch.float8_e4m3fn)


def _exponent(scale):
    return (scale.contiguous().view(torch.int32) >> 23) - 127


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _append(s):
    x = torch.stack([s["k"], s["v"]])  # [2, T, H, D]
    T, H, D = x.shape[1:]
    p8, d16 = s["pages"].shape[3:5]
    page, pool = p8 * 8, s["pages"].shape[1]
    b, t = _tokens_of(s, T)
    pos = s["start"].long()[b] + t
    ids = s["table"].long()[b, pos // page]
    x = x.float()
    amax = torch.zeros(2, pool, H, device=DEV).index_reduce_(1, ids, x.abs().amax(-1), "amax")
    # the first page of each sequence may hold older tokens
    first = s["table"].long()[torch.arange(s["start"].numel(), device=DEV), s["start"].long() // page]
    old = s["start"].long() % page  # how many
    was = _exponent(s["scales"])
    e = _need(amax)
    e[:, first] = torch.where(old[None, :, None] > 0, torch.maximum(e[:, first], was[:, first]), e[:, first])
    touched = torch.zeros(pool, dtype=torch.bool, device=DEV)
    touched[ids] = True
    e = torch.where(touched[None, :, None], e, was)
    # older tokens of those pages follow the larger scale
    raw = s["pages"].view(torch.uint8)
    keep = raw[:, first].view(torch.float8_e4m3fn).float()
    down = _pow2((was - e)[:, first].clamp(min=-120))[..., None, None, None, None]
    tok = torch.arange(page, device=DEV).view(p8, 1, 8, 1)
    redo = tok[None] < old.view(-1, 1, 1, 1, 1)
    raw[:, first] = torch.where(redo[None, :, None], _grid(keep * down).view(torch.uint8), raw[:, first])
    y = _grid(_round4(x) * _pow2(-e[:, ids])[..., None])  # [2, T, H, D]
    o = pos % page
    raw.view(2, pool, H, p8, d16, 8, 16)[:, ids, :, o // 8, :, o % 8] = y.view(torch.uint8).view(2, T, H, d16, 16).permute(1, 0, 2, 3, 4)
    s["scales"].copy_(_pow2(e))
    return {"pages": s["pages"], "scales": s["scales"]}


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _free_pages(refs):
    return torch.argsort((refs != 0).to(torch.uint8), stable=True)  # the free ones first, ascending


def _fork(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    par, chi, page = s["parents"].long(), s["children"].long(), s["pages"].shape[4] * 8
    rows, n = table[par].long(), lens[par].long()
    full, part = n // page, n % page != 0
    new = _free_pages(refs)[(part.cumsum(0) - 1).clamp(min=0)]
    j = torch.arange(table.shape[1], device=DEV)[None]
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    dst = torch.where(part, new, rows[:, 0])
    src = torch.where(part, last, rows[:, 0])
    shared = j < full[:, None]
    refs.index_add_(0, rows.clamp(min=0).flatten(), shared.flatten().to(torch.int32))
    refs[dst] = torch.where(part, torch.ones_like(refs[dst]), refs[dst])
    table[chi] = torch.where(shared, rows, torch.where((j == full[:, None]) & part[:, None], new[:, None], -1)).to(torch.int32)
    lens[chi] = n.to(torch.int32)
    raw = s["pages"].view(torch.uint8)
    raw[:, :, dst] = raw[:, :, src]
    s["scales"][:, :, dst] = s["scales"][:, :, src]


def _extend(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    rows, page = s["children"].long(), s["pages"].shape[4] * 8
    at, n = lens[rows].long(), s["n_new"].long()
    have = _pages_of(at, page)
    need = _pages_of(at + n, page) - have
    ok = (need.sum() <= (refs == 0).sum()) & ((have + need) <= table.shape[1]).all()
    j = torch.arange(-(-s["max_new"] // page) + 1, device=DEV)[None]
    new = _free_pages(refs)[((need.cumsum(0) - need)[:, None] + j).clamp(max=refs.numel() - 1)]
    put = (j < need[:, None]) & ok
    col = (have[:, None] + j).clamp(max=table.shape[1] - 1)
    col, row = torch.where(put, col, 0), rows[:, None].expand_as(put)
    table[row[put], col[put]] = new[put].to(torch.int32)
    refs[new[put]] = 1
    lens[rows] = torch.where(ok, at + n, at).to(torch.int32)
    return torch.where(ok, at, -1).to(torch.int32)


def _free(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    rows, page = s["children"].long(), s["pages"].shape[4] * 8
    held = torch.arange(table.shape[1], device=DEV)[None] < _pages_of(lens[rows].long(), page)[:, None]
    refs.index_add_(0, table[rows].long().clamp(min=0).flatten(), -held.flatten().to(torch.int32))
    table[rows] = -1
    lens[rows] = 0


def _compact(s):
    table, refs = s["table"].clone(), s["refs"].clone()
    page, pool = s["pages"].shape[4] * 8, refs.numel()
    live = refs != 0
    count = live.sum()
    at = torch.arange(pool, device=DEV)
    hole, high = ~live & (at < count), live & (at >= count)
    # the k-th live page behind the front goes to the k-th hole in it
    src, dst = high.nonzero()[:, 0], hole.nonzero()[:, 0]
    to = at.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    held = torch.arange(table.shape[1], device=DEV)[None] < _pages_of(s["lens"].long(), page)[:, None]
    table = torch.where(held, to[table.long().clamp(min=0)].to(torch.int32), table)
    raw = s["pages"].view(torch.uint8)
    raw[:, :, dst] = raw[:, :, src]
    s["scales"][:, :, dst] = s["scales"][:, :, src]
    return {"live": count.to(torch.int32).view(1), "table": table, "refs": refs, "pages": s["pages"], "scales": s["scales"]}


def _sample(s):
    z = s["logits"].float()
    B, V = z.shape
    # values next to a border decide: weights and their running sums in 64 bits
    val, idx = z.sort(dim=1, descending=True, stable=True)
    temp = s["temperature"].double()[:, None]
    x = val.double() - val[:, :1].double()
    w = torch.exp(x / torch.where(temp > 0, temp, torch.ones_like(temp)))
    rank = torch.arange(V, device=DEV)[None]
    keep = (rank == 0) | (temp > 0)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((k <= 0) | (rank < k))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        c = torch.cumsum(w * keep, 1)
        keep = keep & ((p >= 1) | (c - w * keep < p * c[:, -1:]))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None])
    c = torch.cumsum(torch.zeros_like(w).scatter_(1, idx, w * keep), 1)
    return (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1).to(torch.int32)


# --------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("branch", "compact", "sample"):
        return None  # whole numbers, and bytes that are moved
    s = prepare(case, seed)
    z, page, D, H = _sizes(case), case["page"], case["head_dim"], case["kv_heads"]
    if op == "attend":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        G, at = case["heads"] // H, 0
        for b, (start, n) in enumerate(zip(z["start"], z["n"])):
            ids = s["table"][b, :-(-(start + n) // page)].long()
            q = s["q"][at:at + n].double()
            for h in range(H):
                kv = [s["pages"].view(torch.uint8)[c, ids, h].view(torch.float8_e4m3fn).double() for c in (0, 1)]
                k, v = [(x.transpose(2, 3).reshape(len(ids), page, D) * s["scales"][c, ids, h].double()[:, None, None])
                        .reshape(-1, D)[:start + n] for c, x in enumerate(kv)]
                for g in range(h * G, (h + 1) * G):
                    a = q[:, g] @ k.T / math.sqrt(D)
                    if n > 1:
                        later = torch.arange(start + n, device=DEV)[None] > start + torch.arange(n, device=DEV)[:, None]
                        a = a.masked_fill(later, float("-inf"))
                    out[at:at + n, g] = torch.softmax(a, 1) @ v
            at += n
        return out
    # append: each page of each sequence by itself
    pages, scales = s["pages"].double(), s["scales"].double()
    at = 0
    for b, (start, n) in enumerate(zip(z["start"], z["n"])):
        i = 0
        while i < n:
            pid, o = int(s["table"][b, (start + i) // page]), (start + i) % page
            m = min(page - o, n - i)
            x = torch.stack([s["k"][at + i:at + i + m], s["v"][at + i:at + i + m]]).double()  # [2, m, H, D]
            f, e = torch.frexp(x)
            x = torch.ldexp(torch.round(f * 16), e - 4)  # 4 significant bits, ties to even
            top = x.abs().amax((1, 3))
            f, e = torch.frexp(top / 448)  # top / 448 <= 2^E
            e = torch.where(top > 0, torch.where(f == 0.5, e - 1, e), E_MIN).clamp(min=E_MIN).double()
            was = torch.log2(scales[:, pid])
            e = torch.maximum(e, was) if o else e
            old = pages[:, pid].transpose(3, 4).reshape(2, H, page, D)
            down = old[:, :, :o] * torch.exp2(was - e)[..., None, None]
            y = x.transpose(1, 2) * torch.exp2(-e)[..., None, None]
            cut = lambda a: torch.where(a.abs() < 2.0 ** -6, torch.trunc(a * 512) / 512, a)  # noqa: E731
            old = torch.cat([cut(down), cut(y), old[:, :, o + m:]], 2)  # what is not written yet stays
            pages[:, pid] = old.reshape(2, H, page // 8, 8, D // 16, 16).transpose(3, 4)
            scales[:, pid] = torch.exp2(e)
            i += m
        at += n
    return {"pages": pages, "scales": scales}
